"""The library's calls that go through ctypes need no compiled Python module;
the serving operators' calls say so where theirs cannot be loaded."""
import os
import subprocess
import sys

import pytest

from sparse_attention_indexer_logits_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["sparse_attention_indexer_logits_gb300._calls"] = None     # what an import of it meets
import torch
import sparse_attention_indexer_logits_gb300 as pml
assert pml.pml_min_block_table_width(130) == pml.lib().pml_min_block_table_width(130) > 0
assert pml.lib().pml_version() > 0
assert "invalid" in str(pml.PmlError(1, "x"))
try:
    pml.pml_fp8_paged_mqa_logits(*[torch.zeros(1)] * 6, 1, 1)
except ValueError as e:
    assert "CUDA tensor" in str(e), e
else:
    raise AssertionError("not refused")
try:
    pml.pml_rope(torch.zeros((1, 1, 2)), torch.zeros(1), torch.zeros(1))
except RuntimeError as e:
    assert "_calls.so cannot be loaded" in str(e), e
else:
    raise AssertionError("called")
print("fine")
"""


def test_the_older_calls_without_the_module():
    _build.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split()[-1] == "fine", r.stderr


def test_a_failing_module_leaves_the_library(monkeypatch, tmp_path):
    """Without g++ or PyTorch's headers the library is built all the same."""
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "libpml.so"))
    monkeypatch.setattr(_build, "CALLS_PATH", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(_build, "SOURCES", ["schedule.cu"])
    done = []

    def no_headers(*args):
        done.append(args)
        raise RuntimeError("g++ failed on binding.cpp")

    monkeypatch.setattr(_build, "_build_calls", no_headers)
    for _ in range(2):
        with pytest.raises(RuntimeError, match="g.. failed"):
            _build.build()
        assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.CALLS_PATH)
    assert len(done) == 2
