"""How work over caches held in 4 bits is counted, compiled for the host."""
import ctypes
import os
import subprocess

import pytest

from sparse_attention_indexer_logits_gb300 import _build


@pytest.fixture(scope="module")
def W(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("work") / "nvfp4_work.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "nvfp4_work.cu")
    subprocess.run([_build._nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC", "-gencode",
                    "arch=compute_103a,code=sm_103a", "-I", _build.CSRC, "-I", _build.INCLUDE, src, "-o", so],
                   check=True, capture_output=True, text=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("n", [-2 ** 31, -1, 0, 1, 63, 64, 65, 5000, 2 ** 31 - 129, 2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 63,
                               2 ** 31 - 1])
def test_blocks_of_any_length(W, n):
    assert W.blocks(n) == max(0, (n + 63) // 64)
