"""The counts of clusters that a device runs, asked for by several threads at once:
compiled for the host, no GPU."""
import ctypes
import os
import subprocess

import pytest

from sparse_attention_indexer_logits_gb300 import _build


@pytest.fixture
def counts(tmp_path):
    so = str(tmp_path / "cluster_counts.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cluster_counts.cpp")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", "-I", _build.CSRC, src, "-o", so], check=True,
                   capture_output=True, text=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("device,size", [(0, 8), (0, 2), (1, 8), (1, 4)])
def test_a_call_beside_the_first(counts, device, size):
    out = (ctypes.c_int * 4)()
    counts.two_first_calls(device, size, out)
    assert list(out) == [8, 1000 * device + size, 1000 * device + size, 0]


def test_devices_in_turn(counts):
    assert counts.in_turn() == 1


def test_none_is_an_answer(counts):
    asked = ctypes.c_int()
    assert counts.none(ctypes.byref(asked)) == 0 and asked.value == 1
