"""How attention's work is counted and cut, compiled for the host: units of
requests of any length, and ranges that have every tile once."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from sparse_attention_indexer_logits_gb300 import _build

ITEM = 3     # units of an item besides its tiles


@pytest.fixture(scope="module")
def W(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("work") / "attention_work.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "attention_work.cu")
    subprocess.run([_build._nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC", "-gencode",
                    "arch=compute_103a,code=sm_103a", "-I", _build.CSRC, "-I", _build.INCLUDE, src, "-o", so],
                   check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(so)
    lib.request_units.restype = ctypes.c_longlong
    return lib


def units(group, width, causal, window, nq, kv):
    """The same by the definition, in 64 bits: per tile of 2 * (128 / group)
    tokens, the 128-key tiles between the first and the last key that one of
    them may see (at least one), twice where they fill more than a half."""
    half = 128 // group
    t0 = np.arange(0, nq, 2 * half, dtype=np.int64)
    ntok = np.minimum(2 * half, nq - t0)
    pos = kv - nq + t0
    hi = np.full_like(t0, min(kv, 64 * width))
    if causal:
        hi = np.minimum(hi, pos + ntok)
    lo = np.maximum(0, pos - window + 1) if window else np.zeros_like(t0)
    none = hi <= lo
    n = np.where(none, 1, (np.maximum(hi, 1) - 1) // 128 + 1 - lo // 128)
    return int((n * np.where(ntok <= half, 1, 2) + ITEM).sum())


@pytest.mark.parametrize("group,causal,nq,kv", [
    (64, True, 1 << 20, 1 << 20), (128, True, 740000, 740000), (128, False, 530000, 530000),
    (128, True, 1 << 20, 1 << 20), (7, True, 3000000, 9000000), (1, True, 5, 1 << 30), (32, False, 1 << 20, 1 << 24)])
def test_units_of_long_requests(W, group, causal, nq, kv):
    want = units(group, 1 << 25, causal, 0, nq, kv)
    assert W.request_units(group, (1 << 25) - 1, int(causal), 0, nq, kv) == want
    if group >= 64 and (nq == 1 << 20 or not causal):
        assert want > 2 ** 31 - 1


def test_units_of_random_requests(W):
    r = random.Random(0)
    for _ in range(500):
        group, causal = r.choice([1, 2, 5, 8, 16, 33, 64, 65, 128]), r.random() < 0.7
        window, kv = r.choice([0, 0, 1, 64, 1000]), r.choice([0, 1, r.randint(0, 300), r.randint(0, 40000)])
        nq, width = r.choice([0, 1, r.randint(0, 700)]), r.choice([1, 10, 1000])
        assert W.request_units(group, width, int(causal), window, nq, kv) == \
            units(group, width, causal, window, nq, kv), (group, causal, window, kv, nq, width)


def test_ranges_have_every_tile_once(W):
    """Ranges of any size, cut through items as the producer walks them."""
    r = random.Random(1)
    for _ in range(300):
        items = [(r.choice([1, 1, 2, 3, 17, 60]), r.choice([1, 2])) for _ in range(r.randint(1, 12))]
        total = sum(W.item_units(n, c) for n, c in items)
        ctas = r.choice([1, 2, 7, 40, 152])
        cuts = [total * k // ctas for k in range(ctas + 1)]
        seen = []
        for lo, hi in zip(cuts, cuts[1:]):
            base = 0
            for i, (n, c) in enumerate(items):
                u = W.item_units(n, c)
                a, b = max(lo, base) - base, min(hi, base + u) - base
                if a < b:
                    seen += [(i, t) for t in range(W.before(n, c, a), W.before(n, c, b))]
                base += u
        assert seen == [(i, t) for i, (n, _) in enumerate(items) for t in range(n)]


@pytest.mark.parametrize("back", [64, 65, 100, 128, 191, 192, 300])
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("window", [0, 1, 200, 1 << 30, (1 << 30) + 5, 2 ** 31 - 1])
def test_spans_at_the_farthest_positions(W, back, causal, window):
    """Lengths up to the last position that a table can hold, 2^31 - 65, and
    windows past 2^30."""
    width, kv, nq = (1 << 25) - 1, 2 ** 31 - back, 3
    out = (ctypes.c_int * 7)()
    W.span(8, width, causal, window, nq, kv, 0, out)
    t0, ntok, lo, hi, j0, n, cost = out
    there = min(kv, 64 * width)
    want_lo = max(0, kv - nq - window + 1) if window else 0
    assert (t0, ntok, lo, hi, cost) == (0, 3, want_lo, there, 1)
    assert j0 == want_lo // 128 and n == -(-there // 128) - want_lo // 128
