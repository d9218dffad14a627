"""Attention whose logits are far from 0: every row and its log-sum against the
definition in 64 bits, under bounds for fp32 scores of their size."""
import math

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import serving_ref as R
from tests.test_attention_gpu import BF, FP, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


def compare_rows(p, out, lse, scale):
    """A score is a sum of products that are exact in fp32: each further one
    adds a rounding of 2^-23 of their magnitudes' sum at most (the tensor core
    may cut off), `score` in all.  A weight is 2^(c x - c m): off by the two
    scores' errors, the rounding of c m (2^-14 of an exponent where |c m| is
    below 1024, and a difference of fp32 numbers past it) under either of two
    references, and the approximate power, 2^-20: `rel` of the weight.
    Numerator and denominator are off by that, P is rounded once, the output
    once.  The log-sum is off by `rel` and three fp32 roundings of its own
    size."""
    half = torch.finfo(p.dtype).eps / 2
    group, rows = p.hq // p.hkv, 0
    for b in range(len(p.qn)):
        lo, hi = int(p.cu[b]), int(p.cu[b + 1])
        k, v = p.keys(b)
        allowed = torch.arange(p.kvn[b]) <= torch.arange(p.kvn[b] - (hi - lo), p.kvn[b])[:, None]
        for h in range(p.hq):
            q, kk = p.q[lo:hi, h].double(), k[:, h // group].double()
            want, want_lse, mag = R.attention(p.q[lo:hi, h], k[:, h // group], v[:, h // group], allowed, scale)
            size = q.abs() @ kk.abs().T
            more = ((q != 0).double() @ (kk != 0).double().T - 1).clamp(min=0)
            fits = size.amax(1) < 3e38
            score = (scale * size * more * 2.0 ** -23).masked_fill(~allowed, 0.0).amax(1)
            rel = 2 * score + 2 * math.log(2) * 2.0 ** -14 + 2.0 ** -20
            got, got_lse = out[lo:hi, h].cpu().double(), lse[lo:hi, h].cpu().double()
            bound = mag * (half + 2 * rel[:, None]) + half * want.abs() + 1e-7
            err = (got - want).abs()
            assert (err <= bound)[fits].all(), f"request {b} head {h}: {(err / bound)[fits].max():.3g} bounds"
            off = (got_lse - want_lse).abs()
            assert (off <= rel + 3 * 2.0 ** -24 * want_lse.abs() + 1e-6)[fits].all(), f"request {b} head {h}"
            rows += int(fits.sum())
    assert pml.pml_device_status(clear=True) == 0
    return rows


QN, KVN = [3, 40, 1], [150, 333, 20000]


@pytest.mark.parametrize("low", [-80, -130, -200, -1e3, -1e20, -1e36])
def test_some_keys_far_away(low):
    """Every seventh key's scores are thousands above or below the others', and
    grow along the cache: |c m| passes 1024 within a row's tiles and pieces."""
    p = Problem(QN, KVN, 4, 1, 64, BF, seed=5)
    p.q *= 40
    for b, n in enumerate(KVN):
        at = torch.arange(0, n, 7)
        page = p.table[b].long()[at // 64]
        p.k[page, at % 64] = 0
        p.k[page, at % 64, :, 0] = (low * (0.5 + at / n)).to(BF)[:, None]
    p.stale(torch.finfo(BF).min)
    assert compare_rows(p, *p.run(), 64 ** -0.5) == 44 * 4


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("offset", [-3000.0, -1500.0, -700.0, -300.0, 300.0, 700.0, 1500.0, 3000.0])
def test_all_keys_far_away(dtype, dim, offset):
    """All of a row's logits around an offset, their differences of order one."""
    p = Problem(QN, KVN, 4, 2, dim, dtype, seed=6)
    p.k[..., 0] = 128.0
    p.q[..., 0] = offset * dim ** 0.5 / 128.0
    p.stale()
    out, lse = p.run()
    assert compare_rows(p, out, lse, dim ** -0.5) == 44 * 4
    assert ((lse.cpu() / offset - 1).abs() < 0.2).all()


def test_a_long_tail_below_one_large_weight():
    """One key's weight is 2^25 times each of 2^20 others', whose sum is 2.7 %
    of all: fp16 weights must not lose them.  A weight below 2^-21 of the
    largest is off by 2^-32 of it at most (half a step of fp16's subnormals
    under a largest of 2^7)."""
    n, tokens = 2 ** 20, 152 * 256
    k = torch.zeros((n // 64, 64, 1, 64), dtype=FP, device="cuda")
    v = torch.ones_like(k)
    k[0, 0, 0, 0], v[0, 0] = 17.4375, 0.0
    q = torch.zeros((tokens, 1, 64), dtype=FP, device="cuda")
    q[..., 0] = 8.0                             # scores are the keys' first elements
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = torch.empty((tokens, 1), device="cuda")
    out = pml.pml_paged_attention(q, k, v, table, lens, causal=False, lse=lse)
    tail = (n - 1) * math.exp(-17.4375)
    want = tail / (1 + tail)
    # sums of 4096 tiles' sums in fp32: 2^-24 each, cut off by eight steps a
    # tile in tensor memory, 2^-23 each
    rel = 2.0 ** -11 + 2e-4 + 4096 * 8 * 2.0 ** -23
    assert (out.double() - want).abs().max() <= want * (rel + 2.0 ** -11) + n * 2.0 ** -32
    assert (lse.double() - 17.4375 - math.log1p(tail)).abs().max() <= 4096 * 2.0 ** -24 + 1e-4
    assert pml.pml_device_status(clear=True) == 0
