"""Attention over caches held in 4 bits, rows of q whose size times the softmax
scale is past fp32, over keys of zeros: every logit is 0 and the output the mean
of the values, warp by warp (few heads) and by tiles (many)."""
import math

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests.test_nvfp4_attention_gpu import BF, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


@pytest.mark.parametrize("hq", [2, 64])
@pytest.mark.parametrize("kvn", [[300, 4000], [4000]])
def test_keys_of_zeros(hq, kvn):
    p = Problem([2] * len(kvn), kvn, hq, 1, 64, BF, seed=41).stale()
    p.q *= 2.0 ** 100
    p.parts[0].zero_()
    out, lse = p.run(causal=False, softmax_scale=2.0 ** 99)
    assert pml.pml_device_status(clear=True) == 0
    for b, n in enumerate(kvn):
        _, v = p.rows(b, torch.arange(n))
        want, mag = v[:, 0].mean(0), v[:, 0].abs().mean(0)
        rows = slice(2 * b, 2 * b + 2)
        # P is rounded once, the output once; sums of n products at 2^-23 each
        off = (out[rows].cpu().double() - want).abs()
        assert (off <= (2.0 ** -11 + 2.0 ** -20 + n * 2.0 ** -23) * mag + 2.0 ** -8 * want.abs()).all()
        assert (lse[rows].cpu().double() - math.log(n)).abs().max() <= 1e-5
