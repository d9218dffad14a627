"""Attention over caches held in 4 bits, rows of q far below 1 under a softmax
scale that brings their logits back to ordinary sizes: warp by warp (few heads)
and by tiles (many), as the definition in 64 bits."""
import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import serving_ref as R
from tests.test_nvfp4_attention_gpu import BF, Problem, check, check_selected

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


def shrunk(p, first, seed):
    """Each head's rows times a power of two, 2^first .. 2^(first + 7)."""
    size = torch.exp2(torch.linspace(first, first + 7, p.hq).round())[:, None]
    p.q = (torch.randn(p.q.shape, generator=R.gen(seed)) * size).to(BF)
    return p


# (logits of the smallest rows about 1, of the largest about 200)
@pytest.mark.parametrize("first,scale", [(-100, 2.0 ** 97), (-92, 2.0 ** 89), (-80, 2.0 ** 77), (-65, 2.0 ** 62)])
@pytest.mark.parametrize("hq", [4, 64])
@pytest.mark.parametrize("dim", [64, 128])
def test_small_rows_under_a_large_scale(first, scale, hq, dim):
    p = shrunk(Problem([1, 2], [2500, 170], hq, 1, dim, BF, seed=31).stale(), first, 32)
    check(p, *p.run(softmax_scale=scale), scale=scale)


@pytest.mark.parametrize("hq", [4, 64])
def test_one_request_of_many_tokens(hq):
    """Tiles with both halves full, and items that several CTAs share."""
    p = shrunk(Problem([9], [3000], hq, 1, 128, BF, seed=33).stale(), -95, 34)
    check(p, *p.run(softmax_scale=2.0 ** 92), scale=2.0 ** 92, heads=range(0, hq, 1 + hq // 12))


@pytest.mark.parametrize("copies", [1, 300])
def test_lists(copies):
    p = shrunk(Problem([1] * copies, [700] * copies, 64, 1, 128, BF, seed=35, k_scale=4.0), -98, 36)
    sel = torch.randint(-50, 700, (copies, 300), generator=R.gen(37), dtype=torch.int32)
    req = torch.arange(copies, dtype=torch.int32)
    lse = torch.empty((copies, 64), device="cuda")
    out = pml.pml_sparse_attention_nvfp4(*p.device(), req.cuda(), sel.cuda(), lse=lse, softmax_scale=2.0 ** 94,
                                         k_scale=4.0)
    assert pml.pml_device_status(clear=True) == 0
    check_selected(p, req[:8], sel[:8], out, lse, heads=range(0, 64, 7), scale=2.0 ** 94)
