"""Attention over pages where the items of a CTA's range follow each other in
ways that its groups have to keep apart."""
import math

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import serving_ref as R
from tests.test_attention_gpu import BF, FP, Problem, check, check_selected, compare

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


@pytest.mark.parametrize("dim,dtype", [(64, BF), (128, FP)])
def test_items_of_one_tile_after_longer_ones(dim, dtype):
    """One tile leaves a half without work: it comes to that item's end while
    the other half may be at the end of the item before."""
    g = R.gen(31)
    short, longer = torch.randint(1, 129, (700,), generator=g), torch.randint(129, 600, (700,), generator=g)
    kvn = torch.stack([longer, short], 1).flatten().tolist()
    p = Problem([1] * len(kvn), kvn, 4, 2, dim, dtype, seed=32).stale()
    out, lse = p.run(cu=False)
    check(p, out, lse, requests=range(0, len(kvn), 61))
    q, k, v, table, lens = p.device()
    for _ in range(20):
        again = torch.full_like(lse, 77.0)
        assert torch.equal(pml.pml_paged_attention(q, k, v, table, lens, lse=again), out)
        assert torch.equal(again, lse)


@pytest.mark.parametrize("k", [100, 300])
def test_lists_of_a_prompt(k):
    """A list for every token of a prompt: several items a CTA, of one tile and
    of more, some cut between CTAs."""
    g = R.gen(k)
    kvn, tokens = [900, 260], 900
    p = Problem([1, 1], kvn, 64, 1, 64, BF, seed=33).stale()
    p.q = (torch.randn((tokens, 64, 64), generator=g) * 1.5).to(BF)
    req = torch.randint(0, 2, (tokens,), generator=g, dtype=torch.int32)
    sel = torch.randint(-50, 900, (tokens, k), generator=g, dtype=torch.int32)
    q, kc, vc, table, lens = p.device()
    lse = torch.empty((tokens, 64), device="cuda")
    out = pml.pml_sparse_attention(q, kc, vc, table, lens, req.cuda(), sel.cuda(), lse=lse)
    assert pml.pml_device_status(clear=True) == 0
    at = list(range(0, tokens, 37))
    p.q = p.q[at]
    check_selected(p, req[at], sel[at], out[at], lse[at])
    for _ in range(10):
        assert torch.equal(pml.pml_sparse_attention(q, kc, vc, table, lens, req.cuda(), sel.cuda()), out)


@pytest.mark.parametrize("dim,dtype", [(64, FP), (128, BF)])
def test_infinities_in_the_first_tile_of_every_item(dim, dtype):
    """Two new tokens, the last one's values infinite: the first token must not
    see them, so each item's product is added row by row, right after the item
    before has ended."""
    g = R.gen(34)
    kvn = torch.randint(2, 260, (900,), generator=g).tolist()
    p = Problem([2] * len(kvn), kvn, 4, 2, dim, dtype, seed=35).stale()
    for b, n in enumerate(kvn):
        p.v[p.table[b, (n - 1) // 64].long(), (n - 1) % 64, :, b % dim] = math.inf
    out, lse = p.run(cu=False)
    check(p, out, lse, requests=range(0, len(kvn), 71))
    assert torch.isfinite(out[::2]).all()
    q, k, v, table, lens = p.device()
    for _ in range(20):
        assert torch.equal(pml.pml_paged_attention(q, k, v, table, lens), out)


def far_away(window, pages):
    """One token at the last position that a table can hold, its table all
    pages in turn."""
    g = R.gen(36)
    width, kv = 2 ** 25 - 1, 2 ** 31 - 64
    table = (torch.arange(width, device="cuda", dtype=torch.int32) % pages)[None]
    q = torch.randn((1, 2, 64), generator=g).to(BF)
    k, v = (torch.randn((pages, 64, 1, 64), generator=g).to(BF) for _ in range(2))
    lse = torch.empty((1, 2), device="cuda")
    out = pml.pml_paged_attention(q.cuda(), k.cuda(), v.cuda(), table, torch.tensor([kv], dtype=torch.int32).cuda(),
                                  window=window, lse=lse)
    assert pml.pml_device_status(clear=True) == 0
    at = (torch.arange(max(0, kv - window), kv) if window <= 1000 else torch.arange(64 * pages)) % (64 * pages)
    k, v = (c.reshape(-1, 64)[at] for c in (k, v))
    return [(out[:, h], lse[:, h]) + R.attention(q[:, h], k, v, torch.ones((1, len(at)), dtype=torch.bool), 0.125)
            for h in range(2)]


@pytest.mark.parametrize("window", [1, 64, 100, 200, 1000])
def test_the_farthest_position(window):
    for got, lse, want, want_lse, mag in far_away(window, 7):
        compare(got, lse, want, want_lse, mag, BF)


def test_a_window_past_2_to_the_30():
    """Every key of 2^31 counts: one page, 2^25 - 1 times, changes the sum and
    not the average.  A CTA adds up 1.1e5 tiles, each sum rounded in fp32
    (2^-24 each of the running one; in tensor memory eight steps a tile, cut
    off rather than rounded, 2^-23 each)."""
    for got, lse, want, want_lse, mag in far_away(2 ** 31 - 1, 1):
        assert abs(lse.item() - want_lse.item() - math.log(2 ** 25 - 1)) <= 1.2e5 * 2.0 ** -24 + 1e-4
        assert ((got.cpu().double() - want).abs() <= (1e6 * 2.0 ** -23 + 2.0 ** -7) * mag).all()
