"""GPU parity of pml_paged_attention and pml_sparse_attention with the
definitions in 64 bits: single tokens, chunks and mixed batches; head groups
from 1 to 128; causal, windows, neither; empty requests and rows without a
key; layouts, strides and caches past 32 bits; stale slots, infinities and NaN
in masked places; pages and requests out of range; lists with holes."""
import math

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


class Problem:
    def __init__(self, qn, kvn, hq, hkv, dim, dtype, seed, layout="nhd", spare=3):
        g = R.gen(seed)
        self.qn, self.kvn, self.hq, self.hkv, self.dim, self.dtype = qn, kvn, hq, hkv, dim, dtype
        self.table, pages = R.block_table(kvn, g, spare)
        self.q = (torch.randn((sum(qn), hq, dim), generator=g) * 1.5).to(dtype)
        shape = (pages, 64, hkv, dim) if layout == "nhd" else (pages, hkv, 64, dim)
        self.k, self.v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
        if layout == "hnd":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.cu = torch.tensor([0] + list(torch.tensor(qn).cumsum(0)), dtype=torch.int32)
        self.kv_lens = torch.tensor(kvn, dtype=torch.int32)

    def stale(self, value=math.nan):
        """Slots past each request's end hold `value`."""
        for b, n in enumerate(self.kvn):
            if n % 64:
                for c in (self.k, self.v):
                    c[self.table[b, n // 64].long(), n % 64:] = value
        return self

    def keys(self, b):
        p = torch.arange(max(self.kvn[b], 0))
        page = self.table[b].long()[p // 64]
        return self.k[page, p % 64], self.v[page, p % 64]

    def device(self):
        # a transposed cache keeps its layout on the way to the GPU
        def up(c):
            return c.cuda() if c.is_contiguous() else c.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        return self.q.cuda(), up(self.k), up(self.v), self.table.cuda(), self.kv_lens.cuda()

    def run(self, cu=True, **kw):
        q, k, v, table, lens = self.device()
        lse = torch.full(q.shape[:2], 77.0, device="cuda")
        out = pml.pml_paged_attention(q, k, v, table, lens, self.cu.cuda() if cu else None, lse=lse, **kw)
        return out, lse


def compare(got, lse, want, want_lse, mag, dtype, where=""):
    """P is rounded once (half a step of the type), the output once; scores of
    128 exact products summed in fp32 and exponentials add 2e-4 at most."""
    half = torch.finfo(dtype).eps / 2
    got, lse = got.cpu().double(), lse.cpu().double()
    assert not torch.isnan(got[torch.isfinite(want)]).any(), f"NaN {where}"
    fine = torch.isfinite(want)
    err = (got - want)[fine].abs()
    bound = (mag * (half + 2e-4) + half * want.abs() + 1e-7)[fine]
    assert (err <= bound).all(), f"{where}: off by {(err / bound).max():.3g} bounds"
    assert torch.equal(torch.isfinite(got), fine), where
    none = torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(lse), none), where
    assert ((lse - want_lse)[~none & torch.isfinite(want_lse)].abs() <=
            1e-4 + 1e-6 * want_lse[~none & torch.isfinite(want_lse)].abs()).all(), where


def check(p, out, lse, causal=True, window=0, scale=None, requests=None):
    scale = p.dim ** -0.5 if scale is None else scale
    group = p.hq // p.hkv
    for b in range(len(p.qn)) if requests is None else requests:
        lo, hi = int(p.cu[b]), int(p.cu[b + 1])
        if lo == hi:
            continue
        k, v = p.keys(b)
        at = torch.arange(p.kvn[b])
        here = torch.arange(p.kvn[b] - (hi - lo), p.kvn[b])[:, None]
        allowed = (at <= here) if causal else torch.ones((hi - lo, p.kvn[b]), dtype=torch.bool)
        if window:
            allowed = allowed & (at > here - window)
        for h in range(p.hq):
            want, want_lse, mag = R.attention(p.q[lo:hi, h], k[:, h // group], v[:, h // group], allowed, scale)
            compare(out[lo:hi, h], lse[lo:hi, h], want, want_lse, mag, p.dtype, f"request {b} head {h}")
    assert pml.pml_device_status(clear=True) == 0


BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kvn", [[1], [64], [100], [128], [129], [1000], [300, 1, 2500]])
def test_single_tokens(dim, dtype, kvn):
    p = Problem([1] * len(kvn), kvn, 8, 2, dim, dtype, seed=sum(kvn)).stale()
    check(p, *p.run(cu=False))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 4), (10, 2), (7, 1), (16, 1), (33, 1), (64, 1), (65, 1),
                                    (128, 1), (100, 1), (256, 2)])
@pytest.mark.parametrize("q", [1, 3])
def test_head_groups(hq, hkv, q):
    p = Problem([q, q], [200, 77], hq, hkv, 64, BF, seed=hq).stale()
    check(p, *p.run(cu=False))


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("q,kv", [(2, 2), (16, 16), (33, 33), (64, 64), (65, 300), (128, 128), (257, 257),
                                  (500, 500), (100, 1111)])
def test_chunks(dim, q, kv):
    p = Problem([q], [kv], 4, 1, dim, BF, seed=q + kv).stale()
    check(p, *p.run())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window", [0, 1, 60, 64, 130, 700])
@pytest.mark.parametrize("causal", [True, False])
def test_mixed_batches(dtype, window, causal):
    qn, kvn = [1, 0, 130, 70, 1, 5, 0, 300], [900, 50, 130, 700, 1, 64, 0, 421]
    p = Problem(qn, kvn, 6, 2, 64, dtype, seed=window).stale()
    check(p, *p.run(causal=causal, window=window), causal=causal, window=window)


def test_rows_without_a_key():
    qn, kvn = [4, 100, 3, 1, 40], [0, 30, 1, 0, 39]
    p = Problem(qn, kvn, 8, 2, 128, BF, seed=1).stale()
    out, lse = p.run()
    check(p, out, lse)
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all() and (out[4:74] == 0).all()


def test_many_short_requests_and_one_long():
    g = R.gen(0)
    kvn = torch.randint(1, 200, (400,), generator=g).tolist() + [3000]
    p = Problem([1] * 401, kvn, 4, 2, 64, BF, seed=2).stale()
    check(p, *p.run(), requests=list(range(0, 400, 23)) + [400])


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_layouts_strides_and_given_outputs(layout):
    p = Problem([5, 60], [70, 200], 6, 3, 128, FP, seed=4, layout=layout).stale()
    q, k, v, table, lens = p.device()
    # q out of a wider projection, pages apart, a wider table, an output with gaps
    wide = torch.zeros((65, 10, 136), dtype=FP, device="cuda")
    wide[:, 2:8, :128] = q
    kp = torch.full((k.shape[0], 2) + (k.shape[1:] if layout == "nhd" else (3, 64, 128)), math.nan, dtype=FP,
                    device="cuda")
    views = []
    for i, c in enumerate((k, v)):
        dst = kp[:, i] if layout == "nhd" else kp[:, i].transpose(1, 2)
        dst.copy_(c)
        views.append(dst)
    tw = torch.full((2, table.shape[1] + 3), -7, dtype=torch.int32, device="cuda")
    tw[:, :table.shape[1]] = table
    out = torch.full((65, 6, 160), 9.0, dtype=FP, device="cuda")[:, :, :128]
    lse = torch.empty((65, 6), device="cuda")
    ws = pml.pml_attention_workspace(128)
    ws.fill_(255)
    got = pml.pml_paged_attention(wide[:, 2:8, :128], views[0], views[1], tw[:, :table.shape[1]], lens,
                                  p.cu.cuda(), out, lse=lse, workspace=ws, softmax_scale=0.3)
    assert got is out
    check(p, out, lse, scale=0.3)
    assert (out.as_strided((65, 6, 32), out.stride(), 128) == 9.0).all()


@pytest.mark.parametrize("low", [-1e3, -1e20, -1e36, torch.finfo(BF).min])
def test_large_logits_and_types_lowest_values(low):
    """Scores far past the range of exp.  Scores are fp32: a row with one that
    fp32 cannot hold is not judged."""
    p = Problem([3, 40], [150, 333], 4, 1, 64, BF, seed=5)
    p.q *= 40
    p.k[:, ::7] = low
    p.k[:, ::7, :, 1:] = 0
    p.stale(torch.finfo(BF).min)
    out, lse = p.run()
    for b in range(2):
        lo, hi = int(p.cu[b]), int(p.cu[b + 1])
        k, v = p.keys(b)
        allowed = torch.arange(p.kvn[b]) <= torch.arange(p.kvn[b] - (hi - lo), p.kvn[b])[:, None]
        for h in range(4):
            want, want_lse, mag = R.attention(p.q[lo:hi, h], k[:, 0], v[:, 0], allowed, 64 ** -0.5)
            got = out[lo:hi, h].cpu().double()
            fits = (p.q[lo:hi, h].double() @ k[:, 0].double().T).abs().amax(1) < 3e38
            assert torch.isfinite(got[fits]).all()
            # one key holds all the weight (the next score is 1e5 * 2^-8 away)
            big = fits & (want_lse.abs() > 1e5)
            assert ((got - want).abs()[big] <= 2.0 ** -7 * mag[big] + 1e-6).all()
    assert pml.pml_device_status(clear=True) == 0


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
def test_masked_places_never_reach_a_row(value, dtype, dim):
    """The values of late tokens of a chunk hold infinities or NaN: earlier
    rows must not see them, later ones must."""
    p = Problem([300, 9, 1], [300, 200, 100], 2, 1, dim, dtype, seed=6).stale(value)
    for b, pos, d in ((0, 290, 3), (0, 170, 0), (1, 196, dim - 1), (1, 199, 5)):
        p.v[p.table[b, pos // 64].long(), pos % 64, 0, d] = value
        if pos % 2:
            p.k[p.table[b, pos // 64].long(), pos % 64, 0, 0] = 2.0
    out, lse = p.run()
    check(p, out, lse)
    late = out.cpu()
    assert not torch.isfinite(late[290:300, :, 3]).any() and torch.isfinite(late[:290, :, 3]).all()
    assert not torch.isfinite(late[170:300, :, 0]).any()
    # a window's far side
    out, lse = p.run(window=64)
    check(p, out, lse, window=64)


def test_masked_keys_of_nan():
    p = Problem([40], [200], 2, 1, 64, BF, seed=7).stale()
    p.k[p.table[0, 3].long(), 199 - 192] = math.nan     # the last token's key
    out, lse = p.run()
    got = out.cpu()
    assert torch.isfinite(got[:39]).all() and torch.isnan(got[39]).all()
    k, v = p.keys(0)
    k[199] = 0
    want, want_lse, mag = R.attention(p.q[:39, 0], k[:199, 0], v[:199, 0],
                                      torch.arange(199) <= torch.arange(160, 199)[:, None], 0.125)
    compare(out[:39, 0], lse[:39, 0], want, want_lse, mag, BF)


def test_pages_out_of_range_are_flagged():
    p = Problem([1, 2], [200, 100], 4, 1, 64, BF, seed=8)
    good = p.table.clone()
    p.table[0, 1] = 9999
    p.table[1, 0] = -1
    p.run()
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK
    # entries that no row can see are not looked at
    p.table = good.clone()
    p.table[0, :2] = -1
    out, lse = p.run(window=50)
    p.table = good
    check(p, out, lse, window=50)


def test_cache_past_32_bits():
    """Pages more than 2^32 elements into the cache."""
    pages, used = 70000, [0, 3, 69998, 69999, 40000]
    k = torch.empty((pages, 64, 8, 128), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    g = R.gen(9)
    p = Problem([7], [300], 16, 8, 128, BF, seed=9)
    p.table = torch.tensor([used], dtype=torch.int32)
    small_k, small_v = (torch.randn((5, 64, 8, 128), generator=g).to(BF) for _ in range(2))
    for i, u in enumerate(used):
        k[u], v[u] = small_k[i].cuda(), small_v[i].cuda()
    lse = torch.empty((7, 16), device="cuda")
    q, table, lens = p.q.cuda(), p.table.cuda(), p.kv_lens.cuda()
    out = pml.pml_paged_attention(q, k, v, table, lens, p.cu.cuda(), lse=lse)
    sel = torch.arange(299, -1, -1, dtype=torch.int32).repeat(7, 1).cuda()
    out_s = pml.pml_sparse_attention(q, k, v, table, lens, torch.zeros(7, dtype=torch.int32, device="cuda"), sel)
    p.k, p.v, p.table = small_k, small_v, torch.tensor([[0, 1, 2, 3, 4]])
    check(p, out, lse)
    kk, vv = p.keys(0)
    for h in (0, 9):
        want, want_lse, mag = R.attention(p.q[:, h], kk[:, h // 2], vv[:, h // 2],
                                          torch.ones((7, 300), dtype=torch.bool), 128 ** -0.5)
        compare(out_s[:, h], want_lse, want, want_lse, mag, BF)


# ------------------------------------------------------------------ selected positions

def check_selected(p, req, sel, out, lse, scale=None):
    scale = p.dim ** -0.5 if scale is None else scale
    group = p.hq // p.hkv
    for t in range(len(req)):
        b = int(req[t])
        n = p.kvn[b] if 0 <= b < len(p.kvn) else 0
        at = sel[t][(sel[t] >= 0) & (sel[t] < n)].long()
        if len(at):
            page = p.table[b].long()[at // 64]
            k, v = p.k[page, at % 64], p.v[page, at % 64]
        else:
            k = v = torch.zeros((0, p.hkv, p.dim))
        for h in range(p.hq):
            want, want_lse, mag = R.attention(p.q[t:t + 1, h], k[:, h // group], v[:, h // group],
                                              torch.ones((1, len(at)), dtype=torch.bool), scale)
            compare(out[t:t + 1, h], lse[t:t + 1, h], want, want_lse, mag, p.dtype, f"token {t} head {h}")


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("k", [1, 5, 128, 129, 700])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (64, 1)])
def test_selected(dim, dtype, k, hq, hkv):
    g = R.gen(k + hq)
    kvn = [1000, 65, 1, 0, 300]
    p = Problem([1] * 5, kvn, hq, hkv, dim, dtype, seed=k).stale()
    req = torch.tensor([0, 1, 4, 2, 0, 3, 1, -1], dtype=torch.int32)
    p.q = (torch.randn((8, hq, dim), generator=g) * 1.5).to(dtype)
    # holes, repeats and positions that are not there
    sel = torch.randint(-200, 1200, (8, k + 3), generator=g, dtype=torch.int32)
    sel[2, ::2] = -1
    sel[6] = -1
    q, kd, vd, table, lens = p.device()
    lse = torch.empty((8, hq), device="cuda")
    out = pml.pml_sparse_attention(q, kd, vd, table, lens, req.cuda(), sel.cuda()[:, :k], lse=lse)
    assert pml.pml_device_status(clear=True) == 0
    check_selected(p, req, sel[:, :k], out, lse)


def test_selected_layouts_and_bad_places():
    g = R.gen(3)
    p = Problem([1, 1], [500, 400], 6, 2, 64, BF, seed=3, layout="hnd").stale()
    sel = torch.stack([torch.randperm(500, generator=g)[:200], torch.randperm(400, generator=g)[:200]]).int()
    q, k, v, table, lens = p.device()
    both = torch.stack([k.transpose(1, 2), v.transpose(1, 2)], 1)      # [pages, 2, heads, 64, dim]
    lse = torch.empty((2, 6), device="cuda")
    req = torch.tensor([0, 1], dtype=torch.int32)
    out = pml.pml_sparse_attention(q, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), table, lens, req.cuda(),
                                   sel.cuda(), lse=lse)
    check_selected(p, req, sel, out, lse)
    assert pml.pml_device_status(clear=True) == 0
    bad = table.clone()
    bad[0, 2] = 100000
    pml.pml_sparse_attention(q, k, v, bad, lens, req.cuda(), sel.cuda())
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK
    out = pml.pml_sparse_attention(q, k, v, table, lens, torch.tensor([0, 2], dtype=torch.int32).cuda(), sel.cuda())
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_REQUEST
    assert (out[1] == 0).all()
    # rows of 64 that do not start at multiples of 64
    gaps = [torch.full((k.shape[0], 64, 2, 72), math.nan, dtype=BF, device="cuda")[..., :64] for _ in range(2)]
    for dst, c in zip(gaps, (k, v)):
        dst.copy_(c)
    out = pml.pml_sparse_attention(q, gaps[0], gaps[1], table, lens, req.cuda(), sel.cuda(), lse=lse)
    check_selected(p, req, sel, out, lse)


def test_selecting_everything_is_dense_attention():
    p = Problem([1, 1], [777, 130], 8, 1, 128, BF, seed=11).stale()
    g = R.gen(5)
    sel = torch.full((2, 900), -1, dtype=torch.int32)
    sel[0, :777] = torch.randperm(777, generator=g).int()
    sel[1, 100:230] = torch.randperm(130, generator=g).int()
    q, k, v, table, lens = p.device()
    lse = torch.empty((2, 8), device="cuda")
    out = pml.pml_sparse_attention(q, k, v, table, lens, torch.arange(2, dtype=torch.int32).cuda(), sel.cuda(), lse=lse)
    check(p, out, lse)


def test_same_result_every_time_and_captured():
    p = Problem([1, 90, 1], [2500, 700, 40], 8, 2, 128, BF, seed=12).stale()
    q, k, v, table, lens = p.device()
    cu, ws = p.cu.cuda(), pml.pml_attention_workspace(128)
    out = torch.empty_like(q)
    pml.pml_paged_attention(q, k, v, table, lens, cu, out, workspace=ws)
    want = out.clone()
    for _ in range(5):
        out.zero_()
        pml.pml_paged_attention(q, k, v, table, lens, cu, out)
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pml.pml_paged_attention(q, k, v, table, lens, cu, out, workspace=ws)
    out.zero_()
    lens[0] = 1800                     # the graph reads the lengths when it runs
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[1:], want[1:]) and not torch.equal(out[0], want[0])
    p.kvn[0] = 1800
    p.table = table.cpu()
    lse = torch.empty((92, 8), device="cuda")
    check(p, pml.pml_paged_attention(q, k, v, table, lens, cu, lse=lse), lse)
    assert torch.equal(out, pml.pml_paged_attention(q, k, v, table, lens, cu))


def test_memory_of_a_call_on_another_stream():
    """The workspace and output that a call on another stream makes for itself
    are not handed to the current stream's allocations while it runs."""
    p = Problem([1] * 40, [3000] * 40, 8, 2, 128, BF, seed=21)
    q, k, v, table, lens = p.device()
    want = pml.pml_paged_attention(q, k, v, table, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        big = torch.randn((6000, 6000), device="cuda")
        for _ in range(5):
            big = big @ big * 1e-3           # the call waits behind this
    got = pml.pml_paged_attention(q, k, v, table, lens, stream=side)
    size = pml.pml_attention_workspace(128).numel()
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 5000])
def test_windows_past_every_position(window):
    p = Problem([30, 3], [20, 300], 4, 1, 64, BF, seed=22).stale()
    out, lse = p.run(window=window)
    check(p, out, lse)


def test_no_tokens():
    p = Problem([0, 0], [10, 0], 4, 2, 64, BF, seed=13)
    out, _ = p.run()
    assert out.shape == (0, 4, 64)
