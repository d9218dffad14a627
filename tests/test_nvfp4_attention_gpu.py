"""GPU parity of pml_paged_attention_nvfp4 and pml_sparse_attention_nvfp4 with
the definitions in 64 bits over the values that the caches stand for: single
tokens, drafts, chunks and mixed batches; head groups from 1 to 300; causal,
windows, neither; empty requests and rows without a key; layouts; stale slots
and NaN scales in masked places; large logits; bad pages, requests and lists.
Up to 32 rows ((token, head) pairs of a kv head) to a request on average, or 127
in all, run warp by warp, more by tiles: both ways are tested throughout."""
import math

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import nvfp4_ref as N
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
NAN_SCALE = 0x7f


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


class Problem:
    def __init__(self, qn, kvn, hq, hkv, dim, dtype, seed, spare=3, k_scale=1.0, v_scale=1.0, signed=False):
        g = R.gen(seed)
        self.qn, self.kvn, self.hq, self.hkv, self.dim, self.dtype = qn, kvn, hq, hkv, dim, dtype
        self.k_scale, self.v_scale = k_scale, v_scale
        self.table, pages = R.block_table(kvn, g, spare)
        self.q = (torch.randn((sum(qn), hq, dim), generator=g) * 1.5 / k_scale).to(dtype)
        self.parts = []
        for _ in range(2):
            codes, scales = N.quantise(torch.randn((pages, 64, hkv, dim), generator=g).to(FP), 1.0)
            if signed:                       # negative scales negate
                scales |= 128 * torch.randint(0, 2, scales.shape, generator=g, dtype=torch.uint8)
            self.parts += [codes, scales]
        self.cu = torch.tensor([0] + list(torch.tensor(qn).cumsum(0)), dtype=torch.int32)
        self.kv_lens = torch.tensor(kvn, dtype=torch.int32)

    def stale(self):
        """Slots past each request's end hold arbitrary codes under NaN scales."""
        for b, n in enumerate(self.kvn):
            if n % 64:
                page = self.table[b, n // 64].long()
                for i in range(4):
                    self.parts[i][page, n % 64:] = NAN_SCALE if i % 2 else 0x5a
        return self

    def set_scale(self, which, b, pos, head, group, byte):
        page = self.table[b, pos // 64].long()
        self.parts[1 if which == "k" else 3][page, pos % 64, head, group] = byte

    def rows(self, b, at):
        page = self.table[b].long()[at // 64]
        return [N.values(self.parts[i][page, at % 64], self.parts[i + 1][page, at % 64], s)
                for i, s in ((0, self.k_scale), (2, self.v_scale))]

    def device(self):
        return [self.q.cuda(), *(p.cuda() for p in self.parts), self.table.cuda(), self.kv_lens.cuda()]

    def run(self, cu=True, **kw):
        args = self.device()
        lse = torch.full(args[0].shape[:2], 77.0, device="cuda")
        out = pml.pml_paged_attention_nvfp4(*args, self.cu.cuda() if cu else None, lse=lse, k_scale=self.k_scale,
                                            v_scale=self.v_scale, **kw)
        return out, lse


def compare_rows(p, q, k, v, allowed, scale, got, got_lse, where):
    """A score is a sum of products that are exact in fp32, each further one a
    rounding of 2^-23 of their magnitudes' sum (the tensor core may cut off),
    after q's own rounding: fp16 at most 2^-25 of the row's largest element.  A
    weight is off by that, by the rounding of its exponent (2^-14 where that is
    below 1024, else fp32's half step of it) under either of two references, and
    by the approximate power's 2^-20: `rel` of it.  Numerator and denominator are
    off by as much; P is rounded to fp16 once, 2^-11 or, for small ones, 2^-32 of
    the largest weight; the output once.  The log-sum is off by `rel` and three
    roundings of its size."""
    half = torch.finfo(p.dtype).eps / 2
    want, want_lse, mag = R.attention(q, k, v, allowed, scale)
    qd, kd = q.double(), torch.nan_to_num(k.double(), nan=0.0)
    size = qd.abs() @ kd.abs().T
    score = size * (p.dim - 1) * 2.0 ** -23 + 2.0 ** -25 * qd.abs().amax(1, keepdim=True) * kd.abs().sum(1)
    score = (scale * score).masked_fill(~allowed, 0.0)
    logit = (scale * size).masked_fill(~allowed, 0.0)
    score, logit = (x.amax(1) if x.shape[1] else torch.zeros(len(q), dtype=torch.float64) for x in (score, logit))
    rel = 2 * score + 2 * math.log(2) * (2.0 ** -14 + 2.0 ** -23 * logit) + 2.0 ** -20
    got, got_lse = got.cpu().double(), got_lse.cpu().double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), where
    seen = torch.where(allowed.any(0)[:, None], torch.nan_to_num(v.double().abs(), nan=0.0), 0.0)
    tiny = 2.0 ** -32 * seen.sum(0) if len(seen) else 0.0
    bound = mag * (2.0 ** -11 + 2 * rel[:, None]) + tiny + half * want.abs() + torch.finfo(p.dtype).tiny
    err = (got - want).abs()
    assert (err <= bound)[fine].all(), f"{where}: off by {(err / bound)[fine].max():.3g} bounds"
    none = torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(got_lse), none), where
    ok = torch.isfinite(want_lse)
    off = (got_lse - want_lse)[ok].abs()
    assert (off <= rel[ok] + 3 * 2.0 ** -24 * want_lse[ok].abs() + 1e-6).all(), f"{where}: log-sum"


def check(p, out, lse, causal=True, window=0, scale=None, requests=None, heads=None):
    scale = p.dim ** -0.5 if scale is None else scale
    group = p.hq // p.hkv
    for b in range(len(p.qn)) if requests is None else requests:
        lo, hi = int(p.cu[b]), int(p.cu[b + 1])
        if lo == hi:
            continue
        at = torch.arange(max(p.kvn[b], 0))
        k, v = p.rows(b, at)
        here = torch.arange(p.kvn[b] - (hi - lo), p.kvn[b])[:, None]
        allowed = (at <= here) if causal else torch.ones((hi - lo, len(at)), dtype=torch.bool)
        if window:
            allowed = allowed & (at > here - window)
        for h in range(p.hq) if heads is None else heads:
            compare_rows(p, p.q[lo:hi, h], k[:, h // group], v[:, h // group], allowed, scale, out[lo:hi, h], lse[lo:hi, h],
                  f"request {b} head {h}")
    assert pml.pml_device_status(clear=True) == 0


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kvn", [[1], [31], [32], [33], [64], [100], [129], [1000], [300, 1, 2500]])
def test_single_tokens(dim, dtype, kvn):
    p = Problem([1] * len(kvn), kvn, 8, 2, dim, dtype, seed=sum(kvn), signed=True).stale()
    check(p, *p.run(cu=False))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 4), (10, 2), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (33, 1),
                                    (64, 1), (65, 1), (128, 1), (300, 1), (48, 2)])
@pytest.mark.parametrize("q", [1, 3, 11])
def test_head_groups(hq, hkv, q):
    p = Problem([q, q], [200, 77], hq, hkv, 64, BF, seed=hq).stale()
    check(p, *p.run(cu=False))


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("q,kv", [(2, 2), (16, 16), (33, 33), (64, 64), (65, 300), (257, 257), (100, 1111)])
def test_chunks(dim, q, kv):
    p = Problem([q], [kv], 4, 1, dim, BF, seed=q + kv).stale()
    check(p, *p.run())


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window", [0, 1, 31, 60, 64, 130, 700])
@pytest.mark.parametrize("causal", [True, False])
def test_mixed_batches(dtype, window, causal):
    qn, kvn = [1, 0, 130, 70, 1, 5, 0, 300], [900, 50, 130, 700, 1, 64, 0, 421]
    p = Problem(qn, kvn, 6, 2, 64, dtype, seed=window).stale()
    check(p, *p.run(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("k_scale,v_scale", [(0.25, 2.0 ** -6), (2.0 ** 5, 8.0), (2.0 ** -32, 2.0 ** 10)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hq", [6, 42])
def test_scales_of_all_values(k_scale, v_scale, dtype, hq):
    if dtype == FP and k_scale < 1e-3:
        k_scale = 2.0 ** -8                        # q grows by as much
    p = Problem([1, 5], [300, 90], hq, 2, 64, dtype, seed=3, k_scale=k_scale, v_scale=v_scale).stale()
    check(p, *p.run())


@pytest.mark.parametrize("hq", [4, 64])
def test_rows_of_very_different_sizes(hq):
    """bf16 rows of q from 2^-90 to 2^20, a row of zeros and elements far below
    their row's largest."""
    p = Problem([1, 2], [300, 170], hq, 1, 128, BF, seed=19).stale()
    size = torch.exp2(torch.linspace(-90, 3, hq).round())[:, None]
    p.q = (p.q.float() * size).to(BF)
    p.q[0, 1] = 0
    p.q[1, :, ::3] *= 2.0 ** -12
    p.q[2, -1] *= 2.0 ** 17
    check(p, *p.run())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [3, 6, 20])
@pytest.mark.parametrize("window", [0, 1, 31, 33, 64, 130])
@pytest.mark.parametrize("causal", [True, False])
def test_mixed_batches_of_few_tokens(dim, hq, window, causal):
    qn, kvn = [1, 0, 6, 3, 1, 5, 0, 4, 2], [900, 50, 6, 700, 1, 64, 0, 421, 97]
    p = Problem(qn, kvn, hq, 1, dim, FP if hq == 3 else BF, seed=window).stale()
    check(p, *p.run(causal=causal, window=window), causal=causal, window=window)


def test_a_long_chunk_among_single_tokens():
    """More tiles of tokens to a request than a lane counts by itself, few on average."""
    qn = [1] * 60 + [200] + [1] * 20
    kvn = [30 + 7 * i for i in range(60)] + [450] + [90] * 20
    p = Problem(qn, kvn, 6, 2, 64, BF, seed=17).stale()
    check(p, *p.run(), requests=list(range(0, 60, 9)) + [60, 61, 80])


def test_rows_without_a_key_of_many():
    qn, kvn = [4, 100, 3, 1, 40, 2], [0, 30, 1, 0, 39, -5]
    p = Problem(qn, kvn, 8, 2, 128, BF, seed=1).stale()
    out, lse = p.run()
    check(p, out, lse, requests=range(5))
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all() and (out[4:74] == 0).all()
    assert (out[148:] == 0).all() and torch.isneginf(lse[148:]).all()


def test_rows_without_a_key():
    qn, kvn = [4, 5, 3, 1, 6, 2], [0, 2, 1, 0, 4, -5]
    p = Problem(qn, kvn, 8, 2, 128, BF, seed=1).stale()
    out, lse = p.run()
    check(p, out, lse, requests=range(5))
    assert (out[:4] == 0).all() and torch.isneginf(lse[:4]).all() and (out[4:7] == 0).all()
    assert (out[19:] == 0).all() and torch.isneginf(lse[19:]).all()


@pytest.mark.parametrize("hq", [4, 24])
def test_rows_of_no_request_stay(hq):
    p = Problem([2, 3], [40, 100], hq, 1, 64, BF, seed=2)
    p.q = torch.cat([p.q, p.q])
    args = p.device()
    out, lse = torch.full_like(args[0], 9.0), torch.full((10, hq), 9.0, device="cuda")
    pml.pml_paged_attention_nvfp4(*args, p.cu.cuda(), out, lse=lse)
    check(p, out[:5], lse[:5])
    assert (out[5:] == 9.0).all() and (lse[5:] == 9.0).all()


@pytest.mark.parametrize("hq,hkv", [(4, 2), (40, 2)])
def test_many_short_requests_and_one_long(hq, hkv):
    g = R.gen(0)
    kvn = torch.randint(1, 200, (400,), generator=g).tolist() + [3000]
    p = Problem([1] * 401, kvn, hq, hkv, 64, BF, seed=2).stale()
    check(p, *p.run(), requests=list(range(0, 400, 23)) + [400], heads=range(0, hq, 3))


@pytest.mark.parametrize("dim", [64, 128])
def test_more_requests_than_warps(dim):
    """Items of no tiles, one and a few, several to a warp."""
    g = R.gen(1)
    kvn = torch.randint(0, 80, (5000,), generator=g).tolist()
    qn = torch.randint(0, 3, (5000,), generator=g).tolist()
    p = Problem(qn, kvn, 2, 1, dim, FP, seed=4).stale()
    check(p, *p.run(), requests=range(0, 5000, 41))


def test_one_long_request():
    p = Problem([2], [70000], 3, 1, 128, BF, seed=5).stale()
    check(p, *p.run())


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv,q", [(1, 1, 1), (4, 1, 1), (8, 8, 1), (19, 19, 1), (32, 8, 1), (7, 1, 4), (16, 2, 3),
                                      (12, 4, 5), (76, 76, 1), (9, 1, 1)])
@pytest.mark.parametrize("kv,window", [(5, 0), (6, 2), (33, 0), (257, 0), (4000, 0), (5000, 900), (0, 0)])
def test_one_request(dim, hq, hkv, q, kv, window):
    """Few items, each with CTAs of its own; more units than warps, fewer, none."""
    p = Problem([q], [kv], hq, hkv, dim, BF if kv % 2 else FP, seed=kv + hq).stale()
    out, lse = p.run(window=window)
    check(p, out, lse, window=window, heads=range(0, hq, 1 + hq // 10))
    for cu in (True, False):
        again, lse2 = p.run(cu=cu, window=window)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hq", [4, 24])
def test_one_request_of_fewer_tokens_than_rows(hq):
    p = Problem([3], [700], hq, 1, 128, BF, seed=4).stale()
    p.q = torch.cat([p.q, p.q, p.q])
    args = p.device()
    out, lse = torch.full_like(args[0], 9.0), torch.full((9, hq), 9.0, device="cuda")
    pml.pml_paged_attention_nvfp4(*args, p.cu.cuda(), out, lse=lse)
    check(p, out[:3], lse[:3])
    assert (out[3:] == 9.0).all() and (lse[3:] == 9.0).all()
    pml.pml_paged_attention_nvfp4(*args, torch.tensor([4, 7], dtype=torch.int32, device="cuda"), out, lse=lse)
    p.q = p.q[4:7]
    check(p, out[4:7], lse[4:7])


@pytest.mark.parametrize("layout", ["pages", "gaps"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("qn", [[5, 60], [4, 3]])
def test_layouts_strides_and_given_outputs(layout, dim, qn):
    n = sum(qn)
    p = Problem(qn, [70, 200], 6, 3, dim, FP, seed=4).stale()
    q, kc, ks, vc, vs, table, lens = p.device()
    if layout == "pages":
        _, *parts = pml.pml_nvfp4_pages(kc.shape[0], 3, dim)
    else:
        parts = [torch.full((kc.shape[0], 2, 3, 64, w), 0x7f, dtype=torch.uint8, device="cuda")[:, 1, :, :, :n]
                 .transpose(1, 2) for n, w in ((dim // 2, 96), (dim // 16, 16)) * 2]
    for dst, src in zip(parts, (kc, ks, vc, vs)):
        dst.copy_(src)
    parts[1], parts[3] = parts[1].view(torch.float8_e4m3fn), parts[3]
    wide = torch.zeros((n, 10, 136), dtype=FP, device="cuda")
    wide[:, 2:8, :dim] = q
    tw = torch.full((2, table.shape[1] + 3), -7, dtype=torch.int32, device="cuda")
    tw[:, :table.shape[1]] = table
    out = torch.full((n, 6, 160), 9.0, dtype=FP, device="cuda")[:, :, :dim]
    lse = torch.empty((n, 6), device="cuda")
    ws = pml.pml_attention_workspace(dim)
    ws.fill_(255)
    got = pml.pml_paged_attention_nvfp4(wide[:, 2:8, :dim], *parts, tw[:, :table.shape[1]], lens, p.cu.cuda(), out,
                                        lse=lse, workspace=ws, softmax_scale=0.3)
    assert got is out
    check(p, out, lse, scale=0.3)
    assert (out.as_strided((n, 6, 160 - dim), out.stride(), dim) == 9.0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [2, 16])
def test_masked_places_never_reach_a_row(dim, hq):
    """Late tokens of a chunk hold values under NaN scales: earlier rows must not
    see them, later ones must; and a window's far side."""
    p = Problem([300, 9, 1], [300, 200, 100], hq, 1, dim, BF, seed=6).stale()
    last = dim // 16 - 1
    for b, pos, group in ((0, 290, 1), (0, 170, 0), (1, 196, last), (1, 199, 1)):
        p.set_scale("v", b, pos, 0, group, NAN_SCALE)
    out, lse = p.run()
    check(p, out, lse)
    late = out.cpu()
    assert torch.isnan(late[290:300, :, 16:32]).all() and torch.isfinite(late[:290, :, 16:32]).all()
    assert torch.isnan(late[170:300, :, :16]).all() and torch.isfinite(late[:170]).all()
    out, lse = p.run(window=64)
    check(p, out, lse, window=64)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [3, 8])
def test_masked_places_of_few_tokens(dim, hq):
    p = Problem([6, 4, 1], [70, 200, 100], hq, 1, dim, BF, seed=18).stale()
    last = dim // 16 - 1
    for b, pos, group in ((0, 67, 1), (0, 64, 0), (1, 198, last), (1, 150, 2)):
        p.set_scale("v", b, pos, 0, group, NAN_SCALE)
    out, lse = p.run()
    check(p, out, lse)
    got = out.cpu()
    assert torch.isnan(got[3:6, :, 16:32]).all() and torch.isfinite(got[:3, :, 16:32]).all()
    assert torch.isfinite(got[6:8, :, 16 * last:]).all() or last == 2
    out, lse = p.run(window=40)
    check(p, out, lse, window=40)


@pytest.mark.parametrize("hq", [2, 6])
def test_masked_keys_of_nan(hq):
    p = Problem([40], [200], hq, 1, 64, BF, seed=7).stale()
    p.set_scale("k", 0, 199, 0, 2, NAN_SCALE | 128)       # the last token's key
    out, lse = p.run()
    got = out.cpu()
    assert torch.isfinite(got[:39]).all() and torch.isnan(got[39]).all()
    k, v = p.rows(0, torch.arange(199))
    compare_rows(p, p.q[:39, 0], k[:, 0], v[:, 0], torch.arange(199) <= torch.arange(160, 199)[:, None], 0.125, out[:39, 0],
          lse[:39, 0], "rows before")


@pytest.mark.parametrize("factor", [10.0, 300.0, 3e4])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("qn", [[3, 40, 1], [3, 9, 1]])
def test_large_logits(factor, dtype, qn):
    """Scores in the hundreds and thousands that grow along the cache, so that
    the running maximum moves in most tiles."""
    if dtype == FP and factor > 1e4:
        factor = 1e4
    p = Problem(qn, [150, 333, 20000], 4, 1, 64, dtype, seed=8).stale()
    p.q = (torch.randn(p.q.shape, generator=R.gen(9)) * factor).to(dtype)
    # one group of the keys grows with the position
    for b, n in enumerate(p.kvn):
        at = torch.arange(n)
        page = p.table[b].long()[at // 64]
        p.parts[1][page, at % 64, 0, 1] = (0x20 + 0x30 * at // n).to(torch.uint8)
    check(p, *p.run())


@pytest.mark.parametrize("size", [1e4, 1e20, -1e20, 1e34, -1e34])
@pytest.mark.parametrize("hq", [2, 64])
def test_equal_logits_far_from_zero(size, hq):
    """Every key's score is the same number, however large: the output is the mean of
    the values, to P's and the output's roundings."""
    p = Problem([1, 1], [300, 4000], hq, 1, 64, BF, seed=11).stale()
    p.q.fill_(size)
    for b, n in enumerate(p.kvn):
        at = torch.arange(n)
        page = p.table[b].long()[at // 64]
        p.parts[0][page, at % 64] = 0x22                # 1 s
        p.parts[1][page, at % 64] = 0x38                # s = 1
    out, lse = p.run()
    for b, n in enumerate(p.kvn):
        _, v = p.rows(b, torch.arange(n))
        want, mag = v[:, 0].mean(0), v[:, 0].abs().mean(0)
        assert ((out[b].cpu().double() - want).abs() <= 2.0 ** -10 * mag + 2.0 ** -8 * want.abs()).all()
        logit = 64 * 0.125 * float(p.q[0, 0, 0])
        assert (lse[b].cpu().double() - logit - math.log(n)).abs().max() <= 2.0 ** -22 * abs(logit) + 1e-5
    assert pml.pml_device_status(clear=True) == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (24, 1)])
@pytest.mark.parametrize("tokens,k", [(1, 4000), (2, 4000), (9, 1500), (20, 700), (37, 900)])
def test_long_lists_of_few_tokens(dim, hq, hkv, tokens, k):
    """Lists long enough to be split between CTAs."""
    g = R.gen(hq)
    p = Problem([1] * tokens, [5000, 3000, 1, 0] * 9 + [200], hq, hkv, dim, FP, seed=12).stale()
    sel = torch.randint(-100, 5000, (tokens, k), generator=g, dtype=torch.int32)
    req = torch.arange(tokens, dtype=torch.int32)
    lse = torch.empty((tokens, hq), device="cuda")
    out = pml.pml_sparse_attention_nvfp4(*p.device(), req.cuda(), sel.cuda(), lse=lse)
    assert pml.pml_device_status(clear=True) == 0
    check_selected(p, req, sel, out, lse, heads=range(0, hq, 3))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hq", [2, 64, 128])
def test_small_weights_beside_a_large_one(dtype, hq):
    """30000 keys whose weights are e^-8 of the best one's."""
    p = Problem([1], [30000], hq, 1, 64, dtype, seed=10).stale()
    p.q.zero_()
    p.q[..., 0] = 8.0
    p.parts[0][:] = 0
    p.parts[0][..., 0] = 0x0a                            # -1 s in element 0
    p.parts[1][:] = 0x38 + 24                            # s = 8: scores -8 of 0.125 * 8 * 8
    best = p.table[0, 200].long()
    p.parts[0][best, 5, :, 0] = 0
    check(p, *p.run(), heads=range(0, hq, 1 if hq == 2 else 21))


@pytest.mark.parametrize("hq", [4, 64])
def test_pages_out_of_range_are_flagged(hq):
    p = Problem([1, 2], [200, 100], hq, 1, 64, BF, seed=8)
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


@pytest.mark.parametrize("hq", [4, 64])
def test_lengths_past_the_table(hq):
    p = Problem([1, 3], [128, 100], hq, 1, 64, BF, seed=9)
    args = p.device()
    args[-1] = torch.tensor([5000, 100], dtype=torch.int32, device="cuda")
    lse = torch.empty((4, hq), device="cuda")
    out = pml.pml_paged_attention_nvfp4(*args, p.cu.cuda(), lse=lse, causal=False)
    check(p, out, lse, causal=False)


@pytest.mark.parametrize("hq", [16, 64])
def test_cache_past_32_bits(hq):
    pages, used = 70000, [0, 3, 69998, 69999, 40000]
    p = Problem([7], [300], hq, 8, 128, BF, seed=9, spare=0)
    q, *small, _, lens = p.device()
    _, *parts = pml.pml_nvfp4_pages(pages, 8, 128)
    for i, u in enumerate(used):
        for dst, src in zip(parts, small):
            dst[u] = src[p.table[0, i].long()]
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    lse = torch.empty((7, hq), device="cuda")
    out = pml.pml_paged_attention_nvfp4(q, *parts, table, lens, p.cu.cuda(), lse=lse)
    check(p, out, lse, heads=(0, 9))
    sel = torch.arange(299, -1, -1, dtype=torch.int32).repeat(7, 1).cuda()
    out = pml.pml_sparse_attention_nvfp4(q, *parts, table, lens, torch.zeros(7, dtype=torch.int32, device="cuda"), sel,
                                         lse=lse)
    check(p, out, lse, heads=(0, 9), causal=False)


# ------------------------------------------------------------------ selected positions

def check_selected(p, req, sel, out, lse, scale=None, heads=None):
    scale = p.dim ** -0.5 if scale is None else scale
    group = p.hq // p.hkv
    for t in range(len(req)):
        b = int(req[t])
        n = p.kvn[b] if 0 <= b < len(p.kvn) else 0
        at = sel[t][(sel[t] >= 0) & (sel[t] < n)].long()
        k, v = p.rows(max(0, min(b, len(p.kvn) - 1)), at)
        for h in range(p.hq) if heads is None else heads:
            compare_rows(p, p.q[t:t + 1, h], k[:, h // group], v[:, h // group], torch.ones((1, len(at)), dtype=torch.bool),
                  scale, out[t:t + 1, h], lse[t:t + 1, h], f"token {t} head {h}")


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("k", [1, 5, 31, 32, 33, 129, 700])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (64, 1)])
def test_selected(dim, dtype, k, hq, hkv):
    g = R.gen(k + hq)
    kvn = [1000, 65, 1, 0, 300]
    p = Problem([1] * 5, kvn, hq, hkv, dim, dtype, seed=k, k_scale=0.5, v_scale=2.0).stale()
    req = torch.tensor([0, 1, 4, 2, 0, 3, 1, -1], dtype=torch.int32)
    p.q = (torch.randn((8, hq, dim), generator=g) * 3.0).to(dtype)
    # holes, repeats and positions that are not there
    sel = torch.randint(-200, 1200, (8, k + 3), generator=g, dtype=torch.int32)
    sel[2, ::2] = -1
    sel[6] = -1
    q, *rest = p.device()
    lse = torch.empty((8, hq), device="cuda")
    out = pml.pml_sparse_attention_nvfp4(q, *rest, req.cuda(), sel.cuda()[:, :k], lse=lse, k_scale=0.5, v_scale=2.0)
    assert pml.pml_device_status(clear=True) == 0
    check_selected(p, req, sel[:, :k], out, lse, heads=range(0, hq, 1 if hq < 10 else 7))


def test_lists_of_a_prompt():
    g = R.gen(4)
    p = Problem([1, 1], [900, 260], 64, 1, 64, BF, seed=33).stale()
    tokens, k = 900, 300
    p.q = (torch.randn((tokens, 64, 64), generator=g) * 1.5).to(BF)
    req = torch.randint(0, 2, (tokens,), generator=g, dtype=torch.int32)
    sel = torch.randint(-50, 900, (tokens, k), generator=g, dtype=torch.int32)
    args = p.device()
    lse = torch.empty((tokens, 64), device="cuda")
    out = pml.pml_sparse_attention_nvfp4(*args, req.cuda(), sel.cuda(), lse=lse)
    assert pml.pml_device_status(clear=True) == 0
    at = list(range(0, tokens, 37))
    p.q = p.q[at]
    check_selected(p, req[at], sel[at], out[at], lse[at], heads=(0, 15, 16, 63))
    for _ in range(5):
        assert torch.equal(pml.pml_sparse_attention_nvfp4(*args, req.cuda(), sel.cuda()), out)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("k", [129, 700])
def test_selected_by_many_tokens(dim, dtype, k):
    """Enough tokens of 64 heads that their lists go by tiles."""
    g = R.gen(k + 1)
    kvn, tokens = [1000, 65, 1, 0, 300], 1200
    p = Problem([1] * 5, kvn, 64, 1, dim, dtype, seed=k, k_scale=0.5, v_scale=2.0).stale()
    req = torch.tensor([0, 1, 4, 2, 0, 3, 1, -1], dtype=torch.int32).repeat(tokens // 8)
    p.q = (torch.randn((tokens, 64, dim), generator=g) * 3.0).to(dtype)
    sel = torch.randint(-200, 1200, (tokens, k + 3), generator=g, dtype=torch.int32)
    sel[2::8, ::2] = -1
    sel[6::8] = -1
    q, *rest = p.device()
    lse = torch.empty((tokens, 64), device="cuda")
    out = pml.pml_sparse_attention_nvfp4(q, *rest, req.cuda(), sel.cuda()[:, :k], lse=lse, k_scale=0.5, v_scale=2.0)
    assert pml.pml_device_status(clear=True) == 0
    at = [*range(8), *range(403, 1200, 97), 1199]
    p.q = p.q[at]
    check_selected(p, req[at], sel[at][:, :k], out[at], lse[at], heads=(0, 21, 63))


@pytest.mark.parametrize("tokens", [1, 900])
def test_selected_past_32_bits(tokens):
    """More rows to a kv head than warps take alone, over rows far into the cache."""
    p = Problem([1], [300], 64, 1, 128, BF, seed=9, spare=0)
    q, *small, _, lens = p.device()
    pages, used = 600000, [0, 3, 599998, 599999, 40000]
    _, *parts = pml.pml_nvfp4_pages(pages, 1, 128)
    for i, u in enumerate(used):
        for dst, src in zip(parts, small):
            dst[u] = src[p.table[0, i].long()]
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    sel = torch.arange(299, -1, -1, dtype=torch.int32).repeat(tokens, 1)
    lse = torch.empty((tokens, 64), device="cuda")
    out = pml.pml_sparse_attention_nvfp4(q.repeat(tokens, 1, 1), *parts, table, lens,
                                         torch.zeros(tokens, dtype=torch.int32, device="cuda"), sel.cuda(), lse=lse)
    for t in {0, tokens // 2, tokens - 1}:
        check_selected(p, torch.tensor([0]), sel[:1], out[t:t + 1], lse[t:t + 1], heads=(0, 63))


@pytest.mark.parametrize("hq,copies", [(6, 1), (100, 1), (100, 400)])
def test_selected_bad_places_and_nan(hq, copies):
    g = R.gen(3)
    p = Problem([1, 1], [500, 400], hq, 2, 64, BF, seed=3).stale()
    sel = torch.stack([torch.randperm(500, generator=g)[:200], torch.randperm(400, generator=g)[:200]]).int()
    req = torch.tensor([0, 1], dtype=torch.int32)
    heads = range(0, hq, max(1, hq // 9))

    def run(table=None, req=req):
        q, *parts, good, lens = p.device()
        many = lambda t: t.cuda().repeat(copies, *[1] * (t.dim() - 1))  # noqa: E731
        lse = torch.empty((2 * copies, hq), device="cuda")
        out = pml.pml_sparse_attention_nvfp4(many(q), *parts, good if table is None else table, lens, many(req), many(sel),
                                             lse=lse)
        return out, lse

    def check_all(out, lse):
        for i in {0, 2 * (copies // 2), 2 * copies - 2}:
            check_selected(p, req, sel, out[i:i + 2], lse[i:i + 2], heads=heads)

    bad = p.table.clone()
    bad[0, 2] = 100000
    run(table=bad.cuda())
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK
    out, _ = run(req=torch.tensor([0, 2], dtype=torch.int32))
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_REQUEST
    assert (out[1::2] == 0).all()
    # a listed NaN reaches the row, one that is not listed does not
    pos = int(sel[0, 17])
    p.set_scale("v", 0, pos, 0, 1, NAN_SCALE)
    out, lse = run()
    check_all(out, lse)
    assert torch.isnan(out[::2, :hq // 2, 16:32]).all()
    sel[0, 17] = -1
    out, lse = run()
    check_all(out, lse)
    assert torch.isfinite(out).all()


# ------------------------------------------------------------------ as they are used

@pytest.mark.parametrize("chunk", [90, 3])
def test_same_result_every_time_and_captured(chunk):
    p = Problem([1, chunk, 1], [2500, 700, 40], 8, 2, 128, BF, seed=12).stale()
    args = p.device()
    cu, ws = p.cu.cuda(), pml.pml_attention_workspace(128)
    out = torch.empty_like(args[0])
    pml.pml_paged_attention_nvfp4(*args, cu, out, workspace=ws)
    want = out.clone()
    for _ in range(5):
        out.zero_()
        pml.pml_paged_attention_nvfp4(*args, cu, out)
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pml.pml_paged_attention_nvfp4(*args, cu, out, workspace=ws)
    out.zero_()
    args[-1][0] = 1800                     # the graph reads the lengths when it runs
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out[0], want[0])
    p.kvn[0] = 1800                        # (how the keys are shared out depends on all lengths)
    lse = torch.empty((chunk + 2, 8), device="cuda")
    check(p, pml.pml_paged_attention_nvfp4(*args, cu, lse=lse), lse)
    assert torch.equal(out, pml.pml_paged_attention_nvfp4(*args, cu))


def test_one_request_captured():
    p = Problem([2], [3000], 16, 4, 128, BF, seed=25).stale()
    args, cu = p.device(), p.cu.cuda()
    out, ws = torch.empty_like(args[0]), pml.pml_attention_workspace(128)
    pml.pml_paged_attention_nvfp4(*args, cu, out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            pml.pml_paged_attention_nvfp4(*args, cu, out, workspace=ws)
    for n in (2999, 1, 40, 3000):
        args[-1].fill_(n)
        out.fill_(9.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        lse = torch.empty((2, 16), device="cuda")
        assert torch.equal(out, pml.pml_paged_attention_nvfp4(*args, cu, lse=lse))
        p.kvn = [n]
        check(p, out, lse)


def test_memory_of_a_call_on_another_stream():
    p = Problem([1] * 40, [3000] * 40, 8, 2, 128, BF, seed=21)
    args = p.device()
    want = pml.pml_paged_attention_nvfp4(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        big = torch.randn((6000, 6000), device="cuda")
        for _ in range(5):
            big = big @ big * 1e-3           # the call waits behind this
    got = pml.pml_paged_attention_nvfp4(*args, stream=side)
    size = pml.pml_attention_workspace(128).numel()
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(junk) == 4


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 5000])
@pytest.mark.parametrize("qn", [[30, 3], [7, 3]])
def test_windows_past_every_position(window, qn):
    p = Problem(qn, [20, 300], 4, 1, 64, BF, seed=22).stale()
    out, lse = p.run(window=window)
    check(p, out, lse)


def test_no_tokens():
    p = Problem([0, 0], [10, 0], 4, 2, 64, BF, seed=13)
    out, _ = p.run()
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [4, 32, 64])
def test_positions_up_to_the_last(dim, hq):
    """A table as wide as positions go, one page behind all its entries, and a
    window that leaves the end of it."""
    width = (2 ** 31 - 1) // 64
    p = Problem([2], [200], hq, 1, dim, BF, seed=20, spare=0)
    q, *parts, table, _ = p.device()
    wide = table[:, :1].expand(1, width).contiguous()
    lens = torch.tensor([64 * width], dtype=torch.int32, device="cuda")
    lse = torch.empty((2, hq), device="cuda")
    out = pml.pml_paged_attention_nvfp4(q, *parts, wide, lens, lse=lse, window=150)
    assert pml.pml_device_status(clear=True) == 0
    page = p.table[0, 0].long()
    for i in range(2):
        at = torch.arange(64 * width - 2 + i - 149, 64 * width - 1 + i) % 64
        k, v = (N.values(p.parts[c][page, at], p.parts[c + 1][page, at], 1.0) for c in (0, 2))
        for h in range(hq):
            compare_rows(p, p.q[i:i + 1, h], k[:, 0], v[:, 0], torch.ones((1, 150), dtype=torch.bool), dim ** -0.5,
                  out[i:i + 1, h], lse[i:i + 1, h], f"token {i}")


def test_two_captured_graphs_share_a_workspace():
    """Replayed one after the other, whatever the other has left there."""
    few, many = Problem([1] * 9, [700] * 9, 8, 1, 128, BF, seed=23), Problem([30], [900], 8, 1, 128, BF, seed=24)
    ws = pml.pml_attention_workspace(128)
    graphs, outs, want = [], [], []
    for p in (few, many):
        args, cu = p.device(), p.cu.cuda()
        want.append(pml.pml_paged_attention_nvfp4(*args, cu))
        out = torch.zeros_like(args[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pml.pml_paged_attention_nvfp4(*args, cu, out, workspace=ws)
        graphs.append((graph, args, cu))
        outs.append(out)
    for order in ((0, 1), (1, 0, 1, 0)):
        for i in order:
            graphs[i][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_step(dtype):
    """A prompt rotated, written and attended to through the pages read back, then
    a token of each request rotated, written and attended to directly, densely and
    over a list: as 64-bit attention over the values that the caches stand for."""
    g = R.gen(14)
    hq, hkv, dim = 8, 2, 128
    prompt, lens = [150, 70], [151, 71]
    p = Problem([1, 1], lens, hq, hkv, dim, dtype, seed=15, k_scale=2.0, v_scale=0.5)
    inv_freq = torch.pow(10000.0, -torch.arange(dim // 2, dtype=torch.float64) * 2 / dim).cuda()
    _, *parts = pml.pml_nvfp4_pages(int(p.table.max()) + 4, hkv, dim)
    table = p.table.cuda()
    scales = dict(k_scale=2.0, v_scale=0.5)

    def write(counts, ends):
        n = sum(counts)
        x = torch.randn((n, hq + 2 * hkv, dim), generator=g).to(dtype).cuda()
        req = torch.tensor([b for b, c in enumerate(counts) for _ in range(c)], dtype=torch.int32).cuda()
        pos = torch.tensor([e - c + i for c, e in zip(counts, ends) for i in range(c)], dtype=torch.int32).cuda()
        qk = x[:, :hq + hkv]
        pml.pml_rope(qk, pos, inv_freq, qk)
        pml.pml_append_nvfp4(qk[:, hq:], x[:, hq + hkv:], pos, req, *parts, table, **scales)
        return x[:, :hq]

    q = write(prompt, prompt)
    width = table.shape[1]
    out_table = torch.arange(2 * width, dtype=torch.int32, device="cuda").view(2, width)
    k16, v16 = (torch.zeros((2 * width, 64, hkv, dim), dtype=dtype, device="cuda") for _ in range(2))
    cu = torch.tensor([0, 150, 220], dtype=torch.int32, device="cuda")
    now = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    pml.pml_read_nvfp4(*parts, table, now, k16, v16, out_table, **scales)
    through = pml.pml_paged_attention(q, k16, v16, out_table, now, cu)
    lse = torch.empty((220, hq), device="cuda")
    direct = pml.pml_paged_attention_nvfp4(q, *parts, table, now, cu, lse=lse, **scales)
    p.parts, p.qn, p.kvn, p.q, p.cu = [t.cpu() for t in parts], prompt, prompt, q.cpu(), cu.cpu()
    check(p, direct, lse)
    # both within their bounds of the same values: P in the type's half steps, and the output's
    half = torch.finfo(dtype).eps / 2
    assert ((direct - through).abs() <= 2 * (2 * half + 4e-4) * v16.abs().max()).all()
    q = write([1, 1], lens)
    now = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty((2, hq), device="cuda")
    out = pml.pml_paged_attention_nvfp4(q, *parts, table, now, lse=lse, **scales)
    p.parts, p.qn, p.kvn, p.q = [t.cpu() for t in parts], [1, 1], lens, q.cpu()
    p.cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    check(p, out, lse)
    sel = torch.stack([torch.randperm(151, generator=g)[:60], torch.randperm(151, generator=g)[:60]]).int()
    req = torch.arange(2, dtype=torch.int32)
    out = pml.pml_sparse_attention_nvfp4(q, *parts, table, now, req.cuda(), sel.cuda(), lse=lse, **scales)
    check_selected(p, req, sel, out, lse)


def test_refusals():
    p = Problem([1, 1], [100, 50], 4, 2, 64, BF, seed=16)
    q, kc, ks, vc, vs, table, lens = p.device()
    req, sel = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 8), dtype=torch.int32, device="cuda")

    def both(code=None, **over):
        a = dict(q=q, kc=kc, ks=ks, vc=vc, vs=vs, table=table, lens=lens, kw={})
        a.update(over)
        parts = [a[n] for n in ("q", "kc", "ks", "vc", "vs", "table", "lens")]
        for call in (lambda: pml.pml_paged_attention_nvfp4(*parts, **a["kw"]),
                     lambda: pml.pml_sparse_attention_nvfp4(*parts, req, sel, **a["kw"])):
            with pytest.raises(ValueError if code is None else pml.PmlError) as e:
                call()
            if code is not None:
                assert e.value.code == code

    both(q=q.float())
    both(q=q[..., :32])
    both(kc=kc[..., :16])
    both(ks=ks[:, :, :1])
    both(ks=ks.float())
    both(vc=vc[:1])
    both(lens=lens.long())
    both(table=table[:1])
    both(kw=dict(lse=torch.empty(3, device="cuda")))
    both(kw=dict(out=torch.empty_like(q).half()))
    both(1, kw=dict(k_scale=3.0))
    both(1, kw=dict(softmax_scale=0.0))
    both(1, kw=dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")))
    both(1, q=torch.cat([q, q[:, :1]], 1))                  # five heads over two
    both(3, kc=torch.zeros((kc.shape[0], 64, 2, 40), dtype=torch.uint8, device="cuda")[..., :32])
    with pytest.raises(ValueError):
        pml.pml_paged_attention_nvfp4(torch.cat([q, q[:1]]), kc, ks, vc, vs, table, lens)
    with pytest.raises(ValueError):
        pml.pml_sparse_attention_nvfp4(q, kc, ks, vc, vs, table, lens, req, sel[:1])
    with pytest.raises(pml.PmlError):
        pml.pml_paged_attention_nvfp4(q, kc, ks, vc, vs, table, lens, window=-1)
