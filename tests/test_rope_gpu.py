"""GPU parity of pml_rope, pml_rope_append and pml_index_quant_append with the
definitions in 64 bits: layouts, partial heads, odd sizes, strides, types, far
and negative positions, gradients (against the formula and against
differences), padding tokens and bad pages."""
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


def freqs(rot, dtype=torch.float64):
    return torch.pow(10000.0, -2.0 * torch.arange(rot // 2, dtype=torch.float64) / max(rot, 1)).to(dtype)


def check(got, want, size, dtype):
    err = (got.cpu().double() - want).abs()
    bound = R.rope_bound(want, size, dtype)
    assert (err <= bound).all(), f"off by up to {(err - bound).max():.3g} past the bound"


SHAPES = [
    # tokens, heads, dim, rot, offset
    (1, 1, 2, 2, 0), (3, 5, 128, 128, 0), (17, 3, 128, 64, 64), (9, 7, 96, 80, 16),
    (5, 2, 72, 18, 3), (4, 3, 7, 4, 1), (33, 64, 64, 32, 32), (2, 1, 512, 512, 0),
    (700, 4, 256, 64, 0), (6, 2, 40, 0, 0),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rope(shape, interleaved, dtype):
    tokens, heads, dim, rot, offset = shape
    g = R.gen(tokens * 7 + dim)
    x = torch.randn((tokens, heads, dim), generator=g).to(dtype)
    pos = torch.randint(0, 40000, (tokens,), generator=g)
    f = freqs(rot)
    want, size = R.rope(x, pos, f, offset, interleaved, 1.25)
    got = pml.pml_rope(x.cuda(), pos.cuda(), f.cuda(), rot_offset=offset, interleaved=interleaved, mscale=1.25)
    check(got, want, size, dtype)


@pytest.mark.parametrize("pos_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("freq_dtype", [torch.float32, torch.float64])
def test_far_and_negative_positions(pos_dtype, freq_dtype):
    g = R.gen(3)
    far = 2 ** 31 - 1 if pos_dtype == torch.int32 else 2 ** 34 + 12345
    pos = torch.tensor([0, 1, -1, far, -far, 2 ** 24 + 1, 123456789], dtype=pos_dtype)
    f = freqs(64, freq_dtype)
    f[1] = -f[1]                       # a turn the other way
    f[2] = 5.0                         # most of a turn per position
    x = torch.randn((len(pos), 2, 64), generator=g)
    # the reference's own product loses 2^-53 * 2^35 radians at the farthest
    # position and so does step (2^-53 of the frequency): 4e-6 each
    want, size = R.rope(x, pos, f)
    got = pml.pml_rope(x.cuda(), pos.cuda(), f.cuda()).cpu().double()
    slack = pos.double().abs()[:, None, None] * 5.0 * 2.0 ** -51
    assert ((got - want).abs() <= R.rope_bound(want, size, torch.float32) + slack * size).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(dtype, interleaved):
    g = R.gen(5)
    wide = torch.randn((11, 9, 131), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 9000, (11,), generator=g).cuda()
    f = freqs(64).cuda()
    for view in (wide[:, 2:6, :128], wide[:, 1:8:2, 3:131], wide.transpose(0, 1)[:9, :, 1:129],
                 wide[:1].expand(11, 9, 131)[:, :, :128]):
        p = pos[:view.shape[0]]
        want, size = R.rope(view.cpu(), p.cpu(), f.cpu(), 32, interleaved)
        check(pml.pml_rope(view, p, f, rot_offset=32, interleaved=interleaved), want, size, dtype)
    # in place, in a wider tensor: the rest of it stays
    buf, before = wide.clone(), wide.clone()
    view = buf[:, 2:6, :128]
    want, size = R.rope(view.cpu(), pos.cpu(), f.cpu(), 32, interleaved)
    assert pml.pml_rope(view, pos, f, out=view, rot_offset=32, interleaved=interleaved) is view
    check(view, want, size, dtype)
    buf[:, 2:6, :128] = before[:, 2:6, :128]
    assert torch.equal(buf, before)


def test_gradient_is_the_transpose_and_matches_differences():
    g = R.gen(6)
    x, dy = (torch.randn((5, 3, 48), generator=g) for _ in range(2))
    pos = torch.randint(0, 3000, (5,), generator=g)
    f = freqs(32)
    for interleaved in (False, True):
        kw = dict(rot_offset=8, interleaved=interleaved, mscale=1.5)
        dx = pml.pml_rope(dy.cuda(), pos.cuda(), f.cuda(), gradient=True, **kw).cpu().double()
        want, size = R.rope(dy, pos, f, 8, interleaved, 1.5, gradient=True)
        check(dx, want, size, torch.float32)
        # a difference in float64 of the definition along a random direction;
        # the map is linear, so the quotient is exact up to rounding
        d = torch.randn((5, 3, 48), generator=g)
        up, _ = R.rope(x.double() + 1e-3 * d.double(), pos, f, 8, interleaved, 1.5)
        dn, _ = R.rope(x.double() - 1e-3 * d.double(), pos, f, 8, interleaved, 1.5)
        slope = ((up - dn) / 2e-3 * dy.double()).sum()
        # 720 terms of size about 2, each within 2 * ROPE_REL of its own
        assert abs(slope - (dx * d.double()).sum()) <= 1e-8 + R.ROPE_REL * (size * d.double().abs()).sum()


def test_no_tokens():
    out = pml.pml_rope(torch.empty((0, 4, 64), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                       freqs(64).cuda())
    assert out.shape == (0, 4, 64)


# ------------------------------------------------------------------ into the pages

def places(g, lens, counts):
    req = torch.tensor([b for b, n in enumerate(counts) for _ in range(n)], dtype=torch.int32)
    pos = torch.tensor([lens[b] - n + i for b, n in enumerate(counts) for i in range(n)], dtype=torch.int32)
    return req, pos


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hkv,dim,rot,offset,interleaved", [
    (8, 2, 128, 128, 0, False), (6, 3, 64, 32, 32, True), (0, 1, 128, 64, 0, False),
    (5, 1, 40, 12, 4, False), (3, 1, 34, 18, 3, True)])
def test_append(dtype, hq, hkv, dim, rot, offset, interleaved):
    g = R.gen(hq + dim)
    lens, counts = [1, 64, 65, 200, 130], [1, 1, 2, 77, 130]
    req, pos = places(g, lens, counts)
    n = len(req)
    table, pages = R.block_table(lens, g)
    qkv = torch.randn((n, hq + 2 * hkv, dim), generator=g).to(dtype)
    # pages of 64 tokens, heads before tokens in the value cache
    kc = torch.randn((pages, 64, hkv, dim), generator=g).to(dtype)
    vc = torch.randn((pages, hkv, 64, dim), generator=g).to(dtype)
    f = freqs(rot)
    req[3] = -1                      # padding
    pos[7] = -5
    d = qkv.cuda()
    kd, vd = kc.cuda(), vc.cuda().transpose(1, 2)
    q_out = torch.full((n, hq, dim), 7.0, dtype=dtype, device="cuda")
    pml.pml_rope_append(d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:], pos.cuda(), req.cuda(), f.cuda(),
                        kd, vd, table.cuda(), q_out, rot_offset=offset, interleaved=interleaved)
    assert pml.pml_device_status(clear=True) == 0
    real = (req >= 0) & (pos >= 0)
    qw, qs = R.rope(qkv[:, :hq], pos, f, offset, interleaved)
    kw, ks = R.rope(qkv[:, hq:hq + hkv], pos, f, offset, interleaved)
    check(q_out[real.cuda()], qw[real], qs[real], dtype)
    assert (q_out.cpu()[~real] == 7.0).all()
    page = table[req[real].long(), pos[real].long() // 64].long()
    slot = pos[real].long() % 64
    got_k, got_v = kd.cpu(), vd.cpu()
    check(got_k[page, slot], kw[real], ks[real], dtype)
    assert torch.equal(got_v[page, slot], qkv[real][:, hq + hkv:])
    # nothing else changed
    want_k, want_v = kc.clone(), vc.transpose(1, 2).clone()
    want_k[page, slot] = got_k[page, slot]
    want_v[page, slot] = got_v[page, slot]
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v)


def test_append_bad_places():
    g = R.gen(1)
    table = torch.tensor([[3, 99], [-1, 1]], dtype=torch.int32).cuda()
    req = torch.tensor([0, 0, 1, 1, 2, 0], dtype=torch.int32).cuda()
    pos = torch.tensor([5, 70, 1, 64, 0, 128], dtype=torch.int32).cuda()
    x = torch.randn((6, 3, 64), generator=g).bfloat16().cuda()
    kc = torch.zeros((4, 64, 1, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q = pml.pml_rope_append(x[:, :1], x[:, 1:2], x[:, 2:], pos, req, freqs(64).cuda(), kc, vc, table)
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK | pml.STATUS_BAD_REQUEST
    want, size = R.rope(x[:, :1].cpu(), pos.cpu(), freqs(64))
    check(q, want, size, torch.bfloat16)
    assert torch.equal(vc[3, 5], x[0, 2:]) and torch.equal(vc[1, 0], x[3, 2:])
    assert (vc != 0).any(-1).any(-1).sum() == 2 and (kc != 0).any(-1).any(-1).sum() == 2


# ------------------------------------------------------------------ the indexer's rows

def split_fused(kv):
    kv = kv.cpu()
    return (kv[:, :8192].contiguous().view(torch.float8_e4m3fn).reshape(-1, 64, 128).double(),
            kv[:, 8192:].contiguous().view(torch.float32).double())


def check_codes(codes, scale, want, size):
    """Codes within half a step of want / scale, scales those of the rows."""
    amax = want.abs().amax(-1).clamp(min=1e-12)
    off = R.ROPE_REL * size.amax(-1)
    assert ((scale * 448.0 - amax).abs() <= off + 2.0 ** -22 * amax).all()
    # half a step: 2^-4 of the value, 2^-10 of the scale among the subnormals
    bound = 2.0 ** -4 * want.abs() + 2.0 ** -10 * scale[..., None]
    bound = bound + (off + 2.0 ** -21 * amax)[..., None]
    assert ((codes * scale[..., None] - want).abs() <= bound).all()


@pytest.mark.parametrize("heads", [1, 8, 64])
@pytest.mark.parametrize("rot,offset,interleaved", [(64, 0, True), (64, 64, False), (128, 0, False),
                                                    (16, 8, True), (96, 16, False), (0, 0, False)])
def test_index_quant(heads, rot, offset, interleaved):
    g = R.gen(heads + rot)
    lens, counts = [3, 70, 300], [1, 2, 150]
    req, pos = places(g, lens, counts)
    n = len(req)
    table, blocks = R.block_table(lens, g)
    q = (torch.randn((n, heads, 128), generator=g) * torch.rand((n, heads, 1), generator=g) * 9).bfloat16()
    k = torch.randn((n, 128), generator=g).bfloat16()
    q[1, 0] = 0
    k[0] = 0
    w = torch.randn((n, heads), generator=g)
    f = freqs(rot)
    kv0 = torch.randint(0, 120, (blocks, 8448), generator=g, dtype=torch.uint8)
    kv = kv0.cuda()
    req[4] = -1
    qo, wo = pml.pml_index_quant_append(q.cuda(), k.cuda(), w.cuda(), pos.cuda(), req.cuda(), f.cuda(), kv,
                                        table.cuda(), weight_scale=0.125, rot_offset=offset,
                                        interleaved=interleaved)
    assert pml.pml_device_status(clear=True) == 0
    real = req >= 0
    qw, qs = R.rope(q, pos, f, offset, interleaved)
    kw, ks = R.rope(k[:, None], pos, f, offset, interleaved)
    scale = wo.cpu().double() / (w.double() * 0.125)
    check_codes(qo.cpu().double()[real], scale[real], qw[real], qs[real])
    page, slot = table[req[real].long(), pos[real].long() // 64].long(), pos[real].long() % 64
    keys, scales = split_fused(kv)
    check_codes(keys[page, slot], scales[page, slot], kw[real, 0], ks[real, 0])
    # other slots keep their bytes
    old, old_scales = split_fused(kv0)
    keep = torch.ones((blocks, 64), dtype=torch.bool)
    keep[page, slot] = False
    assert torch.equal(keys[keep], old[keep]) and torch.equal(scales[keep], old_scales[keep])


def test_index_quant_without_keys_and_not_numbers():
    g = R.gen(2)
    q = torch.randn((3, 2, 128), generator=g).bfloat16()
    q[0, 0, 5] = math.nan
    q[1, 1, 7] = math.inf
    w = torch.ones((3, 2))
    qo, wo = pml.pml_index_quant_append(q.cuda(), None, w.cuda(), torch.arange(3, dtype=torch.int32).cuda(), None,
                                        freqs(0).cuda(), None, None)
    wo = wo.cpu()
    assert math.isnan(wo[0, 0]) and math.isinf(wo[1, 1]) and torch.isfinite(wo[[0, 1, 2, 2], [1, 0, 0, 1]]).all()


def test_index_feeds_the_logits():
    """q, weights and cache made here give the logits of the unquantised rows,
    to the codes' half steps (2^-4 each for q and k)."""
    g = R.gen(8)
    lens, heads = [90, 200], 16
    req, pos = places(g, lens, lens)
    table, blocks = R.block_table(lens, g)
    n = len(req)
    q, k = torch.randn((n, heads, 128), generator=g).bfloat16(), torch.randn((n, 128), generator=g).bfloat16()
    w = torch.rand((n, heads), generator=g)
    f = freqs(64)
    kv = torch.zeros((blocks, 8448), dtype=torch.uint8, device="cuda")
    qo, wo = pml.pml_index_quant_append(q.cuda(), k.cuda(), w.cuda(), pos.cuda(), req.cuda(), f.cuda(), kv,
                                        table.cuda())
    last = torch.tensor([89, 289])
    logits = torch.zeros((2, 256), device="cuda")
    pml.pml_fp8_paged_mqa_logits(qo[last.cuda()].contiguous(), kv, wo[last.cuda()].contiguous(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), logits, 256, 1)
    kw, _ = R.rope(k[:, None], pos, f)
    qw, _ = R.rope(q, pos, f)
    for b, (lo, hi) in enumerate(((0, 90), (90, 290))):
        dots = qw[last[b]] @ kw[lo:hi, 0].T
        mag = qw[last[b]].abs() @ kw[lo:hi, 0].abs().T
        want = (w[last[b]].double()[:, None] * dots.clamp(min=0)).sum(0)
        bound = (w[last[b]].double()[:, None] * mag).sum(0) * (2 * 2.0 ** -4 + 2.0 ** -8)
        assert ((logits[b, :lens[b]].cpu().double() - want).abs() <= bound).all()


def test_captured_and_on_another_stream():
    g = R.gen(4)
    x = torch.randn((40, 8, 128), generator=g).bfloat16().cuda()
    pos = torch.arange(40, device="cuda")
    f = freqs(128).cuda()
    out = torch.empty_like(x)
    pml.pml_rope(x, pos, f, out)
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pml.pml_rope(x, pos, f, out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    pml.pml_rope(x, pos, f, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
