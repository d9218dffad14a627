"""Argument checks of the C entries over caches held in 4 bits.  No GPU: only
calls that return before touching CUDA."""
import ctypes

import pytest
import torch

from tests.test_serving_abi_cpu import ALIGNMENT, BF16, F32, INVALID, OK, P, UNSUPPORTED, L, caller  # noqa: F401


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("codes", "scales")] + \
        [(n, ctypes.c_int64) for n in ("page", "slot", "head", "s_page", "s_slot", "s_head")] + [("scale", ctypes.c_float)]


def cache(**over):
    c = Cache(P, P, 8192, 128, 64, 1024, 16, 8, 1.0)
    for n, v in over.items():
        setattr(c, n, v)
    return ctypes.addressof(c), c


GOOD = cache()
KV = dict(kc=GOOD[0], vc=GOOD[0], pages=4)
TABLE = dict(bt=P, bts=4, btw=4)


def cache_refusals(call, others=()):
    for name in ("kc", "vc"):
        assert call(**{name: None}) == INVALID
        for over in (dict(codes=None), dict(scales=None), dict(scale=0.0), dict(scale=-2.0), dict(scale=3.0),
                     dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=2.0 ** 33), dict(scale=2.0 ** -33)):
            at, keep = cache(**over)
            assert call(**{name: at}) == INVALID, over
        for over in (dict(codes=P + 8), dict(scales=P + 4), dict(page=8200), dict(slot=72), dict(head=8), dict(slot=0),
                     dict(page=-8192), dict(s_page=1028), dict(s_slot=12), dict(s_head=4), dict(s_slot=0)):
            at, keep = cache(**over)
            assert call(**{name: at}) == ALIGNMENT, over


def test_append(L):  # noqa: F811
    call = caller(L, "pml_append_nvfp4", dict(k=P, kt=256, kh=128, v=P, vt=256, vh=128, dtype=BF16, positions=P, p64=0,
                                              req=P, nreq=2, **KV, **TABLE, tokens=3, kv=2, dim=128, stream=None))
    assert call(tokens=0) == OK and call(tokens=-1) == INVALID and call(kv=0) == INVALID
    assert call(dtype=F32) == UNSUPPORTED and call(dim=96) == UNSUPPORTED and call(kv=8193) == UNSUPPORTED
    for name in ("k", "v", "positions", "req", "bt"):
        assert call(**{name: None}) == INVALID, name
    assert call(pages=0) == INVALID and call(nreq=0) == INVALID and call(btw=0) == INVALID and call(bts=3) == INVALID
    assert call(pages=1 << 31) == INVALID
    for name in ("kt", "kh", "vt", "vh"):
        assert call(**{name: 132}) == ALIGNMENT, name
    assert call(k=P + 8) == ALIGNMENT and call(positions=P + 2) == ALIGNMENT and call(p64=1, positions=P + 4) == ALIGNMENT
    cache_refusals(call)


def test_read(L):  # noqa: F811
    call = caller(L, "pml_read_nvfp4", dict(**KV, bt=P, bts=4, lens=P, batch=2, width=4, ko=P, kp=16384, ks=256, kh=128,
                                            vo=P, vp=16384, vs=256, vh=128, dtype=BF16, opages=8, ot=P, ots=4, kv=2,
                                            dim=128, stream=None))
    assert call(batch=0) == OK and call(width=0) == OK
    assert call(batch=-1) == INVALID and call(width=-1) == INVALID and call(kv=0) == INVALID
    assert call(dtype=F32) == UNSUPPORTED and call(dim=32) == UNSUPPORTED
    for name in ("bt", "lens", "ot", "ko", "vo"):
        assert call(**{name: None}) == INVALID, name
    assert call(pages=0) == INVALID and call(opages=0) == INVALID and call(bts=3) == INVALID and call(ots=3) == INVALID
    for name in ("kp", "ks", "kh", "vp", "vs", "vh"):
        assert call(**{name: 132}) == ALIGNMENT and call(**{name: 0}) == ALIGNMENT, name
    assert call(ko=P + 8) == ALIGNMENT and call(lens=P + 2) == ALIGNMENT and call(ot=P + 2) == ALIGNMENT
    cache_refusals(call)


Q = dict(q=P, qt=4096, qh=128, dtype=BF16)
SIZE = dict(tokens=4, heads=32, kv=2, dim=128, scale=0.1)
TAIL = dict(out=P, ot=4096, oh=128, lse=P, ws=P, wsb=1 << 40, stream=None)


def attention_refusals(call):
    assert call(tokens=0) == OK
    assert call(kv=3) == INVALID and call(heads=0) == INVALID and call(kv=0) == INVALID and call(tokens=-4) == INVALID
    assert call(dtype=F32) == UNSUPPORTED and call(dim=96) == UNSUPPORTED and call(heads=8194) == UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == INVALID
    tiny, huge = cache(scale=2.0 ** -32), cache(scale=2.0 ** 32)
    assert call(kc=tiny[0], scale=1e-22) == INVALID and call(kc=huge[0], scale=1e22) == INVALID
    for name in ("q", "bt", "lens", "out", "ws"):
        assert call(**{name: None}) == INVALID, name
    assert call(pages=0) == INVALID and call(btw=0) == INVALID and call(bts=3) == INVALID
    assert call(btw=1 << 26, bts=1 << 27) == UNSUPPORTED      # 2^32 positions
    for name in ("qt", "qh", "ot", "oh"):
        assert call(**{name: 132}) == ALIGNMENT, name
    for name in ("q", "out", "ws"):
        assert call(**{name: P + 8}) == ALIGNMENT, name
    assert call(lse=P + 2) == ALIGNMENT and call(lens=P + 2) == ALIGNMENT
    cache_refusals(call)


def test_paged_attention(L):  # noqa: F811
    call = caller(L, "pml_paged_attention_nvfp4", dict(**Q, **KV, **TABLE, lens=P, cu=P, batch=2, **SIZE, causal=1,
                                                       window=0, **TAIL))
    attention_refusals(call)
    assert call(batch=-1) == INVALID and call(batch=0) == INVALID and call(batch=16385) == UNSUPPORTED
    assert call(batch=0, tokens=0) == OK
    assert call(cu=None, batch=3) == INVALID and call(window=-1) == INVALID and call(cu=P + 2) == ALIGNMENT


def test_sparse_attention(L):  # noqa: F811
    call = caller(L, "pml_sparse_attention_nvfp4", dict(**Q, **KV, **TABLE, lens=P, req=P, nreq=2, sel=P, sst=64, k=64,
                                                        **SIZE, **TAIL))
    attention_refusals(call)
    assert call(k=0) == INVALID and call(sst=63) == INVALID and call(nreq=0) == INVALID
    assert call(req=None) == INVALID and call(sel=None) == INVALID and call(sel=P + 2) == ALIGNMENT


def test_python_checks():
    import sparse_attention_indexer_logits_gb300 as pml
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    buffer, *parts = pml.pml_nvfp4_pages(3, 1, 64, device="cpu")
    assert buffer.shape == (3, 2 * 64 * 36) and [p.shape[-1] for p in parts] == [32, 4, 32, 4]
    assert all(p.data_ptr() % 16 == 0 and p.stride(1) == p.shape[-1] for p in parts)
    with pytest.raises(ValueError, match="head_dim"):
        pml.pml_nvfp4_pages(3, 1, 96, device="cpu")
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        pml.pml_append_nvfp4(x, x, i, i, *parts, i[None])
    with pytest.raises(ValueError, match="k_codes must be"):
        pml.pml_read_nvfp4(*parts, i[None], i, x, x, i[None])
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pml.pml_paged_attention_nvfp4(x, *parts, i[None], i)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pml.pml_sparse_attention_nvfp4(x, *parts, i[None], i, i, i[None])
