"""Argument checks of the serving operators' C entries and of their Python
calls.  No GPU: only calls that return before touching CUDA."""
import pytest
import torch

P = 0x10000  # a 16-byte aligned stand-in pointer value; never dereferenced
F32, BF16, FP16 = 0, 1, 2
OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from sparse_attention_indexer_logits_gb300 import _build
    _build.build()
    import sparse_attention_indexer_logits_gb300 as pml
    return pml.lib()


def caller(L, name, args):
    """A call with `args` (in order), any of them overridden by name."""
    def call(**over):
        assert set(over) <= set(args), over
        a = dict(args)
        a.update(over)
        return getattr(L, name)(*a.values())
    return call


ROT = dict(positions=P, p64=0)
FREQ = dict(inv_freq=P, f64=1, rot=64, off=0, il=0, ms=1.0)


def test_rope(L):
    call = caller(L, "pml_rope", dict(x=P, xt=1024, xh=128, out=P, ot=1024, oh=128, dtype=BF16, **ROT, **FREQ, grad=0,
                                      tokens=4, heads=8, dim=128, stream=None))
    assert call(tokens=0) == OK and call(heads=0) == OK
    assert call(tokens=-1) == INVALID and call(dim=0) == INVALID
    assert call(dtype=3) == UNSUPPORTED and call(dim=513, rot=0) == UNSUPPORTED
    assert call(x=None) == INVALID and call(out=None) == INVALID and call(positions=None) == INVALID
    assert call(inv_freq=None) == INVALID
    assert call(rot=63) == INVALID and call(rot=130) == INVALID and call(off=66) == INVALID
    assert call(off=-1) == INVALID and call(rot=-2) == INVALID
    assert call(x=P + 1) == ALIGNMENT and call(dtype=F32, out=P + 2) == ALIGNMENT
    assert call(positions=P + 2) == ALIGNMENT and call(p64=1, positions=P + 4) == ALIGNMENT
    assert call(inv_freq=P + 4) == ALIGNMENT


def test_rope_append(L):
    call = caller(L, "pml_rope_append", dict(
        q=P, qt=1024, qh=128, qo=P, qot=1024, qoh=128, k=P, kt=256, kh=128, v=P, vt=256, vh=128, dtype=BF16, **ROT,
        req=P, nreq=2, **FREQ, kc=P, kp=16384, ks=256, kch=128, vc=P, vp=16384, vs=256, vch=128, pages=4, bt=P,
        bts=4, btw=4, tokens=3, heads=8, kv=2, dim=128, stream=None))
    assert call(tokens=0) == OK
    assert call(dtype=F32) == UNSUPPORTED
    assert call(kv=0) == INVALID and call(heads=-1) == INVALID
    for name in ("q", "qo", "k", "v", "kc", "vc", "req", "bt", "positions", "inv_freq"):
        assert call(**{name: None}) == INVALID, name
    assert call(pages=0) == INVALID and call(nreq=0) == INVALID
    assert call(btw=0) == INVALID and call(bts=3) == INVALID
    assert call(kc=P + 1) == ALIGNMENT and call(req=P + 2) == ALIGNMENT


def test_index_quant(L):
    call = caller(L, "pml_index_quant_append", dict(
        q=P, qt=8192, qh=128, k=P, kt=128, w=P, ws=1.0, **ROT, req=P, nreq=2, **FREQ, qo=P, wo=P, kv=P, blocks=4, bt=P,
        bts=4, btw=4, tokens=3, heads=64, stream=None))
    assert call(tokens=0) == OK
    assert call(heads=0) == INVALID and call(heads=1025) == UNSUPPORTED
    assert call(rot=40) == UNSUPPORTED and call(off=4) == UNSUPPORTED
    for name in ("q", "w", "qo", "wo", "kv", "req", "bt", "positions", "inv_freq"):
        assert call(**{name: None}) == INVALID, name
    assert call(blocks=0) == INVALID and call(nreq=0) == INVALID and call(bts=3) == INVALID
    assert call(q=P + 8) == ALIGNMENT and call(k=P + 2) == ALIGNMENT and call(qt=8196) == ALIGNMENT
    assert call(kt=132) == ALIGNMENT and call(qo=P + 8) == ALIGNMENT


KV = dict(q=P, qt=4096, qh=128, kc=P, kp=16384, ks=256, kh=128, vc=P, vp=16384, vs=256, vh=128, dtype=BF16, pages=4,
          bt=P, bts=4, btw=4, lens=P)
SIZE = dict(tokens=4, heads=32, kv=2, dim=128, scale=0.1)
TAIL = dict(out=P, ot=4096, oh=128, lse=P, ws=P, wsb=1 << 40, stream=None)


def attention_refusals(call):
    assert call(tokens=0) == OK
    assert call(kv=3) == INVALID and call(heads=0) == INVALID and call(kv=0) == INVALID and call(tokens=-4) == INVALID
    assert call(dtype=F32) == UNSUPPORTED and call(dim=96) == UNSUPPORTED
    assert call(heads=129, kv=1) == UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=bad) == INVALID
    for name in ("q", "kc", "vc", "bt", "lens", "out", "ws"):
        assert call(**{name: None}) == INVALID, name
    assert call(pages=0) == INVALID and call(btw=0) == INVALID and call(bts=3) == INVALID
    assert call(btw=1 << 26, bts=1 << 27) == UNSUPPORTED      # 2^32 positions
    for name in ("qt", "qh", "kp", "ks", "kh", "vp", "vs", "vh", "ot", "oh"):
        assert call(**{name: 132}) == ALIGNMENT, name
    for name in ("qt", "kp", "ks", "vh"):
        assert call(**{name: 0}) == ALIGNMENT and call(**{name: -128}) == ALIGNMENT, name
    for name in ("q", "kc", "vc", "out", "ws"):
        assert call(**{name: P + 8}) == ALIGNMENT, name
    assert call(lse=P + 2) == ALIGNMENT and call(lens=P + 2) == ALIGNMENT


def test_paged_attention(L):
    call = caller(L, "pml_paged_attention", dict(**KV, cu=P, batch=2, **SIZE, causal=1, window=0, **TAIL))
    attention_refusals(call)
    assert call(batch=-1) == INVALID and call(batch=0) == INVALID and call(batch=16385) == UNSUPPORTED
    assert call(batch=0, tokens=0) == OK
    assert call(cu=None, batch=3) == INVALID and call(window=-1) == INVALID and call(cu=P + 2) == ALIGNMENT


def test_sparse_attention(L):
    call = caller(L, "pml_sparse_attention", dict(**KV, req=P, nreq=2, sel=P, sst=64, k=64, **SIZE, **TAIL))
    attention_refusals(call)
    assert call(k=0) == INVALID and call(sst=63) == INVALID and call(nreq=0) == INVALID
    assert call(req=None) == INVALID and call(sel=None) == INVALID and call(sel=P + 2) == ALIGNMENT


def test_workspace_bytes(L):
    assert L.pml_attention_workspace_bytes(152, 128) == 304 * (32 + 256 * 8 + 256 * 128 * 4)
    assert L.pml_attention_workspace_bytes(152, 96) == 0 and L.pml_attention_workspace_bytes(0, 64) == 0


POOL = dict(refs=P, pages=10, bt=P, bts=4, btw=4, lens=P, rows=3)


def pool_refusals(call):
    assert call(pages=-1) == INVALID and call(rows=-1) == INVALID and call(btw=5) == INVALID
    assert call(refs=None) == INVALID and call(bt=None) == INVALID and call(lens=None) == INVALID
    assert call(refs=P + 2) == ALIGNMENT
    assert call(rows=1 << 20, btw=1 << 12, bts=1 << 12) == UNSUPPORTED


def test_pages(L):
    fork = caller(L, "pml_pages_fork", dict(**POOL, parents=P, children=P, n=2, src=P, dst=P, count=P, stream=None))
    extend = caller(L, "pml_pages_extend", dict(**POOL, new=P, pages_out=P, cap=5, count=P, stream=None))
    free = caller(L, "pml_pages_free", dict(**POOL, list=P, n=2, stream=None))
    compact = caller(L, "pml_pages_compact", dict(**POOL, refs_out=P, bt_out=P, bts_out=4, remap=P, src=P, dst=P, cap=5,
                                                  count=P, stream=None))
    for call in (fork, extend, free, compact):
        pool_refusals(call)
    for name in ("parents", "children", "src", "dst", "count"):
        assert fork(**{name: None}) == INVALID
    assert fork(n=-1) == INVALID and fork(dst=P + 1) == ALIGNMENT
    assert extend(new=None) == INVALID and extend(cap=-1) == INVALID and extend(count=None) == INVALID
    assert free(n=0) == OK and free(list=None) == INVALID and free(n=-1) == INVALID
    assert compact(cap=4) == INVALID and compact(remap=None) == INVALID and compact(bts_out=3) == INVALID
    assert compact(bts_out=5) == INVALID      # in place with another stride
    copy = caller(L, "pml_pages_copy", dict(cache=P, layers=2, ls=4096, pages=10, ps=256, pb=256, src=P, dst=P, count=P,
                                            cap=5, stream=None))
    assert copy(layers=0) == OK and copy(cap=0) == OK and copy(pb=0) == OK and copy(pages=0) == OK
    assert copy(cache=None) == INVALID and copy(count=None) == INVALID and copy(ps=255) == INVALID
    assert copy(src=P + 2) == ALIGNMENT and copy(layers=-1) == INVALID


def test_python_checks():
    import sparse_attention_indexer_logits_gb300 as pml
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        pml.pml_rope(x, i, f)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pml.pml_rope_append(x, x, x, i, i, f, x, x, i)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pml.pml_index_quant_append(x, None, f, i, None, f, None, None)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        pml.pml_paged_attention(x, x, x, i, i)
    with pytest.raises(ValueError, match="ref_counts must be"):
        pml.pml_pages_free(i, i, i, i)
    with pytest.raises(ValueError, match="cache must be"):
        pml.pml_pages_copy(x, i, i, i)
