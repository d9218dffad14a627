"""What the serving calls refuse from Python before anything is launched, and
that nothing they were given has changed."""
import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(*shape, dtype=BF):
    return torch.ones(shape, dtype=dtype, device="cuda")


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def rope():
    return dict(x=rows(3, 4, 64), positions=ints(3), inv_freq=rows(32, dtype=torch.float32), out=rows(3, 4, 64))


def append():
    return dict(q=rows(3, 4, 64), k=rows(3, 2, 64), v=rows(3, 2, 64), positions=ints(3), requests=ints(3),
                inv_freq=rows(32, dtype=torch.float32), k_cache=rows(2, 64, 2, 64), v_cache=rows(2, 64, 2, 64),
                block_table=ints(1, 2), q_out=rows(3, 4, 64))


def index():
    return dict(q=rows(3, 4, 128), k=rows(3, 128), weights=rows(3, 4, dtype=torch.float32), positions=ints(3),
                requests=ints(3), inv_freq=rows(32, dtype=torch.float32),
                kv_fused=torch.zeros((2, 8448), dtype=torch.uint8, device="cuda"), block_table=ints(1, 2),
                q_out=torch.zeros((3, 4, 128), dtype=torch.uint8, device="cuda"),
                w_out=rows(3, 4, dtype=torch.float32))


def dense():
    return dict(q=rows(3, 4, 64), k_cache=rows(2, 64, 2, 64), v_cache=rows(2, 64, 2, 64), block_table=ints(3, 2),
                kv_lens=ints(3), cu_q=ints(4), out=rows(3, 4, 64), lse=rows(3, 4, dtype=torch.float32))


def listed():
    kw = dense()
    del kw["cu_q"]
    return dict(kw, requests=ints(3), selected=ints(3, 8))


def fork():
    return dict(ref_counts=ints(8), block_table=ints(4, 2), seq_lens=ints(4), parents=ints(2), children=ints(2),
                copy_src=ints(2), copy_dst=ints(2), copy_count=ints(1))


def compact():
    return dict(ref_counts=ints(8), block_table=ints(4, 2), seq_lens=ints(4), ref_counts_out=ints(8),
                block_table_out=ints(4, 2), remap=ints(8), copy_src=ints(4), copy_dst=ints(4), copy_count=ints(1))


def copy():
    return dict(cache=rows(2, 8, 16), copy_src=ints(2), copy_dst=ints(2), copy_count=ints(1))


# call, its arguments, what is changed, the refusal
CASES = [
    (pml.pml_rope, rope, "x", lambda t: t.cpu(), "x must be a CUDA tensor"),
    (pml.pml_rope, rope, "x", lambda t: t[0], "x must be .tokens, heads, dim"),
    (pml.pml_rope, rope, "x", lambda t: rows(3, 4, 128)[..., ::2], "unit last stride"),
    (pml.pml_rope, rope, "x", lambda t: t.double(), "float32, bfloat16 or float16"),
    (pml.pml_rope, rope, "positions", lambda t: t.float(), "int32 or int64"),
    (pml.pml_rope, rope, "positions", lambda t: t[:2], "one value per token"),
    (pml.pml_rope, rope, "positions", lambda t: ints(6)[::2], "contiguous"),
    (pml.pml_rope, rope, "inv_freq", lambda t: t.half(), "float32 or float64"),
    (pml.pml_rope, rope, "out", lambda t: t.float(), "type"),
    (pml.pml_rope, rope, "out", lambda t: t[:2], "x's shape"),
    (pml.pml_rope_append, append, "q", lambda t: t.float(), "bfloat16 or float16"),
    (pml.pml_rope_append, append, "k", lambda t: t.half(), "type"),
    (pml.pml_rope_append, append, "v", lambda t: t[:, :1], "k and v"),
    (pml.pml_rope_append, append, "requests", lambda t: t.long(), "requests must be a contiguous CUDA int32"),
    (pml.pml_rope_append, append, "k_cache", lambda t: t[:, :32], "pages, 64, heads, dim"),
    (pml.pml_rope_append, append, "v_cache", lambda t: t[:1], "k_cache and v_cache"),
    (pml.pml_rope_append, append, "block_table", lambda t: t[0], "rows, width"),
    (pml.pml_rope_append, append, "q_out", lambda t: t[..., :32], "q's shape"),
    (pml.pml_index_quant_append, index, "q", lambda t: t.half(), "128"),
    (pml.pml_index_quant_append, index, "weights", lambda t: t[:, :2], "weights must be float32"),
    (pml.pml_index_quant_append, index, "k", lambda t: t[:2], "k must be a CUDA bfloat16"),
    (pml.pml_index_quant_append, index, "requests", lambda t: None, "keys need"),
    (pml.pml_index_quant_append, index, "kv_fused", lambda t: t[:, :8000].contiguous(), "8448-byte"),
    (pml.pml_index_quant_append, index, "q_out", lambda t: t.int(), "1-byte"),
    (pml.pml_index_quant_append, index, "w_out", lambda t: t.t(), "w_out must be float32"),
    (pml.pml_paged_attention, dense, "q", lambda t: t.float(), "bfloat16 or float16"),
    (pml.pml_paged_attention, dense, "kv_lens", lambda t: t[:2], "kv_lens must hold 3"),
    (pml.pml_paged_attention, dense, "cu_q", lambda t: t[:3], "cu_q must hold 4"),
    (pml.pml_paged_attention, dense, "out", lambda t: t[:2], "q's shape"),
    (pml.pml_paged_attention, dense, "lse", lambda t: t.double(), "lse must be"),
    (pml.pml_paged_attention, dense, "workspace", lambda t: torch.zeros(4), "workspace must be"),
    (pml.pml_paged_attention, dense, "window", lambda t: 1 << 40, "window is too large"),
    (pml.pml_sparse_attention, listed, "selected", lambda t: t[:2], "a row per token"),
    (pml.pml_sparse_attention, listed, "selected", lambda t: t.long(), "selected must be"),
    (pml.pml_sparse_attention, listed, "requests", lambda t: t[:2], "requests must hold 3"),
    (pml.pml_pages_fork, fork, "ref_counts", lambda t: t.long(), "ref_counts must be"),
    (pml.pml_pages_fork, fork, "children", lambda t: t[:1], "children must hold 2"),
    (pml.pml_pages_fork, fork, "copy_count", lambda t: ints(2), "copy_count must hold 1"),
    (pml.pml_pages_compact, compact, "block_table_out", lambda t: t[:3], "block_table's shape"),
    (pml.pml_pages_compact, compact, "remap", lambda t: t[:7], "remap must hold 8"),
    (pml.pml_pages_copy, copy, "cache", lambda t: rows(2, 8, 32)[..., ::2], "must be contiguous"),
    (pml.pml_pages_copy, copy, "cache", lambda t: t[0, 0], "cache must be"),
]


@pytest.mark.parametrize("call, make, name, change, message", CASES)
def test_refusals(call, make, name, change, message):
    kw = make()
    kw[name] = change(kw.get(name))
    before = {n: t.clone() for n, t in kw.items() if torch.is_tensor(t)}
    with pytest.raises(ValueError, match=message):
        call(**kw)
    torch.cuda.synchronize()
    assert all(torch.equal(kw[n], t) for n, t in before.items())


@pytest.mark.parametrize("call, make, name", [
    (pml.pml_rope, rope, "positions"), (pml.pml_rope_append, append, "k"), (pml.pml_paged_attention, dense, "kv_lens"),
    (pml.pml_pages_copy, copy, "copy_src")])
def test_what_is_no_tensor(call, make, name):
    kw = make()
    kw[name] = [1, 2, 3]
    with pytest.raises(TypeError, match=f"{name} must be a tensor"):
        call(**kw)


def test_the_library_s_own_refusals_come_through():
    kw = dense()
    with pytest.raises(pml.PmlError, match="invalid argument"):
        pml.pml_paged_attention(**dict(kw, window=-1))
    with pytest.raises(pml.PmlError, match="unsupported"):
        pml.pml_paged_attention(rows(3, 4, 32), rows(2, 64, 2, 32), rows(2, 64, 2, 32), kw["block_table"], kw["kv_lens"])
    with pytest.raises(pml.PmlError, match="invalid argument"):
        pml.pml_paged_attention(**dict(kw, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")))
