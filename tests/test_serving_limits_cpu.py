"""Limits of the serving operators' C entries.  No GPU: only calls that return
before touching CUDA."""
from tests.test_serving_abi_cpu import KV, SIZE, TAIL, P, UNSUPPORTED, INVALID, OK, L, caller  # noqa: F401


def test_longest_list(L):  # noqa: F811
    call = caller(L, "pml_sparse_attention", dict(**KV, req=P, nreq=2, sel=P, sst=2 ** 31, k=64, **SIZE, **TAIL))
    assert call(k=2 ** 31 - 1) == UNSUPPORTED and call(k=2 ** 31 - 255) == UNSUPPORTED
    # the longest one passes on to the next check
    assert call(k=2 ** 31 - 256, q=None) == INVALID


def test_a_step_without_requests(L):  # noqa: F811
    call = caller(L, "pml_sparse_attention", dict(**KV, req=P, nreq=2, sel=P, sst=64, k=64, **SIZE, **TAIL))
    assert call(nreq=0, tokens=0) == OK and call(nreq=0) == INVALID and call(nreq=-1, tokens=0) == INVALID
