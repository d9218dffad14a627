"""Pages held in 4 bits read back where a request's length is near 2^31: it has
the table's positions, and the requests beside it theirs."""
import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests.test_nvfp4_cache_gpu import BF, filled, i32, read_want, same

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


@pytest.mark.parametrize("long", [2 ** 31 - 1, 2 ** 31 - 63, 2 ** 31 - 64])
def test_a_length_near_the_last(long):
    _, parts = filled(9, 2, 64, 14)
    table, out_table = i32([[0, 4, 2], [8, 3, 1], [5, 6, 7]]), i32([[5, 1, 6], [0, 2, 8], [3, 4, 7]])
    out = [torch.full((9, 64, 2, 64), 9.0, dtype=BF, device="cuda") for _ in range(2)]
    want = read_want(parts, table, [70, 192, 0], out, out_table, (1.0, 1.0))
    pml.pml_read_nvfp4(*parts, table.cuda(), i32([70, long, -5]).cuda(), *out, out_table.cuda())
    assert pml.pml_device_status(clear=True) == 0
    assert same(out[0], want[0]) and same(out[1], want[1])
