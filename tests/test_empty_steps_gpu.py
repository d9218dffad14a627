"""Steps without requests or tokens: nothing to do, and not an error."""
import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests.test_serving_checks_gpu import ints, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


@pytest.mark.parametrize("requests", [0, 3])
def test_nothing_to_attend(requests):
    q, cache, table, lens = rows(0, 4, 64), rows(2, 64, 2, 64), ints(requests, 2), ints(requests)
    assert pml.pml_paged_attention(q, cache, cache, table, lens).shape == (0, 4, 64)
    assert pml.pml_paged_attention(q, cache, cache, table, lens, ints(requests + 1)).shape == (0, 4, 64)
    assert pml.pml_sparse_attention(q, cache, cache, table, lens, ints(0), ints(0, 8)).shape == (0, 4, 64)
    assert pml.pml_device_status(clear=True) == 0


@pytest.mark.parametrize("requests", [0, 3])
def test_nothing_to_append(requests):
    f, table = rows(32, dtype=torch.float32), ints(requests, 2)
    cache = rows(2, 64, 2, 64)
    x = rows(0, 4, 64)
    assert pml.pml_rope_append(x, x[:, :2], x[:, :2], ints(0), ints(0), f, cache, cache, table).shape == (0, 4, 64)
    kv = torch.zeros((2, 8448), dtype=torch.uint8, device="cuda")
    q, w = pml.pml_index_quant_append(rows(0, 4, 128), rows(0, 128), rows(0, 4, dtype=torch.float32), ints(0), ints(0),
                                      f, kv, table)
    assert q.shape == (0, 4, 128) and w.shape == (0, 4)
    assert (cache == 1).all() and (kv == 0).all() and pml.pml_device_status(clear=True) == 0


def test_tokens_of_no_request_are_refused():
    with pytest.raises(ValueError, match="divide equally"):
        pml.pml_paged_attention(rows(2, 4, 64), rows(2, 64, 2, 64), rows(2, 64, 2, 64), ints(0, 2), ints(0))
    with pytest.raises(pml.PmlError, match="invalid"):
        pml.pml_sparse_attention(rows(2, 4, 64), rows(2, 64, 2, 64), rows(2, 64, 2, 64), ints(0, 2), ints(0), ints(2),
                                 ints(2, 8))
