"""The calls over caches held in 4 bits refuse tensors and streams of another
device than the current one on the host, and touch nothing."""
from types import SimpleNamespace

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests.test_devices_gpu import elsewhere
from tests.test_serving_checks_gpu import ints, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


def parts():
    _, *p = pml.pml_nvfp4_pages(2, 2, 64)
    return dict(zip(("k_codes", "k_scales", "v_codes", "v_scales"), p))


def append():
    return dict(k=rows(3, 2, 64), v=rows(3, 2, 64), positions=ints(3), requests=ints(3), **parts(),
                block_table=ints(1, 2))


def read():
    return dict(**parts(), block_table=ints(3, 2), kv_lens=ints(3), k_out=rows(6, 64, 2, 64), v_out=rows(6, 64, 2, 64),
                out_table=ints(3, 2))


def dense():
    return dict(q=rows(3, 4, 64), **parts(), block_table=ints(3, 2), kv_lens=ints(3), cu_q=ints(4), out=rows(3, 4, 64),
                lse=rows(3, 4, dtype=torch.float32))


def listed():
    kw = dense()
    del kw["cu_q"]
    return dict(kw, requests=ints(3), selected=ints(3, 8))


CALLS = [(pml.pml_append_nvfp4, append), (pml.pml_read_nvfp4, read), (pml.pml_paged_attention_nvfp4, dense),
         (pml.pml_sparse_attention_nvfp4, listed)]


@pytest.mark.parametrize("call, make", CALLS)
def test_one_tensor_of_another_device(call, make):
    kw = make()
    names = [n for n, t in kw.items() if torch.is_tensor(t)]
    before = {n: kw[n].clone() for n in names}
    for name in names:
        with pytest.raises(ValueError, match="device"):
            call(**dict(kw, **{name: elsewhere(kw[name])}))
    torch.cuda.synchronize()
    assert all(torch.equal(kw[n], t) for n, t in before.items())


@pytest.mark.parametrize("call, make", CALLS)
def test_a_stream_of_another_device(call, make):
    mine = torch.cuda.current_stream()
    with pytest.raises(ValueError, match="stream must be of the current device"):
        call(**make(), stream=SimpleNamespace(cuda_stream=mine.cuda_stream, device_index=1))


@pytest.mark.parametrize("call, make", CALLS)
def test_tensors_that_fit(call, make):
    call(**make())
    assert pml.pml_device_status(clear=True) == 0
