"""Tensors and streams of another device than the current one are refused on
the host.  (No second device is needed: the tensors only say so.)"""
from types import SimpleNamespace

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests.test_serving_checks_gpu import append, compact, copy, dense, fork, index, listed, rope

pytestmark = pytest.mark.gpu

CALLS = [(pml.pml_rope, rope), (pml.pml_rope_append, append), (pml.pml_index_quant_append, index),
         (pml.pml_paged_attention, dense), (pml.pml_sparse_attention, listed), (pml.pml_pages_fork, fork),
         (pml.pml_pages_compact, compact), (pml.pml_pages_copy, copy)]


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another device and holds nothing."""

    @staticmethod
    def __new__(cls, t):
        return torch.Tensor._make_wrapper_subclass(cls, t.shape, dtype=t.dtype, device="cuda:1")

    __torch_dispatch__ = None


def elsewhere(t):
    w = Elsewhere(t)
    assert w.is_cuda and w.get_device() == 1
    return w


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


def test_streams_that_fit():
    kw = rope()
    want = pml.pml_rope(**kw).clone()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.ExternalStream(0),
                   SimpleNamespace(cuda_stream=0)):
        torch.cuda.synchronize()
        kw["out"].zero_()
        torch.cuda.synchronize()
        pml.pml_rope(**kw, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(kw["out"], want)


def test_the_older_calls():
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="seq_lens must be on the current device"):
        pml.pml_schedule(elsewhere(lens), 4)
    with pytest.raises(ValueError, match="logits must be on the current device"):
        pml.pml_topk_logits(elsewhere(torch.zeros((2, 64), device="cuda")), lens, 1, 64, 4)
    assert pml.pml_schedule(lens, 4).shape == (5, 2)
