"""The example's serving loop over K/V caches held in 4 bits: sparse decode with k
past the length gives dense decode over the pages read back, forks go on like
their parents, compaction changes no output."""
import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests.test_serve_example_gpu import example, inputs, prefilled  # noqa: F401

pytestmark = pytest.mark.gpu


def test_selecting_all_is_dense(example):  # noqa: F811
    # (a stack of one layer: a rounding of its outputs may move a later layer's
    # codes across a border)
    x = inputs(3, 1)
    one = [prefilled(example, k=512, kv_bits=4, layers=1) for _ in range(2)]
    for s in one:
        s.extend({0: 1, 1: 1, 2: 1})
    sparse, dense = one[0].step(x, [0, 1, 2], [1, 1, 1]), one[1].step(x, [0, 1, 2], [1, 1, 1], dense=True)
    # P and the output rounded once each in either way, and the projection's sums
    assert (sparse.float() - dense.float()).abs().max() <= 4 * 2.0 ** -8 * dense.float().abs().max()
    assert pml.pml_device_status(clear=True) == 0


def test_forks_and_compaction_change_nothing(example):  # noqa: F811
    s = prefilled(example, kv_bits=4, layers=1)
    s.fork([0, 1, 0], [5, 6, 7])
    rows = [0, 1, 5, 6, 7]
    x = inputs(2, 2)
    for _ in range(3):
        s.extend(dict.fromkeys(rows, 1))
        y = s.step(x[[0, 1, 0, 1, 0]], rows, [1] * 5)
        # (how a row's keys are shared out depends on its place in the batch: P and
        # the output rounded once each from sums in another order)
        for i, j in ((0, 2), (0, 4), (1, 3)):
            assert (y[i].float() - y[j].float()).abs().max() <= 4 * 2.0 ** -8 * y.float().abs().max()
        x = y[:2]
    s.free([0, 6])
    before = [t.clone() for t in (s.refs, s.table, s.lens)]
    keep = [c.clone() for c in (*s.kv, s.index)]
    s.extend(dict.fromkeys([1, 2, 5, 7], 1))
    want = s.step(inputs(4, 3), [1, 2, 5, 7], [1] * 4)
    for t, u in zip((s.refs, s.table, s.lens, *s.kv, s.index), before + keep):
        t.copy_(u)
    s.compact()
    s.extend(dict.fromkeys([1, 2, 5, 7], 1))
    assert torch.equal(s.step(inputs(4, 3), [1, 2, 5, 7], [1] * 4), want)
    assert pml.pml_device_status(clear=True) == 0


def test_main_runs(example, capsys):  # noqa: F811
    example.main(4)
    out = capsys.readouterr().out
    assert "lengths [770, 0, 71, 0, 770]" in out and "status 0" in out
