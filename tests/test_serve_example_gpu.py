"""The example's serving loop: sparse decode with k past the length gives dense
decode, a fork goes on like its parent, and compaction changes no output."""
import importlib.util
import os

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("serve_step", os.path.join(HERE, "..", "examples", "serve_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    pml.pml_device_status(clear=True)
    return m


def prefilled(example, **kw):
    s = example.Server(**kw)
    g = torch.Generator(device="cuda").manual_seed(5)
    prompts = {0: 300, 1: 64, 2: 1}
    for lo, hi in ((0, 200), (200, 300)):
        part = {r: min(n, hi) - lo for r, n in prompts.items() if min(n, hi) > lo}
        s.extend(part)
        s.step(torch.randn((sum(part.values()), 512), generator=g, device="cuda", dtype=torch.bfloat16), list(part),
               list(part.values()), dense=True)
    return s


def inputs(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, 512), generator=g, device="cuda", dtype=torch.bfloat16)


def test_selecting_all_is_dense(example):
    a, b = prefilled(example, k=512), prefilled(example, k=512)
    x = inputs(3, 1)
    for s in (a, b):
        s.extend({0: 1, 1: 1, 2: 1})
    sparse, dense = a.step(x, [0, 1, 2], [1, 1, 1]), b.step(x, [0, 1, 2], [1, 1, 1], dense=True)
    # two layers; each rounds its probabilities and outputs in another order
    assert (sparse.float() - dense.float()).abs().max() <= 8 * 2.0 ** -8 * dense.float().abs().max()
    few = prefilled(example, k=16)
    few.extend({0: 1, 1: 1, 2: 1})
    assert not torch.equal(few.step(x, [0, 1, 2], [1, 1, 1]), sparse)
    assert pml.pml_device_status(clear=True) == 0


def test_forks_and_compaction_change_nothing(example):
    s = prefilled(example)
    s.fork([0, 1, 0], [5, 6, 7])
    rows = [0, 1, 5, 6, 7]
    x = inputs(2, 2)
    for step in range(3):
        s.extend(dict.fromkeys(rows, 1))
        y = s.step(x[[0, 1, 0, 1, 0]], rows, [1] * 5)
        assert torch.equal(y[0], y[2]) and torch.equal(y[0], y[4]) and torch.equal(y[1], y[3])
        x = y[:2]
    s.free([0, 6])
    before = [t.clone() for t in (s.refs, s.table, s.lens)]
    keep = [c.clone() for c in (*s.kv, s.index)]
    s.extend(dict.fromkeys([1, 2, 5, 7], 1))
    want = s.step(inputs(4, 3), [1, 2, 5, 7], [1] * 4)
    # the same step again, from a compacted pool
    for t, u in zip((s.refs, s.table, s.lens, *s.kv, s.index), before + keep):
        t.copy_(u)
    s.compact()
    live = int((s.refs > 0).sum())
    assert (s.refs[:live] > 0).all() and live < int((before[0] > 0).nonzero().max()) + 1
    s.extend(dict.fromkeys([1, 2, 5, 7], 1))
    assert torch.equal(s.step(inputs(4, 3), [1, 2, 5, 7], [1] * 4), want)
    assert pml.pml_device_status(clear=True) == 0


def test_main_runs(example, capsys):
    example.main()
    out = capsys.readouterr().out
    assert "lengths [770, 0, 71, 0, 770]" in out and "status 0" in out
