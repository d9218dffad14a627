"""GPU parity of the pool's bookkeeping with loops over lists, every value
equal: forks (shared, part-full, repeated parents, none free), extending,
freeing, compacting (in place and not), copies of every width, pools of one
page to hundreds of thousands, rows and pages out of range."""
import random

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


def put(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(rnd, lens, pages, width, extra_rows):
    """A pool whose requests hold shuffled pages."""
    ids = list(range(pages))
    rnd.shuffle(ids)
    refs, table, at = [0] * pages, [], 0
    for n in list(lens) + [0] * extra_rows:
        need = -(-n // 64)
        row = ids[at:at + need]
        at += need
        for p in row:
            refs[p] = 1
        table.append(row + [rnd.randrange(pages) for _ in range(width - need)])
    return R.Pool(refs, table, list(lens) + [0] * extra_rows)


class Device:
    def __init__(self, pool):
        self.refs, self.table, self.lens = put(pool.refs), put(pool.table), put(pool.lens)

    def same(self, pool):
        assert self.refs.tolist() == pool.refs
        assert self.table.tolist() == pool.table
        assert self.lens.tolist() == pool.lens


def pad(v, n):
    return v + [-1] * (n - len(v))


@pytest.mark.parametrize("requests,hi,pages,forks,seed", [
    (3, 200, 40, 4, 0), (1, 1, 2, 1, 1), (1, 64, 5, 3, 2), (20, 900, 260, 37, 3), (7, 3000, 700, 1500, 4),
    (300, 200, 5000, 1200, 5), (5, 640, 50, 60, 6)])
def test_fork_then_free(requests, hi, pages, forks, seed):
    rnd = random.Random(seed)
    lens = [rnd.choice([rnd.randint(1, hi), hi // 64 * 64, 0]) for _ in range(requests)]
    pages = max(pages, sum(-(-n // 64) for n in lens) + 1)
    pool = make(rnd, lens, pages, -(-hi // 64) + 1, forks)
    d = Device(pool)
    parents, children = [rnd.randrange(requests) for _ in range(forks)], list(range(requests, requests + forks))
    rnd.shuffle(children)
    src, dst, count = put([5] * forks), put([5] * forks), put([9])
    short = sum(pool.lens[a] % 64 > 0 for a in parents) > len(pool.free_pages())
    moves = pool.fork(parents, children)
    pml.pml_pages_fork(d.refs, d.table, d.lens, put(parents), put(children), src, dst, count)
    d.same(pool)
    assert count.item() == len(moves)
    assert src.tolist() == pad([a for a, _ in moves], forks) and dst.tolist() == pad([b for _, b in moves], forks)
    assert pml.pml_device_status(clear=True) == (pml.STATUS_NO_PAGES if short else 0)
    gone = children[::2]
    pool.free(gone)
    pml.pml_pages_free(d.refs, d.table, d.lens, put(gone))
    d.same(pool)
    assert pml.pml_device_status(clear=True) == 0


@pytest.mark.parametrize("rows,hi,pages,seed", [(1, 10, 3, 0), (9, 700, 200, 1), (1500, 300, 9000, 2),
                                                (40, 2000, 500, 3), (64, 64, 70000, 4)])
def test_extend(rows, hi, pages, seed):
    rnd = random.Random(seed)
    lens = [rnd.randint(0, hi) for _ in range(rows)]
    pages = max(pages, sum(-(-n // 64) for n in lens) + 2)
    width = -(-hi // 64) + 3
    pool = make(rnd, lens, pages, width, 0)
    d = Device(pool)
    for step, (grow, capacity) in enumerate([(1, pages), (130, pages), (64, 5), (100, pages)]):
        want = [n + rnd.randint(-3, grow) for n in pool.lens]
        want = [min(w, width * 64) for w in want]
        refused = 0
        if step == 3:
            want[rnd.randrange(rows)] = width * 64 + 1
            refused = pml.STATUS_BAD_BLOCK
        new, count = put([5] * capacity), put([7])
        total = sum(max(0, -(-w // 64) - -(-n // 64)) for w, n in zip(want, pool.lens) if w <= width * 64)
        none = pml.STATUS_NO_PAGES if total > min(capacity, len(pool.free_pages())) else 0
        taken = pool.extend(want, capacity)
        pml.pml_pages_extend(d.refs, d.table, d.lens, put(want), new, count)
        d.same(pool)
        assert count.item() == len(taken) and new.tolist() == pad(taken, capacity)
        assert pml.pml_device_status(clear=True) == none | refused


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("requests,hi,pages,seed", [(1, 1, 1, 0), (2, 300, 30, 1), (50, 2000, 3000, 2),
                                                    (4, 100, 200000, 3), (30, 500, 0, 4)])
def test_compact(requests, hi, pages, seed, in_place):
    rnd = random.Random(seed)
    lens = [rnd.randint(1, hi) for _ in range(requests)]
    pages = max(pages, sum(-(-n // 64) for n in lens))
    pool = make(rnd, lens, pages, -(-hi // 64) + 1, 2)
    pool.fork([0], [requests]) if pages > sum(-(-n // 64) for n in lens) else None
    d, before = Device(pool), Device(pool)
    room = pages // 2 + 3
    src, dst, count, remap = put([5] * room), put([5] * room), put([9]), put([5] * pages)
    refs, table = (d.refs, d.table) if in_place else (torch.full_like(d.refs, 77), torch.full_like(d.table, 77))
    pml.pml_pages_compact(d.refs, d.table, d.lens, refs, table, remap, src, dst, count)
    moves, want_remap = pool.compact()
    assert refs.tolist() == pool.refs and table.tolist() == pool.table and d.lens.tolist() == pool.lens
    assert remap.tolist() == want_remap and count.item() == len(moves)
    assert src.tolist() == pad([a for a, _ in moves], room) and dst.tolist() == pad([b for _, b in moves], room)
    if not in_place:
        assert torch.equal(d.refs, before.refs) and torch.equal(d.table, before.table)
    assert pml.pml_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype,page", [(torch.bfloat16, (64, 2, 64)), (torch.uint8, (8448,)), (torch.uint8, (7,)),
                                        (torch.float32, (33,)), (torch.int16, (1,)), (torch.uint8, (20004,))])
@pytest.mark.parametrize("layers", [0, 1, 3])
def test_copy(dtype, page, layers):
    g = R.gen(layers)
    shape = ((layers,) if layers else ()) + (40,) + page
    cache = torch.randint(0, 100, shape, generator=g).to(dtype)
    ids = torch.randperm(40, generator=g).tolist()
    src, dst = ids[:15], ids[15:30]
    d = cache.cuda()
    # more entries than the count: the rest is not copied
    pml.pml_pages_copy(d, put(src + ids[30:33]), put(dst + ids[33:36]), put([15]), layers=layers > 0)
    want = cache.clone()
    if layers:
        want[:, dst] = cache[:, src]
    else:
        want[dst] = cache[src]
    assert torch.equal(d.cpu(), want)
    pml.pml_pages_copy(d, put(src), put(dst), put([0]), layers=layers > 0)
    assert torch.equal(d.cpu(), want)
    assert pml.pml_device_status(clear=True) == 0


def test_copy_of_strided_pages_and_past_the_capacity():
    g = R.gen(9)
    wide = torch.randint(0, 100, (2, 10, 3, 32), generator=g, dtype=torch.int32).cuda()
    view, before = wide[:, :, 1], wide.clone()
    pml.pml_pages_copy(view, put([0, 1]), put([8, 9]), put([1000]))
    before[:, 8:, 1] = before[:, :2, 1]
    assert torch.equal(wide, before)


def test_numbers_out_of_range():
    rnd = random.Random(1)
    pool = make(rnd, [100, 64], 10, 3, 2)
    d = Device(pool)
    src, dst, count = put([0] * 3), put([0] * 3), put([0])
    pml.pml_pages_fork(d.refs, d.table, d.lens, put([-1, 0, 4]), put([2, 3, 2]), src, dst, count)
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_REQUEST
    moves = pool.fork([0], [3])
    d.same(pool)
    assert dst.tolist() == [moves[0][1], -1, -1]
    pml.pml_pages_free(d.refs, d.table, d.lens, put([-2, 4]))
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_REQUEST
    d.same(pool)
    # a page outside the pool, and one that nobody holds, are left alone
    d.table[1, 0] = 99
    pml.pml_pages_free(d.refs, d.table, d.lens, put([1]))
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK
    assert d.refs.tolist() == pool.refs and d.lens.tolist()[1] == 0
    cache = torch.arange(10, dtype=torch.int32, device="cuda")[:, None].contiguous()
    pml.pml_pages_copy(cache, put([0, 10, -1, 2]), put([5, 1, 1, -3]), put([4]), layers=False)
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK
    assert cache[:, 0].tolist() == [0, 1, 2, 3, 4, 0, 6, 7, 8, 9]


def test_nothing_to_do():
    d = Device(make(random.Random(0), [5], 2, 1, 0))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    count = put([3])
    pml.pml_pages_fork(d.refs, d.table, d.lens, none, none, none, none, count)
    assert count.item() == 0
    pml.pml_pages_free(d.refs, d.table, d.lens, none)
    pml.pml_pages_copy(torch.zeros((2, 4), device="cuda"), none, none, count, layers=False)
    torch.cuda.synchronize()
    assert pml.pml_device_status(clear=True) == 0
