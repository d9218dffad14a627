"""GPU parity of pml_append_nvfp4 and pml_read_nvfp4 with the definitions in 64
bits, bit for bit: every 16-bit value, ties, scales at both ends of their range,
layouts, padding, bad places, caches past 32 bits, graphs."""
import math

import pytest
import torch

import sparse_attention_indexer_logits_gb300 as pml
from tests import nvfp4_ref as N
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True, scope="module")
def _build():
    import __graft_entry__
    __graft_entry__.build()
    pml.pml_device_status(clear=True)
    yield


def i32(values):
    return torch.tensor(values, dtype=torch.int32)


def filled(pages, heads, dim, seed, layout="pages"):
    """Caches full of arbitrary bytes, in one of three layouts: (the buffers, the four parts)."""
    g = R.gen(seed)
    noise = lambda t: t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))  # noqa: E731
    if layout == "pages":
        buffer, *parts = pml.pml_nvfp4_pages(pages, heads, dim)
        noise(buffer)
        return [buffer], parts
    if layout == "rows":                  # slots before heads, four buffers
        parts = [noise(torch.empty((pages, 64, heads, w), dtype=torch.uint8, device="cuda"))
                 for w in (dim // 2, dim // 16) * 2]
        return parts, parts
    # gaps: rows of 96 and 16 bytes, heads before slots, every other page
    buffers = [noise(torch.empty((pages, 2, heads, 64, w), dtype=torch.uint8, device="cuda")) for w in (96, 16) * 2]
    return buffers, [b[:, 1, :, :, :w].transpose(1, 2) for b, w in zip(buffers, (dim // 2, dim // 16) * 2)]


def append(k, v, pos, req, parts, table, **kw):
    pml.pml_append_nvfp4(k.cuda(), v.cuda(), pos.cuda(), req.cuda(), *parts, table.cuda(), **kw)


# ------------------------------------------------------------------ quantised

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heads,dim", [(8, 128), (1, 64), (3, 128), (5, 64)])
@pytest.mark.parametrize("layout", ["pages", "rows", "gaps"])
def test_append(dtype, heads, dim, layout):
    g = R.gen(heads + dim)
    lens, counts = [1, 64, 65, 200, 130], [1, 1, 2, 77, 130]
    req = i32([b for b, n in enumerate(counts) for _ in range(n)])
    pos = i32([lens[b] - n + i for b, n in enumerate(counts) for i in range(n)])
    req[3], pos[7] = -1, -5                          # padding
    table, pages = R.block_table(lens, g)
    rows = torch.randn((len(req), 2 * heads + 1, dim), generator=g).to(dtype)
    buffers, parts = filled(pages, heads, dim, 1, layout)
    before = [b.clone() for b in buffers]
    want = [p.cpu().clone() for p in parts]
    d = rows.cuda()
    pml.pml_append_nvfp4(d[:, :heads], d[:, heads + 1:], pos.cuda(), req.cuda(), *parts, table.cuda(), k_scale=0.5,
                         v_scale=4.0)
    assert pml.pml_device_status(clear=True) == 0
    real = (req >= 0) & (pos >= 0)
    page = table[req[real].long(), pos[real].long() // 64].long()
    slot = pos[real].long() % 64
    for i, (x, s) in enumerate(((rows[:, :heads], 0.5), (rows[:, heads + 1:], 4.0))):
        codes, scales = N.quantise(x[real], s)
        want[2 * i][page, slot], want[2 * i + 1][page, slot] = codes, scales
    for got, w in zip(parts, want):
        assert torch.equal(got.cpu(), w)
    # what lies between the rows stays
    for buffer, old, part in zip(buffers, before, parts):
        if layout == "gaps":
            part.zero_()
            w = old.clone()
            w[:, 1, :, :, :part.shape[3]] = 0
            assert torch.equal(buffer, w)


def rows_of(values, dim=64):
    """Values as rows, the last one repeated."""
    n = -(-len(values) // dim) * dim
    return torch.cat([values, values[-1:].expand(n - len(values))]).view(-1, 1, dim)


def one_by_one(k, g, dtype):
    """The code and scale bytes of rows [tokens, 1, 64] appended to one request."""
    n = len(k)
    pages = -(-n // 64)
    _, parts = filled(pages, 1, 64, 2)
    append(k.to(dtype), k.to(dtype).flip(0), torch.arange(n), torch.zeros(n, dtype=torch.int32), parts,
           torch.arange(pages, dtype=torch.int32)[None], k_scale=g, v_scale=g)
    assert pml.pml_device_status(clear=True) == 0
    flat = [p.cpu().flatten(0, 1)[:n] for p in parts]
    for i, x in enumerate((k, k.flip(0))):
        codes, scales = N.quantise(x.to(dtype), g)
        assert torch.equal(flat[2 * i + 1], scales), "scales"
        bad = (flat[2 * i] != codes).any(-1).any(-1)
        assert not bad.any(), f"codes of {x[bad][0].tolist()}"


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("g", [1.0, 2.0 ** -32, 2.0 ** 32, 0.125])
def test_every_value(dtype, g):
    """Every 16-bit pattern, infinities and NaN among them, in groups of sixteen
    neighbours, and in groups with patterns of other sizes."""
    bits = torch.arange(65536).to(torch.uint16).view(torch.int16).view(dtype)
    one_by_one(rows_of(bits).to(dtype), g, dtype)
    mixed = bits.view(16, 4096).T.flatten()
    one_by_one(rows_of(mixed), g, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_ties(dtype):
    """Quotients on the borders between codes, and one step of the type to either
    side, under every scale that a largest value of 6 s gives exactly."""
    scale = N.E4M3[1:0x7f]
    if dtype == FP:
        scale = scale[scale >= 2.0 ** -6]            # below, the borders are not fp16 numbers
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    rows = []
    for s in scale.tolist():
        x = (border * s).to(dtype)
        assert torch.equal(x.double(), border * s)
        up = (x.view(torch.int16) + 1).view(dtype)
        down = (x.view(torch.int16) - 1).view(dtype)
        for y in (x, up, down):
            for sign in (1, -1):
                rows.append(torch.cat([y * sign, -y * sign, torch.tensor([6 * s, -6 * s]).to(dtype)]))
    one_by_one(torch.cat(rows).view(-1, 1, 16).repeat(1, 1, 4), 1.0, dtype)


@pytest.mark.parametrize("g", [1.0, 2.0 ** -20, 2.0 ** 20])
def test_sizes(g):
    """Groups from far below the smallest scale to far past the largest."""
    gen = R.gen(3)
    size = torch.exp2(torch.arange(-40, 41).double())[:, None, None]
    k = (torch.randn((81, 1, 64), generator=gen).double() * size * g).to(BF)
    one_by_one(k, g, BF)


def test_append_bad_places():
    g = R.gen(1)
    table = i32([[3, 99], [-1, 1]]).cuda()
    req, pos = i32([0, 0, 1, 1, 2, 0]).cuda(), torch.tensor([5, 70, 1, 64, 0, 128]).cuda()
    x = torch.randn((6, 1, 64), generator=g).bfloat16()
    buffer, *parts = pml.pml_nvfp4_pages(4, 1, 64)
    pml.pml_append_nvfp4(x.cuda(), x.cuda(), pos, req, *parts, table)
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK | pml.STATUS_BAD_REQUEST
    codes, scales = N.quantise(x, 1.0)
    for got, w in zip(parts, (codes, scales) * 2):
        got = got.cpu()
        assert torch.equal(got[3, 5], w[0]) and torch.equal(got[1, 0], w[3])
        got[3, 5], got[1, 0] = 0, 0
        assert (got == 0).all()


# ------------------------------------------------------------------ read back

def read_want(parts, table, lens, out, out_table, scales, width=None):
    """What the outputs have to hold."""
    want = [o.cpu().clone() for o in out]
    for i, (codes, size) in enumerate((parts[:2], parts[2:])):
        v = N.values(codes.cpu(), size.cpu(), scales[i])
        for b, n in enumerate(lens):
            p = torch.arange(max(min(n, 64 * (width or table.shape[1])), 0))
            here, there = table[b].long()[p // 64], out_table[b].long()[p // 64]
            want[i][there, p % 64] = v[here, p % 64].to(want[i].dtype)
    return want


def same(got, want):
    """Equal, NaN with NaN (their signs and payloads aside)."""
    return torch.equal(torch.nan_to_num(got.cpu(), nan=777.0), torch.nan_to_num(want, nan=777.0))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heads,dim", [(8, 128), (1, 64), (3, 128), (5, 64)])
@pytest.mark.parametrize("layout", ["pages", "rows", "gaps"])
def test_read(dtype, heads, dim, layout):
    """Any bytes (negative scales and NaN among them) into pages of any order and layout."""
    g = R.gen(heads)
    lens = [1, 0, 64, 65, 300, -3, 129]
    table, pages = R.block_table(lens, g)
    _, parts = filled(pages, heads, dim, 5, layout)
    out_table = torch.randperm(table.numel() + 2, generator=g)[:table.numel()].view(table.shape).int()
    shape = (table.numel() + 2, 64, heads, dim)
    if layout == "rows":
        out = [torch.full(shape, 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    else:
        out = [torch.full((shape[0], heads, 2, 64, dim + 8), 9.0, dtype=dtype, device="cuda")[:, :, 1, :, :dim]
               .transpose(1, 2) for _ in range(2)]
    scales = (2.0 ** -3, 2.0 ** 2)
    want = read_want(parts, table, lens, out, out_table, scales)
    pml.pml_read_nvfp4(*parts, table.cuda(), i32(lens).cuda(), *out, out_table.cuda(), k_scale=scales[0],
                       v_scale=scales[1])
    assert pml.pml_device_status(clear=True) == 0
    assert same(out[0], want[0]) and same(out[1], want[1])


def test_read_past_a_type_s_range():
    """2688 * 2^8 is past fp16's largest value, 2^-10 * 2^-32 below its smallest."""
    _, parts = filled(2, 1, 64, 6)
    for scale in (2.0 ** 8, 2.0 ** -32):
        out = [torch.zeros((2, 64, 1, 64), dtype=FP, device="cuda") for _ in range(2)]
        table = i32([[0, 1]])
        want = read_want(parts, table, [128], out, table, (scale, scale))
        pml.pml_read_nvfp4(*parts, table.cuda(), i32([128]).cuda(), *out, table.cuda(), k_scale=scale, v_scale=scale)
        assert same(out[0], want[0]) and same(out[1], want[1])


def test_read_bad_pages_and_lengths_past_the_table():
    _, parts = filled(4, 2, 64, 7)
    table, out_table = i32([[0, 4, 2], [-1, 3, 1]]), i32([[5, 1, 6], [0, 2, 7]])
    out = [torch.full((7, 64, 2, 64), 9.0, dtype=BF, device="cuda") for _ in range(2)]
    want = [o.cpu().clone() for o in out]
    for i in range(2):
        v = N.values(parts[2 * i].cpu(), parts[2 * i + 1].cpu(), 1.0).to(BF)
        want[i][5], want[i][6], want[i][2, :6] = v[0], v[2], v[3, :6]
    pml.pml_read_nvfp4(*parts, table.cuda(), i32([5000, 70]).cuda(), *out, out_table.cuda())
    assert pml.pml_device_status(clear=True) == pml.STATUS_BAD_BLOCK
    assert same(out[0], want[0]) and same(out[1], want[1])


def test_many_requests_read():
    g = R.gen(8)
    lens = torch.randint(0, 150, (3001,), generator=g).tolist()
    table, pages = R.block_table(lens, g)
    _, parts = filled(pages, 1, 64, 8)
    out_table = torch.arange(table.numel(), dtype=torch.int32).view(table.shape)
    out = [torch.full((table.numel(), 64, 1, 64), 9.0, dtype=BF, device="cuda") for _ in range(2)]
    want = read_want(parts, table, lens, out, out_table, (1.0, 1.0))
    pml.pml_read_nvfp4(*parts, table.cuda(), i32(lens).cuda(), *out, out_table.cuda())
    assert same(out[0], want[0]) and same(out[1], want[1])


def test_nothing_to_do():
    buffer, *parts = pml.pml_nvfp4_pages(2, 1, 64)
    empty = torch.empty((0, 1, 64), dtype=BF, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    pml.pml_append_nvfp4(empty, empty, none, none, *parts, table)
    out = [torch.full((1, 64, 1, 64), 9.0, dtype=BF, device="cuda") for _ in range(2)]
    pml.pml_read_nvfp4(*parts, table[:0], none, *out, table[:0])
    pml.pml_read_nvfp4(*parts, table, torch.zeros(1, dtype=torch.int32, device="cuda"), *out, table)
    assert (buffer == 0).all() and (out[0] == 9.0).all() and (out[1] == 9.0).all()


def test_caches_past_32_bits():
    """Pages more than 2^32 bytes into the cache, and elements into the output."""
    pages, heads, dim = 70000, 8, 128
    used = [69999, 0, 69998, 40000]
    _, *parts = pml.pml_nvfp4_pages(pages, heads, dim)
    g = R.gen(9)
    rows = torch.randn((200, 2 * heads, dim), generator=g).to(FP)
    table = i32([used])
    pos = torch.arange(10, 210)
    append(rows[:, :heads], rows[:, heads:], pos, torch.zeros(200, dtype=torch.int32), parts, table)
    out = [torch.zeros((70000, 64, heads, dim), dtype=FP, device="cuda") for _ in range(2)]
    out_table = i32([[5, 69999, 68000, 69998]]).cuda()
    pml.pml_read_nvfp4(*parts, table.cuda(), i32([210]).cuda(), *out, out_table)
    assert pml.pml_device_status(clear=True) == 0
    for i, x in enumerate((rows[:, :heads], rows[:, heads:])):
        want = N.values(*N.quantise(x, 1.0), 1.0).to(FP)
        assert torch.equal(out[i][out_table[0].long()].cpu().flatten(0, 1)[10:210], want)


def test_captured_and_on_another_stream():
    g = R.gen(10)
    table, pages = R.block_table([100, 40], g)
    buffer, *parts = pml.pml_nvfp4_pages(pages, 2, 128)
    x = torch.randn((140, 4, 128), generator=g).to(BF).cuda()
    req = i32([0] * 100 + [1] * 40).cuda()
    pos = torch.cat([torch.arange(100), torch.arange(40)]).cuda()
    out = [torch.zeros((pages, 64, 2, 128), dtype=BF, device="cuda") for _ in range(2)]
    table, lens = table.cuda(), i32([100, 40]).cuda()

    def step(stream=None):
        pml.pml_append_nvfp4(x[:, :2], x[:, 2:], pos, req, *parts, table, stream=stream)
        pml.pml_read_nvfp4(*parts, table, lens, *out, table, stream=stream)

    step()
    want, want_out = buffer.clone(), [o.clone() for o in out]
    buffer.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(buffer, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    buffer.zero_()
    [o.zero_() for o in out]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(buffer, want) and all(torch.equal(a, b) for a, b in zip(out, want_out))
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, 2 * b) for a, b in zip(out, want_out))    # twice the scales, the same codes


def test_layers_of_pages_are_copied():
    """A pool's page copies take the caches' buffer, layers in front."""
    buffer, *parts = pml.pml_nvfp4_pages(5, 2, 64, layers=3)
    assert buffer.shape == (3, 5, 2 * 2 * 64 * 36) and parts[0].shape == (3, 5, 64, 2, 32)
    assert parts[3].shape == (3, 5, 64, 2, 4)
    buffer.copy_(torch.randint(0, 256, buffer.shape, dtype=torch.uint8, generator=R.gen(11)))
    want = [p[:, 1].clone() for p in parts]
    pml.pml_pages_copy(buffer, i32([1]).cuda(), i32([4]).cuda(), i32([1]).cuda())
    assert all(torch.equal(p[:, 4], w) for p, w in zip(parts, want))


def test_refusals():
    buffer, *parts = pml.pml_nvfp4_pages(2, 1, 64)
    x = torch.zeros((3, 1, 64), dtype=BF, device="cuda")
    i, table = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    call = lambda k=x, v=x, pos=i, req=i, p=parts, t=table, **kw: pml.pml_append_nvfp4(k, v, pos, req, *p, t, **kw)  # noqa: E731
    for bad in (dict(k=x.float()), dict(v=x.half()), dict(v=x[:2]), dict(pos=i[:2]), dict(pos=i.float()), dict(req=i[:2]),
                dict(t=table.long()), dict(k=x.repeat(1, 2, 1), v=x.repeat(1, 2, 1)),
                dict(p=[parts[0][..., :16], *parts[1:]]), dict(p=[*parts[:3], parts[3].float()]),
                dict(p=[parts[0].view(torch.int8), *parts[1:]])):
        with pytest.raises(ValueError):
            call(**bad)
    for scale in (0.0, -1.0, 3.0, math.inf, math.nan, 2.0 ** 33, 2.0 ** -33):
        with pytest.raises(pml.PmlError) as e:
            call(k_scale=scale)
        assert e.value.code == 1
    with pytest.raises(pml.PmlError) as e:                 # rows that do not start at 16 bytes
        wide = torch.zeros((2, 64, 1, 40), dtype=torch.uint8, device="cuda")[..., :32]
        call(p=[wide, *parts[1:]])
    assert e.value.code == 3
    out = torch.zeros((2, 64, 1, 64), dtype=BF, device="cuda")
    read = lambda p=parts, t=table, n=i[:1], k=out, v=out, o=table: pml.pml_read_nvfp4(*p, t, n, k, v, o)  # noqa: E731
    for bad in (dict(n=i), dict(k=out.float()), dict(v=out.half()), dict(v=out[:1]), dict(o=table[:, :1]),
                dict(k=out[..., :32]), dict(k=out[:, :32])):
        with pytest.raises(ValueError):
            read(**bad)
    assert (buffer == 0).all() and (out == 0).all()
