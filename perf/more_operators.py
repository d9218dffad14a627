"""Operators over K/V caches held in 4 bits, as cases that can be timed.

A cache is pages of 64 tokens addressed through a block table; a token's head of
``dim`` values is ``dim / 2`` bytes of E2M1 codes (element d in byte d / 2, the
low nibble the even one) and ``dim / 16`` E4M3 scales, one for 16 values, all of
a cache times one power of two:

* ``cache``    -- a step's k and v quantised into their pages, and the requests'
  pages read back in 16 bits;
* ``read``     -- pages read back alone;
* ``attend``   -- attention of new tokens over such caches: single tokens, a few
  drafts, mixed batches, and chunks (which attend over the pages read back);
* ``selected`` -- attention over the positions that a list names.

``run`` computes each in elementary torch operations or, where ``own`` is true,
with the library's kernels.  ``exact`` states the same definitions in 64 bits.
"""
import math
import random

import torch

own = False

PAGE = 64                       # tokens of a page
GROUP = 16                      # values of a scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 requests with short contexts: small, where latency counts
        dict(name="cache_step", op="cache", tokens=64, requests=64, hkv=8, dim=128, dtype="bf16", hi=160,
             k_scale=1.0, v_scale=1.0),
        # a prefill step's chunk of five requests, odd lengths
        dict(name="cache_chunk", op="cache", tokens=8190, requests=5, hkv=8, dim=128, dtype="fp16", hi=2500,
             k_scale=0.5, v_scale=0.0625),
        # the contexts of a few requests read back before a chunk attends to them
        dict(name="read_contexts", op="read", requests=7, hkv=4, dim=64, dtype="bf16", lo=9000, hi=32768,
             k_scale=1.0, v_scale=0.25),
        # one short request: the smallest attention call
        dict(name="attend_one", op="attend", kind="tokens", batch=1, q=1, lo=4000, hi=4000, hq=32, hkv=8, dim=128,
             dtype="bf16", window=0, k=0, k_scale=1.0, v_scale=1.0),
        # the decode batch of this repository's benchmark: 64 requests, U[1024, 32768]
        dict(name="attend_tokens", op="attend", kind="tokens", batch=64, q=1, lo=1024, hi=32768, hq=64, hkv=8,
             dim=128, dtype="bf16", window=0, k=0, k_scale=1.0, v_scale=0.25),
        # four draft tokens a request, groups of seven heads
        dict(name="attend_drafts", op="attend", kind="tokens", batch=31, q=4, lo=300, hi=16000, hq=28, hkv=4,
             dim=128, dtype="fp16", window=0, k=0, k_scale=0.5, v_scale=1.0),
        # a mixed step: short chunks, single tokens, empty requests, a sliding window, groups of five
        dict(name="attend_mixed", op="attend", kind="mixed", batch=48, q=40, lo=1, hi=8000, hq=20, hkv=4, dim=64,
             dtype="fp16", window=1500, k=0, k_scale=1.0, v_scale=1.0),
        # a prefill chunk that ends a long context
        dict(name="attend_chunk", op="attend", kind="chunk", batch=1, q=4096, lo=32768, hi=32768, hq=32, hkv=4,
             dim=128, dtype="bf16", window=0, k=0, k_scale=1.0, v_scale=1.0),
        # the 2048 positions that the indexer selected for each of 64 decode tokens
        dict(name="selected_tokens", op="selected", kind="selected", batch=64, q=1, lo=1024, hi=32768, hq=64, hkv=1,
             dim=128, dtype="bf16", window=0, k=2048, k_scale=1.0, v_scale=1.0),
        # a few tokens over fewer positions, some of the requests shorter than the list
        dict(name="selected_few", op="selected", kind="selected", batch=7, q=1, lo=100, hi=5000, hq=16, hkv=2,
             dim=64, dtype="fp16", window=0, k=500, k_scale=2.0, v_scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache", "cache", "read", "attend", "attend", "attend", "attend", "selected", "selected"])
    case = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), dim=rng.choice([64, 128, 128]),
                k_scale=2.0 ** rng.randint(-4, 2), v_scale=2.0 ** rng.randint(-6, 2))
    if op == "cache":
        requests = _log(rng, 1, 200)
        return dict(case, tokens=max(requests, _log(rng, 1, 9000)), requests=requests,
                    hkv=rng.choice([1, 2, 4, 5, 8]), hi=rng.randint(100, 3000))
    if op == "read":
        hi = _log(rng, 30, 40000)
        return dict(case, requests=max(1, min(_log(rng, 1, 100), 200_000 // hi)), hkv=rng.choice([1, 2, 4, 5, 8]),
                    lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi)
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (40, 8), (28, 4), (64, 1), (20, 4), (8, 1), (24, 2)])
    case.update(batch=1, q=1, lo=1, hi=1, hq=hq, hkv=hkv, window=0, k=0)
    if op == "selected":
        case["k"] = rng.choice([37, 64, 500, 1024, 2048])
        case.update(kind="selected", batch=_log(rng, 1, 200), hi=rng.randint(300, 40000))
        case["batch"] = min(case["batch"], max(1, 4_000_000 // (case["k"] * hkv)),
                            max(1, 8_000_000 // (case["hi"] * hkv)))
        return case
    kind = case["kind"] = rng.choice(["tokens", "tokens", "mixed", "chunk"])
    if kind == "tokens":
        case["hi"] = _log(rng, 40, 40000)
        case["batch"] = min(_log(rng, 1, 100), max(1, 8_000_000 // (case["hi"] * hkv)))
        case["q"] = rng.choice([1, 1, 2, 3, 4])
        case["lo"] = max(1, case["hi"] // rng.choice([1, 4, 32]))
    elif kind == "mixed":
        case.update(batch=rng.randint(2, 60), q=rng.randint(2, 50), hi=rng.randint(300, 5000),
                    window=rng.choice([0, rng.randint(1, 2000)]))
    else:
        case["q"] = _log(rng, 100, 4000)
        case["hi"] = case["lo"] = max(case["q"], _log(rng, 500, 33000))
        case["batch"] = max(1, min(4, 40_000_000 // (case["q"] * case["hi"])))
        if hq * case["batch"] * case["q"] * case["hi"] > 4_000_000_000:
            case.update(hq=28, hkv=4, batch=1)
    return case


def _lengths(case):
    """(new tokens, cached tokens with them) of each request: the same for every seed, up to order."""
    r = random.Random("%s %s %s %s" % (case["kind"], case["batch"], case["lo"], case["hi"]))
    pairs = []
    for _ in range(case["batch"]):
        q, kv = case["q"], r.randint(case["lo"], case["hi"])
        if case["kind"] == "mixed":
            c = r.random()
            q = 0 if c < 0.1 else 1 if c < 0.5 else r.randint(2, case["q"])
            kv = q // 2 if r.random() < 0.1 else max(kv, q)   # now and then rows without a key
        pairs.append((q, kv))
    return pairs


def _starts(case):
    """Length of each request before the call's tokens, and its number of new tokens."""
    r = random.Random("%s %s %s" % (case["tokens"], case["requests"], case["hi"]))
    n, b = case["tokens"], case["requests"]
    new = [n * (i + 1) // b - n * i // b for i in range(b)]
    return [(max(0, r.randint(1, max(1, case["hi"])) - c), c) for c in new]


def _read_lengths(case):
    r = random.Random("%s %s %s" % (case["requests"], case["lo"], case["hi"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["requests"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _put(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(rnd, lengths, spare):
    """A block table over shuffled pages that covers `lengths`, and the pool's number of pages."""
    need = [(n + PAGE - 1) // PAGE for n in lengths]
    pages = sum(need) + spare
    ids = list(range(pages))
    rnd.shuffle(ids)
    width = max(max(need), 1)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return _put(rows), pages


def _out_tables(lengths):
    """The pages that a read fills: as many as the requests have, one after another."""
    need = [(n + PAGE - 1) // PAGE for n in lengths]
    width, rows, at = max(max(need), 1), [], 0
    for n in need:
        rows.append(list(range(at, at + n)) + [0] * (width - n))
        at += n
    return _put(rows), max(at, 1)


def _cache(g, pages, hkv, dim, scale):
    """(codes, scales) of a cache of rows like a layer's keys: normal values, each element of a head
    with a size of its own; the heads of a page one after another, its codes before its scales."""
    # (a million rows, repeated over larger caches, so that they are quick to make)
    n = pages * hkv * PAGE
    few = min(n, 1 << 20)
    size = torch.exp(0.5 * torch.randn(dim, generator=g, device="cuda"))
    x = torch.randn((few, dim), generator=g, device="cuda").mul_(size * scale).bfloat16()
    codes, scales = _quantise(x, scale)
    data = torch.empty((pages, hkv * PAGE * (dim // 2 + dim // GROUP)), dtype=torch.uint8, device="cuda")
    cut = hkv * PAGE * dim // 2
    parts = []
    for part, rows, width in ((data[:, :cut], codes, dim // 2), (data[:, cut:], scales.view(torch.uint8), dim // GROUP)):
        view = part.unflatten(1, (hkv, PAGE, width))
        step = max(1, few // (hkv * PAGE))
        for at in range(0, pages, step):
            end = min(pages, at + step)
            view[at:end] = rows[:(end - at) * hkv * PAGE].view(end - at, hkv, PAGE, width)
        parts.append(view.transpose(1, 2))               # [pages, PAGE, hkv, width]
    return parts


def _stale(parts, table, lens):
    """Slots past a request's end hold what earlier users left there: not numbers, for one."""
    last = torch.arange(PAGE, device="cuda")
    rest = lens % PAGE
    page = table.gather(1, (lens // PAGE).clamp(max=table.shape[1] - 1).long()[:, None])[:, 0].long()
    old = (last >= rest[:, None]) & (rest[:, None] > 0)
    for _, scales in parts:
        scales[page] = torch.where(old[:, :, None, None], 0x7f, scales[page].int()).to(torch.uint8)


def prepare(case, seed):
    if case["op"] == "cache":
        return _prepare_cache(case, seed)
    if case["op"] == "read":
        return _prepare_read(case, seed)
    return _prepare_attend(case, seed)


def _prepare_cache(c, seed):
    g, rnd, dt = _gen(seed), random.Random(seed), DTYPES[c["dtype"]]
    pairs = _starts(c)
    rnd.shuffle(pairs)
    lens = [s + n for s, n in pairs]
    table, pages = _tables(rnd, lens, 3)
    # k and v behind the queries in a projection's rows
    kv = torch.randn((c["tokens"], 2 + 2 * c["hkv"], c["dim"]), generator=g, device="cuda")
    kv[:, 2:2 + c["hkv"]] *= c["k_scale"]
    kv[:, 2 + c["hkv"]:] *= c["v_scale"]
    kv = kv.to(dt)
    kc, vc = (_cache(g, pages, c["hkv"], c["dim"], c[n]) for n in ("k_scale", "v_scale"))
    _stale((kc, vc), table, _put(lens))
    out_table, out_pages = _out_tables(lens)
    out = [torch.zeros((out_pages, PAGE, c["hkv"], c["dim"]), dtype=dt, device="cuda") for _ in range(2)]
    return dict(case=c, k=kv[:, 2:2 + c["hkv"]], v=kv[:, 2 + c["hkv"]:],
                request=_put([b for b, (_, n) in enumerate(pairs) for _ in range(n)]),
                positions=_put([s + i for s, n in pairs for i in range(n)]), k_cache=kc, v_cache=vc, table=table,
                kv_lens=_put(lens), out_table=out_table, k_out=out[0], v_out=out[1])


def _prepare_read(c, seed):
    g, rnd, dt = _gen(seed), random.Random(seed), DTYPES[c["dtype"]]
    lens = _read_lengths(c)
    rnd.shuffle(lens)
    table, pages = _tables(rnd, lens, 3)
    kc, vc = (_cache(g, pages, c["hkv"], c["dim"], c[n]) for n in ("k_scale", "v_scale"))
    _stale((kc, vc), table, _put(lens))
    out_table, out_pages = _out_tables(lens)
    out = [torch.zeros((out_pages, PAGE, c["hkv"], c["dim"]), dtype=dt, device="cuda") for _ in range(2)]
    return dict(case=c, k_cache=kc, v_cache=vc, table=table, kv_lens=_put(lens), out_table=out_table, k_out=out[0],
                v_out=out[1])


def _prepare_attend(c, seed):
    g, rnd, dt = _gen(seed), random.Random(seed), DTYPES[c["dtype"]]
    pairs = _lengths(c)
    rnd.shuffle(pairs)
    qn, kvn = [p[0] for p in pairs], [p[1] for p in pairs]
    table, pages = _tables(rnd, kvn, 2)
    q = torch.randn((sum(qn), c["hq"], c["dim"]), generator=g, device="cuda").div_(c["k_scale"]).to(dt)
    kc, vc = (_cache(g, pages, c["hkv"], c["dim"], c[n]) for n in ("k_scale", "v_scale"))
    kv_lens = _put(kvn)
    _stale((kc, vc), table, kv_lens)
    starts = [0]
    for n in qn:
        starts.append(starts[-1] + n)
    s = dict(case=c, q=q, k_cache=kc, v_cache=vc, table=table, kv_lens=kv_lens, cu_q=_put(starts), max_q=max(qn),
             max_kv=max(kvn), scale=c["dim"] ** -0.5, out=torch.empty_like(q),
             lse=torch.empty(q.shape[:2], dtype=torch.float32, device="cuda"))
    if c["kind"] == "selected":
        # the positions in the order of some score, -1 past a short request's end
        score = torch.rand((len(kvn), max(max(kvn), c["k"])), generator=g, device="cuda")
        score.masked_fill_(torch.arange(score.shape[1], device="cuda") >= kv_lens[:, None], -1.0)
        best, at = score.topk(c["k"], dim=1)
        s["selected"] = torch.where(best >= 0, at, -1).to(torch.int32)
        s["request"] = torch.arange(len(kvn), dtype=torch.int32, device="cuda")
    if c["kind"] == "chunk":
        # the 16-bit pages of the chunk's contexts, which such a program keeps for all layers
        s["out_table"], out_pages = _out_tables(kvn)
        s["k16"], s["v16"] = (torch.zeros((out_pages, PAGE, c["hkv"], c["dim"]), dtype=dt, device="cuda")
                              for _ in range(2))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "cache":
        _plain_append(state)
        return _plain_read(state)
    if c["op"] == "read":
        return _plain_read(state)
    return _plain_attend(c, state)


def _own(c, s):
    import sparse_attention_indexer_logits_gb300 as pml
    parts = (*s["k_cache"], *s["v_cache"])
    scales = dict(k_scale=c["k_scale"], v_scale=c["v_scale"])
    if c["op"] in ("cache", "read"):
        if c["op"] == "cache":
            pml.pml_append_nvfp4(s["k"], s["v"], s["positions"], s["request"], *parts, s["table"], **scales)
        pml.pml_read_nvfp4(*parts, s["table"], s["kv_lens"], s["k_out"], s["v_out"], s["out_table"], **scales)
        return dict(k=s["k_out"], v=s["v_out"])
    if c["kind"] == "selected":
        pml.pml_sparse_attention_nvfp4(s["q"], *parts, s["table"], s["kv_lens"], s["request"], s["selected"],
                                       s["out"], softmax_scale=s["scale"], lse=s["lse"], **scales)
    elif c["kind"] == "chunk":
        pml.pml_read_nvfp4(*parts, s["table"], s["kv_lens"], s["k16"], s["v16"], s["out_table"], **scales)
        pml.pml_paged_attention(s["q"], s["k16"], s["v16"], s["out_table"], s["kv_lens"], s["cu_q"], s["out"],
                                softmax_scale=s["scale"], lse=s["lse"])
    else:
        pml.pml_paged_attention_nvfp4(s["q"], *parts, s["table"], s["kv_lens"], s["cu_q"], s["out"],
                                      softmax_scale=s["scale"], window=c["window"], lse=s["lse"], **scales)
    return dict(out=s["out"], lse=s["lse"])


def _quantise(x, scale):
    """Rows [.., dim] as (codes [.., dim / 2], E4M3 scales [.., dim / 16]): the nearest codes, ties to the
    even one.  (Quotients of 16-bit values by a scale's four bits are never rounded onto a border.)"""
    x = x.float().unflatten(-1, (-1, GROUP))
    s = (x.abs().amax(dim=-1) / (6.0 * scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s.float() * scale)[..., None]
    size = torch.where(d > 0, x.abs() / d, 0.0)
    code = (size > 0.25).to(torch.uint8) + (size >= 0.75) + (size > 1.25) + (size >= 1.75) + (size > 2.5)
    code = code + (size >= 3.5) + (size > 5.0)
    code = (code + 8 * (x < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _values(codes, scales, scale):
    """The values, in 32 bits, that codes [.., dim / 2] and scales [.., dim / 16] stand for."""
    table = torch.tensor([*E2M1, *(-v for v in E2M1)], device="cuda")
    x = table[torch.stack((codes & 15, codes >> 4), dim=-1).int()].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float() * scale
    return (x.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _plain_append(s):
    pos = s["positions"].long()
    page = s["table"][s["request"].long(), pos // PAGE].long()
    for x, (codes, scales), g in ((s["k"], s["k_cache"], "k_scale"), (s["v"], s["v_cache"], "v_scale")):
        new, size = _quantise(x, s["case"][g])
        codes[page, pos % PAGE] = new
        scales[page, pos % PAGE] = size.view(torch.uint8)


def _plain_read(s):
    key = torch.arange(s["table"].shape[1] * PAGE, device="cuda")
    request, at = torch.nonzero(key < s["kv_lens"][:, None], as_tuple=True)
    page, to = (s[t][request, at // PAGE].long() for t in ("table", "out_table"))
    for out, (codes, scales), g in ((s["k_out"], s["k_cache"], "k_scale"), (s["v_out"], s["v_cache"], "v_scale")):
        out[to, at % PAGE] = _values(codes[page, at % PAGE], scales[page, at % PAGE].contiguous(), s["case"][g]).to(out.dtype)
    return dict(k=s["k_out"], v=s["v_out"])


def _softmax_rows(score, allowed, v):
    """Rows [.., keys] of scores over values, and the logarithm of their sums; a row that may look
    at nothing gives 0 and -inf."""
    score.masked_fill_(~allowed, float("-inf"))
    top = score.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    score.sub_(top).exp_()
    total = score.sum(dim=-1)
    out = torch.matmul(score, v) / total.clamp(min=1e-30)[..., None]
    return out, top[..., 0] + total.log()


def _rows_at(s, page, slot, there):
    """k and v [.., heads, keys, dim] in 32 bits of the slots, 0 where `there` is false."""
    return [_values(codes[page, slot], scales[page, slot].contiguous(), s["case"][g])
            .masked_fill_(~there[..., None, None], 0.0).transpose(1, 2)
            for (codes, scales), g in ((s["k_cache"], "k_scale"), (s["v_cache"], "v_scale"))]


def _plain_attend(c, s):
    q, table, kv_lens = s["q"], s["table"], s["kv_lens"].long()
    n, hq, dim = q.shape
    hkv, group = c["hkv"], hq // c["hkv"]
    if c["kind"] == "selected":
        at = s["selected"].long()
        fine = (at >= 0) & (at < kv_lens[s["request"].long()][:, None])
        at = at.clamp(min=0)
        page = table[s["request"].long()[:, None], at // PAGE].long()
        k, v = _rows_at(s, page, at % PAGE, fine)                            # [tokens, hkv, k, dim]
        score = torch.matmul(q.float().view(n, hkv, group, dim), k.transpose(2, 3)) * s["scale"]
        out, lse = _softmax_rows(score, fine[:, None, None, :], v)
        return dict(out=out.reshape(n, hq, dim).to(q.dtype), lse=lse.reshape(n, hq))
    # every request padded to the longest
    max_q, max_kv = s["max_q"], s["max_kv"]
    batch = kv_lens.numel()
    start, count = s["cu_q"][:-1].long(), s["cu_q"].diff().long()
    token = (start[:, None] + torch.arange(max_q, device="cuda")).clamp(max=max(n - 1, 0))
    qp = q[token].float().view(batch, max_q, hkv, group, dim).permute(0, 2, 3, 1, 4)
    key = torch.arange(max_kv, device="cuda")
    there = key[None, :] < kv_lens[:, None]
    page = table[:, key // PAGE].long()
    k, v = _rows_at(s, page, key % PAGE, there)                              # [batch, hkv, keys, dim]
    at = (kv_lens - count)[:, None] + torch.arange(max_q, device="cuda")     # position of each query
    allowed = there[:, None, :] & (key <= at[:, :, None])
    if c["window"]:
        allowed &= key > at[:, :, None] - c["window"]
    score = torch.matmul(qp.reshape(batch, hkv, group * max_q, dim), k.transpose(2, 3)).mul_(s["scale"])
    out, lse = _softmax_rows(score.view(batch, hkv, group, max_q, max_kv), allowed[:, None, None], v[:, :, None])
    # back from the padded rows: token t is query t - start of its request
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    i = t - start[b]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, max_q, hq, dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, max_q, hq)
    return dict(out=out[b, i].to(q.dtype), lse=lse[b, i])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    row = c["dim"] // 2 + c["dim"] // GROUP           # bytes of a row of codes and scales
    if c["op"] in ("cache", "read"):
        lens = [s + n for s, n in _starts(c)] if c["op"] == "cache" else _read_lengths(c)
        rows = 2 * c["hkv"] * sum(lens)               # of k and v
        new = 2 * c["hkv"] * c.get("tokens", 0)
        return {"bytes": rows * (row + 2 * c["dim"]) + new * (row + 2 * c["dim"]) + 8 * c.get("tokens", 0)
                + 8 * sum((n + PAGE - 1) // PAGE for n in lens),
                "flops": (rows + 3 * new) * c["dim"]}
    pairs = _lengths(c)
    queries = sum(q for q, _ in pairs)
    if c["kind"] == "selected":
        keys = pairs_done = sum(min(kv, c["k"]) for _, kv in pairs)
        more = 4 * queries * c["k"]
    else:
        w = c["window"]
        span = lambda q, kv: min(kv, (q - 1 + w) if w else kv) if q else 0  # noqa: E731
        keys = sum(span(q, kv) for q, kv in pairs)
        see = lambda at: max(0, min(at + 1, w) if w else at + 1)  # noqa: E731
        pairs_done = sum(see(kv - q + i) for q, kv in pairs for i in range(q))
        more = 4 * keys // PAGE
    return {"bytes": keys * c["hkv"] * row * 2 + queries * c["hq"] * (4 * c["dim"] + 4) + more,
            "flops": pairs_done * c["hq"] * c["dim"] * 4}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] in ("cache", "read"):
        return _exact_read(c, s)
    return _exact_attend(c, s)


def _numbers(codes, scales, scale):
    """The values of codes and scales from their fields: sign, two exponent bits, one of the mantissa;
    four exponent bits and three of the mantissa."""
    code = torch.stack((codes.remainder(16), codes.div(16, rounding_mode="floor")), dim=-1).flatten(-2).double()
    low = code.remainder(8)
    exponent, mantissa = (low / 2).floor(), low.remainder(2)
    size = torch.where(exponent > 0, torch.exp2(exponent - 1) * (1 + mantissa / 2), mantissa / 2)
    byte = scales.double()
    e, m = (byte / 8).floor(), byte.remainder(8)
    s = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m * 2.0 ** -9)
    return torch.where(code >= 8, -size, size) * s.repeat_interleave(GROUP, dim=-1) * scale


def _rounded(x, scale):
    """What rows become when they are held in 4 bits."""
    x = x.double()
    top = x.unflatten(-1, (-1, GROUP)).abs().max(dim=-1).values / (6 * scale)
    step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -40))).clamp(min=-6) - 3)
    s = (torch.round(top / step) * step).clamp(max=448.0)
    d = (s * scale).repeat_interleave(GROUP, dim=-1)
    y = torch.where(d > 0, x / d, 0.0).clamp(-6.0, 6.0)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return torch.round(y / step) * step * d


def _exact_read(c, s):
    outs = {}
    for name, n in (("k", "k_scale"), ("v", "v_scale")):
        out = s[name + "_out"].double().flatten(0, 1)
        codes, scales = (p.flatten(0, 1) for p in s[name + "_cache"])
        new = _rounded(s[name], c[n]) if c["op"] == "cache" else None
        for b, kv in enumerate(s["kv_lens"].tolist()):
            at = torch.arange(kv, device="cuda")
            here, there = (s[t][b, at.div(PAGE, rounding_mode="floor")].long() * PAGE + at % PAGE
                           for t in ("table", "out_table"))
            rows = _numbers(codes[here], scales[here], c[n])
            if new is not None:
                mine = s["request"] == b
                rows[s["positions"][mine].long()] = new[mine]
            out[there] = rows
        outs[name] = out.view(s[name + "_out"].shape)
    return outs


def _exact_attend(c, s):
    n, hq, dim = s["q"].shape
    hkv, group = c["hkv"], hq // c["hkv"]
    if work(c)["flops"] > 3e12:
        return None
    out = torch.zeros((n, hq, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    starts, lens = s["cu_q"].tolist(), s["kv_lens"].tolist()
    for b, kv in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if hi == lo or kv == 0:
            continue
        at = torch.arange(kv, device="cuda")
        if c["kind"] == "selected":
            at = s["selected"][b].long()
            at = at[(at >= 0) & (at < kv)]
        slots = s["table"][b, torch.div(at, PAGE, rounding_mode="floor")].long() * PAGE + at % PAGE
        k, v = (_numbers(codes.flatten(0, 1)[slots], scales.flatten(0, 1)[slots], c[g])       # [keys, hkv, dim]
                for (codes, scales), g in ((s["k_cache"], "k_scale"), (s["v_cache"], "v_scale")))
        here = torch.arange(kv - (hi - lo), kv, device="cuda").unsqueeze(1)
        hidden = (at > here) | ((at <= here - c["window"]) if c["window"] else (at < 0))
        heads = max(1, min(group, 2 ** 29 // max(1, (hi - lo) * at.numel())))
        for h in [h for j in range(hkv) for h in range(j * group, (j + 1) * group, heads)]:
            j = h // group
            end = min(h + heads, (j + 1) * group)
            logit = torch.einsum("qhd,kd->hqk", s["q"][lo:hi, h:end].double(), k[:, j]) * s["scale"]
            if c["kind"] != "selected":
                logit.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(logit, dim=2)
            p = torch.exp(logit - z.clamp(min=-1e300).unsqueeze(2))
            out[lo:hi, h:end], lse[lo:hi, h:end] = (p @ v[:, j]).transpose(0, 1), z.T
    return dict(out=out, lse=lse)
