"""The serving operators around the paged indexer, as cases that can be timed.

Five operators share 64-token pages addressed through a block table:

* ``rope``    -- rotary positions of ``[tokens, heads, dim]`` and their gradient;
* ``append``  -- rotary positions of q and k, with k and v written into the
  pages of a bf16 / fp16 cache;
* ``index``   -- the indexer's inputs: q and k rotated and quantised to e4m3,
  the keys written into the fp8 cache that ``pml_fp8_paged_mqa_logits`` reads;
* ``attend``  -- attention of new tokens over a paged cache: single tokens,
  chunks, mixed batches, or the positions a top-k selected;
* ``pages``   -- forking requests (shared pages, the last one copied), freeing
  them, and compacting the pool.

``run`` computes each in elementary torch operations or, where ``own`` is
true, with the library's kernels.  ``exact`` states the same definitions in 64
bits, token by token or request by request.
"""
import math
import random

import torch

own = False

PAGE = 64                       # tokens of a page
FP8_BLOCK = PAGE * 128 + PAGE * 4   # bytes of an fp8 block: 64 keys, then 64 fp32 scales
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a training step's rotation of the queries, heads wholly rotated
        dict(name="rope_train", op="rope", tokens=16384, heads=32, dim=128, rot=128, offset=0,
             interleaved=False, dtype="bf16", gradient=False, scaled=False, top=16384),
        # its gradient in fp32, frequencies stretched for a long context, odd sizes
        dict(name="rope_grad_long", op="rope", tokens=4099, heads=24, dim=96, rot=80, offset=16,
             interleaved=True, dtype="fp32", gradient=True, scaled=True, top=1000000),
        # one decode step of 64 requests: a small call, where latency counts
        dict(name="append_decode", op="append", tokens=64, requests=64, hq=32, hkv=8, dim=128,
             rot=128, offset=0, interleaved=False, dtype="bf16", hi=2048),
        # a prefill step's chunk, part of each head rotated
        dict(name="append_chunk", op="append", tokens=8190, requests=5, hq=64, hkv=8, dim=128,
             rot=64, offset=64, interleaved=True, dtype="fp16", hi=2500),
        # the indexer's side of a decode step with two tokens for each request
        dict(name="index_decode", op="index", tokens=128, requests=64, heads=64, rot=64, offset=0,
             interleaved=True, hi=2048),
        # the indexer's side of a prefill step
        dict(name="index_chunk", op="index", tokens=8192, requests=4, heads=64, rot=64, offset=64,
             interleaved=False, hi=2600),
        # the decode batch of this repository's benchmark: 64 requests, U[1024, 32768]
        dict(name="attend_decode", op="attend", kind="tokens", batch=64, q=1, lo=1024, hi=32768,
             hq=64, hkv=8, dim=128, dtype="bf16", window=0, k=0),
        # a prefill chunk that ends a long context
        dict(name="attend_chunk", op="attend", kind="chunk", batch=1, q=4096, lo=32768, hi=32768,
             hq=32, hkv=4, dim=128, dtype="bf16", window=0, k=0),
        # a mixed step: chunks, single tokens, empty requests, a sliding window, groups of five
        dict(name="attend_mixed", op="attend", kind="mixed", batch=24, q=500, lo=1, hi=8000, hq=20,
             hkv=4, dim=64, dtype="fp16", window=1500, k=0),
        # the 2048 positions that the indexer selected for each of 64 decode tokens
        dict(name="attend_selected", op="attend", kind="selected", batch=64, q=1, lo=1024, hi=32768,
             hq=64, hkv=1, dim=128, dtype="bf16", window=0, k=2048),
        # parallel samples: requests forked, their last pages copied, then freed
        dict(name="pages_fork", op="pages", kind="fork", requests=96, forks=160, hi=8192,
             page_elems=PAGE * 4 * 128, layers=2, used=0.6),
        # a pool that has run for long, its live pages moved to the front
        dict(name="pages_compact", op="pages", kind="compact", requests=64, forks=0, hi=8192,
             page_elems=PAGE * 4 * 128, layers=4, used=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "index", "attend", "attend", "attend", "pages"])
    if op == "rope":
        dim = rng.choice([64, 72, 96, 128, 192, 256])
        rot = rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)])
        heads = rng.randint(1, 64)
        tokens = min(_log(rng, 1, 30000), 60_000_000 // (heads * dim))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=rot,
                    offset=rng.choice([0, dim - rot]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), gradient=rng.random() < 0.5,
                    scaled=rng.random() < 0.5, top=_log(rng, 2000, 2000000))
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        requests = _log(rng, 1, 200)
        dim = rng.choice([64, 128])
        rot = rng.choice([dim, dim // 2])
        return dict(op=op, tokens=max(requests, _log(rng, 1, 9000)), requests=requests,
                    hq=hkv * rng.randint(1, 8), hkv=hkv, dim=dim, rot=rot,
                    offset=rng.choice([0, dim - rot]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16"]), hi=rng.randint(500, 3000))
    if op == "index":
        requests = _log(rng, 1, 200)
        return dict(op=op, tokens=max(requests, _log(rng, 1, 8500)), requests=requests,
                    heads=rng.choice([8, 16, 32, 64]), rot=rng.choice([32, 64, 128]), offset=0,
                    interleaved=rng.random() < 0.5, hi=rng.randint(500, 3000))
    if op == "pages":
        kind = rng.choice(["fork", "compact"])
        requests = rng.randint(4, 120)
        return dict(op=op, kind=kind, requests=requests,
                    forks=_log(rng, 1, 300) if kind == "fork" else 0, hi=_log(rng, 200, 9000),
                    page_elems=PAGE * rng.choice([1, 2, 4]) * rng.choice([64, 128]),
                    layers=rng.randint(1, 3), used=rng.uniform(0.3, 0.8))
    kind = rng.choice(["tokens", "chunk", "mixed", "selected"])
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (40, 8), (28, 4), (64, 1), (20, 4), (8, 1)])
    case = dict(op=op, kind=kind, batch=1, q=1, lo=1, hi=1, hq=hq, hkv=hkv,
                dim=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                window=0, k=0)
    if kind == "tokens":
        case["hi"] = _log(rng, 40, 40000)
        case["batch"] = min(_log(rng, 1, 100), max(1, 8_000_000 // (case["hi"] * hkv)))
        case["q"] = rng.choice([1, 1, 2, 4])
        case["lo"] = max(1, case["hi"] // rng.choice([1, 4, 32]))
    elif kind == "chunk":
        case["q"] = _log(rng, 16, 4000)
        case["hi"] = case["lo"] = max(case["q"], _log(rng, 500, 33000))
        case["batch"] = max(1, min(4, 40_000_000 // (case["q"] * case["hi"])))
        if hq * case["batch"] * case["q"] * case["hi"] > 4_000_000_000:
            case.update(hq=28, hkv=4, batch=1)
    elif kind == "mixed":
        case.update(batch=rng.randint(2, 30), q=rng.randint(2, 400), hi=rng.randint(300, 5000),
                    window=rng.choice([0, rng.randint(1, 2000)]))
    else:
        case["k"] = rng.choice([64, 500, 1024, 2048])
        case.update(batch=_log(rng, 1, 200), hi=rng.randint(300, 40000))
        case["batch"] = min(case["batch"], max(1, 4_000_000 // (case["k"] * hkv)),
                            max(1, 8_000_000 // (case["hi"] * hkv)))
    return case


def _lengths(case):
    """(new tokens, cached tokens with them) of each request: the same for every seed, up to order."""
    r = random.Random("%s %s %s %s" % (case.get("kind"), case["batch"], case["lo"], case["hi"]))
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


def _page_lengths(case):
    r = random.Random("%s %s" % (case["requests"], case["hi"]))
    return [r.randint(1, case["hi"]) for _ in range(case["requests"])]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _frequencies(rot, scaled):
    """Radians per position of each pair of a head: a geometric series or, stretched for a context
    `factor` times longer, slow pairs divided by `factor`, fast ones kept, a ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = torch.pow(10000.0, -2.0 * i / rot)
    if not scaled:
        return f, 1.0
    factor, context = 32.0, 4096.0
    turns = context * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0


def _tables(rnd, lengths, spare, width=None):
    """A block table over shuffled pages that covers `lengths`, and the pool's number of pages."""
    need = [(n + PAGE - 1) // PAGE for n in lengths]
    pages = sum(need) + spare
    ids = list(range(pages))
    rnd.shuffle(ids)
    width = width or max(max(need), 1)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), pages


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "index": _prepare_index,
            "attend": _prepare_attend, "pages": _prepare_pages}[case["op"]](case, seed)


def _prepare_rope(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    # heads of a wider projection's rows, as a fused q/k/v product leaves them
    x = _normal(g, (c["tokens"], c["heads"] + 8, c["dim"]), dt)[:, :c["heads"]]
    freq, mscale = _frequencies(c["rot"], c["scaled"])
    pos = torch.randint(0, c["top"], (c["tokens"],), generator=g, device="cuda")
    out = torch.empty((c["tokens"], c["heads"], c["dim"]), dtype=dt, device="cuda")
    return dict(case=c, x=x, positions=pos, inv_freq=freq, mscale=mscale, out=out)


def _token_places(c, rnd):
    """(request, position) of each token, requests in a shuffled order, and their final lengths."""
    pairs = _starts(c)
    rnd.shuffle(pairs)
    req = [b for b, (_, n) in enumerate(pairs) for _ in range(n)]
    pos = [s + i for s, n in pairs for i in range(n)]
    put = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return put(req), put(pos), [s + n for s, n in pairs]


def _prepare_append(c, seed):
    g, rnd, dt = _gen(seed), random.Random(seed), DTYPES[c["dtype"]]
    req, pos, lens = _token_places(c, rnd)
    table, pages = _tables(rnd, lens, 3)
    qkv = _normal(g, (c["tokens"], c["hq"] + 2 * c["hkv"], c["dim"]), dt)
    cache = [_normal(g, (pages, PAGE, c["hkv"], c["dim"]), dt) for _ in range(2)]
    freq, _ = _frequencies(c["rot"], False)
    return dict(case=c, q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]],
                v=qkv[:, c["hq"] + c["hkv"]:], positions=pos, request=req, inv_freq=freq,
                k_cache=cache[0], v_cache=cache[1], table=table,
                q_out=torch.empty((c["tokens"], c["hq"], c["dim"]), dtype=dt, device="cuda"))


def _prepare_index(c, seed):
    g, rnd = _gen(seed), random.Random(seed)
    req, pos, lens = _token_places(c, rnd)
    table, pages = _tables(rnd, lens, 3)
    kv = torch.zeros((pages, FP8_BLOCK), dtype=torch.uint8, device="cuda")
    kv[:, :PAGE * 128] = _normal(g, (pages, PAGE * 128), torch.float32, 50.0).to(torch.float8_e4m3fn).view(torch.uint8)
    kv[:, PAGE * 128:] = torch.rand((pages, PAGE), generator=g, device="cuda").view(torch.uint8)
    freq, _ = _frequencies(c["rot"], False)
    n, h = c["tokens"], c["heads"]
    return dict(case=c, q=_normal(g, (n, h, 128), torch.bfloat16), k=_normal(g, (n, 128), torch.bfloat16),
                weights=_normal(g, (n, h), torch.float32), weight_scale=(128.0 * h) ** -0.5,
                positions=pos, request=req, inv_freq=freq, kv_fused=kv, table=table,
                q_out=torch.empty((n, h, 128), dtype=torch.float8_e4m3fn, device="cuda"),
                w_out=torch.empty((n, h), dtype=torch.float32, device="cuda"))


def _prepare_attend(c, seed):
    g, rnd, dt = _gen(seed), random.Random(seed), DTYPES[c["dtype"]]
    pairs = _lengths(c)
    rnd.shuffle(pairs)
    qn, kvn = [p[0] for p in pairs], [p[1] for p in pairs]
    table, pages = _tables(rnd, kvn, 2)
    q = _normal(g, (sum(qn), c["hq"], c["dim"]), dt, 1.5)
    k, v = (_normal(g, (pages, PAGE, c["hkv"], c["dim"]), dt) for _ in range(2))
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kv_lens = put(kvn)
    # slots past a request's end hold what earlier users left there: not numbers, for one
    last = torch.arange(PAGE, device="cuda")
    for cache in (k, v):
        part = kv_lens % PAGE
        page = table.gather(1, (kv_lens // PAGE).clamp(max=table.shape[1] - 1).long()[:, None])[:, 0].long()
        stale = (last >= part[:, None]) & (part[:, None] > 0)
        cache[page] = torch.where(stale[:, :, None, None], float("nan"), cache[page])
    starts = [0]
    for n in qn:
        starts.append(starts[-1] + n)
    s = dict(case=c, q=q, k_cache=k, v_cache=v, table=table, kv_lens=kv_lens, cu_q=put(starts),
             max_q=max(qn), max_kv=max(kvn), scale=c["dim"] ** -0.5,
             out=torch.empty_like(q), lse=torch.empty(q.shape[:2], dtype=torch.float32, device="cuda"))
    if c["kind"] == "selected":
        # the positions in the order of some score, -1 past a short request's end
        score = torch.rand((len(kvn), max(max(kvn), c["k"])), generator=g, device="cuda")
        score.masked_fill_(torch.arange(score.shape[1], device="cuda") >= kv_lens[:, None], -1.0)
        best, at = score.topk(c["k"], dim=1)
        s["selected"] = torch.where(best >= 0, at, -1).to(torch.int32)
        s["request"] = torch.arange(len(kvn), dtype=torch.int32, device="cuda")
    return s


def _prepare_pages(c, seed):
    g, rnd = _gen(seed), random.Random(seed)
    lens = _page_lengths(c)
    rnd.shuffle(lens)
    live = sum((n + PAGE - 1) // PAGE for n in lens)
    spare = max(int(live / c["used"]) - live, c["forks"] + 1)
    table, pages = _tables(rnd, lens + [0] * c["forks"], spare, max(lens) // PAGE + 2)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    used = torch.arange(table.shape[1], device="cuda") < torch.tensor(
        [(n + PAGE - 1) // PAGE for n in lens] + [0] * c["forks"], device="cuda")[:, None]
    refs[table[used].long()] = 1
    cache = torch.randn((c["layers"], pages, c["page_elems"]), generator=g, device="cuda", dtype=torch.bfloat16)
    put = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=c, refs=refs, table=table, lens=put(lens + [0] * c["forks"]), cache=cache)
    room = c["forks"] if c["kind"] == "fork" else (pages + 1) // 2
    for name in ("src", "dst"):
        s[name] = torch.full((room,), -1, dtype=torch.int32, device="cuda")
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["kind"] == "fork":
        s["parents"] = put([rnd.randrange(c["requests"]) for _ in range(c["forks"])])
        s["children"] = put([c["requests"] + i for i in range(c["forks"])])
    else:
        s["refs_out"], s["table_out"] = torch.empty_like(refs), torch.empty_like(table)
        s["remap"] = torch.empty_like(refs)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"rope": _plain_rope, "append": _plain_append, "index": _plain_index,
            "attend": _plain_attend, "pages": _plain_pages}[c["op"]](c, state)


def _own(c, s):
    import sparse_attention_indexer_logits_gb300 as pml
    if c["op"] == "rope":
        return pml.pml_rope(s["x"], s["positions"], s["inv_freq"], s["out"], rot_offset=c["offset"],
                            interleaved=c["interleaved"], mscale=s["mscale"], gradient=c["gradient"])
    if c["op"] == "append":
        pml.pml_rope_append(s["q"], s["k"], s["v"], s["positions"], s["request"], s["inv_freq"],
                            s["k_cache"], s["v_cache"], s["table"], s["q_out"],
                            rot_offset=c["offset"], interleaved=c["interleaved"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if c["op"] == "index":
        pml.pml_index_quant_append(s["q"], s["k"], s["weights"], s["positions"], s["request"],
                                   s["inv_freq"], s["kv_fused"], s["table"], s["q_out"], s["w_out"],
                                   weight_scale=s["weight_scale"], rot_offset=c["offset"],
                                   interleaved=c["interleaved"])
        return _index_outputs(s["q_out"], s["w_out"], s["kv_fused"])
    if c["op"] == "attend":
        if c["kind"] == "selected":
            pml.pml_sparse_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                                     s["request"], s["selected"], s["out"], softmax_scale=s["scale"],
                                     lse=s["lse"])
        else:
            pml.pml_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                                    s["cu_q"], s["out"], softmax_scale=s["scale"], causal=True,
                                    window=c["window"], lse=s["lse"])
        return dict(out=s["out"], lse=s["lse"])
    if c["kind"] == "fork":
        pml.pml_pages_fork(s["refs"], s["table"], s["lens"], s["parents"], s["children"], s["src"],
                           s["dst"], s["count"])
        pml.pml_pages_copy(s["cache"], s["src"], s["dst"], s["count"])
        pml.pml_pages_free(s["refs"], s["table"], s["lens"], s["children"])
        return _pages_outputs(s, s["refs"], s["table"])
    pml.pml_pages_compact(s["refs"], s["table"], s["lens"], s["refs_out"], s["table_out"], s["remap"],
                          s["src"], s["dst"], s["count"])
    pml.pml_pages_copy(s["cache"], s["src"], s["dst"], s["count"])
    return dict(_pages_outputs(s, s["refs_out"], s["table_out"]), remap=s["remap"])


def _index_outputs(q, w, kv):
    return dict(q=q, weights=w, keys=kv[:, :PAGE * 128].view(torch.float8_e4m3fn),
                scales=kv[:, PAGE * 128:].view(torch.float32))


def _pages_outputs(s, refs, table):
    return dict(src=s["src"], dst=s["dst"], count=s["count"], refs=refs, table=table, lens=s["lens"],
                cache=s["cache"].view(torch.int16))


def _rotate(x, positions, inv_freq, offset, interleaved, mscale=1.0, gradient=False):
    """x [tokens, heads, dim] in 32 bits, its pairs turned by position * frequency."""
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq[None, :]
    cos, sin = ((f(angle) * mscale).float()[:, None, :] for f in (torch.cos, torch.sin))
    if gradient:
        sin = -sin
    x = x.float()
    y = x.clone()
    part = x[..., offset:offset + rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        y[..., offset:offset + rot:2] = a * cos - b * sin
        y[..., offset + 1:offset + rot:2] = b * cos + a * sin
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        y[..., offset:offset + rot // 2] = a * cos - b * sin
        y[..., offset + rot // 2:offset + rot] = b * cos + a * sin
    return y


def _plain_rope(c, s):
    return _rotate(s["x"], s["positions"], s["inv_freq"], c["offset"], c["interleaved"], s["mscale"],
                   c["gradient"]).to(s["x"].dtype)


def _plain_append(c, s):
    q, k = (_rotate(s[n], s["positions"], s["inv_freq"], c["offset"], c["interleaved"]).to(s[n].dtype)
            for n in ("q", "k"))
    pos = s["positions"].long()
    page = s["table"][s["request"].long(), pos // PAGE].long()
    s["k_cache"][page, pos % PAGE] = k
    s["v_cache"][page, pos % PAGE] = s["v"]
    return dict(q=q, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _quantise(x):
    """e4m3 codes and scales of rows: the largest magnitude of a row becomes 448."""
    scale = x.abs().amax(dim=-1).clamp(min=1e-12) / 448.0
    return (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _plain_index(c, s):
    q, qs = _quantise(_rotate(s["q"], s["positions"], s["inv_freq"], c["offset"], c["interleaved"]))
    k, ks = _quantise(_rotate(s["k"][:, None], s["positions"], s["inv_freq"], c["offset"], c["interleaved"])[:, 0])
    pos = s["positions"].long()
    page = s["table"][s["request"].long(), pos // PAGE].long()
    keys = s["kv_fused"][:, :PAGE * 128].view(-1, PAGE, 128)
    keys[page, pos % PAGE] = k.view(torch.uint8)
    s["kv_fused"][:, PAGE * 128:].view(torch.float32)[page, pos % PAGE] = ks
    return _index_outputs(q, s["weights"] * qs * s["weight_scale"], s["kv_fused"])


def _softmax_rows(score, allowed, v):
    """Rows [.., keys] of scores over values, and the logarithm of their sums; a row that may look
    at nothing gives 0 and -inf."""
    score.masked_fill_(~allowed, float("-inf"))
    top = score.amax(dim=-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    score.sub_(top).exp_()
    total = score.sum(dim=-1)
    out = torch.matmul(score, v) / total.clamp(min=1e-30)[..., None]
    return out, top[..., 0] + total.log()


def _plain_attend(c, s):
    q, table, kv_lens = s["q"], s["table"], s["kv_lens"].long()
    n, hq, dim = q.shape
    hkv, group = c["hkv"], hq // c["hkv"]
    if c["kind"] == "selected":
        at = s["selected"].long()
        fine = (at >= 0) & (at < kv_lens[s["request"].long()][:, None])
        at = at.clamp(min=0)
        page = table[s["request"].long()[:, None], at // PAGE].long()
        k, v = (s[x][page, at % PAGE].float().masked_fill_(~fine[:, :, None, None], 0.0).transpose(1, 2)
                for x in ("k_cache", "v_cache"))                        # [tokens, hkv, k, dim]
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
    k, v = (s[x][page, key % PAGE].float().masked_fill_(~there[:, :, None, None], 0.0).transpose(1, 2)
            for x in ("k_cache", "v_cache"))                            # [batch, hkv, keys, dim]
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


def _copy_pages(s):
    ok = s["src"] >= 0
    s["cache"][:, s["dst"][ok].long()] = s["cache"][:, s["src"][ok].long()]


def _first(values, keep, room):
    """The kept values in order, then -1."""
    got = torch.full((room,), -1, dtype=torch.int32, device="cuda")
    kept = values[keep]
    got[:kept.numel()] = kept.to(torch.int32)
    return got


def _plain_pages(c, s):
    refs, table, lens = s["refs"], s["table"], s["lens"]
    col = torch.arange(table.shape[1], device="cuda")
    if c["kind"] == "compact":
        ids = torch.arange(refs.numel(), device="cuda")
        live = refs > 0
        total = live.sum()
        src, dst = ids[live & (ids >= total)], ids[~live & (ids < total)]
        remap = torch.where(live, ids, -1)
        remap[src] = dst
        s["refs_out"].zero_()
        s["refs_out"][remap[live]] = refs[live]
        used = col < ((lens + PAGE - 1) // PAGE)[:, None]
        s["table_out"].copy_(torch.where(used, remap[table.long()].to(torch.int32), table))
        s["remap"].copy_(remap)
        room = s["src"].numel()
        s["src"].copy_(_first(src, slice(None), room))
        s["dst"].copy_(_first(dst, slice(None), room))
        s["count"].fill_(src.numel())
        _copy_pages(s)
        return dict(_pages_outputs(s, s["refs_out"], s["table_out"]), remap=s["remap"])
    parents, children = s["parents"].long(), s["children"].long()
    # fork: full pages shared, a part page replaced by the lowest free page
    n = lens[parents]
    full, part = n // PAGE, n % PAGE > 0
    free = torch.argsort(refs > 0, stable=True)
    rank = (part.cumsum(0) - 1).clamp(min=0)
    new = free[rank].to(torch.int32)
    ok = ~part | (rank < (refs == 0).sum())
    rows = table[parents]
    shared = (col < full[:, None]) & ok[:, None]
    mine = (col == full[:, None]) & (part & ok)[:, None]
    old = rows.gather(1, full.long()[:, None])[:, 0]
    table[children] = torch.where(shared, rows, torch.where(mine, new[:, None], table[children]))
    lens[children] = torch.where(ok, n, 0)
    refs.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    copied = part & ok
    refs[new[copied].long()] = 1
    s["src"].copy_(_first(old, copied, len(old)))
    s["dst"].copy_(_first(new, copied, len(new)))
    s["count"].copy_(copied.sum())
    _copy_pages(s)
    # free the children again
    used = col < ((lens[children] + PAGE - 1) // PAGE)[:, None]
    gone = table[children][used]
    refs.index_add_(0, gone.long(), -torch.ones_like(gone))
    lens[children] = 0
    return _pages_outputs(s, refs, table)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}.get(c.get("dtype"), 2)
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        return {"bytes": 2 * n * size + 8 * c["tokens"], "flops": 3 * n}
    if c["op"] == "append":
        n = c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["dim"]
        return {"bytes": 2 * n * size + 12 * c["tokens"], "flops": 3 * n}
    if c["op"] == "index":
        rows = c["tokens"] * (c["heads"] + 1)
        return {"bytes": rows * (128 * 3 + 8) + 12 * c["tokens"], "flops": rows * 128 * 5}
    if c["op"] == "pages":
        lens = _page_lengths(c)
        live = sum((n + PAGE - 1) // PAGE for n in lens)
        width = max(lens) // PAGE + 2
        spare = max(int(live / c["used"]) - live, c["forks"] + 1)
        page = c["page_elems"] * 2 * c["layers"]
        if c["kind"] == "fork":
            return {"bytes": c["forks"] * (2 * page + 12 * width) + 8 * (live + spare), "flops": 0}
        moved = live * spare // (live + spare)
        return {"bytes": moved * 2 * page + 8 * c["requests"] * width + 12 * (live + spare), "flops": 0}
    pairs = _lengths(c)
    row = c["dim"] * size
    queries = sum(q for q, _ in pairs)
    if c["kind"] == "selected":
        keys = sum(min(kv, c["k"]) for _, kv in pairs)
        pairs_done = keys
        more = 4 * queries * c["k"]
    else:
        w = c["window"]
        span = lambda q, kv: min(kv, (q - 1 + w) if w else kv) if q else 0  # noqa: E731
        keys = sum(span(q, kv) for q, kv in pairs)
        see = lambda at: max(0, min(at + 1, w) if w else at + 1)  # noqa: E731
        pairs_done = sum(see(kv - q + i) for q, kv in pairs for i in range(q))
        more = 4 * keys // PAGE
    return {"bytes": keys * c["hkv"] * row * 2 + queries * c["hq"] * (2 * row + 4) + more,
            "flops": pairs_done * c["hq"] * c["dim"] * 4}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "index": _exact_index,
            "attend": _exact_attend}[c["op"]](c, s)


def _turned(x, positions, inv_freq, offset, interleaved, mscale=1.0, sign=1.0):
    """Each pair as a complex number times mscale * e^(i position frequency)."""
    y, half = x.double().clone(), inv_freq.numel()
    turn = torch.polar(torch.full((), mscale, dtype=torch.float64, device="cuda"),
                       sign * positions.double().unsqueeze(1) * inv_freq).unsqueeze(1)
    part = y[..., offset:offset + 2 * half]
    pair = part.unflatten(-1, (half, 2)) if interleaved else part.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    y[..., offset:offset + 2 * half] = (z if interleaved else z.transpose(-1, -2)).flatten(-2)
    return y


def _exact_rope(c, s):
    return _turned(s["x"], s["positions"], s["inv_freq"], c["offset"], c["interleaved"], s["mscale"],
                   -1.0 if c["gradient"] else 1.0)


def _slots(s):
    pos = s["positions"].long()
    return s["table"][s["request"].long(), pos.div(PAGE, rounding_mode="floor")].long() * PAGE + pos % PAGE


def _exact_append(c, s):
    q, k = (_turned(s[n], s["positions"], s["inv_freq"], c["offset"], c["interleaved"]) for n in ("q", "k"))
    caches = []
    for cache, new in ((s["k_cache"], k), (s["v_cache"], s["v"].double())):
        flat = cache.double().flatten(0, 1)
        flat[_slots(s)] = new
        caches.append(flat.view(cache.shape))
    return dict(q=q, k_cache=caches[0], v_cache=caches[1])


def _exact_index(c, s):
    q = _turned(s["q"], s["positions"], s["inv_freq"], c["offset"], c["interleaved"])
    k = _turned(s["k"].unsqueeze(1), s["positions"], s["inv_freq"], c["offset"], c["interleaved"]).squeeze(1)
    qs, ks = (x.abs().max(dim=-1).values / 448.0 for x in (q, k))
    old = _index_outputs(None, None, s["kv_fused"])
    keys, scales = old["keys"].double().view(-1, 128), old["scales"].double().flatten()
    keys[_slots(s)] = k / ks[:, None]
    scales[_slots(s)] = ks
    return dict(q=q / qs[..., None], weights=s["weights"].double() * qs * s["weight_scale"],
                keys=keys.view(old["keys"].shape), scales=scales.view(old["scales"].shape))


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
        k, v = (s[x].flatten(0, 1)[slots].double() for x in ("k_cache", "v_cache"))   # [keys, hkv, dim]
        here = torch.arange(kv - (hi - lo), kv, device="cuda").unsqueeze(1)
        hidden = (at > here) | ((at <= here - c["window"]) if c["window"] else (at < 0))
        for h in range(hq):
            logit = (s["q"][lo:hi, h].double() @ k[:, h // group].T) * s["scale"]
            if c["kind"] != "selected":
                logit[hidden] = -math.inf
            z = torch.logsumexp(logit, dim=1)
            p = torch.exp(logit - z.clamp(min=-1e300).unsqueeze(1))
            out[lo:hi, h], lse[lo:hi, h] = p @ v[:, h // group], z
    return dict(out=out, lse=lse)
