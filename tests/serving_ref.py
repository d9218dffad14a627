"""Plain 64-bit definitions of the serving operators, for the GPU tests, and
the pool bookkeeping in loops."""
from __future__ import annotations

import math

import torch

PAGE = 64


def gen(seed: int) -> torch.Generator:
    return torch.Generator(device="cpu").manual_seed(seed)


def rope(x, positions, inv_freq, offset=0, interleaved=False, mscale=1.0, gradient=False):
    """(rotated x, |a| + |b| of each element's pair), in float64."""
    y = x.double().clone()
    size = y.abs()
    rot = 2 * inv_freq.numel()
    t = positions.double()[:, None] * inv_freq.double()[None, :]
    cos, sin = (mscale * torch.cos(t))[:, None], (mscale * torch.sin(t))[:, None]
    if gradient:
        sin = -sin
    part = y[..., offset:offset + rot]
    if interleaved:
        sel = [(slice(0, None, 2)), (slice(1, None, 2))]
    else:
        sel = [slice(0, rot // 2), slice(rot // 2, rot)]
    a, b = part[..., sel[0]].clone(), part[..., sel[1]].clone()
    part[..., sel[0]] = a * cos - b * sin
    part[..., sel[1]] = b * cos + a * sin
    mag = size[..., offset:offset + rot]
    total = mscale * (a.abs() + b.abs())
    mag[..., sel[0]] = total
    mag[..., sel[1]] = total
    return y, size


# cosine and sine are off by at most 2^-26 of a turn (9.4e-8 radians) plus two
# ulps of sincospif and the product with mscale (2^-23 + 2^-24 of one), and a
# product, a fused product and sum round twice more: 4.5e-7 of |a| + |b|
ROPE_REL = 4.5e-7


def rope_bound(y, size, dtype):
    return ROPE_REL * size + (torch.finfo(dtype).eps / 2) * (y.abs() + ROPE_REL * size) + \
        torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def block_table(lens, g, spare=2, width=None):
    """A table over shuffled pages, and the number of pages."""
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=g).tolist()
    width = width or max(need + [1])
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32).reshape(len(lens), width), pages


def attention(q, k, v, allowed, scale):
    """q [rows, dim], k and v [keys, dim], allowed [rows, keys]: output, log of
    the sum, and the weighted magnitudes sum_j p_j |v_j| that errors scale with."""
    s = (q.double() @ k.double().T) * scale
    s = s.masked_fill(~allowed, -math.inf)
    if s.shape[1] == 0:
        s = torch.full((s.shape[0], 1), -math.inf, dtype=torch.float64)
        v, allowed = torch.zeros((1, v.shape[1])), torch.zeros((s.shape[0], 1), dtype=torch.bool)
    top = s.amax(1).clamp(min=-1e300)
    e = torch.exp(s - top[:, None])
    total = e.sum(1)
    lse = top + total.log()
    p = e / total.clamp(min=1e-300)[:, None]
    vv = torch.where(allowed.any(0)[:, None], v.double(), 0.0)
    # a masked key contributes nothing, whatever its value holds
    bad = ~torch.isfinite(vv)
    out = p @ vv.masked_fill(bad, 0.0)
    mag = p @ vv.masked_fill(bad, 0.0).abs()
    if bad.any():
        for j in torch.nonzero(bad.any(1))[:, 0].tolist():
            rows = allowed[:, j]
            out[rows] += (p[rows, j][:, None] * v[j].double()[None, :]).masked_fill(~bad[j], 0.0)
    return out, lse, mag


class Pool:
    """The pages' bookkeeping in plain loops (lists of ints)."""

    def __init__(self, refs, table, lens):
        self.refs, self.table, self.lens = list(refs), [list(r) for r in table], list(lens)

    def free_pages(self):
        return [p for p, c in enumerate(self.refs) if c == 0]

    def fork(self, parents, children):
        free, moves = self.free_pages(), []
        failed = False
        for a, b in zip(parents, children):
            n = self.lens[a]
            full, part = n // PAGE, n % PAGE > 0
            if part and (failed or not free):
                failed = True
                self.lens[b] = 0
                continue
            for c in range(full):
                self.table[b][c] = self.table[a][c]
                self.refs[self.table[a][c]] += 1
            if part:
                p = free.pop(0)
                moves.append((self.table[a][full], p))
                self.table[b][full] = p
                self.refs[p] = 1
            self.lens[b] = n
        return moves

    def extend(self, want, capacity):
        free = self.free_pages()[:capacity]
        taken, failed = [], False
        for i, n in enumerate(want):
            have = -(-self.lens[i] // PAGE)
            need = max(0, -(-n // PAGE) - have)
            if -(-n // PAGE) > len(self.table[i]):
                continue
            if need:
                if failed or need > len(free):
                    failed = True
                    continue
                for c in range(need):
                    p = free.pop(0)
                    self.table[i][have + c] = p
                    self.refs[p] = 1
                    taken.append(p)
            self.lens[i] = max(self.lens[i], n)
        return taken

    def free(self, rows):
        for b in rows:
            for c in range(-(-self.lens[b] // PAGE)):
                self.refs[self.table[b][c]] -= 1
            self.lens[b] = 0

    def compact(self):
        live = [p for p, c in enumerate(self.refs) if c > 0]
        n = len(live)
        src = [p for p in live if p >= n]
        dst = [p for p in range(n) if self.refs[p] == 0]
        remap = [p if c > 0 else -1 for p, c in enumerate(self.refs)]
        for a, b in zip(src, dst):
            remap[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        for i, row in enumerate(self.table):
            for c in range(-(-self.lens[i] // PAGE)):
                row[c] = remap[row[c]]
        return list(zip(src, dst)), remap
