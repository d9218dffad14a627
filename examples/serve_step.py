"""A serving step with sparse attention, from the library's calls.

A small attention stack (random weights) serves a few requests over one pool of
64-token pages: prompts are prefilled in chunks with dense attention; decode
steps score the cached positions with the indexer, keep the best k and attend
to those; a request is forked into samples that share its pages; finished ones
are freed and the pool is compacted.

Per layer and step the calls are

    pml_rope_append         q rotated, k and v into their pages
    pml_index_quant_append  the indexer's q and key, rotated and quantised
    pml_paged_attention     (prefill)
    pml_fp8_paged_mqa_logits, pml_topk_logits, pml_sparse_attention   (decode)

and, between steps, pml_pages_extend / _fork / _copy / _free / _compact.

    python examples/serve_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import sparse_attention_indexer_logits_gb300 as pml  # noqa: E402

PAGE = 64


class Server:
    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, dim=128, index_heads=16, rot=64, k=256,
                 rows=16, pages=256, max_context=2048, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.layers, self.heads, self.kv_heads, self.dim = layers, heads, kv_heads, dim
        self.index_heads, self.k, self.max_context, self.rows = index_heads, k, max_context, rows
        out = (heads + 2 * kv_heads) * dim + (index_heads + 1) * 128 + index_heads
        self.w_in = [rand(hidden, out) * hidden ** -0.5 for _ in range(layers)]
        self.w_out = [rand(heads * dim, hidden) * (heads * dim) ** -0.5 for _ in range(layers)]
        self.inv_freq = torch.pow(10000.0, -torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        # the caches of all layers, and the pool that hands out their pages
        self.kv = [torch.zeros((layers, pages, PAGE, kv_heads, dim), device="cuda", dtype=torch.bfloat16)
                   for _ in range(2)]
        self.index = torch.zeros((layers, pages, 8448), device="cuda", dtype=torch.uint8)
        i32 = lambda *s: torch.zeros(s, device="cuda", dtype=torch.int32)  # noqa: E731
        self.refs, self.lens = i32(pages), i32(rows)
        self.table = i32(rows, max_context // PAGE)
        self.src, self.dst, self.count, self.remap = i32(pages), i32(pages), i32(1), i32(pages)
        self.new_pages, self.logits = i32(pages), torch.empty((rows, max_context), device="cuda")
        self.workspace = pml.pml_attention_workspace(dim)

    # ---------------------------------------------------------------- the pool

    def extend(self, more: dict[int, int]):
        """Room for `more[row]` tokens; the rows' lengths grow by them."""
        want = self.lens.clone()
        for row, n in more.items():
            want[row] += n
        pml.pml_pages_extend(self.refs, self.table, self.lens, want, self.new_pages, self.count)

    def _copy(self, n):
        for cache in (*self.kv, self.index):
            pml.pml_pages_copy(cache, self.src[:n], self.dst[:n], self.count)

    def fork(self, parents, children):
        """Rows `children` become copies of rows `parents`, sharing full pages."""
        put = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
        n = len(parents)
        pml.pml_pages_fork(self.refs, self.table, self.lens, put(parents), put(children), self.src[:n], self.dst[:n],
                           self.count)
        self._copy(n)

    def free(self, rows):
        pml.pml_pages_free(self.refs, self.table, self.lens, torch.tensor(rows, device="cuda", dtype=torch.int32))

    def compact(self):
        """The pages in use move to the front of the pool."""
        pml.pml_pages_compact(self.refs, self.table, self.lens, self.refs, self.table, self.remap, self.src, self.dst,
                              self.count)
        self._copy(self.src.numel())

    # ---------------------------------------------------------------- a step

    def step(self, x, rows, counts, dense=False):
        """`counts[i]` new tokens of row `rows[i]`, their hidden states one after
        another in `x`, whose room `extend` has made: the stack's output.  A
        decode step (one token each) attends to the indexer's k best positions
        unless `dense`."""
        put = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
        at = put(rows).long()
        lens, table = self.lens[at].contiguous(), self.table[at].contiguous()
        starts = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
        request = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), put(counts).long())
        position = (torch.arange(x.shape[0], device="cuda") - starts[request] + lens[request]
                    - put(counts)[request]).to(torch.int32)
        request = request.to(torch.int32)
        decode = not dense and all(c == 1 for c in counts)
        h, kv, d, ih = self.heads, self.kv_heads, self.dim, self.index_heads
        for layer in range(self.layers):
            y = x @ self.w_in[layer]
            q, k, v, qi, ki, w = y.split([h * d, kv * d, kv * d, ih * 128, 128, ih], dim=1)
            q, k, v = (t.unflatten(1, (-1, d)) for t in (q, k, v))
            kc, vc = self.kv[0][layer], self.kv[1][layer]
            q = pml.pml_rope_append(q, k, v, position, request, self.inv_freq, kc, vc, table)
            qi, w = pml.pml_index_quant_append(qi.unflatten(1, (ih, 128)), ki, w.float().contiguous(), position,
                                               request, self.inv_freq, self.index[layer], table,
                                               weight_scale=(128 * ih) ** -0.5, interleaved=True)
            if decode:
                logits = self.logits[:len(rows)]
                pml.pml_fp8_paged_mqa_logits(qi, self.index[layer], w, lens, table, logits, self.max_context, 1)
                best, _ = pml.pml_topk_logits(logits, lens, 1, self.max_context, self.k)
                o = pml.pml_sparse_attention(q, kc, vc, table, lens, request, best, workspace=self.workspace)
            else:
                o = pml.pml_paged_attention(q, kc, vc, table, lens, starts, workspace=self.workspace)
            x = x + o.flatten(1) @ self.w_out[layer]
        return x


def main():
    torch.manual_seed(0)
    s = Server()
    prompts = {0: 700, 1: 130, 2: 1}
    hidden = s.w_in[0].shape[0]
    inputs = {r: torch.randn((n, hidden), device="cuda", dtype=torch.bfloat16) for r, n in prompts.items()}
    # prefill, at most 256 tokens of a request at a time
    done = dict.fromkeys(prompts, 0)
    while any(done[r] < n for r, n in prompts.items()):
        part = {r: min(256, n - done[r]) for r, n in prompts.items() if done[r] < n}
        s.extend(part)
        s.step(torch.cat([inputs[r][done[r]:done[r] + c] for r, c in part.items()]), list(part), list(part.values()),
               dense=True)
        for r, c in part.items():
            done[r] += c
    # two samples of request 0, then a few decode steps of all five
    s.fork([0, 0], [3, 4])
    rows = [0, 1, 2, 3, 4]
    x = torch.randn((5, hidden), device="cuda", dtype=torch.bfloat16)
    for _ in range(70):
        s.extend(dict.fromkeys(rows, 1))
        x = torch.nn.functional.normalize(s.step(x, rows, [1] * 5).float(), dim=1).bfloat16() * hidden ** 0.5
    used = int((s.refs > 0).sum())
    s.free([1, 3])
    s.compact()
    live = int((s.refs > 0).sum())
    print(f"lengths {s.lens.tolist()[:5]}, pages {used} -> {live}, highest in use "
          f"{int(torch.nonzero(s.refs).max())}, status {pml.pml_device_status()}")


if __name__ == "__main__":
    main()
