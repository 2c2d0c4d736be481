"""The attention block of one verification step of speculative decoding, on quantised weights.

Several requests, each with an adapter of its own (or none), have a tree of drafted tokens to verify:

    qkv = x @ dequant(Wqkv) + bias, plus the requests' adapters on it      (antiquant_matmul, lora_matmul)
    q, k turned by position; k and v appended to the requests' pages       (rope)
    attention of the drafted tokens over their pages                       (tree_attention)
    y = attention @ dequant(Wo), plus the requests' adapters on it         (antiquant_matmul, lora_matmul)

A drafted token's position is the context's length plus its depth in the tree; its cache row is the next free one
of its request.  Everything is prepared once: a step writes the new tokens, trees and lengths into the same
tensors and calls ``step()``, which enqueues kernels only (and may be captured into a HIP graph).

    python examples/verify_step.py
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import weight_quantized_gemm_amd as W  # noqa: E402


class VerifyStep:
    """contexts: cached tokens of each request; parents: for each request, its drafted tokens' parents (-1: the
    context's last token); adapters: the adapter of each request, -1 for none.  The caches of keys and
    values start with random contents in place of the contexts' tokens."""

    def __init__(self, contexts, parents, adapters, *, heads=8, kv_heads=2, dim=64, page=16, rank=16, seed=0,
                 dtype=torch.bfloat16, device="cuda:0"):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).to(device)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
        hidden, kv, out = heads * dim, kv_heads * dim, heads * dim
        width = hidden + 2 * kv
        self.contexts, self.parents, self.adapters = contexts, parents, adapters
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        counts = [len(p) for p in parents]
        tokens = sum(counts)
        count = max(max(adapters) + 1, 1)  # (one that nobody has, where nobody has any)

        # weights: int8 with a scale per column; adapters (rank, in) and (out, rank)
        codes = lambda k, n: torch.randint(-127, 128, (k, n), generator=g, dtype=torch.int8).to(device)
        self.x = normal(tokens, hidden)
        self.w_qkv, self.s_qkv = codes(hidden, width), normal(width, std=0.1).abs() * (hidden ** -0.5 / 16)
        self.w_out, self.s_out = codes(hidden, out), normal(out, std=0.1).abs() * (hidden ** -0.5 / 16)
        self.bias = normal(width, std=0.1)
        self.a_qkv, self.b_qkv = normal(count, rank, hidden, std=hidden ** -0.5), normal(count, width, rank, std=0.1)
        self.a_out, self.b_out = normal(count, rank, hidden, std=hidden ** -0.5), normal(count, out, rank, std=0.1)
        self.scale = torch.full((count,), 2.0, device=device)
        self.indices = ints([a for a, c in zip(adapters, counts) for _ in range(c)])

        # pages of the requests in any order, with room for the drafted tokens
        need = [-(-(c + t) // page) for c, t in zip(contexts, counts)]
        pages = torch.randperm(sum(need) + 4, generator=g)
        table, at = torch.zeros(len(need), max(need), dtype=torch.int32), 0
        for i, n in enumerate(need):
            table[i, :n] = pages[at:at + n].int()
            at += n
        self.k_cache, self.v_cache = (normal(len(pages) * page, kv_heads, dim) for _ in range(2))
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + c)
        depth, slots = [], []
        for i, (context, tree) in enumerate(zip(contexts, parents)):
            mine = []
            for j, p in enumerate(tree):
                mine.append(0 if p < 0 else mine[p] + 1)
                slots.append(int(table[i, (context + j) // page]) * page + (context + j) % page)
            depth += [context + d for d in mine]
        self.positions, self.slots = ints(depth), ints(slots)
        self.table, self.lens, self.starts = table.to(device), ints(contexts), ints(starts)
        self.mask = W.tree_mask_from_parents([p for tree in parents for p in tree], starts, device=device)
        self.inv_freq, self.attention_factor = W.rope_frequencies(dim, scaling="ramp", factor=4.0, original_length=4096,
                                                                  device=device)

        self.qkv_call = W.AntiquantMatmul(self.x, self.w_qkv, self.s_qkv, None, self.bias)
        qkv = self.qkv_call.out
        self.qkv_adapters = W.LoraMatmul(self.x, self.a_qkv, self.b_qkv, self.indices, self.scale, x3=qkv, out=qkv)
        q = qkv[:, :hidden].unflatten(1, (heads, dim))
        k = qkv[:, hidden:hidden + kv].unflatten(1, (kv_heads, dim))
        v = qkv[:, hidden + kv:].unflatten(1, (kv_heads, dim))
        self.rope_call = W.Rope(q, k, v, self.positions, self.inv_freq, slots=self.slots,
                                attention_factor=self.attention_factor, q_out=q, k_out=self.k_cache, v_out=self.v_cache)
        self.attention_call = W.TreeAttention(q, self.k_cache, self.v_cache, self.table, self.lens, self.starts, self.mask,
                                              page_size=page)
        seen = self.attention_call.out.flatten(1)
        self.out_call = W.AntiquantMatmul(seen, self.w_out, self.s_out)
        self.out_adapters = W.LoraMatmul(seen, self.a_out, self.b_out, self.indices, self.scale, x3=self.out_call.out,
                                         out=self.out_call.out)
        self.calls = [self.qkv_call, self.qkv_adapters, self.rope_call, self.attention_call, self.out_call,
                      self.out_adapters]

    def step(self, stream=None):
        for call in self.calls:
            call(stream)
        return self.out_call.out

    def plain(self):
        """The same block in fp64 on the CPU, request by request; reads the caches as they stand."""
        d = lambda t: t.double().cpu()
        hidden, kv = self.heads * self.dim, self.kv_heads * self.dim

        def project(x, w, s, a, b):
            y = d(x) @ (d(w) * d(s))
            for t, i in enumerate(self.indices.tolist()):
                if i >= 0:
                    y[t] += float(self.scale[i]) * ((d(x)[t] @ d(a)[i].t()) @ d(b)[i].t())
            return y

        qkv = project(self.x, self.w_qkv, self.s_qkv, self.a_qkv, self.b_qkv) + d(self.bias)
        w = d(self.positions)[:, None] * d(self.inv_freq)
        turn = torch.polar(torch.full_like(w, self.attention_factor), w)[:, None]

        def rotated(t, heads):
            t = t.unflatten(1, (heads, self.dim))
            z = torch.complex(t[..., :self.dim // 2], t[..., self.dim // 2:]) * turn
            return torch.cat((z.real, z.imag), -1)

        q, k = rotated(qkv[:, :hidden], self.heads), rotated(qkv[:, hidden:hidden + kv], self.kv_heads)
        v = qkv[:, hidden + kv:].unflatten(1, (self.kv_heads, self.dim))
        k_cache, v_cache = d(self.k_cache), d(self.v_cache)
        slots = self.slots.cpu().long()
        k_cache[slots], v_cache[slots] = k, v
        seen = torch.empty(q.shape, dtype=torch.float64)
        group, at = self.heads // self.kv_heads, 0
        for i, (context, tree) in enumerate(zip(self.contexts, self.parents)):
            j = torch.arange(context + len(tree))
            rows = self.table.cpu()[i, j // self.page].long() * self.page + j % self.page
            for t, _ in enumerate(tree):
                path, p = [], t
                while p >= 0:
                    path.append(context + p)
                    p = tree[p]
                pick = rows[torch.tensor(list(range(context)) + path)]
                for h in range(self.heads):
                    s = (k_cache[pick, h // group] @ q[at, h]) * self.dim ** -0.5
                    seen[at, h] = s.softmax(0) @ v_cache[pick, h // group]
                at += 1
        return project(seen.flatten(1), self.w_out, self.s_out, self.a_out, self.b_out)


def main():
    step = VerifyStep([37, 500, 0, 130], [[-1, 0, 0, 1, 2], [-1], [-1, 0, 1], [-1, -1, 0, 1, 1, 4, 5]], [0, -1, 1, 0])
    want = step.plain()
    got = step.step()
    torch.cuda.synchronize()
    off = float((got.double().cpu() - want).norm() / want.norm())
    print(f"{got.shape[0]} drafted tokens of {len(step.contexts)} requests: relative error against fp64 {off:.2e}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.step()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    graph.replay()
    begin.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"one replay of the captured step: {begin.elapsed_time(end) * 10:.1f} us")
    return off


if __name__ == "__main__":
    main()
