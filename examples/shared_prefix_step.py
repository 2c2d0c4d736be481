"""One layer's attention and the verification of a speculative step, for requests that share a prompt.

Each request has the shared prompt's keys before its own, and brings its last decided token and a tree of drafted ones:

    tables = starts, positions, cache rows, tree mask and new pages from the requests' lengths      (step_layout)
    qkv    = x @ dequant(Wqkv)                                                                       (antiquant_matmul)
    q, k normed by head and turned by position; k and v appended to the requests' pages             (norm_rope)
    attention over the prompt, by rows of all requests together, and over each one's own pages       (prefix_attention)
    p      = softmax(attention @ dequant(Wout)), the probabilities after each token                  (antiquant_matmul)
    the drafted tokens that p accepts, and the token that follows                                    (verify_drafts)

Everything is prepared once: a step writes the new tokens, lengths and random numbers into the same tensors and
calls ``step()``, which copies nothing to the host (and may be captured into a HIP graph).

    python examples/shared_prefix_step.py
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import weight_quantized_gemm_amd as W  # noqa: E402


class SharedPrefixStep:
    """prefix: tokens of the shared prompt; contexts: further cached tokens of each request; parents: for each request, the
    parents of its tokens, the first of which is its last decided one (parent -1) and the root of its drafts; room:
    tokens that a captured step has room for.  The caches start with random contents in place of the cached tokens."""

    def __init__(self, prefix, contexts, parents, *, heads=8, kv_heads=2, dim=64, page=16, vocab=512, room=None, seed=0,
                 dtype=torch.bfloat16, device="cuda:0"):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dtype).to(device)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
        hidden, kv = heads * dim, kv_heads * dim
        counts = [len(p) for p in parents]
        tokens = sum(counts) if room is None else room
        self.prefix, self.contexts, self.parents, self.counts = prefix, contexts, parents, counts
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page

        codes = lambda k, n: torch.randint(-127, 128, (k, n), generator=g, dtype=torch.int8).to(device)
        self.x = normal(tokens, hidden)
        self.w_qkv, self.s_qkv = codes(hidden, hidden + 2 * kv), normal(hidden + 2 * kv, std=0.1).abs() * (hidden ** -0.5 / 8)
        self.w_out, self.s_out = codes(hidden, vocab), normal(vocab).abs() * (hidden ** -0.5 / 8)
        self.q_weight, self.k_weight = 1 + normal(dim, std=0.1), 1 + normal(dim, std=0.1)

        # pages: the prompt's, the requests', and a stack of free ones
        shared, have = -(-prefix // page), [-(-c // page) for c in contexts]
        need = sum(-(-(c + t) // page) - h for c, t, h in zip(contexts, counts, have))
        ids = torch.randperm(shared + sum(have) + need + 4, generator=g).int()
        self.prefix_table = ids[None, :shared].clone().to(device)
        width = max(-(-(c + t) // page) for c, t in zip(contexts, counts))
        table, at = torch.full((len(contexts), width), -1, dtype=torch.int32), shared
        for i, h in enumerate(have):
            table[i, :h] = ids[at:at + h]
            at += h
        self.table, self.free = table.to(device), ids[at:].clone().to(device)
        self.free_count = ints([len(self.free)])
        self.k_cache, self.v_cache = (normal(len(ids) * page, kv_heads, dim) for _ in range(2))

        rest = tokens - sum(counts)
        self.lens, self.new = ints(contexts), ints(counts)
        self.tokens = torch.randint(0, vocab, (tokens,), generator=g).int().to(device)
        self.accept, self.sample = (torch.rand(n, generator=g).to(device) for n in (tokens, len(contexts)))
        self.up = ints([p for tree in parents for p in tree] + [-1] * rest)
        self.layout_call = W.StepLayout(self.lens, self.new, self.table, self.free, self.free_count, tokens=tokens,
                                        page_size=page, position_offsets=ints([prefix] * len(contexts)),
                                        parents=self.up, mask_words=-(-max(counts) // 32))
        t = self.tables = self.layout_call.out
        self.qkv_call = W.AntiquantMatmul(self.x, self.w_qkv, self.s_qkv)
        qkv = self.qkv_call.out
        q = qkv[:, :hidden].unflatten(1, (heads, dim))
        k = qkv[:, hidden:hidden + kv].unflatten(1, (kv_heads, dim))
        v = qkv[:, hidden + kv:].unflatten(1, (kv_heads, dim))
        self.inv_freq = W.rope_frequencies(dim, device=device)[0]
        self.rope_call = W.NormRope(q, k, v, t.positions, self.inv_freq, q_weight=self.q_weight, k_weight=self.k_weight,
                                    slots=t.slots, q_out=q, k_out=self.k_cache, v_out=self.v_cache)
        self.attention_call = W.PrefixAttention(q, self.k_cache, self.v_cache, self.prefix_table, ints([prefix]),
                                                ints([0, len(contexts)]), self.table, self.lens, t.q_starts, t.tree_mask,
                                                page_size=page)
        self.attention_call.out.zero_()  # rows of no request stay as they are
        self.out_call = W.AntiquantMatmul(self.attention_call.out.flatten(1), self.w_out, self.s_out)
        self.probabilities = torch.empty(tokens, vocab, device=device)
        self.verify_call = W.VerifyDrafts(self.probabilities, self.tokens, t.q_starts, self.accept, self.sample,
                                          parents=self.up, depth=max(max(counts) - 1, 1))

    def step(self, stream=None):
        """(accepted, counts, next tokens) of each request."""
        for call in (self.layout_call, self.qkv_call, self.rope_call, self.attention_call, self.out_call):
            call(stream)
        torch.softmax(self.out_call.out, -1, dtype=torch.float32, out=self.probabilities)
        return self.verify_call(stream)

    def plain(self):
        """The probabilities in fp64 on the CPU, token by token; reads the caches as they stand before a step."""
        d = lambda t: t.double().cpu()
        hidden, kv, page = self.heads * self.dim, self.kv_heads * self.dim, self.page
        n = sum(self.counts)
        qkv = d(self.x)[:n] @ (d(self.w_qkv) * d(self.s_qkv))
        j = torch.arange(self.prefix)
        k_cache, v_cache = d(self.k_cache), d(self.v_cache)
        shared = self.prefix_table.cpu()[0, j // page].long() * page + j % page
        group, half, out, at = self.heads // self.kv_heads, self.dim // 2, [], 0
        normed = lambda x, w: x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * d(w)
        for i, (context, tree) in enumerate(zip(self.contexts, self.parents)):
            j = torch.arange(-(-context // page) * page)[:context]
            rows = self.table.cpu()[i, j // page].long() * page + j % page
            keys, values = [], []  # of the request's tokens
            for t, p in enumerate(tree):
                path, up = [t], p
                while up >= 0:
                    path.append(up)
                    up = tree[up]
                w = (self.prefix + context + len(path) - 1) * d(self.inv_freq)
                turn = torch.polar(torch.ones_like(w), w)

                def turned(x):
                    z = torch.complex(x[..., :half], x[..., half:]) * turn
                    return torch.cat((z.real, z.imag), -1)

                y = qkv[at + t]
                q = turned(normed(y[:hidden].view(self.heads, self.dim), self.q_weight))
                keys.append(turned(normed(y[hidden:hidden + kv].view(self.kv_heads, self.dim), self.k_weight)))
                values.append(y[hidden + kv:].view(self.kv_heads, self.dim))
                k = torch.cat((k_cache[shared], k_cache[rows], torch.stack([keys[x] for x in path])))
                v = torch.cat((v_cache[shared], v_cache[rows], torch.stack([values[x] for x in path])))
                seen = []
                for h in range(self.heads):
                    s = (k[:, h // group] @ q[h]) * self.dim ** -0.5
                    seen.append(s.softmax(0) @ v[:, h // group])
                out.append(torch.cat(seen))
            at += len(tree)
        return (torch.stack(out) @ (d(self.w_out) * d(self.s_out))).softmax(-1)


def main():
    step = SharedPrefixStep(700, [37, 0, 130, 64], [[-1, 0, 0, 1, 2], [-1], [-1, 0, 1], [-1, 0, 0, 1, 1, 4, 5]])
    want = step.plain()
    accepted, counts, following = step.step()
    torch.cuda.synchronize()
    off = float((step.probabilities.double().cpu() - want).norm() / want.norm())
    print(f"{len(want)} tokens of {len(step.counts)} requests: relative error of the probabilities against fp64 {off:.2e}")
    print("accepted", counts.tolist(), "next", following.tolist(), "pages left", step.tables.free_left.tolist())
    return off


if __name__ == "__main__":
    main()
