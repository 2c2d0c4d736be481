"""Cases for timing and checking the operators around a serving step's attention: the paged layout of a step
from the requests' lengths, norms of the heads of q and k with rotary positions of one or several axes and the append
to the cache, attention of a batch that shares a long prefix, and the verification of drafted tokens against the
target's probabilities.

`run` computes an operator either in its plain form (elementary torch operations in 32 bits, in 64 for angles, long
sums and what is compared with random numbers, rounded once at the end) or, where the module's `own` is true,
through this package's prepared calls.  `exact` computes the same outputs from the operators' definitions in 64 bits.

    layout:     starts, request, position and cache row of each token of a step, its row of the tree mask, and the new
                pages of each request, taken from a stack of free ones
    norm_rope:  x <- x / sqrt(mean(x^2) + eps) * weight for each head of q and k, then turned by position (a pair of
                elements by the position along its axis); k and v written to the rows of the cache that `slots` names
    prefix:     softmax(scale * q K^T) V over the keys of a prefix that a group of sequences shares and those
                of the sequence's own; a drafted token sees those drafted tokens that its row of the mask names
    verify:     a request's drafted tokens, in their order: the child x of the last accepted token is taken if
                u * q(x) < r(x), r being the target's probabilities and q the draft's (without a draft's: u * what
                is left < r(x)); a refusal leaves r <- max(r - q, 0), scaled to 1 (without: r(x) <- 0).  Then a token
                from what is left, the first whose running sum passes a random share of the whole
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token for each request of a decode batch
        {"name": "layout-decode-48", "op": "layout", "requests": 48, "tokens": 1, "context": 4096, "page": 16,
         "tree": False, "prompts": False},
        # trees of up to 48 drafted tokens behind a shared prefix
        {"name": "layout-trees-64x48", "op": "layout", "requests": 64, "tokens": 48, "context": 2000, "page": 32,
         "tree": True, "prompts": False},
        # continuous batching at its largest: prompts' pieces among thousands of single tokens
        {"name": "layout-mixed-4096", "op": "layout", "requests": 4096, "tokens": 700, "context": 3000, "page": 16,
         "tree": False, "prompts": True},
        # the smallest decode batch
        {"name": "norm-rope-decode-8", "op": "norm_rope", "tokens": 8, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "layout": "half", "axes": 1, "positions": 4096, "dtype": "bf16"},
        # a piece of video: time, height and width; an odd number of tokens, smaller heads
        {"name": "norm-rope-video-6001", "op": "norm_rope", "tokens": 6001, "heads": 16, "kv_heads": 16, "dim": 96,
         "rotary": 96, "layout": "interleaved", "axes": 3, "positions": 1000, "dtype": "fp16"},
        # prompts of a long context
        {"name": "norm-rope-prompts-16384", "op": "norm_rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "layout": "half", "axes": 1, "positions": 131072, "dtype": "bf16"},
        # a few requests behind a short system prompt: the latency of a decode step
        {"name": "prefix-decode-8", "op": "prefix", "seqs": 8, "groups": 1, "prefix": 2000, "context": 100, "tokens": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "mask": False, "dtype": "bf16"},
        # a decode batch behind a long document
        {"name": "prefix-decode-64", "op": "prefix", "seqs": 64, "groups": 1, "prefix": 32768, "context": 1000,
         "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 32, "mask": False, "dtype": "fp16"},
        # trees of drafted tokens of requests that share two prefixes
        {"name": "prefix-trees-32x16", "op": "prefix", "seqs": 32, "groups": 2, "prefix": 16001, "context": 500,
         "tokens": 16, "heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "mask": True, "dtype": "bf16"},
        # one request, four drafted tokens
        {"name": "verify-chain-1x5", "op": "verify", "seqs": 1, "tokens": 5, "vocab": 32000, "tree": False, "draft": True,
         "dtype": "fp32"},
        # trees of the draft's best tokens, which come without probabilities; an odd vocabulary
        {"name": "verify-trees-16x24", "op": "verify", "seqs": 16, "tokens": 24, "vocab": 50257, "tree": True,
         "draft": False, "dtype": "fp32"},
        # a decode batch with eight sampled drafts each over a large vocabulary
        {"name": "verify-chains-64x9", "op": "verify", "seqs": 64, "tokens": 9, "vocab": 131072, "tree": False,
         "draft": True, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _plain_cost(c):
    """What bounds a case's plain form, or the making of its inputs."""
    if c["op"] == "layout":
        return sum(_new_tokens(c)) * (2 + c["tokens"] if c["tree"] else 1)
    if c["op"] == "norm_rope":
        return c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    if c["op"] == "verify":
        return c["seqs"] * c["tokens"] * c["vocab"] * (2 if c["draft"] else 1)
    return (c["seqs"] * (c["context"] + c["tokens"]) * (c["heads"] * c["tokens"] + c["kv_heads"] * c["dim"])
            + c["prefix"] * (c["heads"] * c["tokens"] * c["seqs"] + c["groups"] * c["kv_heads"] * c["dim"]))


def draw(rng: random.Random):
    op = rng.choice(["layout", "norm_rope", "prefix", "verify"])
    most = [c for c in listed() if c["op"] == op]
    limit = {m: max(work(c)[m] for c in most) for m in ("bytes", "flops")}
    limit["plain"] = max(_plain_cost(c) for c in most)
    while True:
        dtype = rng.choice(["bf16", "fp16"])
        kv = rng.choice([1, 2, 4, 8])
        if op == "layout":
            tree = rng.random() < 0.5
            c = {"op": op, "requests": _log_int(rng, 1, 4096), "tokens": _log_int(rng, 1, 100 if tree else 2000),
                 "context": _log_int(rng, 1, 8192), "page": rng.choice([1, 16, 24, 32, 64, 128]), "tree": tree,
                 "prompts": not tree and rng.random() < 0.5}
        elif op == "norm_rope":
            dim = rng.choice([64, 80, 96, 128, 256])
            c = {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv,
                 "dim": dim, "rotary": rng.choice([dim, dim // 2, 20]), "layout": rng.choice(["half", "interleaved"]),
                 "axes": rng.choice([1, 1, 2, 3]), "positions": _log_int(rng, 1024, 131072), "dtype": dtype}
        elif op == "prefix":
            seqs = _log_int(rng, 1, 128)
            c = {"op": op, "seqs": seqs, "groups": rng.randint(1, min(seqs, 4)), "prefix": _log_int(rng, 1, 65536),
                 "context": _log_int(rng, 1, 4096), "tokens": _log_int(rng, 1, 32),
                 "heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv, "dim": rng.choice([64, 128, 128, 256]),
                 "page": rng.choice([16, 24, 32, 64, 128]), "mask": rng.random() < 0.6, "dtype": dtype}
        else:
            c = {"op": op, "seqs": _log_int(rng, 1, 64), "tokens": _log_int(rng, 1, 40),
                 "vocab": _log_int(rng, 1000, 200000), "tree": rng.random() < 0.4, "draft": rng.random() < 0.6,
                 "dtype": rng.choice(["fp32", "fp32", "bf16"])}
        w = work(c)
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"] and _plain_cost(c) <= limit["plain"]:
            return c


# ------------------------------------------------------------------------------------------------ what a case holds

def _new_tokens(c):
    """New tokens of each request: a few have none; with prompts, every 16th brings a long piece of one."""
    def count(i):
        if i % 11 == 7:
            return 0
        if c["prompts"]:
            return 1 + (i * 37) % c["tokens"] if i % 16 == 0 else 1
        return max(1, c["tokens"] - i % 5)
    return [count(i) for i in range(c["requests"])]


def _cached(c):
    """Cached tokens of each request before the step: ragged."""
    return [0 if i % 16 == 0 else (c["context"] * (1 + i * 29 % 64)) // 64 for i in range(c["requests"])]


def _lengths(c):
    """Own context and new tokens of each sequence: ragged, the longest first."""
    b = c["seqs"]
    return ([c["context"] - c["context"] * 3 * i // (4 * b) for i in range(b)],
            [max(1, c["tokens"] - i % 5) for i in range(b)])


def _groups(c):
    """Where the sequences of each prefix begin, and the prefixes' lengths."""
    n = c["groups"]
    return [c["seqs"] * g // n for g in range(n + 1)], [c["prefix"] - c["prefix"] * g // (2 * n) for g in range(n)]


def _words(c):
    return -(-c["tokens"] // 32)


def work(c):
    if c["op"] == "layout":
        new, ctx, page = _new_tokens(c), _cached(c), c["page"]
        pages = sum(-(-(x + t) // page) - -(-x // page) for x, t in zip(ctx, new))
        n = sum(new)
        return {"bytes": 4 * (3 * len(new) + n * (3 + (1 + _words(c) if c["tree"] else 0)) + 2 * pages), "flops": 8 * n}
    if c["op"] == "norm_rope":
        heads = c["heads"] + 2 * c["kv_heads"]
        turned = c["tokens"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 2 * 2 * c["tokens"] * heads * c["dim"], "flops": turned * (3 * c["rotary"] + 4 * c["dim"])}
    if c["op"] == "verify":
        size = 4 if c["dtype"] == "fp32" else 2  # of each request, one row of the target's and one of the draft's
        rows = c["seqs"] * (2 if c["draft"] else 1)
        return {"bytes": size * rows * c["vocab"] + 16 * c["seqs"] * c["tokens"], "flops": 3 * rows * c["vocab"]}
    ctx, tok = _lengths(c)
    first, lens = _groups(c)
    keys = sum(ctx) + sum(tok) + sum(lens)
    seen = sum(t * (x + 1) for x, t in zip(ctx, tok))
    seen += sum(n * sum(tok[lo:hi]) for n, lo, hi in zip(lens, first, first[1:]))
    return {"bytes": 2 * (2 * keys * c["kv_heads"] * c["dim"] + 2 * sum(tok) * c["heads"] * c["dim"]),
            "flops": 4 * c["heads"] * c["dim"] * seen}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    s = {"case": dict(c)}
    {"layout": _prepare_layout, "norm_rope": _prepare_norm_rope, "prefix": _prepare_prefix,
     "verify": _prepare_verify}[c["op"]](c, s, g, rng)
    return s


def _prepare_layout(c, s, g, rng):
    new, ctx, page = _new_tokens(c), _cached(c), c["page"]
    order = list(range(len(new)))
    rng.shuffle(order)
    new, ctx = [new[i] for i in order], [ctx[i] for i in order]
    if c["prompts"]:
        ctx = [x + rng.randint(0, page) for x in ctx]
    have = [-(-x // page) for x in ctx]
    width = max(-(-(x + t) // page) for x, t in zip(ctx, new)) + 1
    need = sum(-(-(x + t) // page) - h for x, t, h in zip(ctx, new, have))
    s["tokens"] = sum(new) + 5  # a captured step's room, not all of it used
    ids = torch.randperm(sum(have) + need + 9, generator=g, device="cuda").int()
    at = _ints(_starts(have))
    col = torch.arange(width, device="cuda")
    mine = col < _ints(have)[:, None]
    s["table"] = torch.where(mine, ids[(at[:-1, None] + col).clamp(max=len(ids) - 1)], -1).int()
    s["free_pages"], s["free_count"] = ids[sum(have):].clone(), _ints([need + 9])
    s["context_lens"], s["new_lens"] = _ints(ctx), _ints(new)
    s["offsets"] = s["parents"] = None
    if c["tree"]:
        s["offsets"] = _ints([rng.choice([0, 1000, 5000]) for _ in new])
        s["parents"] = _ints([p for t in new for p in _tree(rng, t)] + [-1] * 5)
    if own:
        import weight_quantized_gemm_amd as W
        s["call"] = W.StepLayout(s["context_lens"], s["new_lens"], s["table"], s["free_pages"], s["free_count"],
                                 tokens=s["tokens"], page_size=page, position_offsets=s["offsets"], parents=s["parents"],
                                 mask_words=_words(c) if c["tree"] else None)


def _tree(rng, n):
    """Parents of the n tokens of a request: the first is its last decided one, the others are drafts."""
    return [-1 if j == 0 else rng.randint(max(0, j - 6), j - 1) for j in range(n)]


def _prepare_norm_rope(c, s, g, rng):
    t, h, kv, d, dt = c["tokens"], c["heads"], c["kv_heads"], c["dim"], DTYPES[c["dtype"]]
    qkv = torch.randn(t, (h + 2 * kv) * d, generator=g, device="cuda", dtype=dt)
    qkv *= 2.0  # one projection's output; q, k and v are views of it
    s["q"] = qkv[:, :h * d].unflatten(1, (h, d))
    s["k"] = qkv[:, h * d:(h + kv) * d].unflatten(1, (kv, d))
    s["v"] = qkv[:, (h + kv) * d:].unflatten(1, (kv, d))
    s["q_weight"], s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda").to(dt) for _ in range(2))
    pairs, axes = c["rotary"] // 2, c["axes"]
    s["axes"] = None
    shape = (t,)
    if axes > 1:  # as many pairs for each axis, the first the most
        cut = [pairs * i // (axes + 1) for i in range(2, axes + 1)]
        s["axes"] = _ints([sum(j >= x for x in cut) for j in range(pairs)])
        shape = (axes, t)
    s["positions"] = torch.randint(0, c["positions"], shape, generator=g, device="cuda", dtype=torch.int32)
    s["inv_freq"] = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().cuda()
    rows = t + t // 2 + 1
    s["slots"] = torch.randperm(rows, generator=g, device="cuda")[:t].int()
    s["k_cache"], s["v_cache"] = (torch.zeros(rows, kv, d, device="cuda", dtype=dt) for _ in range(2))
    s["q_out"] = torch.empty(t, h, d, device="cuda", dtype=dt)
    if own:
        import weight_quantized_gemm_amd as W
        s["call"] = W.NormRope(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=EPS, axes=s["axes"], slots=s["slots"],
                               interleaved=c["layout"] == "interleaved", q_out=s["q_out"], k_out=s["k_cache"],
                               v_out=s["v_cache"])


def _prepare_prefix(c, s, g, rng):
    dt, page, kv, d = DTYPES[c["dtype"]], c["page"], c["kv_heads"], c["dim"]
    ctx, tok = _lengths(c)
    order = list(range(c["seqs"]))
    rng.shuffle(order)
    ctx, tok = [ctx[i] for i in order], [tok[i] for i in order]
    first, shared = _groups(c)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt) * std

    need = [-(-n // page) for n in shared] + [-(-(x + t) // page) for x, t in zip(ctx, tok)]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device="cuda").int()
    s["prefix_table"] = torch.zeros(c["groups"], max(need[:c["groups"]]), dtype=torch.int32, device="cuda")
    s["block_table"] = torch.zeros(c["seqs"], max(need[c["groups"]:]) + 1, dtype=torch.int32, device="cuda")
    at = 0
    for i, x in enumerate(need):
        row = s["prefix_table"][i] if i < c["groups"] else s["block_table"][i - c["groups"]]
        row[:x] = ids[at:at + x]
        at += x
    s["q"] = normal(sum(tok), c["heads"], d, std=1.5)
    s["k_cache"], s["v_cache"] = normal(pages * page, kv, d), normal(pages * page, kv, d)
    s["prefix_lens"], s["prefix_starts"] = _ints(shared), _ints(first)
    s["context_lens"], s["q_starts"] = _ints(ctx), _ints(_starts(tok))
    s["mask"] = None
    if c["mask"]:  # a random tree for each sequence: a token sees its parent's row and itself
        rows = []
        for t in tok:
            seen = []
            for j in range(t):
                p = rng.randint(max(-1, j - 8), j - 1)
                seen.append((seen[p] if p >= 0 else 0) | 1 << j)
            rows += [[v - (v >> 31 << 32)] for v in seen]
        s["mask"] = _ints(rows)
    s["scale"] = d ** -0.5
    # the same in the form that the plain computation takes: sequence of each token, tokens of each group
    s["seq_of"] = torch.arange(c["seqs"], device="cuda").repeat_interleave(_ints(tok).long())
    starts = _starts(tok)
    s["rows_of"] = [(starts[a], starts[b]) for a, b in zip(first, first[1:])]
    s["shared"] = shared
    if own:
        import weight_quantized_gemm_amd as W
        s["call"] = W.PrefixAttention(s["q"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_lens"],
                                      s["prefix_starts"], s["block_table"], s["context_lens"], s["q_starts"], s["mask"],
                                      page_size=page, scale=s["scale"])


def _prepare_verify(c, s, g, rng):
    b, width, vocab, dt = c["seqs"], c["tokens"], c["vocab"], DTYPES[c["dtype"]]
    tok = [max(1, width - i % 5) for i in range(b)]
    rng.shuffle(tok)
    starts = _starts(tok)
    n = starts[-1]
    logits = 5.0 * torch.randn(n, vocab, generator=g, device="cuda")
    s["target"] = logits.softmax(-1).to(dt)
    draft = logits.add_(torch.randn(n, vocab, generator=g, device="cuda"), alpha=0.7).softmax(-1).to(dt)
    del logits
    s["parents"] = None
    rows = [[-1] + list(range(t - 1)) for t in tok]
    if c["tree"]:
        rows = [_tree(rng, t) for t in tok]
        s["parents"] = _ints([p for r in rows for p in r])
    parent = torch.tensor([lo + max(p, 0) for lo, r in zip(starts, rows) for p in r], device="cuda")
    if c["draft"]:  # drawn from the draft's probabilities after the parent
        u = torch.rand(n, 1, generator=g, device="cuda")
        tokens = torch.empty(n, dtype=torch.int32, device="cuda")
        for lo in range(0, n, 64):
            cum = draft[parent[lo:lo + 64]].float().cumsum(-1)
            tokens[lo:lo + 64] = (cum < u[lo:lo + 64] * cum[:, -1:]).sum(-1).clamp(max=vocab - 1).int()
    else:  # the draft's best ones, the first child's the very best
        best = draft.float().topk(8).indices
        rank = torch.tensor([min(r[1:j].count(r[j]), 7) for r in rows for j in range(len(r))], device="cuda")
        tokens = best[parent, rank].int()
    s["tokens"], s["q_starts"] = tokens, _ints(starts)
    s["draft"] = draft if c["draft"] else None
    s["accept_random"] = torch.rand(n, generator=g, device="cuda")
    s["sample_random"] = torch.rand(b, generator=g, device="cuda")
    s["depth"] = max(1, width - 1)
    if own:
        import weight_quantized_gemm_amd as W
        s["call"] = W.VerifyDrafts(s["target"], s["tokens"], s["q_starts"], s["accept_random"], s["sample_random"],
                                   draft=s["draft"], parents=s["parents"], depth=s["depth"])


# ----------------------------------------------------------------------------------------------------- the operators

def run(s):
    op = s["case"]["op"]
    if own:
        out = s["call"]()
        if op == "layout":
            return {"q_starts": out.q_starts, "requests": out.requests, "positions": out.positions, "slots": out.slots,
                    "tree_mask": out.tree_mask, "free_left": out.free_left, "table": s["table"]}
        if op == "norm_rope":
            return {"q": out[0], "k_cache": out[1], "v_cache": out[2]}
        if op == "verify":
            return {"accepted": out[0], "counts": out[1], "next": out[2]}
        return out
    return {"layout": _layout, "norm_rope": _norm_rope, "prefix": _prefix, "verify": _verify}[op](s)


def _layout(s):
    c, n, page, table = s["case"], s["tokens"], s["case"]["page"], s["table"]
    ctx, new = s["context_lens"].long(), s["new_lens"].long()
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    starts = torch.cat((zero, new.cumsum(0)))
    have = (ctx + page - 1) // page
    want = (ctx + new + page - 1) // page
    taken = torch.cat((zero, (want - have).cumsum(0)))
    # new pages, from the top of the stack
    free, count = s["free_pages"], s["free_count"].long()
    col = torch.arange(table.shape[1], device="cuda")
    at = count - 1 - (taken[:-1, None] + col - have[:, None])
    page_id = torch.where(at >= 0, free[at.clamp(0, len(free) - 1)], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < want[:, None]), page_id, table))
    # tokens
    t = torch.arange(n, device="cuda")
    req = torch.searchsorted(starts[1:], t, right=True)
    live = req < len(new)
    req = req.clamp(max=len(new) - 1)
    place = t - starts[req]
    key = ctx[req] + place
    entry = table[req, (key // page).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & (entry >= 0), entry * page + key % page, -1)
    depth, mask = place, None
    if c["tree"]:
        words = _words(c)
        bits = torch.zeros(n, 32 * words, dtype=torch.bool, device="cuda")
        depth, node, up = torch.zeros_like(place), place, s["parents"].long()
        for _ in range(c["tokens"]):
            on = live & (node >= 0)
            bits |= on[:, None] & (node[:, None] == torch.arange(32 * words, device="cuda"))
            node = torch.where(on, up[(starts[req] + node).clamp(0, n - 1)], -1)
            depth = depth + (node >= 0)
        mask = (bits.unflatten(1, (words, 32)).long() << torch.arange(32, device="cuda")).sum(-1)
        mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).int()
    offset = 0 if s["offsets"] is None else s["offsets"].long()[req]
    return {"q_starts": starts.int(), "requests": torch.where(live, req, -1).int(),
            "positions": torch.where(live, offset + ctx[req] + depth, 0).int(), "slots": slots.int(), "tree_mask": mask,
            "free_left": (count - taken[-1:]).int(), "table": table}


def _normed(x, weight):
    x = x.float()
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.float()


def _norm_rope(s):
    c, dt, pairs = s["case"], s["q"].dtype, s["case"]["rotary"] // 2
    pos = s["positions"] if s["axes"] is None else s["positions"].t()[:, s["axes"].long()]
    angle = pos.double().reshape(pos.shape[0], -1) * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        turn, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
        if c["layout"] == "interleaved":
            u, w = turn[..., 0::2], turn[..., 1::2]
            turn = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
        else:
            u, w = turn[..., :pairs], turn[..., pairs:]
            turn = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
        return torch.cat((turn, rest), -1).to(dt)

    s["q_out"].copy_(turned(_normed(s["q"], s["q_weight"])))
    s["k_cache"][s["slots"].long()] = turned(_normed(s["k"], s["k_weight"]))
    s["v_cache"][s["slots"].long()] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _prefix(s):
    c, q = s["case"], s["q"]
    page, kv, d, width, seqs = c["page"], c["kv_heads"], c["dim"], c["tokens"], c["seqs"]
    group = c["heads"] // kv
    ctx, starts, seq = s["context_lens"].long(), s["q_starts"].long(), s["seq_of"]
    n = q.shape[0]
    place = torch.arange(n, device="cuda") - starts[seq]
    # queries by cached head: (kv, n, group, d)
    rows = (q.float() * s["scale"]).reshape(n, kv, group, d).transpose(0, 1)
    # scores over each sequence's own keys, padded to the longest: (seqs, kv, width, group, span)
    span = c["context"] + width
    key = torch.arange(span, device="cuda")
    table = s["block_table"].long()
    slot = table.gather(1, (key // page).clamp(max=table.shape[1] - 1).expand(seqs, span)) * page + key % page
    k, v = (s[x][slot].float().transpose(1, 2) for x in ("k_cache", "v_cache"))
    padded = torch.zeros(seqs, width, kv, group, d, device="cuda")
    padded[seq, place] = rows.transpose(0, 1)
    padded = padded.permute(0, 2, 1, 3, 4).reshape(seqs, kv, width * group, d)
    mine = (padded @ k.transpose(2, 3).contiguous()).unflatten(2, (width, group))
    j = key - ctx[:, None]
    at = torch.arange(width, device="cuda")
    if s["mask"] is None:
        sees = j[:, None] <= at[:, None]
    else:
        bits = torch.zeros(seqs, width, 32, dtype=torch.bool, device="cuda")
        bits[seq, place] = (s["mask"] >> torch.arange(32, device="cuda") & 1).bool()
        sees = (j < 0)[:, None] | bits.gather(2, j[:, None].clamp(0, 31).expand(-1, width, -1))
    sees = sees & (j < (starts[1:] - starts[:-1])[:, None])[:, None]
    mine.masked_fill_(~sees[:, None, :, None], -math.inf)
    mine = mine.permute(0, 2, 1, 3, 4)[seq, place].transpose(0, 1)  # (kv, n, group, span)
    out = torch.empty(kv, n, group, d, device="cuda")
    for i, (lo, hi) in enumerate(s["rows_of"]):
        at = torch.arange(s["shared"][i], device="cuda")
        slot = s["prefix_table"][i].long()[at // page] * page + at % page
        pk, pv = (s[x][slot].float().transpose(0, 1) for x in ("k_cache", "v_cache"))
        shared = (rows[:, lo:hi].flatten(1, 2) @ pk.transpose(1, 2).contiguous()).unflatten(1, (hi - lo, group))
        own_part = mine[:, lo:hi]
        top = torch.maximum(shared.amax(-1, keepdim=True), own_part.amax(-1, keepdim=True))
        shared, own_part = (shared - top).exp_(), (own_part - top).exp_()
        total = shared.sum(-1, keepdim=True) + own_part.sum(-1, keepdim=True)
        o = (shared.flatten(1, 2) @ pv).unflatten(1, (hi - lo, group))
        # the own part's products by sequence, padded as above
        p = torch.zeros(seqs, width, kv, group, span, device="cuda")
        p[seq[lo:hi], place[lo:hi]] = own_part.transpose(0, 1)
        own_o = (p.permute(0, 2, 1, 3, 4).flatten(2, 3) @ v).unflatten(2, (width, group))
        o += own_o.permute(0, 2, 1, 3, 4)[seq[lo:hi], place[lo:hi]].transpose(0, 1)
        out[:, lo:hi] = o / total
    return out.transpose(0, 1).reshape(q.shape).to(q.dtype)


def _verify(s):
    c, target, draft, tokens = s["case"], s["target"], s["draft"], s["tokens"].long()
    seqs, width, n, vocab = c["seqs"], c["tokens"], s["tokens"].shape[0], c["vocab"]
    starts = s["q_starts"].long()
    count = starts[1:] - starts[:-1]
    starts = starts[:-1]
    cur, depth = starts.clone(), torch.zeros_like(starts)
    accepted = torch.full((seqs, s["depth"] + 1), -1, dtype=torch.long, device="cuda")
    refused = torch.full((seqs, width), -1, dtype=torch.long, device="cuda")  # tokens, since the last accepted one
    lost = torch.zeros(seqs, dtype=torch.float64, device="cuda")             # their probabilities
    whole = draft is not None and s["parents"] is not None
    left = target[cur].double() if whole else None
    for j in range(1, width):
        row = (starts + j).clamp(max=n - 1)
        parent = s["parents"][row].long() if s["parents"] is not None else torch.full_like(row, j - 1)
        test = (count > j) & (starts + parent == cur)
        x, u = tokens[row], s["accept_random"][row].double()
        p = left.gather(1, x[:, None])[:, 0] if whole else target[cur, x].double()
        if draft is None:
            p = torch.where((refused == x[:, None]).any(-1), 0.0, p)
            yes = test & (u * (1 - lost) < p)
        else:
            yes = test & (u * draft[cur, x].double() < p)
        no = test & ~yes
        if whole:
            rest = (left - draft[cur].double()).clamp(min=0)
            total = rest.sum(-1, keepdim=True)
            rest = torch.where(total > 0, rest / total, 0.0)
            left = torch.where(no[:, None], rest, left)
        refused[:, j] = torch.where(no, x, refused[:, j])
        refused = torch.where(yes[:, None], -1, refused)
        lost = torch.where(yes, 0.0, torch.where(no, lost + p, lost))
        depth = depth + yes
        accepted[:, 1:] = torch.where(yes[:, None] & (torch.arange(1, s["depth"] + 1, device="cuda") == depth[:, None]), j,
                                      accepted[:, 1:])
        cur = torch.where(yes, row, cur)
        if whole:
            left = torch.where(yes[:, None], target[cur].double(), left)
    full = target[cur].double()
    if whole:
        rest = left
    elif draft is not None:
        rest = torch.where((refused >= 0).any(-1)[:, None], (full - draft[cur].double()).clamp(min=0), full)
    else:
        rest = torch.cat((full, torch.zeros(seqs, 1, dtype=torch.float64, device="cuda")), 1)
        rest = rest.scatter(1, torch.where(refused >= 0, refused, vocab), 0.0)[:, :vocab]
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, full)
    cum = rest.cumsum(-1)
    token = (cum <= s["sample_random"].double()[:, None] * cum[:, -1:]).sum(-1)
    last = torch.where(rest > 0, torch.arange(vocab, device="cuda"), -1).amax(-1)
    return {"accepted": accepted[:, 1:].int(), "counts": depth.int(), "next": torch.minimum(token, last).int()}


# ------------------------------------------------------------------------------------- the definitions, in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return {"layout": _exact_layout, "norm_rope": _exact_norm_rope, "prefix": _exact_prefix,
            "verify": _exact_verify}[c["op"]](c, s)


def _exact_layout(c, s):
    page, n = c["page"], s["tokens"]
    ctx, new, table = s["context_lens"].tolist(), s["new_lens"].tolist(), s["table"].tolist()
    stack = s["free_pages"].tolist()[:int(s["free_count"])]
    parents = s["parents"].tolist() if c["tree"] else None
    offsets = [0] * len(ctx) if s["offsets"] is None else s["offsets"].tolist()
    starts, req, pos, slots, masks = [0], [], [], [], []
    for b, (x, t) in enumerate(zip(ctx, new)):
        seen, depth = [], []
        for j in range(t):
            at, r = divmod(x + j, page)
            if r == 0:
                table[b][at] = stack.pop() if stack else -1
            slots.append(table[b][at] * page + r if table[b][at] >= 0 else -1)
            req.append(b)
            if parents is None:
                pos.append(offsets[b] + x + j)
                continue
            p = parents[starts[-1] + j]
            seen.append((seen[p] if p >= 0 else 0) | 1 << j)
            depth.append(depth[p] + 1 if p >= 0 else 0)
            pos.append(offsets[b] + x + depth[j])
            w = [seen[j] >> 32 * i & 0xffffffff for i in range(_words(c))]
            masks.append([v - (v >> 31 << 32) for v in w])
        starts.append(starts[-1] + t)
    rest = n - len(req)
    return {"q_starts": _ints(starts), "requests": _ints(req + [-1] * rest), "positions": _ints(pos + [0] * rest),
            "slots": _ints(slots + [-1] * rest),
            "tree_mask": _ints(masks + [[0] * _words(c)] * rest) if c["tree"] else None, "free_left": _ints([len(stack)]),
            "table": _ints(table)}


def _exact_norm_rope(c, s):
    pairs = c["rotary"] // 2
    one, two = ((slice(0, c["rotary"], 2), slice(1, c["rotary"], 2)) if c["layout"] == "interleaved" else
                (slice(0, pairs), slice(pairs, c["rotary"])))
    angle = torch.empty(c["tokens"], pairs, dtype=torch.float64, device="cuda")
    for j in range(pairs):
        pos = s["positions"] if s["axes"] is None else s["positions"][int(s["axes"][j])]
        angle[:, j] = pos.double() * float(s["inv_freq"][j])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        x = x / ((x * x).sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * s[name + "_weight"].double()
        z = torch.complex(x[..., one], x[..., two]) * turn
        x[..., one], x[..., two] = z.real, z.imag
        out[name] = x
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache[s["slots"].long()], v_cache[s["slots"].long()] = out["k"], s["v"].double()
    return {"q": out["q"], "k_cache": k_cache, "v_cache": v_cache}


def _exact_prefix(c, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, group, page = s["q_starts"].tolist(), c["heads"] // c["kv_heads"], c["page"]
    first, shared = s["prefix_starts"].tolist(), s["prefix_lens"].tolist()
    for i, ctx in enumerate(s["context_lens"].tolist()):
        lo, hi = starts[i], starts[i + 1]
        t = hi - lo
        g = sum(i >= x for x in first[1:])
        at = torch.arange(shared[g], device="cuda")
        slots = [s["prefix_table"][g].long()[at // page] * page + at % page]
        at = torch.arange(ctx + t, device="cuda")
        slots.append(s["block_table"][i].long()[at // page] * page + at % page)
        slots = torch.cat(slots)
        draft = torch.ones(t, t, dtype=torch.bool, device="cuda").tril()
        if s["mask"] is not None:
            draft = (s["mask"][lo:hi].long() >> torch.arange(t, device="cuda") & 1) == 1
        for h in range(c["kv_heads"]):
            q = s["q"][lo:hi, h * group:(h + 1) * group].double().flatten(0, 1)
            score = ((q @ s["k_cache"][slots, h].double().t()) * s["scale"]).unflatten(0, (t, group))
            score[..., -t:] = score[..., -t:].masked_fill(~draft[:, None], -math.inf)
            o = score.softmax(-1).flatten(0, 1) @ s["v_cache"][slots, h].double()
            out[lo:hi, h * group:(h + 1) * group] = o.unflatten(0, (t, group))
    return out


def _exact_verify(c, s):
    tokens, starts = s["tokens"].tolist(), s["q_starts"].tolist()
    u_accept, u_sample = s["accept_random"].tolist(), s["sample_random"].tolist()
    accepted, counts, following = [], [], []
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        children = [[] for _ in range(hi - lo)]
        for j in range(1, hi - lo):
            children[j - 1 if s["parents"] is None else int(s["parents"][lo + j])].append(j)
        node, path = 0, []
        while True:
            left, taken, gone = s["target"][lo + node].double(), None, 0.0
            for j in children[node]:
                x, u = tokens[lo + j], u_accept[lo + j]
                if s["draft"] is None:
                    if u * (1.0 - gone) < float(left[x]):
                        taken = j
                        break
                    gone += float(left[x])
                    left[x] = 0.0
                else:
                    q = s["draft"][lo + node].double()
                    if u * float(q[x]) < float(left[x]):
                        taken = j
                        break
                    left = (left - q).clamp(min=0)
                    total = float(left.sum())
                    left = left / total if total > 0 else left * 0
            if taken is None:
                break
            node = taken
            path.append(node)
        if not float(left.sum()) > 0:
            left = s["target"][lo + node].double()
        cum = left.cumsum(0)
        past = (cum > u_sample[b] * cum[-1]).nonzero()
        following.append(int(past[0]) if len(past) else int((left > 0).nonzero()[-1]))
        counts.append(len(path))
        accepted.append(path + [-1] * (s["depth"] - len(path)))
    return {"accepted": _ints(accepted), "counts": _ints(counts), "next": _ints(following)}
