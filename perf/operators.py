"""Cases for timing and checking the operators of a serving step that run beside the weight-quantized
projections: low-rank adapters of many requests added to a projection's output, rotary positions with the
append to the cache, and attention for a tree of drafted tokens over that paged cache.

`run` computes an operator either in its plain form (elementary torch operations in 32 bits, rounded once at
the end) or, where the module's `own` is true, through this package's prepared calls.  `exact` computes the same
outputs from the operators' definitions in 64 bits.

    adapters:  out[t] = x3[t] + scale[i] * (x1[t] @ a[i]^T) @ b[i]^T,   i = the adapter of token t (none: x3[t])
    rope:      q, k rotated by position; k and v written to the rows of the cache that `slots` names
    tree:      softmax(scale * q K^T) V over a sequence's cached keys; a drafted token sees the whole context and
               those drafted tokens that its row of the mask names
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one request, one token: the latency of a single decode step with its adapter
        {"name": "adapters-one-token", "op": "adapters", "tokens": 1, "requests": 1, "adapters": 4, "rank": 16,
         "k": 4096, "n": 4096, "dtype": "bf16"},
        # a decode batch, one token each, twice as many requests as adapters
        {"name": "adapters-decode-64", "op": "adapters", "tokens": 64, "requests": 64, "adapters": 32, "rank": 32,
         "k": 8192, "n": 8192, "dtype": "fp16"},
        # continuous batching: some prompts' pieces among many single tokens, an odd token count
        {"name": "adapters-mixed-777", "op": "adapters", "tokens": 777, "requests": 40, "adapters": 16, "rank": 64,
         "k": 8192, "n": 2048, "dtype": "bf16"},
        # prompts of a dozen requests at once
        {"name": "adapters-prompts-16384", "op": "adapters", "tokens": 16384, "requests": 12, "adapters": 8,
         "rank": 64, "k": 4096, "n": 8192, "dtype": "bf16"},
        # the smallest decode batch
        {"name": "rope-decode-4", "op": "rope", "tokens": 4, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "layout": "half", "positions": 4096, "scaling": 1.0, "dtype": "bf16"},
        # a large decode batch, adjacent pairs, half of each head rotated
        {"name": "rope-decode-509", "op": "rope", "tokens": 509, "heads": 32, "kv_heads": 32, "dim": 128,
         "rotary": 64, "layout": "interleaved", "positions": 32768, "scaling": 1.0, "dtype": "fp16"},
        # prompts, frequencies scaled for a long context
        {"name": "rope-prompts-16384", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "layout": "half", "positions": 131072, "scaling": 8.0, "dtype": "bf16"},
        # one request, one token, a short context: the latency of a single decode step
        {"name": "tree-one-token", "op": "tree", "seqs": 1, "context": 1000, "tokens": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "mask": False, "dtype": "bf16"},
        # trees of up to 16 tokens over small heads, as many cached heads as query heads
        {"name": "tree-batch-16x16", "op": "tree", "seqs": 16, "context": 4096, "tokens": 16, "heads": 16,
         "kv_heads": 16, "dim": 64, "page": 16, "mask": True, "dtype": "bf16"},
        # a plain decode batch of ragged contexts
        {"name": "tree-decode-64", "op": "tree", "seqs": 64, "context": 8192, "tokens": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 32, "mask": False, "dtype": "fp16"},
        # one request with a very long context
        {"name": "tree-long-131072", "op": "tree", "seqs": 1, "context": 131072, "tokens": 29, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "mask": True, "dtype": "bf16"},
        # wide trees for several requests, eight query heads to a cached one
        {"name": "tree-wide-8x64", "op": "tree", "seqs": 8, "context": 16384, "tokens": 64, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 128, "mask": True, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _plain_cost(c):
    """What bounds a case's plain form: the products over all adapters, or the padded scores and keys."""
    if c["op"] == "adapters":
        return c["tokens"] * c["adapters"] * c["rank"] * (c["k"] + c["n"])
    if c["op"] == "rope":
        return c["tokens"] * (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    keys = c["seqs"] * (c["context"] + c["tokens"])
    return keys * (c["heads"] * c["tokens"] + c["kv_heads"] * c["dim"])


def draw(rng: random.Random):
    op = rng.choice(["adapters", "rope", "tree"])
    most = [c for c in listed() if c["op"] == op]
    limit = {m: max(work(c)[m] for c in most) for m in ("bytes", "flops")}
    limit["plain"] = max(_plain_cost(c) for c in most)
    while True:
        dtype = rng.choice(["bf16", "fp16"])
        if op == "adapters":
            tokens = _log_int(rng, 1, 16384)
            c = {"op": op, "tokens": tokens, "requests": _log_int(rng, 1, min(tokens, 256)),
                 "adapters": _log_int(rng, 1, 64), "rank": 8 * _log_int(rng, 1, 16), "k": 32 * _log_int(rng, 8, 256),
                 "n": 32 * _log_int(rng, 8, 256), "dtype": dtype}
        elif op == "rope":
            kv = rng.choice([1, 2, 4, 8])
            dim = rng.choice([64, 96, 128, 256])
            c = {"op": op, "tokens": _log_int(rng, 1, 16384), "heads": kv * rng.choice([1, 2, 4, 7, 8]),
                 "kv_heads": kv, "dim": dim, "rotary": rng.choice([dim, dim // 2, 32]),
                 "layout": rng.choice(["half", "interleaved"]), "positions": _log_int(rng, 1024, 131072),
                 "scaling": rng.choice([1.0, 4.0, 8.0]), "dtype": dtype}
        else:
            kv = rng.choice([1, 2, 4, 8])
            c = {"op": op, "seqs": _log_int(rng, 1, 64), "context": _log_int(rng, 1, 131072),
                 "tokens": _log_int(rng, 1, 64), "heads": kv * rng.choice([1, 2, 4, 7, 8]), "kv_heads": kv,
                 "dim": rng.choice([64, 128]), "page": rng.choice([16, 24, 32, 64, 128, 256]),
                 "mask": rng.random() < 0.7, "dtype": dtype}
        w = work(c)
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"] and _plain_cost(c) <= limit["plain"]:
            return c


# ------------------------------------------------------------------------------------------------ what a case holds

def _ranks(c):
    """Adapters of three ranks in one stack, as requests bring them."""
    return [c["rank"] if j % 3 == 0 else max(1, c["rank"] // 2) if j % 3 == 1 else max(1, c["rank"] - 3)
            for j in range(c["adapters"])]


def _adapter_of(c):
    """The adapter of each request; every eighth request has none."""
    return [-1 if i % 8 == 7 else i % c["adapters"] for i in range(c["requests"])]


def _lengths(c):
    """Context and drafted tokens of each sequence: ragged, the longest first."""
    b = c["seqs"]
    return ([c["context"] - c["context"] * 3 * i // (4 * b) for i in range(b)],
            [max(1, c["tokens"] - i % 5) for i in range(b)])


def work(c):
    if c["op"] == "adapters":
        ranks = _ranks(c)
        used = sorted({a for a in _adapter_of(c) if a >= 0})
        weights = sum(ranks[a] for a in used) * (c["k"] + c["n"])
        rank = sum(ranks[a] for a in used) / max(1, len(used))
        share = sum(a >= 0 for a in _adapter_of(c)) / c["requests"]
        return {"bytes": 2 * (weights + c["tokens"] * (c["k"] * share + 2 * c["n"])),
                "flops": 2 * c["tokens"] * share * rank * (c["k"] + c["n"])}
    if c["op"] == "rope":
        heads = c["heads"] + 2 * c["kv_heads"]
        return {"bytes": 2 * 2 * c["tokens"] * heads * c["dim"],
                "flops": 3 * c["tokens"] * (c["heads"] + c["kv_heads"]) * c["rotary"]}
    ctx, tok = _lengths(c)
    keys = sum(ctx) + sum(tok)
    return {"bytes": 2 * (2 * keys * c["kv_heads"] * c["dim"] + 2 * sum(tok) * c["heads"] * c["dim"]),
            "flops": 4 * c["heads"] * c["dim"] * sum(t * (x + 1) for x, t in zip(ctx, tok))}


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    dt = DTYPES[c["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt) * std

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    s = {"case": dict(c)}
    if c["op"] == "adapters":
        m, r, k, n = c["tokens"], c["rank"], c["k"], c["n"]
        s["x1"] = normal(m, k)
        s["a"] = normal(c["adapters"], r, k, std=k ** -0.5)
        s["b"] = normal(c["adapters"], n, r, std=0.5 * r ** -0.5)
        s["scale"] = torch.tensor([rng.choice([0.5, 1.0, 2.0]) for _ in range(c["adapters"])], device="cuda")
        s["ranks"] = ints(_ranks(c))
        s["x3"] = normal(m, n)  # what the shared projection gave
        # a request's tokens stand together; where there are more tokens than requests, a quarter of the
        # requests (one at least) are prompts and the rest bring one token each
        count = c["requests"]
        lens = [1] * count
        prompts = rng.sample(range(count), max(1, count // 4))
        cuts = sorted(rng.randint(0, m - count) for _ in range(len(prompts) - 1))
        for p, lo, hi in zip(prompts, [0] + cuts, cuts + [m - count]):
            lens[p] += hi - lo
        of = _adapter_of(c)
        rng.shuffle(of)
        s["indices"] = ints(of).repeat_interleave(ints(lens).long()).int()
        if own:
            import weight_quantized_gemm_amd as W
            s["call"] = W.LoraMatmul(s["x1"], s["a"], s["b"], s["indices"], s["scale"], ranks=s["ranks"], x3=s["x3"])
    elif c["op"] == "rope":
        t, h, kv, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        qkv = normal(t, (h + 2 * kv) * d)  # one projection's output; q, k and v are views of it
        s["q"] = qkv[:, :h * d].unflatten(1, (h, d))
        s["k"] = qkv[:, h * d:(h + kv) * d].unflatten(1, (kv, d))
        s["v"] = qkv[:, (h + kv) * d:].unflatten(1, (kv, d))
        s["positions"] = torch.randint(0, c["positions"], (t,), generator=g, device="cuda", dtype=torch.int32)
        pairs = c["rotary"] // 2
        freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs) / c["scaling"]
        s["inv_freq"] = freq.float().cuda()
        s["attention_factor"] = 1.0 + 0.1 * math.log(c["scaling"])
        s["slots"] = torch.randperm(t + t // 2 + 1, generator=g, device="cuda")[:t].int()
        s["k_cache"], s["v_cache"] = (torch.zeros(t + t // 2 + 1, kv, d, device="cuda", dtype=dt) for _ in range(2))
        s["q_out"] = torch.empty(t, h, d, device="cuda", dtype=dt)
        if own:
            import weight_quantized_gemm_amd as W
            s["call"] = W.Rope(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], slots=s["slots"],
                               interleaved=c["layout"] == "interleaved", attention_factor=s["attention_factor"],
                               q_out=s["q_out"], k_out=s["k_cache"], v_out=s["v_cache"])
    else:
        ctx, tok = _lengths(c)
        order = list(range(c["seqs"]))
        rng.shuffle(order)
        ctx, tok = [ctx[i] for i in order], [tok[i] for i in order]
        page, kv, d = c["page"], c["kv_heads"], c["dim"]
        need = [-(-(x + t) // page) for x, t in zip(ctx, tok)]
        pages = sum(need) + 3
        ids = torch.randperm(pages, generator=g, device="cuda").int()
        table = torch.zeros(c["seqs"], max(need) + 1, dtype=torch.int32, device="cuda")
        at = 0
        for i, x in enumerate(need):
            table[i, :x] = ids[at:at + x]
            at += x
        s["q"] = normal(sum(tok), c["heads"], d, std=1.5)
        s["k_cache"], s["v_cache"] = normal(pages * page, kv, d), normal(pages * page, kv, d)
        s["block_table"], s["context_lens"] = table, ints(ctx)
        starts = [0]
        for t in tok:
            starts.append(starts[-1] + t)
        s["q_starts"] = ints(starts)
        s["mask"] = None
        if c["mask"]:  # a random tree for each sequence: a token sees its parent's row and itself
            words = -(-c["tokens"] // 32)
            rows = []
            for t in tok:
                seen = []
                for j in range(t):
                    p = rng.randint(max(-1, j - 8), j - 1)
                    seen.append((seen[p] if p >= 0 else 0) | 1 << j)
                rows += [[(v >> 32 * w & 0xffffffff) - (v >> 32 * w + 31 & 1) * (1 << 32) for w in range(words)]
                         for v in seen]
            s["mask"] = ints(rows)
        s["scale"] = d ** -0.5
        # the same in the form that the plain computation takes: sequence and place of each query token
        s["seq_of"] = torch.arange(c["seqs"], device="cuda").repeat_interleave(ints(tok).long())
        if own:
            import weight_quantized_gemm_amd as W
            s["call"] = W.TreeAttention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["context_lens"],
                                        s["q_starts"], s["mask"], page_size=page, scale=s["scale"])
    return s


# ----------------------------------------------------------------------------------------------------- the operators

def run(s):
    if own:
        out = s["call"]()
        return {"q": out[0], "k_cache": out[1], "v_cache": out[2]} if s["case"]["op"] == "rope" else out
    return {"adapters": _adapters, "rope": _rope, "tree": _tree}[s["case"]["op"]](s)


def _adapters(s):
    a, b, x3 = s["a"], s["b"], s["x3"]
    count, r, k = a.shape
    h = (s["x1"].float() @ a.float().reshape(count * r, k).t()).reshape(-1, count, r)  # through every adapter
    mine = s["indices"][:, None] == torch.arange(count, device="cuda")
    keep = mine[:, :, None] & (torch.arange(r, device="cuda") < s["ranks"][:, None])
    h = torch.where(keep, h * s["scale"][:, None], 0.0)
    y = h.reshape(-1, count * r) @ b.float().transpose(1, 2).reshape(count * r, -1)
    return (x3.float() + y).to(x3.dtype)


def _rotated(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    turn, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        u, w = turn[..., 0::2], turn[..., 1::2]
    else:
        u, w = turn[..., :rot // 2], turn[..., rot // 2:]
    u, w = u * cos - w * sin, w * cos + u * sin
    turn = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turn, rest), -1)


def _rope(s):
    interleaved, dt = s["case"]["layout"] == "interleaved", s["q"].dtype
    angle = s["positions"].float()[:, None, None] * s["inv_freq"]
    cos, sin = angle.cos() * s["attention_factor"], angle.sin() * s["attention_factor"]
    s["q_out"].copy_(_rotated(s["q"], cos, sin, interleaved).to(dt))
    s["k_cache"][s["slots"].long()] = _rotated(s["k"], cos, sin, interleaved).to(dt)
    s["v_cache"][s["slots"].long()] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _tree(s):
    c, q, table = s["case"], s["q"], s["block_table"]
    page, kv, d = c["page"], c["kv_heads"], c["dim"]
    group, width, seqs = c["heads"] // kv, c["tokens"], c["seqs"]
    ctx, starts, seq = s["context_lens"].long(), s["q_starts"].long(), s["seq_of"]
    place = torch.arange(q.shape[0], device="cuda") - starts[seq]
    span = c["context"] + width
    key = torch.arange(span, device="cuda")
    # keys of each sequence, padded to the longest: (seqs, kv, span, d)
    slot = table.long().gather(1, (key // page).clamp(max=table.shape[1] - 1).expand(seqs, span)) * page + key % page
    k = s["k_cache"][slot].float().transpose(1, 2)
    v = s["v_cache"][slot].float().transpose(1, 2)
    # queries padded to the widest tree: (seqs, kv, width * group, d)
    padded = torch.zeros(seqs, width, kv, group, d, device="cuda")
    padded[seq, place] = q.float().reshape(-1, kv, group, d)
    padded = padded.permute(0, 2, 1, 3, 4).reshape(seqs, kv, width * group, d)
    score = (padded * s["scale"]) @ k.transpose(2, 3).contiguous()
    # what each token sees: the context, and drafted tokens by the mask (none: those up to itself)
    j = key - ctx[:, None]
    if s["mask"] is None:
        row = torch.arange(width, device="cuda")
        sees = j[:, None] <= row[:, None]
    else:
        bits = torch.zeros(seqs, width, 32 * s["mask"].shape[1], dtype=torch.bool, device="cuda")
        bits[seq, place] = (s["mask"][:, :, None] >> torch.arange(32, device="cuda") & 1).bool().flatten(1)
        sees = (j < 0)[:, None] | bits.gather(2, j[:, None].clamp(0, bits.shape[2] - 1).expand(-1, width, -1))
    count = starts[1:] - starts[:-1]
    sees = sees & (j < count[:, None])[:, None]
    score = score.unflatten(2, (width, group)).masked_fill_(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = (score - top).exp_()
    total = p.sum(-1)
    o = (p.flatten(2, 3) @ v).unflatten(2, (width, group))
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return o.permute(0, 2, 1, 3, 4)[seq, place].reshape(q.shape).to(q.dtype)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "adapters":
        if c["tokens"] * c["rank"] * (c["k"] + c["n"]) > 1 << 42:
            return None
        y = s["x3"].double()
        for i, rank in enumerate(s["ranks"].tolist()):
            rows = (s["indices"] == i).nonzero()[:, 0]
            if len(rows):
                h = s["x1"][rows].double() @ s["a"][i, :rank].double().t()
                y[rows] += float(s["scale"][i]) * (h @ s["b"][i, :, :rank].double().t())
        return y
    if c["op"] == "rope":
        angle = s["positions"].double()[:, None] * s["inv_freq"].double()
        turn = torch.polar(torch.full_like(angle, s["attention_factor"]), angle)[:, None]
        out = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            pairs = c["rotary"] // 2
            one, two = ((slice(0, c["rotary"], 2), slice(1, c["rotary"], 2)) if c["layout"] == "interleaved" else
                        (slice(0, pairs), slice(pairs, c["rotary"])))
            z = torch.complex(x[..., one], x[..., two]) * turn
            x[..., one], x[..., two] = z.real, z.imag
            out[name] = x
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_cache[s["slots"].long()], v_cache[s["slots"].long()] = out["k"], s["v"].double()
        return {"q": out["q"], "k_cache": k_cache, "v_cache": v_cache}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts, group = s["q_starts"].tolist(), c["heads"] // c["kv_heads"]
    for i, ctx in enumerate(s["context_lens"].tolist()):
        lo, hi = starts[i], starts[i + 1]
        t = hi - lo
        at = torch.arange(ctx + t, device="cuda")
        slot = s["block_table"][i].long()[at // c["page"]] * c["page"] + at % c["page"]
        draft = torch.ones(t, t, dtype=torch.bool, device="cuda").tril()
        if s["mask"] is not None:
            words = s["mask"][lo:hi].long()
            place = torch.arange(t, device="cuda")
            draft = (words[:, place // 32] >> place % 32 & 1) == 1
        for h in range(c["kv_heads"]):
            q = s["q"][lo:hi, h * group:(h + 1) * group].double().transpose(0, 1)
            score = (q @ s["k_cache"][slot, h].double().t()) * s["scale"]
            score[..., ctx:] = score[..., ctx:].masked_fill(~draft, -math.inf)
            out[lo:hi, h * group:(h + 1) * group] = (score.softmax(-1) @ s["v_cache"][slot, h].double()).transpose(0, 1)
    return out
