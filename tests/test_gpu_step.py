"""The serving operators around a step's attention against plain computations in 64 bits (GPU).

Layouts and verified tokens are whole numbers and have to be equal.  Error bounds of the others, from the formats (u: half
a step of the 16-bit type, 2^-8 with bf16's 8-bit significand and 2^-11 with fp16's 11-bit one; e = 2^-24):

* every result is rounded once: u |result|, and half the smallest subnormal, of fp16 2^-25, of bf16 2^-134 (a head of
  numbers far apart has some that leave bf16: 2^-200 becomes 0);
* norm_rope: a sum of 16 products a lane and up to 5 additions across lanes, 21 e, which the root halves; the mean and eps
  e; root and division 7 e; the weight's two products 2 e; sine and cosine (reduced in fp64) 5 e with the factor; the
  turn's product and sum 2 e: 28 e < 2^-19 of factor (|u| + |v|), u and v being the normed elements that turn together;
* prefix_attention, as in test_gpu_serve.py: weights as two 16-bit terms (taken as one, u), scores whose error ds =
  2 (d + 4) e scale |q| |k| moves each weight and the sum by it, fp32 sums: (u + 4 ds + 2 (keys + 8) e) sum p |v|.
"""
import math

import pytest
import torch

import weight_quantized_gemm_amd as W
from test_gpu_serve import DEV, DTYPES, E, SUB, U, close, gen, rnd, say

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def ints(v, *shape):
    t = torch.tensor(v, dtype=torch.int32, device=DEV)
    return t.reshape(shape) if shape else t


# --------------------------------------------------------------------------------------------- layout

def layout_ref(ctx, new, table, stack, n, page, offsets=None, parents=None, words=None):
    """Token by token, with a stack that is popped."""
    table, stack, short = [list(r) for r in table], list(stack), 0
    starts, req, pos, slots, masks = [0], [], [], [], []
    for b, (x, t) in enumerate(zip(ctx, new)):
        x, t = max(x, 0), min(max(t, 0), n - starts[-1])
        width = len(table[b])
        seen, depth = [], []
        for j in range(t):
            at, r = divmod(x + j, page)
            if r == 0 and at < width:
                short += not stack
                table[b][at] = stack.pop() if stack else -1
            entry = table[b][at] if at < width else -1
            slots.append(entry * page + r if entry >= 0 and entry * page + r < 2 ** 31 else -1)
            req.append(b)
            p = -1 if parents is None else parents[starts[-1] + j]
            up = 0 <= p < j
            seen.append((seen[p] if up else 0) | 1 << j)
            depth.append(j if parents is None else depth[p] + 1 if up else 0)
            pos.append(min(x + depth[j] + (offsets[b] if offsets else 0), 2 ** 31 - 1))
            if parents is not None:
                w = [seen[j] >> 32 * i & 0xffffffff for i in range(words)]
                masks.append([v - (v >> 31 << 32) for v in w])
        starts.append(starts[-1] + t)
    rest = n - len(req)
    return dict(q_starts=starts, requests=req + [-1] * rest, positions=pos + [0] * rest, slots=slots + [-1] * rest,
                tree_mask=masks + [[0] * words] * rest if parents is not None else None, free_left=[len(stack) - short],
                table=table)


def check_layout(ctx, new, table, free, count, n, page, offsets=None, parents=None, words=None, what=""):
    want = layout_ref(ctx, new, table, free[:max(0, min(count, len(free)))], n, page, offsets, parents, words)
    B, width = len(ctx), len(table[0]) if table else 3
    t = ints(table, B, width) if B else torch.zeros(0, width, dtype=torch.int32, device=DEV)
    kw = dict(tokens=n, page_size=page, position_offsets=ints(offsets, B) if offsets is not None else None,
              parents=ints(parents, n) if parents is not None else None, mask_words=words)
    call = W.StepLayout(ints(ctx, B), ints(new, B), t, ints(free, len(free)), ints([count]), **kw)
    for again in range(2):  # the same inputs, the pages of the first call in the table: the same answer
        for o in call.out:
            if o is not None:
                o.fill_(-99)
        out = call()
        for name in ("q_starts", "requests", "positions", "slots", "tree_mask", "free_left"):
            got = getattr(out, name)
            if want[name] is None:
                assert got is None
                continue
            assert torch.equal(got.cpu(), torch.tensor(want[name], dtype=torch.int32).reshape(got.shape)), (what, name, again)
        assert torch.equal(t.cpu(), torch.tensor(want["table"], dtype=torch.int32).reshape(t.shape)), (what, again)
    return out


def layout_case(seed, B, most, page, context=300, prompts=False, tree=False, slack=3, width=None, short=0):
    g = gen(seed)
    r = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).tolist()
    new = r(0, most, B)
    if prompts:
        new = [x if i % 9 == 0 else min(x, 1) for i, x in enumerate(new)]
    ctx = r(0, context, B)
    have = [-(-x // page) for x in ctx]
    need = sum(-(-(x + t) // page) - h for x, t, h in zip(ctx, new, have))
    width = max([-(-(x + t) // page) for x, t in zip(ctx, new)], default=0) + 1 if width is None else width
    ids = torch.randperm(sum(have) + need + 4, generator=g).tolist()
    table, at = [], 0
    for h in have:
        table.append((ids[at:at + h] + [-5] * width)[:width])
        at += h
    n = sum(new) + slack
    parents = None
    if tree:
        parents = [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for t in new for j in range(t)] + [0] * slack
    return dict(ctx=ctx, new=new, table=table, free=ids[at:], count=need + 4 - short, n=n, page=page,
                offsets=r(0, 10000, B) if tree else None, parents=parents,
                words=max(1, -(-max(new, default=0) // 32)) if tree else None)


@pytest.mark.parametrize("case", [
    (1, 1, 1), (1, 40, 16), (3, 5, 1), (48, 1, 16), (64, 48, 32, 300, False, True), (7, 100, 24, 2000, False, True),
    (257, 9, 64), (4096, 2, 16), (4097, 3, 7), (9000, 3, 16, 300, False, True), (500, 700, 16, 300, True),
], ids=str)
def test_layout(case):
    say("layout", case)
    check_layout(**layout_case(11, *case), what=case)


def test_layout_ends_of_the_ranges():
    say("layout ends")
    check_layout([], [], [], [1, 2], 2, 5, 16, what="no requests")
    check_layout([5, 6], [0, 0], [[1], [2]], [], 0, 0, 16, what="no tokens")
    check_layout([5, 0], [2, 3], [[1, 4], [2, 4]], [7, 8, 9], 3, 9, 4, what="count")
    for count in (-3, 99):  # clamped to the stack there is
        check_layout([5, 0], [2, 3], [[1, 4], [2, 4]], [7, 8, 9], count, 9, 4, what=count)
    check_layout([-7, 3], [-1, 3], [[1, 4], [2, 4]], [7, 8, 9], 3, 9, 4, what="negative lengths")
    c = layout_case(3, 40, 9, 4)
    for n in (0, 1, 57, sum(c["new"]) - 1):  # room for fewer tokens than there are
        check_layout(**{**c, "n": n}, what=n)
    check_layout(**layout_case(4, 40, 30, 4, short=60), what="not enough pages")
    check_layout(**layout_case(5, 40, 30, 4, width=9, context=40), what="a table too narrow")
    check_layout([0, 10], [3, 3], [[], []], [7, 8], 2, 8, 4, what="no table")
    # rows of the cache past 2^31, positions past 2^31
    big = 1 << 20
    check_layout([3, 2 * big - 1], [2, 2], [[2047, -1, -1], [0, 2048, -1]], [2049, 2046], 2, 6, big, what="2^31")
    check_layout([100, 3], [2, 1], [[1], [2]], [], 0, 3, 128, offsets=[2 ** 31 - 101, -50], what="positions")


def test_layout_more_tokens_than_passes():
    """So many tokens that a workgroup takes several passes of them, with parents that are staged anew for each."""
    say("layout passes")
    check_layout(**layout_case(21, 200, 3000, 16, tree=False), what="passes")
    new, n = [1300] * 250, 250 * 1300 + 7
    parents = [j - 1 if j % 1000 else max(j - 1, 0) - 900 * (j > 0) if j else -1 for _ in new for j in range(1300)] + [0] * 7
    check_layout([5] * 250, new, [[3] + [-1] * 90] * 250, list(range(25000)), 25000, n, 16, None, parents, 3, what="trees")
    check_layout(**layout_case(22, 1500, 1500, 16), what="wide passes")


def test_layout_trees():
    say("layout trees")
    # parents that are none, deep chains (longer than what stands in LDS), a mask with too few words or none
    new, n = [6, 3], 9
    check_layout([4, 9], new, [[1, 2, 3]] * 2, [5, 6], 2, n, 8, [0, 0], [-1, 0, 5, 2, -9, 100, 0, 0, 3], 1, what="parents")
    deep = [2000, 1500, 40]
    parents = [j - 1 for t in deep for j in range(t)]
    for words in (0, 1, 40, 63, 70):
        check_layout([1, 2, 3], deep, [[-1] * 140] * 3, list(range(300)), 300, sum(deep), 16, [7, 8, 9], parents, words,
                     what=words)


def test_layout_feeds_the_step():
    """Its tables are what rope and tree_attention take: the same outputs as from tables made by hand."""
    say("layout step")
    page, lens = 16, [(37, 5), (0, 3), (128, 1), (15, 9)]
    g = gen(5)
    n = sum(t for _, t in lens)
    parents = [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for _, t in lens for j in range(t)]
    table = torch.full((4, 10), -1, dtype=torch.int32)
    at = 0
    for b, (c, _) in enumerate(lens):
        for p in range(-(-c // page)):
            table[b, p] = at
            at += 1
    free = list(range(at, at + 8))
    table = table.to(DEV)
    out = W.step_layout(ints([c for c, _ in lens]), ints([t for _, t in lens]), table, ints(free), ints([8]), tokens=n,
                        page_size=page, parents=ints(parents), mask_words=1)
    assert torch.equal(out.tree_mask, W.tree_mask_from_parents(parents, out.q_starts.tolist(), device=DEV))
    q, k, v = (rnd(g, n, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2))
    kc, vc = (rnd(g, (at + 8) * page, 2, 64, dtype=torch.bfloat16) for _ in range(2))
    freq = W.rope_frequencies(64, device=DEV)[0]
    kw = dict(slots=out.slots, k_out=kc, v_out=vc)
    q2, _, _ = W.rope(q, k, v, out.positions, freq, **kw)
    assert torch.equal(vc[out.slots.long()], v) and out.slots.unique().numel() == n
    o = W.tree_attention(q2, kc, vc, table, ints([c for c, _ in lens]), out.q_starts, out.tree_mask, page_size=page)
    assert torch.isfinite(o).all()


# ------------------------------------------------------------------------------------------ norm_rope

def norm_ref(x, weight, pos, freq, axes, eps, interleaved, factor):
    """(result, bound) of heads x (T, h, d); weight None: no norm."""
    dt, y = x.dtype, x.double().cpu()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double().cpu()
    half = freq.shape[0]
    pos, freq = pos.double().cpu(), freq.double().cpu()
    if axes is None:
        w = pos.reshape(-1, 1) * freq
    else:
        ax = axes.cpu().long()
        ok = (ax >= 0) & (ax < pos.shape[0])
        w = torch.where(ok, pos.t()[:, ax.clamp(0, pos.shape[0] - 1)], 0.0) * freq
    c, s = factor * w.cos()[:, None], factor * w.sin()[:, None]
    one = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
    two = one + (1 if interleaved else half)
    u, v = y[..., one], y[..., two]
    ref, mag = y.clone(), y.abs()
    ref[..., one], ref[..., two] = u * c - v * s, v * c + u * s
    both = (u.abs() + v.abs()) * abs(factor)
    mag[..., one], mag[..., two] = both, both
    bound = U[dt] * ref.abs() + max(SUB[dt], 2.0 ** -134) + 2.0 ** -19 * mag
    if weight is None:  # elements that do not turn are copied
        rest = torch.ones(x.shape[-1], dtype=torch.bool)
        rest[one], rest[two] = False, False
        bound[..., rest] = 0
    return ref, bound


NORM = [  # T, hq, hkv, d, rot, interleaved, axes, weights (q, k), slots
    (1, 1, 1, 8, 2, False, 1, "16", False),
    (1, 32, 8, 128, 128, False, 1, "16", True),
    (3, 4, 2, 64, 64, False, 1, "32", True),
    (5, 7, 1, 96, 96, True, 3, "16", True),
    (17, 16, 16, 80, 80, False, 3, "16", True),     # 5 pieces of a half, 10 of a head
    (33, 8, 2, 128, 64, False, 2, "16", False),
    (9, 3, 3, 256, 256, False, 1, "16", True),
    (9, 3, 3, 256, 128, False, 1, "32", True),      # 24 units of a head
    (21, 5, 5, 64, 20, False, 1, "16", True),       # halves of 10
    (21, 5, 5, 64, 20, True, 2, "16", False),
    (8, 2, 1, 256, 250, False, 3, "32", True),
    (8, 2, 1, 24, 6, True, 1, "16", True),
    (300, 1, 1, 32, 32, False, 1, "16", True),
    (130, 28, 4, 128, 128, True, 1, "q", True),
    (64, 6, 2, 72, 72, False, 16, "k", True),       # halves of 36
    (11, 4, 2, 128, 128, False, 2, "none", True),
]


def norm_case(i, dt, T, hq, hkv, d, rot, interleaved, axes, weights, slots):
    g = gen(200 + i)
    qkv = rnd(g, T, (hq + 2 * hkv) * d + 8, dtype=dt, std=2.0)
    cut = [hq * d, (hq + hkv) * d, (hq + 2 * hkv) * d]
    c = dict(q=qkv[:, :cut[0]].unflatten(1, (hq, d)), k=qkv[:, cut[0]:cut[1]].unflatten(1, (hkv, d)),
             v=qkv[:, cut[1]:cut[2]].unflatten(1, (hkv, d)))
    kind = torch.float32 if weights == "32" else dt
    w = lambda: (1 + 0.3 * torch.randn(d, generator=g)).to(kind).to(DEV)
    c["q_weight"] = w() if weights in ("16", "32", "q") else None
    c["k_weight"] = w() if weights in ("16", "32", "k") else None
    c["axes"] = None
    shape = (T,)
    if axes > 1:
        shape = (axes, T)
        c["axes"] = torch.randint(-1 if i % 2 else 0, axes + (i % 2), (rot // 2,), generator=g).int().to(DEV)
    c["positions"] = torch.randint(0, 131072, shape, generator=g).int().to(DEV)
    c["inv_freq"] = W.rope_frequencies(rot, device=DEV)[0]
    c["slots"] = None
    if slots:
        c["slots"] = torch.randperm(T + 7, generator=g)[:T].int().to(DEV)
        c["k_out"], c["v_out"] = (torch.full((T + 7, hkv, d), 5.0, dtype=dt, device=DEV) for _ in range(2))
    c["interleaved"], c["attention_factor"], c["eps"] = interleaved, 1.0 + 0.25 * (i % 2), 10.0 ** -(5 + i % 3)
    return c


def norm_check(c, out, what):
    names = dict(pos=c["positions"], freq=c["inv_freq"], axes=c["axes"], eps=c["eps"], interleaved=c["interleaved"],
                 factor=c["attention_factor"])
    T = c["q"].shape[0]
    ref, bound = norm_ref(c["q"], c["q_weight"], **names)
    close(out[0], ref, bound, (what, "q"))
    rows = torch.arange(T, device=DEV) if c["slots"] is None else c["slots"].long()
    keep = (rows >= 0) & (rows < out[1].shape[0])
    ref, bound = norm_ref(c["k"], c["k_weight"], **names)
    keep_cpu = keep.cpu()
    close(out[1][rows[keep]], ref[keep_cpu], bound[keep_cpu], (what, "k"))
    assert torch.equal(out[2][rows[keep]], c["v"][keep])
    if c["slots"] is not None:
        others = torch.ones(out[1].shape[0], dtype=torch.bool, device=DEV)
        others[rows[keep]] = False
        assert (out[1][others] == 5).all() and (out[2][others] == 5).all()


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("i", range(len(NORM)))
def test_norm_rope(i, dt):
    say("norm_rope", i, NORM[i], dt)
    c = norm_case(i, dt, *NORM[i])
    norm_check(c, W.norm_rope(**c), NORM[i])


def test_norm_rope_in_place_and_dropped_slots():
    say("norm_rope in place")
    for i in (1, 4, 8, 3):
        c = norm_case(i, torch.bfloat16, *NORM[i][:8], False)
        want = W.norm_rope(**c)
        q, k = c["q"].clone(), c["k"].clone()
        got = W.norm_rope(**{**c, "q": q, "k": k, "q_out": q, "k_out": k})
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        c = norm_case(i, torch.bfloat16, *NORM[i][:8], True)
        c["slots"][0] = -1
        c["slots"][-1] = 10 ** 9
        norm_check(c, W.norm_rope(**c), i)
    c = norm_case(2, torch.float16, *NORM[2])
    out = W.norm_rope(c["q"], None, None, c["positions"], c["inv_freq"], q_weight=c["q_weight"])
    assert out[1] is None and out[2] is None
    ref, bound = norm_ref(c["q"], c["q_weight"], c["positions"], c["inv_freq"], None, 1e-6, False, 1.0)
    close(out[0], ref, bound, "q alone")
    for t in W.norm_rope(c["q"][:0], c["k"][:0], c["v"][:0], c["positions"][:0], c["inv_freq"], q_weight=c["q_weight"])[:1]:
        assert t.shape == (0, 4, 64)


@pytest.mark.parametrize("i", [1, 4, 6, 8, 9])
def test_norm_rope_sizes_of_numbers(i):
    """Heads of zeros, of numbers whose squares leave fp32 (bf16), of tiny ones, and infinities and NaN, which stay in
    their heads."""
    say("norm_rope numbers", i)
    T, hq, hkv, d, rot, inter = 4, 6, 2, *NORM[i][3:6]
    c = norm_case(i, torch.bfloat16, T, hq, hkv, d, rot, inter, 1, "16", True)
    c["q"] = c["q"].clone()
    c["q"][0, 0] = 0
    c["q"][0, 1] *= 2.0 ** 120
    c["q"][1, 2, 1:] *= 2.0 ** -100
    c["q"][1, 2, 0] = 2.0 ** 100
    c["q"][2, 1] *= 2.0 ** -60
    c["eps"] = 1e-30
    norm_check(c, W.norm_rope(**c), "finite")
    clean = W.norm_rope(**c)[0].clone()
    c["q"][3, 0, 1], c["q"][3, 2, d - 1] = NAN, INF
    out = W.norm_rope(**c)[0]
    same = torch.ones(T, hq, dtype=torch.bool, device=DEV)
    same[3, 0] = same[3, 2] = False
    assert torch.equal(out[same], clean[same])
    assert torch.isnan(out[3, 0]).all()
    ref, _ = norm_ref(c["q"][3:], c["q_weight"], c["positions"][3:], c["inv_freq"], None, c["eps"], inter, 1.25 if i % 2 else 1.0)
    assert torch.equal(torch.isnan(out[3, 2]).cpu(), torch.isnan(ref[0, 2])) and torch.isnan(ref[0, 2]).any()


@pytest.mark.parametrize("i", [1, 4, 6])
@pytest.mark.parametrize("far", [18, -18])
def test_norm_rope_weights_far_from_one(i, far):
    """Heads of 2^(3 far) under weights (fp32) of 2^(-5 far): the root's inverse times the weight leaves fp32's normal
    numbers, the result does not."""
    say("norm_rope far weights", i, far)
    T, hq, hkv, d, rot, inter = 4, 6, 2, *NORM[i][3:6]
    c = norm_case(i, torch.bfloat16, T, hq, hkv, d, rot, inter, 1, "32", True)
    c["q"], c["q_weight"] = c["q"] * 2.0 ** (3 * far), torch.ones(d, device=DEV) * 2.0 ** (-5 * far)
    c["eps"] = 1e-36
    norm_check(c, W.norm_rope(**c), "far")


def test_norm_rope_large():
    """More heads in a row than one workgroup has, 64-bit offsets, far positions."""
    say("norm_rope large")
    dt, T, h, d = torch.bfloat16, 4, 2, 128
    wide = torch.zeros(T, (1 << 30) + 1024, dtype=dt, device=DEV)
    q = wide[:, 1 << 30:(1 << 30) + h * d].unflatten(1, (h, d))
    g = gen(3)
    q.copy_(rnd(g, T, h, d, dtype=dt))
    weight = rnd(g, d, dtype=dt)
    pos = ints([0, 2 ** 31 - 1, -2 ** 31, 12345])
    freq = W.rope_frequencies(d, device=DEV)[0]
    out = torch.empty(T, h, d, dtype=dt, device=DEV)
    W.norm_rope(q, None, None, pos, freq, q_weight=weight, q_out=q)
    W.norm_rope(rnd(gen(3), T, h, d, dtype=dt), None, None, pos, freq, q_weight=weight, q_out=out)
    assert torch.equal(out, q)
    ref, bound = norm_ref(rnd(gen(3), T, h, d, dtype=dt), weight, pos, freq, None, 1e-6, False, 1.0)
    close(out, ref, bound, "far")


# --------------------------------------------------------------------------------------------- prefix

def prefix_case(seed, dt, prefixes, seqs, hq, hkv, d, page, mask=None, before=0, after=0, std=1.0, narrow=0):
    """prefixes: (length, sequences) of each group; seqs: (own context, tokens) of each sequence, before and
    after of them in no group.  Rows of the cache that no key has hold NaN."""
    g = gen(seed)
    need = [-(-n // page) for n, _ in prefixes] + [-(-(c + t) // page) for c, t in seqs]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g)
    kc, vc = (torch.full((pages * page, hkv, d), NAN, dtype=dt, device=DEV) for _ in range(2))
    G = len(prefixes)
    ptable = torch.full((G, max(need[:G], default=0) + 1), -7, dtype=torch.int32)
    table = torch.full((len(seqs), max(max(need[G:], default=0) + 1 - narrow, 0)), -7, dtype=torch.int32)
    at = 0
    for i, x in enumerate(need):
        own = ids[at:at + x]
        at += x
        keys = prefixes[i][0] if i < G else sum(seqs[i - G])
        row = ptable[i] if i < G else table[i - G]
        row[:x] = own[:len(row)].int()
        j = torch.arange(keys)
        slots = (own[j // page] * page + j % page).to(DEV) if keys else j.to(DEV)
        kc[slots], vc[slots] = rnd(g, keys, hkv, d, dtype=dt), rnd(g, keys, hkv, d, dtype=dt)
    starts, first = [0], [before]
    for _, t in seqs:
        starts.append(starts[-1] + t)
    for _, n in prefixes:
        first.append(first[-1] + n)
    assert first[-1] + after == len(seqs)
    n = starts[-1]
    c = dict(q=rnd(g, n, hq, d, dtype=dt, std=std), k=kc, v=vc, ptable=ptable.to(DEV), table=table.to(DEV), page=page,
             plens=ints([x for x, _ in prefixes], G), pstarts=ints(first), context=ints([x for x, _ in seqs]),
             starts=ints(starts), mask=None, seqs=seqs, prefixes=prefixes, first=first)
    if mask == "tree":
        parents = [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for _, t in seqs for j in range(t)]
        c["mask"] = W.tree_mask_from_parents(parents, starts, device=DEV)
    elif mask == "random":
        words = max(1, -(-max(t for _, t in seqs) // 32))
        c["mask"] = torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=g).int().to(DEV)
    return c


def prefix_run(c, **kw):
    return W.prefix_attention(c["q"], c["k"], c["v"], c["ptable"], c["plens"], c["pstarts"], c["table"], c["context"],
                              c["starts"], c["mask"], page_size=c["page"], **kw)


def prefix_ref(c, scale=None):
    """(result, bound): keys that a row does not see are left out, not multiplied by 0."""
    q, dt = c["q"].double().cpu(), c["q"].dtype
    k, v = c["k"].double().cpu(), c["v"].double().cpu()
    ptable, table, page = c["ptable"].cpu(), c["table"].cpu(), c["page"]
    n, hq, d = q.shape
    hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    pages = k.shape[0] // page
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    starts = c["starts"].tolist()

    def rows_of(entries, keys):
        j = torch.arange(min(max(keys, 0), len(entries) * page))
        pg = entries[j // page].long()
        on = (pg >= 0) & (pg < pages)
        return torch.where(on, pg * page + j % page, -1)

    for b, (ctx, t) in enumerate(c["seqs"]):
        g = [i for i in range(len(c["prefixes"])) if c["first"][i] <= b < c["first"][i + 1]]
        shared = rows_of(ptable[g[0]], c["prefixes"][g[0]][0]) if g else torch.zeros(0, dtype=torch.long)
        ctx = max(ctx, 0)
        mine = rows_of(table[b], ctx + t)
        dr = torch.arange(len(mine)) - ctx
        for i in range(t):
            row = starts[b] + i
            if c["mask"] is None:
                sees = dr <= i
            else:
                words = c["mask"][row].cpu().long()
                w = (dr // 32).clamp(0, max(len(words) - 1, 0))
                bit = (words[w] >> (dr % 32) & 1) == 1 if len(words) else torch.zeros(len(dr), dtype=torch.bool)
                sees = (dr < 0) | ((dr // 32 < len(words)) & bit)
            pick = torch.cat((shared, torch.where(sees, mine, -1)))
            pick = pick[pick >= 0]
            if not len(pick):
                continue
            for h in range(hkv):
                rows = slice(h * hq // hkv, (h + 1) * hq // hkv)
                s = scale * (q[row, rows] @ k[pick, h].t())
                p = s.softmax(-1)
                out[row, rows] = p @ v[pick, h]
                ds = (2 * (d + 4) * E * abs(scale) * (q[row, rows].abs() @ k[pick, h].abs().t())).amax(-1, keepdim=True)
                mag = p @ v[pick, h].abs()
                low = SUB[dt] * v[pick, h].abs().sum(0) * p.amax(-1, keepdim=True)
                bound[row, rows] = (U[dt] * out[row, rows].abs() + SUB[dt] + low
                                    + (U[dt] + 4 * ds + 2 * (len(pick) + 8) * E) * mag)
    return out, bound


PREFIX = [  # prefixes, seqs, hq, hkv, d, page, mask, before, after
    ([(1, 1)], [(0, 1)], 1, 1, 64, 1, None, 0, 0),
    ([(100, 2)], [(5, 1), (0, 1)], 4, 4, 128, 16, "tree", 0, 0),
    ([(2000, 8)], [(30 + 7 * i, 1) for i in range(8)], 32, 8, 128, 16, None, 0, 0),
    ([(700, 3), (0, 2), (33, 0), (129, 4)], [(i * 11 % 40, 1 + i % 3) for i in range(9)], 6, 2, 64, 24, "tree", 0, 0),
    ([(515, 4)], [(20, 9), (0, 16), (300, 0), (64, 5), (1000, 3), (7, 2)], 8, 2, 128, 32, "tree", 1, 1),
    ([(3000, 40)], [(i % 50, 2) for i in range(40)], 8, 1, 64, 16, "tree", 0, 0),      # 640 rows
    ([(1000, 12), (777, 12)], [(100, 5)] * 24, 16, 4, 128, 64, "random", 0, 0),         # 240 rows
    ([(4097, 5)], [(40, 3)] * 5, 14, 2, 128, 128, None, 0, 0),                          # 105 rows
    ([(600, 6)], [(25, 4)] * 6, 4, 2, 256, 16, "tree", 0, 0),
    ([(90, 2)] * 70, [(3, 1)] * 140, 2, 2, 64, 8, None, 0, 0),                          # more groups than a wave
    ([(50, 3)], [(20, 33), (5, 64), (100, 40)], 7, 1, 128, 16, "tree", 0, 0),
    ([], [(30, 2), (0, 3)], 4, 2, 64, 16, None, 0, 2),
    ([(20000, 2)], [(3, 1), (900, 1)], 8, 8, 64, 64, None, 0, 0),
]


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("i", range(len(PREFIX)))
def test_prefix(i, dt):
    say("prefix", i, str(PREFIX[i])[:120], dt)
    prefixes, seqs, hq, hkv, d, page, mask, before, after = PREFIX[i]
    c = prefix_case(300 + i, dt, prefixes, seqs, hq, hkv, d, page, mask, before, after, std=1.0 + i % 3)
    out = prefix_run(c)
    ref, bound = prefix_ref(c)
    close(out, ref, bound, i)
    assert torch.equal(prefix_run(c), out)  # no order of execution shows


def test_prefix_without_prefixes_is_tree_attention():
    say("prefix none")
    c = prefix_case(5, torch.bfloat16, [], [(700, 3), (20, 9), (0, 1)], 8, 2, 128, 16, "tree", 0, 3)
    plain = W.tree_attention(c["q"], c["k"], c["v"], c["table"], c["context"], c["starts"], c["mask"], page_size=16)
    ref, bound = prefix_ref(c)
    close(prefix_run(c), ref, bound, "none")
    close(plain, ref, bound, "tree")


def test_prefix_rows_and_keys_that_nothing_has():
    """Prefixes and contexts of no length, empty rows of the mask, keys on no page, tokens of no sequence."""
    say("prefix nothing")
    seqs = [(0, 3), (40, 2), (0, 2)]
    c = prefix_case(7, torch.bfloat16, [(0, 1), (70, 1)], seqs, 4, 2, 64, 16, "tree", 0, 1)
    c["mask"][:] = 0
    ref, bound = prefix_ref(c)
    out = prefix_run(c)
    close(out, ref, bound, "empty rows")
    assert not out[:3].any() and not out[5:].any() and out[3:5].any()
    c["mask"] = torch.empty(7, 0, dtype=torch.int32, device=DEV)  # no drafted token is seen
    ref, bound = prefix_ref(c)
    close(prefix_run(c), ref, bound, "no words")
    c["plens"][:] = -3
    c["prefixes"] = [(-3, 1), (-3, 1)]
    ref, bound = prefix_ref(c)
    close(prefix_run(c), ref, bound, "negative")
    # pages outside the cache; a table narrower than the keys; a table of no width
    c = prefix_case(8, torch.float16, [(200, 2)], [(50, 2), (33, 4)], 4, 4, 128, 16, None, narrow=2)
    c["ptable"][0, 3], c["ptable"][0, 5], c["table"][1, 0] = -1, 10 ** 6, 10 ** 6
    ref, bound = prefix_ref(c)
    close(prefix_run(c), ref, bound, "lost pages")
    c["table"] = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    ref, bound = prefix_ref(c)
    close(prefix_run(c), ref, bound, "no table")
    c["ptable"][:] = -1
    assert not prefix_run(c).any()
    # rows of no sequence are left as they were
    c = prefix_case(9, torch.bfloat16, [(64, 2)], [(5, 3), (9, 3)], 2, 1, 64, 16)
    c["starts"][:] = ints([1, 3, 5])
    out = torch.full_like(c["q"], 9.0)
    prefix_run(c, out=out)
    assert (out[0] == 9).all() and (out[5:] == 9).all() and not (out[1:5] == 9).all(dim=-1).any()
    c["starts"][:] = ints([0, 3, 99])  # clamped to the rows there are
    full = prefix_run(c)
    assert torch.isfinite(full).all()


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,d,n", [(2, 64, 3), (16, 128, 6), (2, 256, 4)])
def test_prefix_infinities(hq, d, n, dt):
    """Infinities and NaN among the prefix's values reach all who see them, and no other group; among own keys
    only their own sequence."""
    say("prefix infinities", hq, d, n, dt)
    seqs = [(20 + i, 2) for i in range(2 * n)]
    c = prefix_case(21, dt, [(150, n), (90, n)], seqs, hq, 1, d, 16)
    clean = prefix_run(c)
    slot = lambda t, b, j: int(c[t][b, j // 16]) * 16 + j % 16
    c["v"][slot("ptable", 0, 40), 0, 3] = INF
    c["v"][slot("ptable", 0, 149), 0, 5] = -INF
    c["v"][slot("ptable", 0, 7), 0, 6] = NAN
    c["v"][slot("table", n + 1, 4), 0, 9] = INF
    c["k"][slot("table", n + 2, 1)] = NAN
    out = prefix_run(c)
    assert (out[:2 * n, :, 3] == INF).all() and (out[:2 * n, :, 5] == -INF).all() and torch.isnan(out[:2 * n, :, 6]).all()
    rest = [x for x in range(d) if x not in (3, 5, 6)]
    close(out[:2 * n][..., rest], *[t[:2 * n][..., rest] for t in prefix_ref({**c, "v": torch.nan_to_num(c["v"], 0, 0, 0)})],
          "finite columns")
    one = slice(2 * (n + 1), 2 * (n + 2))
    assert (out[one, :, 9] == INF).all() and torch.isfinite(out[one][..., 10:]).all()
    two = slice(2 * (n + 2), 2 * (n + 3))
    assert torch.isnan(out[two]).all()
    others = torch.ones(4 * n, dtype=torch.bool, device=DEV)
    others[:2 * n] = others[one] = others[two] = False
    assert torch.equal(out[others], clean[others])


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
def test_prefix_scores_far_apart(dt):
    """The prefix's scores stand hundreds above the own ones or below, row by row; scales of either sign."""
    say("prefix far", dt)
    c = prefix_case(31, dt, [(900, 6)], [(60, 3)] * 6, 8, 2, 128, 16)
    c["q"][::2] *= 20
    slots = c["ptable"][0, torch.arange(900, device=DEV) // 16].long() * 16 + torch.arange(900, device=DEV) % 16
    c["k"][slots[::3]] *= 3
    for scale in (None, 1.0, -0.5, 0.0):
        ref, bound = prefix_ref(c, scale)
        close(prefix_run(c, scale=scale), ref, bound, scale)


def test_prefix_workspace_and_starts_that_do_not_ascend():
    """Nothing is written outside the output and the workspace, whose contents are not read, and the next call is
    right."""
    say("prefix starts")
    for n, hq in ((24, 8), (2, 8), (40, 2)):
        c = prefix_case(41, torch.bfloat16, [(300, 2), (100, 2), (50, 2)], [(70, n), (5, 1), (40, 2), (0, 1), (9, 3), (8, 1)],
                        hq, 2, 64, 16)
        call = W.PrefixAttention(c["q"], c["k"], c["v"], c["ptable"], c["plens"], c["pstarts"], c["table"], c["context"],
                                 c["starts"], page_size=16)
        size = call.workspace_size
        ws = torch.full((size + (1 << 20),), 0xff, dtype=torch.uint8, device=DEV)
        good = prefix_run(c, workspace=ws).clone()
        ref, bound = prefix_ref(c)
        close(good, ref, bound, n)
        total = c["q"].shape[0]
        for starts, first in (([0, total] * 3 + [0], [0, 2, 4, 6]), (c["starts"].tolist(), [4, 0, 6, 2]),
                              ([total] * 7, [6, 6, 0, 6]), ([0, total, 0, total, 0, total, 0], [0, 6, 0, 6])):
            prefix_run({**c, "starts": ints(starts), "pstarts": ints(first)}, workspace=ws)
            assert (ws[size:] == 0xff).all()
        assert torch.equal(prefix_run(c, workspace=ws), good)
        with pytest.raises(ValueError):
            prefix_run(c, workspace=ws[:size - 1])


def test_prefix_strides():
    """q as a slice of a projection, K and V interleaved in one cache, output heads first."""
    say("prefix strides")
    dt = torch.bfloat16
    c = prefix_case(31, dt, [(300, 2)], [(100, 5), (40, 6)], 4, 2, 128, 16, "tree")
    ref, bound = prefix_ref(c)
    both = torch.stack((c["k"], c["v"]), 1)
    wide = torch.cat((c["q"].flatten(1), torch.full((11, 24), NAN, dtype=dt, device=DEV)), 1)
    out = torch.empty(4, 11, 128, dtype=dt, device=DEV).transpose(0, 1)
    got = prefix_run({**c, "q": wide[:, :512].unflatten(1, (4, 128)), "k": both[:, 0], "v": both[:, 1]}, out=out)
    close(got, ref, bound, "strides")


# --------------------------------------------------------------------------------------------- verify

def verify_ref(c):
    """From the definition, in fp64 on the CPU, request by request."""
    target, draft = c["target"].double().cpu(), None if c["draft"] is None else c["draft"].double().cpu()
    pos = lambda t: torch.where(t > 0, t, 0.0)  # negative numbers and NaN are 0
    tokens, starts, V = c["tokens"].tolist(), [min(max(s, 0), target.shape[0]) for s in c["starts"].tolist()], target.shape[1]
    parents = None if c["parents"] is None else c["parents"].tolist()
    ua, us = c["accept"].double().tolist(), c["sample"].double().tolist()
    accepted, counts, following = [], [], []
    for b, (lo, hi) in enumerate(zip(starts, starts[1:])):
        n, path, node = min(max(hi - lo, 0), 1024), [], 0
        if n == 0:
            accepted.append([-1] * c["depth"])
            counts.append(0)
            following.append(-1)
            continue
        kids = [[] for _ in range(n)]
        for j in range(1, n):
            p = j - 1 if parents is None else parents[lo + j]
            if 0 <= p < j:
                kids[p].append(j)
        while True:
            left, gone, taken = pos(target[lo + node]), 0.0, None
            full = left.clone()
            if len(path) < c["depth"]:
                for j in kids[node]:
                    x = tokens[lo + j]
                    px = float(left[x]) if 0 <= x < V else 0.0
                    if draft is None:
                        if ua[lo + j] * (1.0 - gone) < px:
                            taken = j
                            break
                        gone += px
                        if 0 <= x < V:
                            left[x] = 0.0
                    else:
                        q = pos(draft[lo + node])
                        if ua[lo + j] * (float(q[x]) if 0 <= x < V else 0.0) < px:
                            taken = j
                            break
                        left = pos(left - q)
                        total = float(left.sum())
                        left = left / total if total > 0 else torch.zeros_like(left)
            if taken is None:
                break
            path.append(taken)
            node = taken
        if not float(left.sum()) > 0:
            left = full
        cum = left.cumsum(0)
        u = us[b]
        past = (cum > max(u, 0.0) * cum[-1]).nonzero() if u == u else []
        last = (left > 0).nonzero()
        following.append(int(past[0]) if len(past) else int(last[-1]) if len(last) else -1)
        counts.append(len(path))
        accepted.append(path + [-1] * (c["depth"] - len(path)))
    return accepted, counts, following


def verify_run(c, **kw):
    return W.verify_drafts(c["target"], c["tokens"], c["starts"], c["accept"], c["sample"], depth=c["depth"],
                           draft=c["draft"], parents=c["parents"], **kw)


def verify_check(c, what=""):
    out = verify_run(c)
    accepted, counts, following = verify_ref(c)
    assert out[1].tolist() == counts, (what, "counts")
    assert out[0].tolist() == accepted, (what, "accepted")
    assert out[2].tolist() == following, (what, "next")
    again = verify_run(c)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    return out


def verify_case(seed, lens, V, tree, draft, dt=torch.float32, depth=None, stride=0, near=0.7, sharp=4.0):
    g = gen(seed)
    n = sum(lens)
    starts = [0]
    for t in lens:
        starts.append(starts[-1] + t)
    logits = sharp * torch.randn(n, V, generator=g)
    p = logits.softmax(-1)
    q = (logits + near * torch.randn(n, V, generator=g)).softmax(-1)

    def put(t):
        room = torch.full((n, V + stride), NAN, dtype=dt, device=DEV)
        room[:, :V] = t.to(dt).to(DEV)
        return room[:, :V]

    parents = [int(torch.randint(max(0, j - 5), j, (1,), generator=g)) if j else -1 for t in lens for j in range(t)]
    rows = [lo + (max(parents[lo + j], 0) if tree else max(j - 1, 0)) for lo, t in zip(starts, lens) for j in range(t)]
    if n:
        tokens = torch.multinomial(q[rows], 1, generator=g)[:, 0] if draft else q[rows].topk(min(4, V)).indices.gather(
            1, torch.randint(0, min(4, V), (n, 1), generator=g))[:, 0]
    else:
        tokens = torch.zeros(0)
    return dict(target=put(p), draft=put(q) if draft else None, tokens=tokens.int().to(DEV), starts=ints(starts),
                parents=ints(parents, n) if tree else None, accept=torch.rand(n, generator=g).to(DEV),
                sample=torch.rand(len(lens), generator=g).to(DEV), depth=max(lens, default=1) if depth is None else depth)


VERIFY = [  # lens, V
    ([1], 1), ([5], 100), ([3, 1, 0, 7, 2], 33), ([9] * 20, 1000), ([24] * 6, 5003), ([70, 130, 1], 300), ([4, 6], 32000),
    ([2] * 300, 64), ([5, 5], 200001),
]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("draft", [False, True], ids=["given", "drawn"])
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("i", range(len(VERIFY)))
def test_verify(i, tree, draft, dt):
    say("verify", i, VERIFY[i][0][:6], VERIFY[i][1], tree, draft, dt)
    for seed in range(3 if VERIFY[i][1] < 10000 else 1):
        verify_check(verify_case(400 + 10 * i + seed, *VERIFY[i], tree, draft, dt, stride=i % 3), VERIFY[i])


def test_verify_ends_of_the_ranges():
    say("verify ends")
    for tree in (False, True):
        for draft in (False, True):
            what = (tree, draft)
            c = verify_case(50, [6, 4, 9, 3], 120, tree, draft, near=0.2)
            for depth in (0, 1, 2):  # a path cut short: the token follows the last one accepted
                verify_check({**c, "depth": depth}, (what, depth))
            verify_check({**c, "accept": torch.zeros_like(c["accept"])}, (what, "all"))
            verify_check({**c, "accept": torch.full_like(c["accept"], 1.0)}, (what, "u = 1"))
            verify_check({**c, "accept": torch.full_like(c["accept"], 1e9)}, (what, "none"))
            verify_check({**c, "accept": torch.full_like(c["accept"], NAN)}, (what, "NaN"))
            for u in (0.0, -1.0, 1.0, 2.0, NAN, 1 - 2.0 ** -24):
                verify_check({**c, "sample": torch.full_like(c["sample"], u)}, (what, u))
            tokens = c["tokens"].clone()
            tokens[1], tokens[7], tokens[12] = -1, 120, 2 ** 31 - 1
            verify_check({**c, "tokens": tokens}, (what, "tokens"))
            for starts in ([0, 6, 6, 6, 22], [2, 5, 9, 9, 9], [0, 6, 10, 19, 500], [-5, 6, 10, 19, 22]):
                verify_check({**c, "starts": ints(starts)}, (what, starts))
    c = verify_case(51, [6, 7], 90, True, False)
    c["parents"][:] = ints([-1, 0, 0, -1, 9, 3, 0, 0, 0, 0, -7, 5, 100])
    verify_check(c, "parents")
    verify_check({**verify_case(51, [6, 7], 90, True, True), "parents": c["parents"]}, "parents, drawn")
    out = W.verify_drafts(c["target"], c["tokens"], c["starts"][:1], c["accept"], c["sample"][:0], depth=3)
    assert out[0].shape == (0, 3) and out[1].shape == (0,)
    none = verify_case(52, [0, 0], 10, False, True)
    assert verify_check(none)[2].tolist() == [-1, -1]


def test_verify_rows_that_hold_nothing():
    """Rows of zeros, of negative numbers and NaN; nothing left after a refusal (the draft's row is the target's, or has
    all of it); all children refused; the same token among siblings."""
    say("verify rows")
    for tree in (False, True):
        c = verify_case(60, [4, 4, 4, 4, 4], 2000, tree, True)
        c["target"][0:4] = 0
        c["target"][4:8] = NAN
        c["target"][8:12, ::2] = -1.0
        c["target"][12:16, 5] = NAN
        c["draft"][12:16, 7] = -3.0
        c["draft"][16:20] = c["target"][16:20]
        c["accept"][:] = 1.0
        verify_check(c, tree)
        verify_check({**c, "draft": None}, tree)
        c["draft"] = torch.ones_like(c["target"])
        verify_check(c, (tree, "all"))
        c["target"][:] = 0
        c["target"][:, 1234] = 1.0
        for u in (0.0, 0.3, 1.0):
            c["accept"][:] = u
            verify_check(c, (tree, u))
            verify_check({**c, "draft": None}, (tree, u))
            c["tokens"][:] = 1234
            verify_check(c, (tree, u))
            verify_check({**c, "draft": None}, (tree, u))
    c = verify_case(61, [40, 40], 50, True, False)  # many siblings, few tokens
    c["parents"] = ints([-1] + [0] * 39, 40).repeat(2)
    c["tokens"] = torch.randint(0, 6, (80,), generator=gen(62)).int().to(DEV)
    c["accept"][:] = 0.999
    verify_check(c, "siblings")
    c = verify_case(61, [40, 40], 50, True, True, near=3.0)
    c["parents"] = ints([-1] + [0] * 39, 40).repeat(2)
    c["accept"][:] = torch.rand(80, generator=gen(63)).to(DEV) * 0.5 + 0.5
    verify_check(c, "siblings, drawn")


def test_verify_long_requests():
    """More tokens than a wave's lanes and than are looked at; paths that go all the way."""
    say("verify long")
    for tree in (False, True):
        for draft in (False, True):
            c = verify_case(70, [1100, 200], 40, tree, draft, near=0.01)
            c["accept"] *= 0.9
            if not draft:
                c["accept"] *= 0.01
            out = verify_check(c, (tree, draft))
            assert int(out[1].max()) >= 3


def test_verify_beyond_4_gib():
    say("verify 64-bit offsets")
    V, n = 1 << 24, 80
    c = verify_case(80, [3, 2], 1000, False, True)
    wide = torch.zeros(n, V, device=DEV)
    q = torch.zeros(n, V, device=DEV)
    wide[-5:, 5000000:5001000], q[-5:, 5000000:5001000] = c["target"], c["draft"]
    want = verify_run(c)
    tokens = torch.cat((torch.zeros(n - 5, dtype=torch.int32, device=DEV), c["tokens"] + 5000000))
    accept = torch.cat((torch.zeros(n - 5, device=DEV), c["accept"]))
    out = W.verify_drafts(wide, tokens, c["starts"] + (n - 5), accept, c["sample"], depth=c["depth"], draft=q)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(out[2], want[2] + 5000000)


def test_verify_distribution():
    """The first token of a chain with one draft is distributed as the target's row: with random numbers on a regular
    grid, each token's share of 16384 requests is within the grid's steps of its probability (256 accept numbers, 64
    sample numbers; the draft's tokens in their proportion, 1/64 each)."""
    say("verify distribution")
    V, g = 4, gen(90)
    p, q = torch.tensor([0.5, 0.25, 0.125, 0.125]), torch.tensor([0.25, 0.25, 0.25, 0.25])
    grid = torch.cartesian_prod(torch.arange(4.0), (torch.arange(64) + 0.5) / 64, (torch.arange(64) + 0.5) / 64)
    B = grid.shape[0]
    target = p.repeat(2 * B, 1).to(DEV)
    tokens = torch.stack((torch.zeros(B), grid[:, 0]), 1).flatten().int().to(DEV)
    accept = torch.stack((torch.zeros(B), grid[:, 1]), 1).flatten().float().to(DEV)
    out = W.verify_drafts(target, tokens, torch.arange(0, 2 * B + 1, 2, device=DEV, dtype=torch.int32), accept,
                          grid[:, 2].float().to(DEV), depth=1, draft=q.repeat(2 * B, 1).to(DEV))
    first = torch.where(out[1] > 0, tokens[1::2], out[2]).cpu()
    for x in range(V):
        assert abs(float((first == x).double().mean()) - float(p[x])) <= 1 / 64


# -------------------------------------------------------------------------------------- the calls themselves

def make_calls():
    lc = layout_case(91, 30, 6, 16, tree=True)
    lay = W.StepLayout(ints(lc["ctx"]), ints(lc["new"]), ints(lc["table"]), ints(lc["free"]), ints([lc["count"]]),
                       tokens=lc["n"], page_size=16, parents=ints(lc["parents"]), mask_words=lc["words"])
    nc = norm_case(5, torch.float16, *NORM[5])
    no = W.NormRope(**nc)
    pc = prefix_case(92, torch.bfloat16, [(900, 4), (300, 2)], [(50, 6)] * 6, 8, 2, 128, 16, "tree")
    pr = W.PrefixAttention(pc["q"], pc["k"], pc["v"], pc["ptable"], pc["plens"], pc["pstarts"], pc["table"], pc["context"],
                           pc["starts"], pc["mask"], page_size=16)
    calls = [lay, no, pr]
    randoms = []
    for tree, draft in ((False, True), (True, False), (True, True)):
        vc = verify_case(93, [7] * 9, 3001, tree, draft)
        calls.append(W.VerifyDrafts(vc["target"], vc["tokens"], vc["starts"], vc["accept"], vc["sample"], depth=6,
                                    draft=vc["draft"], parents=vc["parents"]))
        randoms += [vc["accept"], vc["sample"]]
    return calls, (nc["q"], pc["q"]), randoms


def flat(out):
    return [x.clone() for x in (out if isinstance(out, tuple) else (out,)) if x is not None]


def test_step_calls_on_another_stream():
    say("step streams")
    calls, _, _ = make_calls()
    plain = [flat(c()) for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for c, want in zip(calls, plain):
        for o in (c.out if isinstance(c.out, tuple) else (c.out,)):
            if o is not None:
                o.fill_(1)
        side.wait_stream(torch.cuda.current_stream())
        c(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(flat(c.out), want))
        assert all(torch.equal(a, b) for a, b in zip(flat(c(side.cuda_stream)), want))
        side.synchronize()


def test_step_calls_in_a_graph():
    """Captured once, replayed over new inputs written into the same tensors, with the same calls made eagerly between
    the replays."""
    say("step graph")
    calls, inputs, randoms = make_calls()
    for c in calls:
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for step in range(4):
        for x in inputs:
            x.copy_(torch.randn(x.shape, generator=gen(70 + step)).to(x.dtype))
        for x in randoms:
            x.copy_(torch.rand(x.shape, generator=gen(80 + step)))
        graph.replay()
        got = [flat(c.out) for c in calls]
        torch.cuda.synchronize()
        want = [flat(c()) for c in calls]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_step_workspaces_given():
    """Contents of the workspace are not read; one too small is refused."""
    say("step workspace")
    c = verify_case(95, [7] * 9, 3001, True, True)
    want = verify_run(c)
    size = W.VerifyDrafts(c["target"], c["tokens"], c["starts"], c["accept"], c["sample"], depth=c["depth"],
                          draft=c["draft"], parents=c["parents"]).workspace_size
    ws = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(verify_run(c, workspace=ws), want))
    assert (ws[size:] == 0xff).all()
    with pytest.raises(ValueError):
        verify_run(c, workspace=ws[:size - 1])
