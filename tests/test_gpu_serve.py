"""The serving operators against plain fp64 computations (GPU).

Error bounds, from the formats (u: rounding to the 16-bit type, 2^-8 with bf16's 8-bit significand and 2^-11 with
fp16's 11-bit one; e = 2^-24):

* every result is rounded once: u |result|, and half the smallest subnormal of fp16, 2^-25;
* adapters: fp32 sums of k and r products with their own roundings, and h as a sum of two 16-bit
  numbers (2^-16 of it in bf16): (2^-16 + 2 (k + r + 8) e) |scale| (|x| |A|^T) |B|^T;
* rope: angles reduced in fp64, then fp32 sine, cosine and three roundings: 2^-21 factor (|u| + |v|);
* tree: weights rounded to 16 bits (u, and in fp16 2^-25 of the largest weight), scores whose error ds =
  2 (d + 4) e scale |q| |k| moves each weight and the sum by it, fp32 sums: (u + 4 ds + 2 (keys + 8) e) sum p |v|.
"""
import math

import numpy as np
import pytest
import torch

import weight_quantized_gemm_amd as W

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SUB = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
DTYPES = [torch.bfloat16, torch.float16]
DEV = "cuda:0"


def say(*what):
    print("[gpu-case]", *what, flush=True)


def close(got, ref, bound, what):
    got, ref = got.double().cpu(), ref.cpu()
    bound = bound.cpu()
    assert got.shape == ref.shape
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    assert torch.equal(got[~fin & ~torch.isnan(ref)], ref[~fin & ~torch.isnan(ref)]), what
    err = (got - ref).abs()[fin]
    over = err > bound[fin]
    assert not over.any(), (what, float((err / bound[fin].clamp(min=1e-300)).max()), int(over.sum()))


def rnd(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float32) * std).to(dtype).to(DEV)


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------------- adapters

def lora_ref(x1, a, b, idx, scale, ranks, x3):
    """(result, bound) in fp64 on the GPU."""
    x, dt = x1.reshape(-1, x1.shape[-1]).double(), x1.dtype
    n = b.shape[1]
    y = torch.zeros(x.shape[0], n, dtype=torch.float64, device=DEV) if x3 is None else x3.reshape(-1, n).double().clone()
    mag = torch.zeros_like(y)
    for i in range(a.shape[0]):
        rows = (idx == i).nonzero()[:, 0]
        if not len(rows):
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        s = 1.0 if scale is None else float(scale[i])
        h = x[rows] @ a[i, :r].double().t().contiguous()
        y[rows] += s * (h @ b[i, :, :r].double().t().contiguous())
        hm = x[rows].abs() @ a[i, :r].double().abs().t().contiguous()
        mag[rows] = abs(s) * (hm @ b[i, :, :r].double().abs().t().contiguous())
    k, r = a.shape[2], a.shape[1]
    bound = U[dt] * y.abs() + SUB[dt] + (2.0 ** -16 + 2 * (k + r + 8) * E) * mag
    shape = tuple(x1.shape[:-1]) + (n,)
    return y.reshape(shape), bound.reshape(shape)


def lora_case(seed, dt, m, L, r, k, n, *, order="runs", ranks=False, scale=True, x3=True):
    g = gen(seed)
    c = dict(x1=rnd(g, m, k, dtype=dt), a=rnd(g, L, r, k, dtype=dt, std=k ** -0.5), b=rnd(g, L, n, r, dtype=dt, std=r ** -0.5))
    idx = torch.randint(-1, L, (m,), generator=g)
    if order == "runs":
        idx = idx.sort().values
    elif order == "one":
        idx = torch.full((m,), L - 1)
    c["indices"] = idx.int().to(DEV)
    c["scale"] = (torch.rand(L, generator=g) * 4 - 2).to(DEV) if scale else None
    c["ranks"] = torch.randint(0, r + 1, (L,), generator=g).int().to(DEV) if ranks else None
    c["x3"] = rnd(g, m, n, dtype=dt) if x3 else None
    return c


def lora_run(c, **kw):
    return W.lora_matmul(c["x1"], c["a"], c["b"], c["indices"], c["scale"], ranks=c["ranks"], x3=c["x3"], **kw)


LORA = [  # m, L, r, k, n, order, ranks, scale, x3
    (1, 1, 8, 8, 8, "one", False, False, False),
    (1, 4, 16, 4096, 4096, "one", True, True, True),
    (2, 3, 24, 40, 136, "mixed", True, True, True),
    (15, 16, 64, 264, 256, "mixed", False, True, True),
    (16, 2, 72, 520, 72, "mixed", True, True, False),
    (17, 40, 16, 1000, 328, "mixed", False, False, True),
    (63, 8, 256, 2048, 64, "runs", True, True, True),
    (64, 100, 32, 4104, 1032, "mixed", False, True, True),
    (65, 3, 136, 96, 4096, "mixed", True, True, True),
    (333, 7, 16, 8192, 200, "runs", True, True, True),
    (1024, 1, 8, 72, 1000, "one", False, True, False),
    (1025, 5, 64, 1032, 520, "runs", True, True, True),
    (1100, 200, 40, 128, 264, "mixed", True, True, True),
    (2049, 5, 64, 1032, 520, "runs", True, True, True),
    (2100, 200, 40, 128, 264, "mixed", True, True, True),
    (2111, 3, 16, 72, 136, "mixed", True, False, False),
    (4099, 6, 256, 512, 256, "runs", False, True, True),
    (20000, 4, 24, 4104, 72, "runs", True, True, True),
]


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", LORA, ids=lambda c: "m%d_L%d_r%d_k%d_n%d_%s" % c[:6])
def test_lora(case, dt):
    m, L, r, k, n, order, ranks, scale, x3 = case
    say("lora", case, dt)
    c = lora_case(m * 7 + r, dt, m, L, r, k, n, order=order, ranks=ranks, scale=scale, x3=x3)
    y = lora_run(c)
    ref, bound = lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], c["ranks"], c["x3"])
    close(y, ref, bound, case)


def test_lora_indices_out_of_range_and_none():
    say("lora no adapters")
    for m in (5, 1500, 2500):
        c = lora_case(3, torch.bfloat16, m, 3, 16, 64, 72)
        c["indices"] = torch.tensor([-1, 3, 2 ** 31 - 1, -2 ** 31, 7], dtype=torch.int32, device=DEV).repeat(m // 5)
        assert torch.equal(lora_run(c), c["x3"])
        c["x3"] = None
        assert not lora_run(c).any()


def test_lora_past_the_rank_and_other_rows_do_not_matter():
    """NaN in rows of a and columns of b past an adapter's rank, in adapters that are not used, and
    infinities in a neighbour's row leave a row's bits as they are."""
    say("lora isolation")
    for dt in DTYPES:
        for m in (37, 1200, 2200):
            c = lora_case(11, dt, m, 6, 40, 264, 136, order="mixed")
            c["ranks"] = torch.tensor([0, 3, 8, 21, 39, 40], dtype=torch.int32, device=DEV)
            c["indices"] = torch.where(c["indices"] == 4, -1, c["indices"]).int()
            clean = lora_run(c)
            for i, r in enumerate(c["ranks"].tolist()):
                c["a"][i, r:] = float("nan")
                c["b"][i, :, r:] = float("nan")
            c["a"][4] = float("inf")
            c["b"][4] = float("nan")
            assert torch.equal(lora_run(c), clean)
            bad = (c["indices"] == 5).nonzero()[0, 0]
            c["x1"][bad, 5] = float("inf")
            y = lora_run(c)
            keep = torch.arange(m, device=DEV) != bad
            assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[bad]).all()


def test_lora_equal_calls_give_equal_bits():
    """Mixed adapters in more windows than there are lists of work items."""
    say("lora repeats")
    for m, L, r, k, n in [(9001, 12, 16, 1024, 136), (4099, 64, 64, 512, 72), (700, 8, 32, 4096, 264)]:
        c = lora_case(17, torch.bfloat16, m, L, r, k, n, order="mixed")
        first = lora_run(c)
        for _ in range(8):
            assert torch.equal(lora_run(c), first), m
        ref, bound = lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], None, c["x3"])
        close(first, ref, bound, m)


def test_lora_first_product_beyond_fp16():
    """h passes fp16's range while the result is back inside it."""
    say("lora large h")
    c = lora_case(5, torch.float16, 40, 2, 16, 512, 64, order="mixed")
    c["x1"] *= 60
    c["a"] *= 800
    c["scale"] = torch.tensor([2.0 ** -16, 2.0 ** -17], device=DEV)
    ref, bound = lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], None, c["x3"])
    assert (c["x1"].float() @ c["a"][0].float().t()).abs().max() > 70000
    close(lora_run(c), ref, bound, "large h")


def test_lora_strides_in_place_and_shapes():
    say("lora strides")
    dt = torch.bfloat16
    for m in (20, 1030, 2060):
        c = lora_case(7, dt, m, 4, 24, 136, 72, order="mixed", ranks=True)
        ref, bound = lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], c["ranks"], c["x3"])
        wide_x = torch.full((m, 136 + 24), float("nan"), dtype=dt, device=DEV)
        wide_x[:, 16:152] = c["x1"]
        wide_y = torch.full((m, 72 + 40), 7.0, dtype=dt, device=DEV)
        wide_y[:, 8:80] = c["x3"]
        y = wide_y[:, 8:80]
        out = W.lora_matmul(wide_x[:, 16:152], c["a"], c["b"], c["indices"], c["scale"], ranks=c["ranks"], x3=y, out=y)
        assert out is y
        close(y, ref, bound, "slices, in place")
        assert (wide_y[:, :8] == 7).all() and (wide_y[:, 80:] == 7).all()
        # one row for all of x3; (b, s, .) shapes
        c["x3"] = c["x3"][:1].expand(m, 72)
        ref, bound = lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], c["ranks"], c["x3"])
        close(lora_run(c), ref, bound, "expanded x3")
        y3 = W.lora_matmul(c["x1"].view(2, m // 2, -1), c["a"], c["b"], c["indices"], c["scale"], ranks=c["ranks"],
                           x3=c["x3"].reshape(2, m // 2, 72))
        close(y3.view(m, 72), ref, bound, "3-D")


def test_lora_no_tokens():
    c = lora_case(7, torch.bfloat16, 0, 4, 24, 136, 72)
    assert lora_run(c).shape == (0, 72)


# ----------------------------------------------------------------------------------------------- rope

def rope_ref(x, positions, inv_freq, interleaved, factor):
    x = x.double()
    pairs = len(inv_freq)
    w = positions.double()[:, None] * inv_freq.double()
    c, s = (torch.cos(w) * factor)[:, None], (torch.sin(w) * factor)[:, None]
    one, two = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., one], y[..., two] = x[..., one] * c - x[..., two] * s, x[..., two] * c + x[..., one] * s
    mag[..., one] = mag[..., two] = (x[..., one].abs() + x[..., two].abs()) * abs(factor)
    return y, mag


def rope_bound(y, mag, dt):
    return torch.where(mag > 0, U[dt] * y.abs() + SUB[dt] + 2.0 ** -21 * mag, 0.0)


ROPE = [  # T, hq, hkv, d, rot, max position
    (1, 1, 1, 8, 2, 10), (1, 32, 8, 128, 128, 4096), (3, 4, 2, 64, 64, 100), (5, 3, 1, 96, 40, 131072),
    (7, 7, 7, 72, 6, 2 ** 31 - 1), (33, 8, 1, 256, 256, 1 << 20), (64, 1, 1, 8, 8, 5), (129, 14, 2, 128, 64, 40000),
    (513, 2, 2, 16, 14, 1000), (1000, 5, 1, 40, 32, 100000), (2000, 1, 1, 8, 6, 77),
]


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "T%d_h%d_%d_d%d_rot%d_p%d" % c)
def test_rope(case, interleaved, dt):
    T, hq, hkv, d, rot, most = case
    say("rope", case, interleaved, dt)
    g = gen(T + d)
    qkv = rnd(g, T, (hq + 2 * hkv) * d, dtype=dt)
    q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([hq * d, hkv * d, hkv * d], 1))
    pos = torch.randint(0, most, (T,), generator=g).int().to(DEV)
    pos[-1] = most - 1
    if T > 2:
        pos[1] = -5
    freq, _ = W.rope_frequencies(rot, device=DEV)
    factor = 1.25
    qr, qm = rope_ref(q, pos, freq, interleaved, factor)
    kr, km = rope_ref(k, pos, freq, interleaved, factor)
    # fresh outputs
    qo, ko, vo = W.rope(q, k, v, pos, freq, interleaved=interleaved, attention_factor=factor)
    close(qo, qr, rope_bound(qr, qm, dt), "q")
    close(ko, kr, rope_bound(kr, km, dt), "k")
    assert torch.equal(vo, v)
    # into a cache: rows given, one token dropped below and one above
    S = T + 9
    slots = torch.randperm(S, generator=g)[:T].int().to(DEV)
    if T > 4:
        slots[2], slots[3] = -1, S
    kc, vc = (torch.full((S, hkv, d), 3.0, dtype=dt, device=DEV) for _ in range(2))
    qo2, _, _ = W.rope(q, k, v, pos, freq, slots=slots, interleaved=interleaved, attention_factor=factor, k_out=kc, v_out=vc)
    assert torch.equal(qo2, qo)
    ek, ev = torch.full_like(kc, 3.0), torch.full_like(vc, 3.0)
    ok = (slots >= 0) & (slots < S)
    ek[slots[ok].long()], ev[slots[ok].long()] = ko[ok], v[ok]
    assert torch.equal(kc, ek) and torch.equal(vc, ev)
    # q alone, and in place
    assert torch.equal(W.rope(q, None, None, pos, freq, interleaved=interleaved, attention_factor=factor)[0], qo)
    W.rope(q, k, None, pos, freq, interleaved=interleaved, attention_factor=factor, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, vo)


def test_rope_head_major_and_empty():
    """q given as a transposed (hq, T, d) tensor, k's head shared by all (stride 0), no tokens."""
    say("rope strides")
    dt, g = torch.float16, gen(4)
    q = rnd(g, 6, 50, 64, dtype=dt).transpose(0, 1)
    k = rnd(g, 50, 1, 64, dtype=dt).expand(50, 3, 64)
    pos = torch.arange(50, dtype=torch.int32, device=DEV)
    freq, _ = W.rope_frequencies(64, device=DEV)
    qo, ko, _ = W.rope(q, k, None, pos, freq, q_out=torch.empty(6, 50, 64, dtype=dt, device=DEV).transpose(0, 1))
    for got, src in ((qo, q), (ko, k)):
        ref, mag = rope_ref(src, pos, freq, False, 1.0)
        close(got, ref, rope_bound(ref, mag, dt), "strided")
    assert W.rope(q[:0], k[:0], k[:0], pos[:0], freq)[0].shape == (0, 6, 64)


# ----------------------------------------------------------------------------------------------- tree

def tree_case(seed, dt, lens, hq, hkv, d, page, mask="tree", *, std=1.0, spare=2, width=None):
    """lens: (context, tokens) of each sequence.  Slots no sequence has hold NaN."""
    g = gen(seed)
    rng = np.random.default_rng(seed)
    need = [-(-(c + t) // page) for c, t in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=g)
    wide = max(need) + 1 if width is None else width
    table = torch.full((len(lens), wide), -7, dtype=torch.int32)
    kc, vc = (torch.full((pages * page, hkv, d), float("nan"), dtype=dt, device=DEV) for _ in range(2))
    at = 0
    for b, (c, t) in enumerate(lens):
        own = ids[at:at + need[b]]
        at += need[b]
        put = min(need[b], wide)
        table[b, :put] = own[:put].int()
        j = torch.arange(c + t)
        slots = (own[j // page] * page + j % page).to(DEV) if c + t else j.to(DEV)
        kc[slots], vc[slots] = rnd(g, c + t, hkv, d, dtype=dt), rnd(g, c + t, hkv, d, dtype=dt)
    starts = np.cumsum([0] + [t for _, t in lens]).tolist()
    n = starts[-1]
    c = dict(q=rnd(g, n, hq, d, dtype=dt, std=std), k=kc, v=vc, table=table.to(DEV), page=page, lens=lens,
             context=torch.tensor([x for x, _ in lens], dtype=torch.int32, device=DEV),
             starts=torch.tensor(starts, dtype=torch.int32, device=DEV), mask=None)
    if mask == "tree":
        parents = [int(rng.integers(-1, j)) if j else -1 for _, t in lens for j in range(t)]
        c["mask"] = W.tree_mask_from_parents(parents, starts, device=DEV)
    elif mask == "random":
        words = max(1, -(-max(t for _, t in lens) // 32))
        c["mask"] = torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=g).int().to(DEV)
    return c


def tree_run(c, **kw):
    return W.tree_attention(c["q"], c["k"], c["v"], c["table"], c["context"], c["starts"], c["mask"], page_size=c["page"],
                            **kw)


def tree_ref(c, scale=None):
    """(result, bound): keys that a row does not see are left out, not multiplied by 0."""
    q, dt = c["q"].double().cpu(), c["q"].dtype
    k, v, table = c["k"].cpu(), c["v"].cpu(), c["table"].cpu()
    n, hq, d = q.shape
    hkv = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    pages = k.shape[0] // c["page"]
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    starts = c["starts"].tolist()
    for b, (ctx, t) in enumerate(c["lens"]):
        keys = min(ctx + t, table.shape[1] * c["page"])
        j = torch.arange(keys)
        pg = table[b, j // c["page"]].long()
        on = (pg >= 0) & (pg < pages)
        slot = torch.where(on, pg * c["page"] + j % c["page"], 0)
        kd, vd = k[slot].double(), v[slot].double()
        for i in range(t):
            row = starts[b] + i
            dr = j - ctx
            if c["mask"] is None:
                sees = dr <= i
            else:
                words = c["mask"][row].cpu().long()
                w = (dr // 32).clamp(0, len(words) - 1)
                sees = (dr < 0) | ((dr // 32 < len(words)) & ((words[w] >> (dr % 32) & 1) == 1))
            pick = (sees & on).nonzero()[:, 0]
            if not len(pick):
                continue
            for h in range(hkv):
                rows = slice(h * hq // hkv, (h + 1) * hq // hkv)
                s = scale * (q[row, rows] @ kd[pick, h].t())
                p = s.softmax(-1)
                out[row, rows] = p @ vd[pick, h]
                ds = (2 * (d + 4) * E * abs(scale) * (q[row, rows].abs() @ kd[pick, h].abs().t())).amax(-1, keepdim=True)
                mag = p @ vd[pick, h].abs()
                low = SUB[dt] * vd[pick, h].abs().sum(0) * p.amax(-1, keepdim=True)
                bound[row, rows] = (U[dt] * out[row, rows].abs() + SUB[dt] + low
                                    + (U[dt] + 4 * ds + 2 * (len(pick) + 8) * E) * mag)
    return out, bound


TREE = [  # lens, hq, hkv, d, page, mask
    ([(0, 1)], 1, 1, 64, 1, None),
    ([(0, 1)], 4, 4, 128, 16, "tree"),
    ([(1000, 1)], 32, 8, 128, 16, None),
    ([(31, 1), (32, 1), (33, 1), (127, 1), (128, 1), (129, 1)], 6, 2, 128, 7, None),
    ([(0, 9), (5, 0), (300, 7), (0, 1), (64, 16)], 8, 2, 64, 24, "tree"),
    ([(5000, 5), (1, 3)], 3, 1, 128, 16, "tree"),
    ([(2043, 40), (4095, 33)], 8, 8, 64, 128, "tree"),
    ([(100, 33), (7, 64), (513, 65)], 7, 1, 128, 16, "random"),
    ([(257, 10)] * 3, 40, 8, 128, 32, "tree"),
    ([(77, 100)], 16, 2, 64, 5, None),
    ([(300, 20), (17, 3)], 4, 2, 256, 16, "tree"),
    ([(1500, 2)], 16, 1, 256, 64, None),
    ([(3 * i % 50, 1 + i % 3) for i in range(150)], 2, 1, 64, 8, "tree"),
]


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("i", range(len(TREE)))
def test_tree(i, dt):
    lens, hq, hkv, d, page, mask = TREE[i]
    say("tree", i, str(TREE[i])[:120], dt)
    c = tree_case(100 + i, dt, lens, hq, hkv, d, page, mask, std=1.0 + i % 3)
    out = tree_run(c)
    ref, bound = tree_ref(c)
    close(out, ref, bound, TREE[i])
    assert torch.equal(tree_run(c), out)  # no order of execution shows


def test_tree_rows_and_keys_that_nothing_has():
    """Rows of a mask that is empty, keys past the table's width or on no page, queries of no
    sequence, negative lengths."""
    say("tree nothing")
    c = tree_case(7, torch.bfloat16, [(0, 4), (90, 3)], 4, 2, 64, 16, "random")
    c["mask"][1] = 0
    c["mask"][4:] = 0
    out = tree_run(c)
    ref, bound = tree_ref(c)
    close(out, ref, bound, "empty rows")
    assert not out[1].any()
    c["mask"] = torch.empty(7, 0, dtype=torch.int32, device=DEV)  # no drafted token is seen
    assert not tree_run(c)[:4].any()
    c = tree_case(8, torch.float16, [(200, 5), (60, 2)], 4, 4, 128, 16, "tree", width=9)
    c["table"][0, 3], c["table"][1, 2] = -1, 10 ** 6
    ref, bound = tree_ref(c)
    close(tree_run(c), ref, bound, "lost pages")
    c["table"][:] = -1
    assert not tree_run(c).any()
    c = tree_case(9, torch.bfloat16, [(0, 3), (0, 2)], 2, 1, 64, 16, "tree")
    c["context"][:] = torch.tensor([-5, 0], device=DEV)
    ref, bound = tree_ref(c)
    close(tree_run(c), ref, bound, "negative context")
    c["starts"][1:] = torch.tensor([2, 99], device=DEV)  # clamped to the 5 rows there are
    c["lens"] = [(0, 2), (0, 3)]
    c["mask"] = None
    out = torch.full_like(c["q"], 9.0)
    W.tree_attention(c["q"], c["k"], c["v"], c["table"], c["context"], c["starts"], None, page_size=16, out=out)
    assert torch.isfinite(out[:2]).all()
    c["starts"][:] = torch.tensor([1, 3, 3], device=DEV)
    out = torch.full_like(c["q"], 9.0)
    W.tree_attention(c["q"], c["k"], c["v"], c["table"], c["context"], c["starts"], None, page_size=16, out=out)
    assert (out[0] == 9).all() and (out[3:] == 9).all() and not (out[1:3] == 9).all()


def test_tree_unseen_values_have_no_part():
    """NaN and infinities in K and V of drafted tokens: rows that do not see them keep their bits,
    rows that do get what the formula gives."""
    say("tree not finite")
    nan, inf = float("nan"), float("inf")
    for dt in DTYPES:
        for hq, hkv, d, tokens in ((4, 2, 64, 6), (8, 1, 128, 9), (2, 2, 256, 5), (16, 2, 128, 12)):
            c = tree_case(21, dt, [(70, tokens), (3, tokens)], hq, hkv, d, 16, "tree")
            c["mask"][:] = torch.tensor([(1 << (i % tokens)) | 1 for i in range(2 * tokens)], device=DEV)[:, None]
            clean = tree_run(c)
            for b, ctx in enumerate((70, 3)):
                slot = lambda j: int(c["table"][b, (ctx + j) // 16]) * 16 + (ctx + j) % 16
                c["v"][slot(1), :, 3], c["v"][slot(1), :, 5], c["v"][slot(1), 0, d - 1] = nan, inf, -inf
                c["k"][slot(2)] = nan
                c["v"][slot(2)] = inf
                c["v"][slot(3), :, 0:40] = -inf
            out = tree_run(c)
            rows = torch.tensor([i % tokens not in (1, 2, 3) for i in range(2 * tokens)], device=DEV)
            assert torch.equal(out[rows], clean[rows])
            for i in range(2 * tokens):
                if i % tokens == 1:
                    assert torch.isnan(out[i, :, 3]).all() and (out[i, :, 5] == inf).all()
                    assert (out[i, :hq // hkv, d - 1] == -inf).all() and torch.isfinite(out[i, :, 6:d - 1]).all()
                if i % tokens == 2:
                    assert torch.isnan(out[i]).all()
                if i % tokens == 3:
                    assert (out[i, :, :40] == -inf).all() and torch.isfinite(out[i, :, 40:]).all()


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,tokens", [(2, 3), (8, 4), (8, 9), (16, 12), (16, 40)])
def test_tree_scores_that_jump(dt, hq, tokens):
    """Each row's scores jump by hundreds at a key of its own, anywhere in a long context and in any order, so
    that what has been summed before has to shrink to nothing: every place of a tile in turn."""
    say("tree jumps", dt, hq, tokens)
    c = tree_case(81, dt, [(1500, tokens)], hq, 1, 128, 16, None)
    g = gen(82)
    rows = tokens * hq
    unit = torch.nn.functional.normalize(torch.randn(rows, 128, generator=g), dim=-1)
    c["q"] = (40 * unit).view(tokens, hq, 128).to(dt).to(DEV)
    key = torch.randperm(1500, generator=g)[:rows]
    slot = c["table"].cpu()[0, key // 16].long() * 16 + key % 16
    c["k"] *= 0.05
    c["k"][slot.to(DEV), 0] = (60 * unit).to(dt).to(DEV)
    ref, bound = tree_ref(c)
    close(tree_run(c), ref, bound, "jumps")
    # the same scores growing slowly, past the slack again and again
    ramp = torch.arange(1500) / 1500.0
    slots = (c["table"].cpu()[0, torch.arange(1500) // 16].long() * 16 + torch.arange(1500) % 16).to(DEV)
    c["q"] = (torch.ones(tokens, hq, 128) * 0.5).to(dt).to(DEV)
    c["k"][slots, 0] = (ramp[:, None] * 30 * torch.ones(1500, 128)).to(dt).to(DEV)
    ref, bound = tree_ref(c)
    close(tree_run(c), ref, bound, "ramp")


def test_tree_starts_that_do_not_ascend():
    """More row tiles than ascending starts can make: nothing is written outside the output and the
    workspace, and the next call is right."""
    say("tree starts")
    for tokens, hq in ((64, 8), (2, 8)):
        c = tree_case(31, torch.bfloat16, [(70, tokens)] + [(40, 0)] * 7, hq, 2, 64, 16, mask=None)
        call = W.TreeAttention(c["q"], c["k"], c["v"], c["table"], c["context"], c["starts"], page_size=16)
        size = call.workspace_size
        ws = torch.full((size + (1 << 20),), 90, dtype=torch.uint8, device=DEV)
        good = tree_run(c, workspace=ws).clone()
        ref, bound = tree_ref(c)
        close(good, ref, bound, tokens)
        odd = dict(c, starts=torch.tensor([0, tokens] * 4 + [0], dtype=torch.int32, device=DEV))
        tree_run(odd, workspace=ws)
        assert (ws[size:] == 90).all()
        assert torch.equal(tree_run(c, workspace=ws), good)


def test_tree_strides():
    """q as a slice of a projection, K and V interleaved in one cache, output heads first."""
    say("tree strides")
    dt = torch.bfloat16
    c = tree_case(31, dt, [(100, 5), (40, 6)], 4, 2, 128, 16, "tree")
    ref, bound = tree_ref(c)
    both = torch.stack((c["k"], c["v"]), 1)
    wide = torch.cat((c["q"].flatten(1), torch.full((11, 24), float("nan"), dtype=dt, device=DEV)), 1)
    out = torch.empty(4, 11, 128, dtype=dt, device=DEV).transpose(0, 1)
    got = W.tree_attention(wide[:, :512].unflatten(1, (4, 128)), both[:, 0], both[:, 1], c["table"], c["context"],
                           c["starts"], c["mask"], page_size=16, out=out)
    close(got, ref, bound, "strides")


def test_tree_cache_beyond_4_gib():
    say("tree 64-bit offsets")
    dt, hkv, d, page = torch.bfloat16, 8, 128, 16
    S = (1 << 21) + 64 * page
    kc, vc = (torch.zeros(S, hkv, d, dtype=dt, device=DEV) for _ in range(2))
    g = gen(41)
    kc[-1024:], vc[-1024:] = rnd(g, 1024, hkv, d, dtype=dt), rnd(g, 1024, hkv, d, dtype=dt)
    table = (S // page - 1 - torch.arange(64)).int()[None].to(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    q = rnd(g, 2, 16, d, dtype=dt)
    out = W.tree_attention(q, kc, vc, table, i32(1000), i32(0, 2), page_size=page)
    c = dict(q=q, k=kc[-1024:].clone(), v=vc[-1024:].clone(), table=(63 - torch.arange(64)).int()[None].to(DEV), page=page,
             lens=[(1000, 2)], mask=None, starts=i32(0, 2))
    ref, bound = tree_ref(c)
    close(out, ref, bound, "beyond 4 GiB")


def test_tree_scale_and_no_tokens():
    c = tree_case(51, torch.float16, [(50, 4)], 2, 1, 64, 16, "tree")
    for scale in (0.0, 0.5, -0.3):
        ref, bound = tree_ref(c, scale)
        close(tree_run(c, scale=scale), ref, bound, scale)
    empty = W.tree_attention(c["q"][:0], c["k"], c["v"], c["table"][:0], c["context"][:0], c["starts"][:1], page_size=16)
    assert empty.shape == (0, 2, 64)


# -------------------------------------------------------------------------------------- the calls themselves

def make_calls():
    c = lora_case(61, torch.bfloat16, 70, 5, 24, 264, 136, order="mixed", ranks=True)
    lo = W.LoraMatmul(c["x1"], c["a"], c["b"], c["indices"], c["scale"], ranks=c["ranks"], x3=c["x3"])
    g = gen(62)
    q, k, v = (rnd(g, 9, h, 64, dtype=torch.float16) for h in (4, 2, 2))
    ro = W.Rope(q, k, v, torch.arange(9, dtype=torch.int32, device=DEV), W.rope_frequencies(64, device=DEV)[0])
    t = tree_case(63, torch.bfloat16, [(700, 8), (3000, 8)], 8, 2, 128, 16, "tree")
    tr = W.TreeAttention(t["q"], t["k"], t["v"], t["table"], t["context"], t["starts"], t["mask"], page_size=16)
    return [lo, ro, tr], (c["x1"], q, t["q"])


def flat(out):
    return [x.clone() for x in (out if isinstance(out, tuple) else (out,))]


def test_serve_calls_on_another_stream():
    say("serve streams")
    calls, _ = make_calls()
    plain = [flat(c()) for c in calls]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for c, want in zip(calls, plain):
        for o in (c.out if isinstance(c.out, tuple) else (c.out,)):
            o.fill_(1.0)
        side.wait_stream(torch.cuda.current_stream())
        c(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(flat(c.out), want))
        assert all(torch.equal(a, b) for a, b in zip(flat(c(side.cuda_stream)), want))
        side.synchronize()


def test_serve_calls_in_a_graph():
    """Captured once, replayed over new inputs written into the same tensors."""
    say("serve graph")
    calls, inputs = make_calls()
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
        graph.replay()
        got = [flat(c.out) for c in calls]
        torch.cuda.synchronize()
        want = [flat(c()) for c in calls]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_serve_workspace_given():
    say("serve workspace")
    c = lora_case(71, torch.bfloat16, 33, 3, 16, 128, 64)
    size = W.LoraMatmul(c["x1"], c["a"], c["b"], c["indices"], x3=c["x3"]).workspace_size
    want = W.lora_matmul(c["x1"], c["a"], c["b"], c["indices"], x3=c["x3"])
    ws = torch.full((size // 4 + 64,), float("nan"), device=DEV)
    got = W.lora_matmul(c["x1"], c["a"], c["b"], c["indices"], x3=c["x3"], workspace=ws)
    assert torch.equal(got, want)
    with pytest.raises(ValueError):
        W.lora_matmul(c["x1"], c["a"], c["b"], c["indices"], x3=c["x3"], workspace=ws[:4])
    t = tree_case(72, torch.bfloat16, [(700, 8)], 8, 2, 128, 16, "tree")
    want = tree_run(t)
    size = W.TreeAttention(t["q"], t["k"], t["v"], t["table"], t["context"], t["starts"], t["mask"],
                           page_size=16).workspace_size
    ws = torch.full((size // 4,), float("nan"), device=DEV)
    assert torch.equal(tree_run(t, workspace=ws), want)
