"""Further cases of the serving operators around a step's attention (GPU): many refused drafts, tables made by hand, large
eps, and a bound of prefix attention that is narrower than test_gpu_step.py's."""
import pytest
import torch

import weight_quantized_gemm_amd as W
from test_gpu_serve import DEV, DTYPES, E, SUB, U, close, gen, rnd, say
from test_gpu_step import (NORM, ints, layout_ref, norm_case, norm_check, prefix_case, prefix_run, verify_case,
                           verify_check)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------------------------- layout

@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
def test_layout_feeds_rope_and_attention(dt):
    """rope and tree_attention over the layout's tables give, bit for bit, what they give over tables made by hand, in the
    cache's rows too."""
    say("layout by hand", dt)
    page, ctx, new, rest = 16, [37, 0, 128, 15, 31], [5, 3, 1, 9, 2], 4
    g = gen(740)
    parents = [int(torch.randint(-1, j, (1,), generator=g)) if j else -1 for t in new for j in range(t)] + [0] * rest
    have = [-(-x // page) for x in ctx]
    ids = torch.randperm(sum(have) + 9, generator=g).tolist()
    table, at = [], 0
    for h in have:
        table.append((ids[at:at + h] + [-1] * 10)[:10])
        at += h
    n, free = sum(new) + rest, ids[at:]
    hand = layout_ref(ctx, new, table, free, n, page, [7] * 5, parents, 1)
    given = ints(table)
    out = W.step_layout(ints(ctx), ints(new), given, ints(free), ints([len(free)]), tokens=n, page_size=page,
                        position_offsets=ints([7] * 5), parents=ints(parents), mask_words=1)
    q, k, v = (rnd(g, n, h, 64, dtype=dt) for h in (4, 2, 2))
    caches = [rnd(g, len(ids) * page, 2, 64, dtype=dt) for _ in range(2)]
    freq = W.rope_frequencies(64, device=DEV)[0]

    def step(positions, slots, table, starts, mask):
        kc, vc = (c.clone() for c in caches)
        turned = W.rope(q, k, v, positions, freq, slots=slots, k_out=kc, v_out=vc)[0]
        o = torch.zeros_like(q)
        W.tree_attention(turned, kc, vc, table, ints(ctx), starts, mask, page_size=page, out=o)
        return turned, kc, vc, o

    want = step(ints(hand["positions"]), ints(hand["slots"]), ints(hand["table"]), ints(hand["q_starts"]), ints(hand["tree_mask"]))
    got = step(out.positions, out.slots, given, out.q_starts, out.tree_mask)
    for name, a, b in zip(("q", "k cache", "v cache", "output"), got, want):
        assert torch.equal(a, b), name
    assert not torch.equal(want[1], caches[0]) and want[3][:sum(new)].any(dim=-1).all() and not want[3][sum(new):].any()


# ------------------------------------------------------------------------------------------ norm_rope

@pytest.mark.parametrize("i", [1, 4, 6, 8, 9])
@pytest.mark.parametrize("size,eps", [(64, 2.0 ** 126), (66, 2.0 ** 127), (61, 2.0 ** 128 - 2.0 ** 104), (63, 2.0 ** 126),
                                      (64, 1e-6), (0, 2.0 ** 126), (-63, 2.0 ** -126), (-66, 2.0 ** -126)])
def test_norm_rope_eps_beside_large_heads(i, size, eps):
    """Heads (bf16) whose squares, or their mean with eps, leave fp32 upwards, or its normal numbers downwards: eps is as
    large as they are."""
    say("norm_rope eps", i, size, eps)
    T, hq, hkv, d, rot, inter = 4, 6, 2, *NORM[i][3:6]
    c = norm_case(i, torch.bfloat16, T, hq, hkv, d, rot, inter, 1, "16", True)
    c["q"], c["eps"] = c["q"] * 2.0 ** size, eps
    norm_check(c, W.norm_rope(**c), (i, size, eps))


# --------------------------------------------------------------------------------------------- prefix

def narrow_ref(c, dt):
    """(result, bound, result of weights rounded to one 16-bit term) of tokens that see the whole prefix and their own
    sequence's keys up to themselves.

    u = U: the result's rounding, u |out|.  A weight enters both sums as two 16-bit terms, off by u^2 of it (and in fp16, where the
    second term may be subnormal, by 2^-32 of the largest), in the sum of products and in the sum below it: 2 u^2 mag,
    mag = sum p |v|, and 2^-31 of the largest weight times sum |v|.  Scores of d products in fp32, ds = 2 (d + 4) e scale
    |q| |k| with e = 2^-24, move each weight and the sum: 4 ds mag.  The exponent's argument (below 8: scores here are
    below 1, and fp16's base is 7 lower) and exp2 itself: 10 e a weight, 20 e mag.  2 n products to a sum, both sums: 4 n e mag;
    joining waves and parts: 20 e mag.  One 16-bit term would be off by up to u of each weight."""
    q, k, v = (c[x].double().cpu() for x in ("q", "k", "v"))
    ptable, table, page, starts = c["ptable"].cpu().long(), c["table"].cpu().long(), c["page"], c["starts"].tolist()
    n, hq, d = q.shape
    hkv, u, low = k.shape[1], U[dt], 0 if dt == torch.bfloat16 else 7
    out, bound, one = (torch.zeros_like(q) for _ in range(3))
    for b, (ctx, t) in enumerate(c["seqs"]):
        g = [i for i in range(len(c["prefixes"])) if c["first"][i] <= b < c["first"][i + 1]][0]
        j = torch.arange(c["prefixes"][g][0])
        shared = ptable[g, j // page] * page + j % page
        for i in range(t):
            j = torch.arange(ctx + i + 1)
            rows = torch.cat((shared, table[b, j // page] * page + j % page))
            for h in range(hkv):
                mine = slice(h * hq // hkv, (h + 1) * hq // hkv)
                x, kk, vv = q[starts[b] + i, mine], k[rows, h], v[rows, h]
                s = d ** -0.5 * x @ kk.t()
                p = s.softmax(-1)
                assert (s.amax(-1) - s.amin(-1)).max() < 1
                out[starts[b] + i, mine] = p @ vv
                mag = p @ vv.abs()
                ds = (2 * (d + 4) * E * d ** -0.5 * (x.abs() @ kk.abs().t())).amax(-1, keepdim=True)
                sub = 2.0 ** -31 * p.amax(-1, keepdim=True) * vv.abs().sum(0) if low else 0.0
                bound[starts[b] + i, mine] = (u * out[starts[b] + i, mine].abs() + SUB[dt] + sub
                                              + (2 * u * u + 4 * ds + (4 * len(rows) + 40) * E) * mag)
                w = (2.0 ** low * (s - s.amax(-1, keepdim=True)).exp()).to(dt).double()
                one[starts[b] + i, mine] = w @ vv / w.sum(-1, keepdim=True)
    return out, bound, one


@pytest.mark.parametrize("dt", DTYPES, ids=["bf16", "fp16"])
@pytest.mark.parametrize("prefixes,seqs,hq,hkv,d", [
    ([(9, 2), (11, 2)], [(3, 1), (0, 2), (7, 1), (2, 2)], 8, 2, 64),    # waves that split the keys
    ([(13, 4)], [(3, 1), (0, 2), (7, 1), (2, 2)], 8, 2, 128),
    ([(6, 8)], [(1 + i, 2) for i in range(8)], 8, 4, 256),
    ([(12, 16)], [(i % 5, 2) for i in range(16)], 8, 1, 128),           # waves that split the rows: 256 of them
    ([(10, 9)], [(i % 5, 3) for i in range(9)], 8, 2, 64),              # 108
    ([(10, 4)], [(3, 17)] * 4, 8, 2, 128),                              # and the own keys' 68
], ids=str)
def test_prefix_weights_have_two_terms(prefixes, seqs, hq, hkv, d, dt):
    """Few keys of nearly equal weights: where values cancel, one 16-bit term a weight would show, as it does in the
    plain computation with weights rounded once."""
    say("prefix narrow", prefixes, hq, hkv, d, dt)
    c = prefix_case(750, dt, prefixes, seqs, hq, hkv, d, 16, std=2.0 ** -6)
    ref, bound, one = narrow_ref(c, dt)
    assert ((one - ref).abs() > bound).any()
    close(prefix_run(c), ref, bound, (prefixes, d))


# --------------------------------------------------------------------------------------------- verify

@pytest.mark.parametrize("most", [4, 40, 1000])
def test_verify_many_siblings(most):
    """Children of one token that are refused one after the other before one is accepted, and the residual they leave; random
    numbers past 1, so that few are accepted."""
    say("verify many siblings", most)
    paths = []
    for seed in range(4):
        c = verify_case(700 + seed, [200, 90, 300], 257, True, True, near=3.0)
        c["parents"] = ints([-1 if j == 0 else j // 40 * 40 if j % 40 else max(j - 3, 0) for n in (200, 90, 300) for j in range(n)])
        c["accept"] = (most * torch.rand(590, generator=gen(710 + seed))).to(DEV)
        paths += verify_check(c, (most, seed))[0].tolist()
    assert any(p[0] > 3 for p in paths)  # the children of token 0 are 1 to 39


def test_verify_refusals_take_a_pass_each():
    """1023 refused children of one token over a vocabulary of 65536, half of which the draft never gives: a refusal is one
    pass over two rows of 256 KB, which one compute unit reads in well under 100 us.  0.5 s is five times that for all;
    work that grew with the square of the refusals, an fp64 division for each element and each refusal before it, would
    be 65536 * 1023^2 / 2 = 3.4e10 of them, at 1e10 a second on one compute unit."""
    say("verify a pass each")
    n, V = 1024, 65536
    c = verify_case(720, [8], V, True, True)
    p, q = c["target"][:1], c["draft"][:1].clone()
    q[:, ::2] = 0
    q /= q.sum()
    tokens = torch.multinomial(q[0].cpu(), n, replacement=True, generator=gen(721)).int().to(DEV)
    c = dict(target=p.repeat(n, 1), draft=q.repeat(n, 1), tokens=tokens, starts=ints([0, n]), parents=ints([-1] + [0] * (n - 1)),
             accept=torch.full((n,), 1e9, device=DEV), sample=torch.tensor([0.4], device=DEV), depth=4)
    out = verify_check(c, "all refused")
    assert out[1].tolist() == [0] and out[2].item() % 2 == 0  # what the draft never gives is what is left
    call = W.VerifyDrafts(c["target"], c["tokens"], c["starts"], c["accept"], c["sample"], depth=4, draft=c["draft"],
                          parents=c["parents"])
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    call()
    end.record()
    torch.cuda.synchronize()
    print(f"1023 refusals: {begin.elapsed_time(end):.2f} ms", flush=True)
    assert begin.elapsed_time(end) < 500
