"""Further cases of the serving operators around a step's attention (GPU): many refused drafts, and tables made by hand."""
import pytest
import torch

import weight_quantized_gemm_amd as W
from test_gpu_serve import DEV, DTYPES, gen, rnd, say
from test_gpu_step import ints, layout_ref, verify_case, verify_check

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
