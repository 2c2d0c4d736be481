"""The serving operators where variants, tiles and types meet their ends (GPU); references and bounds are those
of test_gpu_serve.py."""
import math

import pytest
import torch

import test_gpu_serve as base
import weight_quantized_gemm_amd as W

pytestmark = pytest.mark.gpu

DEV, DTYPES = base.DEV, base.DTYPES
say, close, gen, rnd = base.say, base.close, base.gen, base.rnd
tree_case, tree_run, tree_ref = base.tree_case, base.tree_run, base.tree_ref
IDS = ["bf16", "fp16"]


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (14, 2, 64), (4, 1, 128), (8, 2, 256)])
def test_tree_long_sequences_among_short_ones(hq, hkv, d, dt):
    """One sequence of several tiles whose height its neighbours' single tokens chose, each tile's keys shared by
    several workgroups: every row is joined from its own tile's parts."""
    say("tree uneven", hq, hkv, d, dt)
    c = tree_case(91, dt, [(300, 5), (310, 1), (290, 1), (305, 1), (297, 1)], hq, hkv, d, 16, None)
    ref, bound = tree_ref(c)
    for _ in range(5):
        out = torch.full_like(c["q"], 9.0)
        close(tree_run(c, out=out), ref, bound, (hq, hkv, d))


@pytest.mark.parametrize("which", range(3), ids=["adapters", "rope", "tree"])
def test_calls_dropped_while_in_flight_on_another_stream(which):
    """Memory that a call owns is not handed out again before the call has ended there."""
    say("serve dropped", which)
    call = base.make_calls()[0][which]
    want = base.flat(call())
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        call = base.make_calls()[0][which]
        outs = [t for t in (call.out if isinstance(call.out, tuple) else (call.out,))]
        own = outs[0] if which == 1 else call.workspace
        at, shape, kind = own.data_ptr(), own.shape, own.dtype
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        call(handle)
        held = [] if which == 1 else outs
        del call, own, outs
        for _ in range(32):  # of the size that was just given back, on the stream that it was allocated on
            again = torch.zeros(shape, dtype=kind, device=DEV)
            assert again.data_ptr() != at
            held.append(again)
        side.synchronize()
        if which != 1:
            assert torch.equal(held[0], want[0])


@pytest.mark.parametrize("rows", [1, 8, 32, 48, 112, 200])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
def test_tree_small_weights_count(dt, d, rows):
    """Every 32nd key has the largest score and a value of 0; the result is what the others, 2^-17 to 2^-25 of it, add.
    Scores are exact here.  A weight is off by 2^-8 (bf16) or 2^-11 (fp16) of it, or 2^-32 of the largest
    (fp16), and by the 2^-21 of its base-2 exponent's rounding."""
    say("tree small weights", dt, d, rows)
    keys = 1024
    g = gen(97)
    c = tree_case(97, dt, [(keys - 1, 1)], rows, 1, d, 16, None)
    c["q"].zero_()
    c["q"][:, :, 0] = 1.0
    order = torch.arange(keys)
    slot = (c["table"].cpu()[0, order // 16].long() * 16 + order % 16).to(DEV)
    score = -(96 + torch.randint(0, 44, (keys,), generator=g)).float() / 8  # -12 to -17.4
    score[::32] = 0.0
    c["k"].zero_()
    c["k"][slot, 0, 0] = score.to(dt).to(DEV)
    v = 1000 + 1000 * torch.rand(keys, d, generator=g)
    v[::32] = 0.0
    c["v"][slot, 0] = v.to(dt).to(DEV)
    p = score.double().softmax(0)
    vd = c["v"][slot, 0].double().cpu()
    ref = (p @ vd).expand(1, rows, d)
    low = 2.0 ** -32 * float(p.max()) * vd.sum(0) if dt == torch.float16 else 0.0
    close(tree_run(c, scale=1.0), ref, 2 * base.U[dt] * ref + base.SUB[dt] + low + 2.0 ** -20 * ref, rows)


# hq, hkv, d, tokens: every tile height, number of waves and head size that a call may get
VARIANTS = [(4, 2, 64, 3), (8, 2, 64, 7), (8, 2, 64, 11), (8, 1, 64, 13), (16, 1, 64, 12), (4, 2, 128, 3), (8, 2, 128, 7),
            (8, 2, 128, 11), (8, 1, 128, 13), (16, 1, 128, 12), (4, 2, 256, 3), (16, 1, 256, 4)]
VIDS = ["h%d_%d_d%d_t%d" % v for v in VARIANTS]


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("variant", VARIANTS, ids=VIDS)
def test_tree_infinities_of_the_context(variant, dt):
    """Infinities in V give infinities of their sign, both signs or a NaN give NaN, wherever the key stands and
    however little its weight is; other columns and other cached heads stay what they are."""
    hq, hkv, d, tokens = variant
    say("tree seen infinities", variant, dt)
    c = tree_case(111, dt, [(500, tokens), (300, tokens)], hq, hkv, d, 16, "tree", std=3.0)
    clean = tree_run(c)
    odd = torch.zeros(hkv, d, dtype=torch.bool)
    g = gen(112)
    for b, ctx in enumerate((500, 300)):
        for key in (0, 31, 32, 33, 100, 127, 128, 250, ctx - 1, ctx):
            slot = int(c["table"][b, key // 16]) * 16 + key % 16
            h, col = int(torch.randint(0, hkv, (), generator=g)), int(torch.randint(0, d // 2, (), generator=g))
            c["v"][slot, h, col] = (float("inf"), -float("inf"), float("nan"))[key % 3 if key < 128 else 0]
            odd[h, col] = True
    out = tree_run(c)
    ref, bound = tree_ref(c)
    close(out, ref, bound, variant)
    assert torch.isinf(out).any()
    same = ~odd.repeat_interleave(hq // hkv, 0).to(DEV)
    # (bases do not move between the two ways: the same weights, up to the rounding of their sums)
    assert torch.isfinite(out[:, same]).all() and (out[:, same] - clean[:, same]).abs().max() < 0.1


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("variant", VARIANTS, ids=VIDS)
def test_tree_is_off_by_its_last_rounding(variant, dt):
    """In the root mean square the result is off by what rounding the exact one once gives.  The rest are weights of
    two 16-bit terms, 2^-16 (bf16) or 2^-22 (fp16) of each, and scores of about 10 whose fp32 sums are off by a
    few 2^-24 of that, 2^-18 of a weight: a hundredth of the rounding to 2^-8 or 2^-11, which adds in the
    squares.  One 16-bit term would add another rounding of the result's own size, a factor of 1.4."""
    hq, hkv, d, tokens = variant
    say("tree rms", variant, dt)
    c = tree_case(121, dt, [(700, tokens), (400, tokens)], hq, hkv, d, 16, "tree")
    ref, _ = tree_ref(c)
    rms = lambda x: float(x.square().mean().sqrt())
    assert rms(tree_run(c).double().cpu() - ref) < 1.05 * rms(ref.to(dt).double() - ref)


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("m", [3, 70, 2100])
@pytest.mark.parametrize("r", [16, 32, 72])
def test_lora_numbers_far_below_the_largest(r, m, dt):
    """One rank's first product is 2^16 to 2^22 times the others, and most columns of b are 0 there.  First products
    are exact here; they are off by 2^-16 of each in bf16, and in fp16 by 2^-39 of the largest, 2^-17 of any."""
    say("lora far below", r, m, dt)
    g = gen(131)
    k, n = 64, 136
    x1 = torch.zeros(m, k)
    x1[:, 0] = 2.0 ** torch.randint(-1, 2, (m,), generator=g)
    a = torch.zeros(2, r, k)
    a[:, :, 0] = 2.0 ** torch.empty(2, r).uniform_(-10, -4, generator=g)
    a[0, 5, 0], a[1, 1, 0] = 4096.0, 2048.0
    b = torch.randn(2, n, r, generator=g)
    b[0, 8:, 5], b[1, 8:, 1] = 0.0, 0.0
    c = dict(x1=x1.to(dt).to(DEV), a=a.to(dt).to(DEV), b=b.to(dt).to(DEV), x3=None, ranks=None,
             indices=torch.randint(0, 2, (m,), generator=g).int().to(DEV), scale=torch.tensor([64.0, -32.0], device=DEV))
    ref, bound = base.lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], None, None)
    if dt == torch.float16:  # the few columns that meet the large rank may pass the type's range
        ref = torch.where(ref.abs() >= 65520, ref.sign() * math.inf, ref)
    close(base.lora_run(c), ref, bound, (r, m))


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,r,n", [(1, 8, 8), (40, 16, 136), (300, 32, 264), (70, 136, 72), (2100, 16, 136), (2300, 200, 72)])
def test_lora_infinities_of_b(m, r, n, dt):
    """An infinity of b gives infinities in its column for the tokens of its adapter, of the sign that the first product
    has, both signs a NaN; every other element is what it was."""
    say("lora infinite b", m, r, n, dt)
    c = base.lora_case(141, dt, m, 3, r, 520, n, order="mixed" if m > 1 else "one", ranks=m > 1)
    clean = base.lora_run(c)
    c["b"][0, 3, 1], c["b"][1, n - 1, r // 2], c["b"][2, 5, 0] = math.inf, -math.inf, math.inf
    c["b"][2, 0, 0], c["b"][2, 0, 2] = math.inf, -math.inf
    ref, bound = base.lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], c["ranks"], c["x3"])
    out = base.lora_run(c)
    close(out, ref, bound, (m, r, n))
    fin = torch.isfinite(ref).to(DEV)
    assert torch.equal(out[fin], clean[fin]) and not fin.all()


def test_lora_sums_that_a_factor_brings_back():
    """bf16 reaches 2^127: a tiny first product against huge numbers of b passes fp32 between the row's factor and
    its return, not in the result."""
    say("lora factor")
    for m in (20, 2100):
        c = base.lora_case(142, torch.bfloat16, m, 2, 24, 64, 72, order="mixed")
        c["x1"] *= 2.0 ** -60
        c["a"] *= 2.0 ** -40
        c["b"] = (c["b"].sign() * 2.0 ** 127 * 1.5).to(torch.bfloat16)
        ref, bound = base.lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], None, c["x3"])
        close(base.lora_run(c), ref, bound, m)


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("variant", VARIANTS, ids=VIDS)
def test_tree_every_variant_where_nothing_is_seen(variant, dt):
    """Empty rows of a mask, pages that do not exist, a table narrower than the context, scales of either sign and zero,
    scores of -inf: in each kernel and head size."""
    hq, hkv, d, tokens = variant
    say("tree variants", variant, dt)
    c = tree_case(151, dt, [(200, tokens), (60, tokens), (0, tokens)], hq, hkv, d, 16, "random", width=13)
    c["mask"][1], c["mask"][2 * tokens + 1] = 0, 0
    c["table"][0, 3], c["table"][1, 2] = -1, 10 ** 6
    for scale in (None, 0.0, -0.3):
        ref, bound = tree_ref(c, scale)
        out = tree_run(c, scale=scale)
        close(out, ref, bound, (variant, scale))
        assert torch.equal(tree_run(c, scale=scale), out)
    assert not out[2 * tokens + 1].any()
    for key in range(60 + tokens):  # what the second sequence sees is -inf in one column that its queries multiply
        slot = int(c["table"][1, key // 16]) * 16 + key % 16
        if 0 <= slot < c["k"].shape[0]:
            c["k"][slot, :, 7] = -math.inf
    c["q"][:, :, 7] = 1.0
    out = tree_run(c)
    assert not out[tokens:2 * tokens].any() and torch.isfinite(out).all()
    c["table"][:] = -1
    assert not tree_run(c).any()


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("variant", VARIANTS, ids=VIDS)
def test_tree_every_variant_unseen_values(variant, dt):
    """NaN and infinities in K and V of drafted tokens that one token in turn sees."""
    hq, hkv, d, tokens = variant
    say("tree variants unseen", variant, dt)
    nan, inf = math.nan, math.inf
    c = tree_case(161, dt, [(70, tokens), (3, tokens)], hq, hkv, d, 16, "tree")
    c["mask"][:] = torch.tensor([(1 << (i % tokens)) | 1 for i in range(2 * tokens)], device=DEV)[:, None]
    clean = tree_run(c)
    for b, ctx in enumerate((70, 3)):
        one, two = (int(c["table"][b, (ctx + j) // 16]) * 16 + (ctx + j) % 16 for j in (1, 2))
        c["v"][one, :, 3], c["v"][one, :, 5], c["v"][one, 0, d - 1] = nan, inf, -inf
        c["k"][two], c["v"][two] = nan, inf
    out = tree_run(c)
    for i in range(2 * tokens):
        if i % tokens == 1:
            assert torch.isnan(out[i, :, 3]).all() and (out[i, :, 5] == inf).all()
            assert (out[i, :hq // hkv, d - 1] == -inf).all() and torch.isfinite(out[i, :, 6:d - 1]).all()
        elif i % tokens == 2:
            assert torch.isnan(out[i]).all()
        else:
            assert torch.equal(out[i], clean[i])


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([(100, 200), (900, 1), (33, 1), (0, 1), (700, 2)], 8, 2, 64), ([(0, 300), (1000, 1), (50, 3)], 4, 4, 64),
    ([(40, 90), (500, 1), (500, 1)], 8, 2, 128), ([(300, 150), (20, 1)], 6, 2, 128), ([(10, 70), (900, 1)], 4, 2, 256),
    ([(500, 1)] * 40 + [(64, 64)], 4, 1, 128)])
def test_tree_pieces_of_prompts_among_single_tokens(lens, hq, hkv, d, dt):
    """Sequences of unlike token counts: one tile height, from the average, for all of them."""
    say("tree unlike", str(lens)[:60], hq, hkv, d, dt)
    for mask in (None, "tree"):
        c = tree_case(171, dt, lens, hq, hkv, d, 16, mask)
        ref, bound = tree_ref(c)
        close(tree_run(c), ref, bound, mask)


@pytest.mark.parametrize("dt", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,r,k,n", [(1, 16, 4096, 4096), (64, 32, 1024, 520), (777, 64, 512, 264), (3000, 72, 520, 136)])
def test_lora_is_off_by_its_last_rounding(m, r, k, n, dt):
    """In the root mean square, as for the attention: terms to 2^-16 (bf16) and 2^-22 (fp16) of the first product, and
    sums of some thousand fp32 products, whose roundings add to a few 2^-22 of their size."""
    say("lora rms", m, r, k, n, dt)
    c = base.lora_case(181, dt, m, 4, r, k, n, order="mixed" if m > 1 else "one", x3=False)
    ref, _ = base.lora_ref(c["x1"], c["a"], c["b"], c["indices"], c["scale"], None, None)
    rms = lambda x: float(x.square().mean().sqrt())
    assert rms(base.lora_run(c).double() - ref) < 1.05 * rms(ref.to(dt).double() - ref)


def test_verify_step_without_adapters():
    """The example's block where no request has an adapter."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    from verify_step import VerifyStep
    say("verify step without adapters")
    step = VerifyStep([40, 3], [[-1, 0, 0], [-1]], [-1, -1])
    want = step.plain()
    got = step.step().double().cpu()
    assert float((got - want).norm() / want.norm()) < 8 * 2.0 ** -9  # as in test_gpu_verify_step.py
