"""Host side of the serving operators: argument rules through the C ABI, the binding's helpers, and the
division that the kernels use (CPU; every refused call returns before any device work)."""
import ctypes
import itertools
import math
import os
import re
import shutil
import subprocess

import pytest

import weight_quantized_gemm_amd as W
from weight_quantized_gemm_amd import make_desc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, INVALID = W.WQ_OK, W.WQ_ERR_PARAM_NULLPTR, W.WQ_ERR_PARAM_INVALID
BF, HF, F32, I32, I8 = W.WQ_BF16, W.WQ_F16, W.WQ_F32, W.WQ_I32, W.WQ_I8
_fresh = itertools.count(0x10000000, 0x1000000)


def D(shape, dt, ptr=None, strides=None):
    return make_desc(shape, dt, next(_fresh) if ptr is None else ptr, strides)


def ref(d):
    return ctypes.byref(d) if d is not None else None


def test_header_binding_and_library_agree(wqlib):
    src = open(os.path.join(ROOT, "include", "wqserve.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"^\s*int\s+(wq_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(W.SERVE_EXPORTS)
    if not os.environ.get("WQ_HOST_LIBRARY"):
        assert all(hasattr(wqlib, n) for n in names)


# ------------------------------------------------------------------------------------------- adapters

def lora_args(m=6, k=64, L=3, r=16, n=40, dt=BF):
    return dict(x1=D([m, k], dt), a=D([L, r, k], dt), b=D([L, n, r], dt), indices=D([m], I32), scale=D([L], F32),
                ranks=D([L], I32), x3=D([m, n], dt), output=D([m, n], dt))


def lora(wqlib, ws=True, **kw):
    args = {**lora_args(), **kw}
    size = ctypes.c_uint64(123)
    st = wqlib.wq_lora_matmul_get_workspace_size(*map(ref, args.values()), ctypes.byref(size) if ws else None)
    return (st, size.value) if st == OK else st


def test_lora_accepts(wqlib):
    st, size = lora(wqlib)
    assert st == OK and size >= 6 * 16 * 4 and size % 256 == 0
    assert lora(wqlib, scale=None, ranks=None, x3=None)[0] == OK
    assert lora(wqlib, **lora_args(dt=HF))[0] == OK
    st, size = lora(wqlib, **lora_args(m=0))
    assert (st, size) == (OK, 0)
    # 3-D, strided rows, one row for all of x3, x3 in place
    assert lora(wqlib, x1=D([2, 3, 64], BF, strides=[264, 88, 1]), x3=D([2, 3, 40], BF), output=D([2, 3, 40], BF))[0] == OK
    assert lora(wqlib, x3=D([6, 40], BF, strides=[0, 1]))[0] == OK
    y = D([6, 40], BF, strides=[48, 1])
    assert lora(wqlib, x3=y, output=y)[0] == OK
    assert lora(wqlib, indices=D([6], I32, ptr=0x10004), ranks=D([3], I32, ptr=0x2000c))[0] == OK
    big = lora_args(m=1 << 28, L=65535, r=256, k=65528, n=4096)
    st, size = lora(wqlib, **big)
    assert st == OK and size >= (1 << 28) * 256 * 4


def test_lora_refuses(wqlib):
    for name in ("x1", "a", "b", "indices", "output"):
        assert lora(wqlib, **{name: None}) == NULLPTR
    assert lora(wqlib, ws=False) == NULLPTR
    for name, d in lora_args().items():
        null = D([d.shape[i] for i in range(d.ndim)], d.dtype, ptr=0)
        assert lora(wqlib, **{name: null}) == NULLPTR, name
        wrong = D([d.shape[i] for i in range(d.ndim)], I8)
        assert lora(wqlib, **{name: wrong}) == INVALID, name
        if d.dtype == BF:
            other = D([d.shape[i] for i in range(d.ndim)], HF)
            assert lora(wqlib, **{name: other}) == INVALID, name
        grown = D([d.shape[i] + (8 if i == 0 else 0) for i in range(d.ndim)], d.dtype)
        assert lora(wqlib, **{name: grown}) == INVALID, name
        flat = D([8] * (4 - d.ndim), d.dtype)
        assert lora(wqlib, **{name: flat}) == INVALID, name
    for bad in (dict(k=60), dict(k=0), dict(k=65536), dict(r=4), dict(r=20), dict(r=264), dict(n=12), dict(n=0),
                dict(n=(1 << 22) + 8), dict(L=0), dict(L=65536), dict(m=(1 << 28) + 1)):
        assert lora(wqlib, **lora_args(**bad)) == INVALID, bad
    # layouts: misaligned, odd strides, overlapping output rows, a 3-D form whose rows do not fold
    assert lora(wqlib, x1=D([6, 64], BF, ptr=0x10008)) == INVALID
    assert lora(wqlib, indices=D([6], I32, ptr=0x10002)) == INVALID
    for s in ([68, 1], [-64, 1], [64, 2], [1 << 41, 1]):
        assert lora(wqlib, x1=D([6, 64], BF, strides=s)) == INVALID, s
    assert lora(wqlib, output=D([6, 40], BF, strides=[32, 1])) == INVALID
    assert lora(wqlib, output=D([6, 40], BF, strides=[0, 1])) == INVALID
    assert lora(wqlib, **lora_args(m=1 << 28, n=1 << 22)) == INVALID  # an output of more than 2^40 elements
    assert lora(wqlib, x1=D([2, 3, 64], BF, strides=[256, 64, 1]), x3=D([2, 3, 40], BF),
                output=D([2, 3, 40], BF)) == INVALID
    assert lora(wqlib, a=D([3, 16, 64], BF, strides=[1024, 72, 1])) == INVALID
    assert lora(wqlib, b=D([3, 40, 16], BF, strides=[640, 1, 40])) == INVALID
    # aliases
    y = D([6, 64], BF)
    assert lora(wqlib, x1=y, output=D([6, 40], BF, ptr=y.data)) == INVALID
    assert lora(wqlib, x3=D([6, 40], BF, ptr=y.data, strides=[48, 1]), output=D([6, 40], BF, ptr=y.data)) == INVALID


def test_lora_workspace_is_checked(wqlib):
    args = lora_args()
    size = lora(wqlib, **args)[1]
    call = lambda ws, n: wqlib.wq_lora_matmul(*map(ref, args.values()), ctypes.c_void_p(ws), n, None)
    assert call(0x100000, size - 1) == INVALID
    assert call(0, size) == NULLPTR
    assert call(0x100010, size) == INVALID
    none = {**lora_args(m=0)}
    assert wqlib.wq_lora_matmul(*map(ref, none.values()), None, 0, None) == OK


# ----------------------------------------------------------------------------------------------- rope

def rope_args(T=5, hq=4, hkv=2, d=64, rot=64, S=9, dt=HF):
    return dict(q=D([T, hq, d], dt), k=D([T, hkv, d], dt), v=D([T, hkv, d], dt), positions=D([T], I32),
                inv_freq=D([rot // 2], F32), slots=D([T], I32), layout=0, factor=1.0, q_out=D([T, hq, d], dt),
                k_out=D([S, hkv, d], dt), v_out=D([S, hkv, d], dt))


def rope(wqlib, **kw):
    a = {**rope_args(), **kw}
    a = [ref(x) if isinstance(x, W.WqTensor) or x is None else x for x in a.values()]
    return wqlib.wq_rope(*a, None)


def test_rope_accepts_no_tokens(wqlib):
    assert rope(wqlib, **rope_args(T=0)) == OK
    assert rope(wqlib, **{**rope_args(T=0), "k": None, "v": None, "slots": None, "k_out": None, "v_out": None}) == OK
    assert rope(wqlib, **rope_args(T=0, hq=1, hkv=1, d=8, rot=2, S=0)) == OK


def test_rope_refuses(wqlib):
    for name in ("q", "positions", "inv_freq", "q_out", "k_out", "v_out"):
        assert rope(wqlib, **{name: None}) == NULLPTR, name
    for name, d in rope_args().items():
        if not isinstance(d, W.WqTensor):
            continue
        shape = [d.shape[i] for i in range(d.ndim)]
        assert rope(wqlib, **{name: D(shape, d.dtype, ptr=0)}) == NULLPTR, name
        assert rope(wqlib, **{name: D(shape, I8)}) == INVALID, name
        if d.dtype == HF:
            assert rope(wqlib, **{name: D(shape, BF)}) == INVALID, name
            assert rope(wqlib, **{name: D(shape, HF, ptr=0x10008)}) == INVALID, name
            assert rope(wqlib, **{name: D(shape, HF, strides=[4 * shape[1] * 64, 68, 1])}) == INVALID, name
            assert rope(wqlib, **{name: D(shape[:2] + [72], HF)}) == INVALID, name
            assert rope(wqlib, **{name: D(shape[:2], HF)}) == INVALID, name
        if name not in ("inv_freq",):
            assert rope(wqlib, **{name: D([shape[0] + 1] + shape[1:], d.dtype)}) == INVALID, name
    assert rope(wqlib, layout=2) == INVALID and rope(wqlib, layout=-1) == INVALID
    assert rope(wqlib, factor=math.inf) == INVALID and rope(wqlib, factor=math.nan) == INVALID
    for bad in (dict(rot=66), dict(rot=0), dict(d=60), dict(d=264), dict(d=0, rot=0), dict(hq=0), dict(hkv=0),
                dict(hq=65536)):
        assert rope(wqlib, **rope_args(**bad)) == INVALID, bad
    # v, slots or outputs without k or v; rows without slots are the tokens'
    assert rope(wqlib, k=None) == INVALID
    assert rope(wqlib, k=None, v=None, k_out=None, v_out=None) == INVALID
    assert rope(wqlib, v=None) == INVALID
    assert rope(wqlib, slots=None) == INVALID
    # overlapping rows and aliases
    assert rope(wqlib, q_out=D([5, 4, 64], HF, strides=[192, 64, 1])) == INVALID
    a = rope_args()
    assert rope(wqlib, **{**a, "k_out": D([9, 2, 64], HF, ptr=a["k"].data)}) == INVALID
    assert rope(wqlib, **{**a, "v_out": D([9, 2, 64], HF, ptr=a["k_out"].data)}) == INVALID
    assert rope(wqlib, **{**a, "q_out": D([5, 4, 64], HF, ptr=a["q"].data, strides=[512, 64, 1])}) == INVALID
    assert rope(wqlib, **{**a, "q_out": D([5, 4, 64], HF, ptr=a["k"].data)}) == INVALID


# ----------------------------------------------------------------------------------------------- tree

def tree_args(N=7, B=3, hq=8, hkv=2, d=128, page=16, pages=20, width=6, words=1, dt=BF):
    return dict(q=D([N, hq, d], dt), k_cache=D([pages * page, hkv, d], dt), v_cache=D([pages * page, hkv, d], dt),
                block_table=D([B, width], I32), context_lens=D([B], I32), q_starts=D([B + 1], I32),
                tree_mask=D([N, words], I32), page_size=page, output=D([N, hq, d], dt))


def tree(wqlib, ws=True, **kw):
    a = {**tree_args(), **kw}
    a = [ref(x) if isinstance(x, W.WqTensor) or x is None else x for x in a.values()]
    size = ctypes.c_uint64(123)
    st = wqlib.wq_tree_attention_get_workspace_size(*a, ctypes.byref(size) if ws else None)
    return (st, size.value) if st == OK else st


def test_tree_accepts(wqlib):
    st, size = tree(wqlib)
    assert st == OK and size % 256 == 0 and size > 0
    assert tree(wqlib, tree_mask=None)[0] == OK
    assert tree(wqlib, tree_mask=D([7, 0], I32, ptr=0))[0] == OK
    assert tree(wqlib, **tree_args(d=64, hkv=8))[0] == OK and tree(wqlib, **tree_args(d=256, dt=HF))[0] == OK
    assert tree(wqlib, **tree_args(N=0))[0:2] == (OK, 0) and tree(wqlib, **tree_args(B=0))[0:2] == (OK, 0)
    assert tree(wqlib, **tree_args(pages=0))[0] == OK and tree(wqlib, **tree_args(width=0))[0] == OK
    assert tree(wqlib, **tree_args(page=1, pages=300))[0] == OK
    both = [20 * 16, 2, 128]
    assert tree(wqlib, k_cache=D(both, BF, strides=[512, 128, 1]), v_cache=D(both, BF, strides=[512, 128, 1]))[0] == OK
    assert tree(wqlib, q=D([7, 8, 128], BF, strides=[2048, 128, 1]))[0] == OK
    # a workspace of some megabytes whatever the lengths, and notes of a few bytes a query token
    for kw in (dict(N=1 << 24, B=65535, width=127, page=1 << 20, pages=2047), dict(N=64, B=1, width=1 << 17)):
        st, size = tree(wqlib, **tree_args(**kw))
        assert st == OK and size <= (66 << 20) + 2 * kw["N"]


def test_tree_longest_tables(wqlib):
    assert tree(wqlib, **tree_args(page=1 << 16, width=32767, pages=4))[0] == OK
    assert tree(wqlib, **tree_args(page=1 << 15, width=65535, pages=4)) == INVALID
    assert tree(wqlib, **tree_args(page=1, width=(1 << 31) - 65535, pages=4)) == INVALID
    assert tree(wqlib, **tree_args(page=1, width=(1 << 31) - 65536, pages=4))[0] == OK


def test_tree_refuses(wqlib):
    for name in ("q", "k_cache", "v_cache", "block_table", "context_lens", "q_starts", "output"):
        assert tree(wqlib, **{name: None}) == NULLPTR, name
    assert tree(wqlib, ws=False) == NULLPTR
    for name, d in tree_args().items():
        if not isinstance(d, W.WqTensor):
            continue
        shape = [d.shape[i] for i in range(d.ndim)]
        assert tree(wqlib, **{name: D(shape, d.dtype, ptr=0)}) == NULLPTR, name
        assert tree(wqlib, **{name: D(shape, F32)}) == INVALID, name
        assert tree(wqlib, **{name: D([shape[0] + 1] + shape[1:], d.dtype)}) == INVALID, name
        if d.dtype == BF:
            assert tree(wqlib, **{name: D(shape, HF)}) == INVALID, name
            assert tree(wqlib, **{name: D(shape, BF, ptr=0x10008)}) == INVALID, name
            assert tree(wqlib, **{name: D(shape, BF, strides=[1028, 128, 1])}) == INVALID, name
            assert tree(wqlib, **{name: D(shape, BF, strides=[1024, -128, 1])}) == INVALID, name
            assert tree(wqlib, **{name: D(shape, BF, strides=[1024, 128, 2])}) == INVALID, name
        else:
            assert tree(wqlib, **{name: D(shape, I32, ptr=0x10002)}) == INVALID, name
    for bad in (dict(d=96), dict(d=512), dict(hq=7), dict(hkv=3), dict(hkv=0), dict(hq=2, hkv=4), dict(N=(1 << 24) + 1), dict(N=1 << 22, hq=512),
                dict(B=65536), dict(width=1 << 27), dict(words=(1 << 20) + 1)):
        assert tree(wqlib, **tree_args(**bad)) == INVALID, bad
    for page in (0, -16, 7, (1 << 20) + 1):
        assert tree(wqlib, page_size=page) == INVALID, page
    assert tree(wqlib, k_cache=D([320, 2, 128], BF, strides=[1 << 31, 128, 1])) == INVALID
    assert tree(wqlib, output=D([7, 8, 128], BF, strides=[512, 128, 1])) == INVALID
    a = tree_args()
    assert tree(wqlib, **{**a, "output": a["q"]}) == INVALID
    assert tree(wqlib, **{**a, "output": D([7, 8, 128], BF, ptr=a["v_cache"].data)}) == INVALID


def test_tree_scale_and_workspace_are_checked(wqlib):
    a = tree_args()
    size = tree(wqlib, **a)[1]
    t = [ref(x) for x in list(a.values())[:7]]

    def call(scale, ws, n):
        return wqlib.wq_tree_attention(*t, 16, scale, ref(a["output"]), ctypes.c_void_p(ws), n, None)
    assert call(math.nan, 0x100000, size) == INVALID and call(math.inf, 0x100000, size) == INVALID
    assert call(1.0, 0x100000, size - 1) == INVALID
    assert call(1.0, 0, size) == NULLPTR
    assert call(1.0, 0x100080, size) == INVALID


# -------------------------------------------------------------------------------------------- helpers

def test_rope_frequencies():
    f, s = W.rope_frequencies(8, 10000.0)
    assert s == 1.0 and [round(float(x), 7) for x in f] == [1.0, 0.1, 0.01, 0.001]
    f4, s = W.rope_frequencies(8, scaling="linear", factor=4.0)
    assert s == 1.0 and all(abs(float(a) * 4 - float(b)) < 1e-7 for a, b in zip(f4, f))
    fb, _ = W.rope_frequencies(8, scaling="base", factor=4.0)
    assert float(fb[0]) == 1.0 and abs(float(fb[3]) / (float(f[3]) / 4) - 1) < 1e-6
    fr, s = W.rope_frequencies(128, scaling="ramp", factor=8.0, original_length=4096)
    f, _ = W.rope_frequencies(128)
    assert abs(s - (0.1 * math.log(8) + 1)) < 1e-12
    assert float(fr[0]) == float(f[0]) and abs(float(fr[-1]) / (float(f[-1]) / 8) - 1) < 1e-6
    turns = [4096 * float(x) / (2 * math.pi) for x in f]
    for a, b, t in zip(fr, f, turns):
        if t > 33:
            assert float(a) == float(b)
        if t < 0.9:
            assert abs(float(a) / (float(b) / 8) - 1) < 1e-6
        assert float(b) / 8 * 0.999999 <= float(a) <= float(b) * 1.000001
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="ramp", factor=2.0)):
        with pytest.raises(ValueError):
            W.rope_frequencies(**bad)


def test_tree_mask_from_parents():
    m = W.tree_mask_from_parents([-1, 0, 0, 2, -1, 0], [0, 4, 4, 6])
    assert m.tolist() == [[1], [3], [5], [13], [1], [3]]
    chain = W.tree_mask_from_parents(list(range(-1, 69)), [0, 70])
    assert chain.shape == (70, 3)
    assert chain[31].tolist() == [-1, 0, 0] and chain[63].tolist() == [-1, -1, 0] and chain[69].tolist() == [-1, -1, 63]
    assert W.tree_mask_from_parents([], [0]).shape == (0, 1)
    for parents, starts in (([0], [0, 1]), ([-1, 1], [0, 2]), ([-2], [0, 1]), ([-1], [0, 2]), ([-1, -1], [1, 2]),
                            ([-1, -1], [0, 3, 2])):
        with pytest.raises(ValueError):
            W.tree_mask_from_parents(parents, starts)


MAIN = r"""
#include <cstdio>
#include "serve_problem.h"
int main() {
  const uint32_t top = 0x7fffffffu;
  auto check = [&](uint32_t d) {
    const wq::FastDiv f = wq::fast_div(d);
    auto q = [&](uint32_t x) { return f.d == 1 ? x : (uint32_t)(((uint64_t)x * f.mul) >> 32) >> f.shift; };
    auto bad = [&](uint32_t x) { return q(x) != x / d; };
    for (uint32_t x = 0; x < 3000; ++x)
      if (bad(x) || bad(top - x)) return std::printf("%u / %u\n", x, d), false;
    for (uint64_t k = 1; k * d <= top; k += 1 + k / 8)  // around multiples
      for (int e = -1; e <= 1; ++e)
        if (k * d + e <= top && bad((uint32_t)(k * d + e))) return std::printf("%lu x %u\n", (unsigned long)k, d), false;
    return true;
  };
  for (uint32_t d = 1; d < 5000; ++d) if (!check(d)) return 1;
  for (int s = 10; s < 31; ++s)
    for (int e = -3; e <= 3; ++e) if (!check((1u << s) + e)) return 1;
  return check(top) && check(top - 1) && check(1000003u) && check(715827883u) ? 0 : 1;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_division_by_multiplication(tmp_path):
    """fast_div against / for small and boundary divisors, near 0, near 2^31 and around multiples; built
    with the sanitizers, with the validation code that it lives in."""
    csrc = os.path.join(ROOT, "weight_quantized_gemm_amd", "csrc")
    main, exe = tmp_path / "main.cpp", tmp_path / "main"
    main.write_text(MAIN)
    b = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I", csrc, str(main),
                        os.path.join(csrc, "serve_validate.cpp"), os.path.join(csrc, "serve_plan.cpp"), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert b.returncode == 0, b.stderr[-3000:]
    env = {k: v for k, v in os.environ.items() if k != "LD_PRELOAD"}
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr[-3000:]
