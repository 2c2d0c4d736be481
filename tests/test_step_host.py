"""Host side of the serving operators around a step's attention: argument rules through the C ABI, workspace sizes and
the binding's helpers (CPU; every refused call returns before any device work)."""
import ctypes
import itertools

import pytest

import weight_quantized_gemm_amd as W
from weight_quantized_gemm_amd import make_desc

OK, NULLPTR, INVALID = W.WQ_OK, W.WQ_ERR_PARAM_NULLPTR, W.WQ_ERR_PARAM_INVALID
BF, HF, F32, I32, I8 = W.WQ_BF16, W.WQ_F16, W.WQ_F32, W.WQ_I32, W.WQ_I8
_fresh = itertools.count(0x10000000, 0x1000000)


def D(shape, dt, ptr=None, strides=None):
    return make_desc(shape, dt, next(_fresh) if ptr is None else ptr, strides)


def ref(x):
    return ctypes.byref(x) if isinstance(x, W.WqTensor) else x


def like(d, dt=None, ptr=None, grow=None):
    shape = [d.shape[i] for i in range(d.ndim)]
    if grow is not None:
        shape[grow] += 8
    return D(shape, d.dtype if dt is None else dt, ptr)


def refuses_each(call, args, required):
    """What holds of every tensor: a null descriptor where it is required, null data, another type, another shape."""
    for name in required:
        assert call(**{**args, name: None}) == NULLPTR, name
    for name, d in args.items():
        if not isinstance(d, W.WqTensor):
            continue
        assert call(**{**args, name: like(d, ptr=0)}) == NULLPTR, name
        assert call(**{**args, name: like(d, I8)}) == INVALID, name
        if d.ndim < 3:
            assert call(**{**args, name: D([4] * (d.ndim + 1), d.dtype)}) == INVALID, name
        if d.ndim > 1:
            assert call(**{**args, name: D([4] * (d.ndim - 1), d.dtype)}) == INVALID, name


# ------------------------------------------------------------------------------------------ norm_rope

def norm_args(T=0, hq=4, hkv=2, d=64, rot=64, S=9, A=3, dt=HF):
    return dict(q=D([T, hq, d], dt), k=D([T, hkv, d], dt), v=D([T, hkv, d], dt), positions=D([A, T], I32),
                inv_freq=D([rot // 2], F32), axes=D([rot // 2], I32), q_weight=D([d], dt), k_weight=D([d], F32), eps=1e-6,
                slots=D([T], I32), layout=0, factor=1.0, q_out=D([T, hq, d], dt), k_out=D([S, hkv, d], dt),
                v_out=D([S, hkv, d], dt))


def norm(wqlib, **kw):
    return wqlib.wq_norm_rope(*[ref(x) for x in {**norm_args(), **kw}.values()], None)


def test_norm_rope_accepts_no_tokens(wqlib):
    """(A call with tokens would launch.)"""
    assert norm(wqlib) == OK
    assert norm(wqlib, q_weight=None, k_weight=None) == OK
    assert norm(wqlib, axes=None, positions=D([0], I32)) == OK
    assert norm(wqlib, positions=D([0], I32)) == OK
    assert norm(wqlib, **norm_args(dt=BF)) == OK
    assert norm(wqlib, k=None, v=None, k_weight=None, slots=None, k_out=None, v_out=None) == OK


def test_norm_rope_smallest_eps(wqlib):
    """eps is fp32's smallest normal number at least: the root of a head of zeros is finite."""
    args = norm_args(T=5)
    assert norm(wqlib, **{**args, "eps": 2.0 ** -127}) == INVALID
    assert norm(wqlib, eps=2.0 ** -126) == OK


def test_norm_rope_refuses(wqlib):
    args = norm_args(T=5)
    call = lambda **kw: norm(wqlib, **kw)
    refuses_each(call, args, ("q", "positions", "inv_freq", "q_out", "k_out", "v_out"))
    for name in ("q", "k", "v", "positions", "inv_freq", "axes", "q_weight", "k_weight", "slots", "q_out"):
        bad = like(args[name], grow=args[name].ndim - 1)
        assert call(**{**args, name: bad}) == INVALID, name
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert call(**{**args, "eps": eps}) == INVALID, eps
    assert call(**{**args, "layout": 2}) == INVALID
    assert call(**{**args, "factor": float("inf")}) == INVALID
    assert call(**{**args, "axes": None}) == INVALID                      # positions of three axes
    assert call(**{**args, "positions": D([17, 5], I32)}) == INVALID
    assert call(**{**args, "positions": D([0, 5], I32)}) == INVALID
    assert call(**{**args, "positions": D([3, 5], I32, strides=[8, 1])}) == INVALID
    assert call(**{**args, "q_weight": D([64], BF)}) == INVALID           # another 16-bit type
    assert call(**{**args, "q_weight": D([64], HF, ptr=0x10008)}) == INVALID
    assert call(**{**args, "k": None, "v": None, "slots": None, "k_out": None, "v_out": None}) == INVALID  # a weight of no k
    for name in ("axes", "q_weight", "k_weight", "positions", "slots", "inv_freq"):
        d = args[name]
        assert call(**{**args, name: like(d, ptr=args["q_out"].data)}) == INVALID, name


# --------------------------------------------------------------------------------------------- layout

def layout_args(B=3, N=12, width=5, F=20, words=2, page=16):
    return dict(context=D([B], I32), new=D([B], I32), table=D([B, width], I32), free=D([F], I32), count=D([1], I32),
                offsets=D([B], I32), parents=D([N], I32), page=page, q_starts=D([B + 1], I32), requests=D([N], I32),
                positions=D([N], I32), slots=D([N], I32), mask=D([N, words], I32), left=D([1], I32))


def layout(wqlib, **kw):
    return wqlib.wq_step_layout(*[ref(x) for x in {**layout_args(), **kw}.values()], None)


def test_layout_refuses(wqlib):
    args = layout_args()
    call = lambda **kw: layout(wqlib, **kw)
    refuses_each(call, args, ("context", "new", "table", "free", "count", "q_starts", "positions", "slots", "left", "mask"))
    for name in ("context", "new", "count", "offsets", "parents", "q_starts", "requests", "positions", "mask", "left"):
        assert call(**{**args, name: like(args[name], grow=0)}) == INVALID, name
    for page in (0, -1, (1 << 20) + 1):
        assert call(page=page) == INVALID
    assert call(parents=None) == INVALID                                  # a mask without parents
    assert call(table=D([3, 1 << 27], I32)) == INVALID                    # 2^31 keys
    assert call(**layout_args(B=65536)) == INVALID
    assert call(**layout_args(N=(1 << 24) + 1)) == INVALID
    assert call(table=D([3, 5], I32, strides=[8, 1])) == INVALID
    assert call(slots=D([12], I32, ptr=0x10002)) == INVALID
    for out in ("q_starts", "requests", "positions", "slots", "mask", "left", "table"):
        for other in ("context", "new", "free", "count", "offsets", "parents", "slots"):
            if other != out:
                at = args[other].data
                assert call(**{**args, out: like(args[out], ptr=at)}) == INVALID, (out, other)
    assert call(left=args["count"], count=args["count"]) == INVALID       # the very same descriptor


# --------------------------------------------------------------------------------------------- prefix

def prefix_args(N=6, hq=8, hkv=2, d=128, B=3, width=4, G=2, wide=9, page=16, S=640, words=1, dt=BF):
    return dict(q=D([N, hq, d], dt), k=D([S, hkv, d], dt), v=D([S, hkv, d], dt), ptable=D([G, wide], I32), plens=D([G], I32),
                pstarts=D([G + 1], I32), table=D([B, width], I32), context=D([B], I32), starts=D([B + 1], I32),
                mask=D([N, words], I32), page=page, out=D([N, hq, d], dt))


def prefix_size(wqlib, ws=True, **kw):
    size = ctypes.c_uint64(99)
    st = wqlib.wq_prefix_attention_get_workspace_size(*[ref(x) for x in {**prefix_args(), **kw}.values()],
                                                      ctypes.byref(size) if ws else None)
    return (st, size.value) if st == OK else st


def test_prefix_accepts(wqlib):
    st, size = prefix_size(wqlib)
    assert st == OK and size > 0 and size % 256 == 0
    assert prefix_size(wqlib, mask=None)[0] == OK
    assert prefix_size(wqlib, **prefix_args(N=0)) == (OK, 0)
    assert prefix_size(wqlib, **prefix_args(B=0)) == (OK, 0)
    st, none = prefix_size(wqlib, **prefix_args(G=0))
    assert st == OK and 0 < none < size
    for d in (64, 128, 256):
        for n in (1, 5, 100, 3000):
            assert prefix_size(wqlib, **prefix_args(N=n, d=d))[0] == OK
    assert prefix_size(wqlib, **prefix_args(wide=1000000, G=65535))[0] == OK


def test_prefix_refuses(wqlib):
    args = prefix_args()
    call = lambda **kw: prefix_size(wqlib, **kw)
    assert call(ws=False) == NULLPTR
    refuses_each(call, args, ("q", "k", "v", "ptable", "plens", "pstarts", "table", "context", "starts", "out"))
    for name in ("plens", "pstarts", "context", "starts", "mask", "out", "k"):
        assert call(**{**args, name: like(args[name], grow=0)}) == INVALID, name
    assert call(**prefix_args(d=96)) == INVALID
    assert call(**prefix_args(hq=7)) == INVALID
    assert call(**prefix_args(G=65536)) == INVALID
    assert call(ptable=D([2, 1 << 27], I32)) == INVALID
    assert call(ptable=D([2, 9], I32, strides=[16, 1])) == INVALID
    assert call(page=0) == INVALID
    assert call(page=24) == INVALID  # 640 rows are no whole pages
    for name in ("ptable", "plens", "pstarts", "table", "q", "k", "v"):
        assert call(**{**args, name: like(args[name], ptr=args["out"].data)}) == INVALID, name


def test_prefix_workspace_and_scale_are_checked(wqlib):
    a = prefix_args()
    size = prefix_size(wqlib, **a)[1]
    names = [x for x in a if x not in ("page", "out")]
    call = lambda ws, n, scale=0.1: wqlib.wq_prefix_attention(*[ref(a[x]) for x in names], 16, scale, ref(a["out"]),
                                                              ctypes.c_void_p(ws), n, None)
    assert call(0x100000, size - 1) == INVALID
    assert call(0, size) == NULLPTR
    assert call(0x100080, size) == INVALID
    for scale in (float("nan"), float("inf"), 3e38):
        assert call(0x100000, size, scale) == INVALID


# --------------------------------------------------------------------------------------------- verify

def verify_args(N=9, V=100, B=2, depth=4, dt=F32):
    return dict(target=D([N, V], dt), draft=D([N, V], dt), tokens=D([N], I32), parents=D([N], I32), starts=D([B + 1], I32),
                accept=D([N], F32), sample=D([B], F32), accepted=D([B, depth], I32), counts=D([B], I32), next=D([B], I32))


def verify_size(wqlib, ws=True, **kw):
    size = ctypes.c_uint64(99)
    st = wqlib.wq_verify_drafts_get_workspace_size(*[ref(x) for x in {**verify_args(), **kw}.values()],
                                                   ctypes.byref(size) if ws else None)
    return (st, size.value) if st == OK else st


def test_verify_accepts(wqlib):
    st, size = verify_size(wqlib)
    assert st == OK and size > 0 and size % 256 == 0
    for dt in (F32, HF, BF):
        assert verify_size(wqlib, **verify_args(dt=dt))[0] == OK
    assert verify_size(wqlib, draft=None, parents=None)[0] == OK
    assert verify_size(wqlib, **verify_args(B=0)) == (OK, 0)
    assert verify_size(wqlib, **verify_args(N=0))[0] == OK
    assert verify_size(wqlib, **verify_args(depth=0))[0] == OK
    assert verify_size(wqlib, target=D([9, 100], F32, ptr=0x10004, strides=[101, 1]))[0] == OK
    # a chunk for each thread that joins them, whatever the sizes
    for V in (1, 1023, 1024, 1025, 50257, 1 << 20, 1 << 24):
        for B in (1, 3, 64, 1000, 65535):
            st, size = verify_size(wqlib, **verify_args(V=V, B=B))
            assert st == OK and 16 * B <= size <= 256 * 4 + 16 * B * (1 + 1024) + 8 * 9


def test_verify_refuses(wqlib):
    args = verify_args()
    call = lambda **kw: verify_size(wqlib, **kw)
    assert call(ws=False) == NULLPTR
    refuses_each(call, args, ("target", "tokens", "starts", "accept", "sample", "accepted", "counts", "next"))
    for name, d in args.items():
        assert call(**{**args, name: like(d, grow=0)}) == INVALID, name
    assert call(draft=D([9, 100], BF)) == INVALID
    assert call(draft=D([9, 99], F32)) == INVALID
    assert call(**verify_args(V=0)) == INVALID
    assert call(**verify_args(V=(1 << 24) + 1)) == INVALID
    assert call(**verify_args(B=65536)) == INVALID
    assert call(**verify_args(depth=(1 << 20) + 1)) == INVALID
    for strides in ([99, 1], [100, 2], [-100, 1], [0, 1]):
        assert call(target=D([9, 100], F32, strides=strides)) == INVALID, strides
    assert call(target=D([9, 100], F32, ptr=0x10002)) == INVALID
    for out in ("accepted", "counts", "next"):
        for other in ("target", "draft", "tokens", "parents", "starts", "accept", "sample"):
            assert call(**{**args, out: like(args[out], ptr=args[other].data)}) == INVALID, (out, other)
    assert call(**{**args, "counts": args["next"]}) == INVALID


def test_verify_workspace_is_checked(wqlib):
    a = verify_args()
    size = verify_size(wqlib, **a)[1]
    call = lambda ws, n: wqlib.wq_verify_drafts(*[ref(x) for x in a.values()], ctypes.c_void_p(ws), n, None)
    assert call(0x100000, size - 1) == INVALID
    assert call(0, size) == NULLPTR
    assert call(0x100010, size) == INVALID
    none = verify_args(B=0)
    assert wqlib.wq_verify_drafts(*[ref(x) for x in none.values()], None, 0, None) == OK


# -------------------------------------------------------------------------------------------- binding

def test_tensors_off_the_device_are_refused():
    torch = pytest.importorskip("torch")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="on a GPU"):
        W.NormRope(z(4, 2, 64), None, None, i(4), torch.ones(32), q_weight=z(64))
    with pytest.raises(ValueError, match="on a GPU"):
        W.StepLayout(i(2), i(2), i(2, 3), i(9), i(1), tokens=4, page_size=16)
    with pytest.raises(ValueError, match="on a GPU"):
        W.PrefixAttention(z(4, 2, 64), z(16, 2, 64), z(16, 2, 64), i(1, 1), i(1), i(2), i(1, 1), i(1), i(2), page_size=16)
    with pytest.raises(ValueError, match="on a GPU"):
        W.VerifyDrafts(torch.ones(3, 8), i(3), i(2), torch.ones(3), torch.ones(1), depth=2)
    with pytest.raises(ValueError, match="words"):
        W.StepLayout(i(2), i(2), i(2, 3), i(9), i(1), tokens=4, page_size=16, parents=i(4))
    with pytest.raises(ValueError, match="columns"):
        W.VerifyDrafts(torch.ones(3, 8), i(3), i(2), torch.ones(3), torch.ones(1), depth=2, accepted=i(1, 3))


def test_rope_axes():
    assert W.rope_axes([2, 1, 3]).tolist() == [0, 0, 1, 2, 2, 2]
    assert W.rope_axes([2, 1, 3], mixed=True).tolist() == [0, 1, 2, 0, 2, 2]
    assert W.rope_axes([0, 2]).tolist() == [1, 1]
    for bad in ([], [0, 0], [3, -1]):
        with pytest.raises(ValueError):
            W.rope_axes(bad)
