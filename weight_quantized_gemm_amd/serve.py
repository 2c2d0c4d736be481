"""The serving operators of ``libwqgemm.so`` (``include/wqserve.h``): low-rank adapters of many
requests beside a shared projection, rotary positions with the append to a paged cache, and
attention for a tree of drafted tokens over that cache.

Like the rest of the binding this only marshals arguments: each operator is a prepared call (a
class: descriptors, outputs and workspace settled once, a call only enqueues kernels) and a
one-shot function of the same arguments.  A prepared call reads its tensors anew each time, so
a serving loop writes the next step's tokens, indices and lengths into the same tensors; it
holds references to them, and their storage must not change.  Calls of one prepared call share its
output and workspace: on several streams they are ordered by the caller, like all uses of a
tensor.  It may be dropped while its calls are in flight, but not before the last replay of a graph
that captured one.
"""
from __future__ import annotations

import ctypes
import math

from . import (_alloc_on, _check, _desc, _ref, _stream_handle, _torch, lib)

SERVE_EXPORTS = ("wq_lora_matmul_get_workspace_size", "wq_lora_matmul", "wq_rope",
                 "wq_tree_attention_get_workspace_size", "wq_tree_attention", "wq_norm_rope", "wq_step_layout",
                 "wq_prefix_attention_get_workspace_size", "wq_prefix_attention",
                 "wq_verify_drafts_get_workspace_size", "wq_verify_drafts")
WQ_ROPE_HALF, WQ_ROPE_INTERLEAVED = 0, 1


def _same_device(named, device):
    """Every tensor lives on `device`, a GPU (the kernels read their pointers there)."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU, not on {device}")
    for name, t in named.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _handle(stream, device):
    """The raw handle of `stream`.  torch's current stream is asked for by its handle: making a stream
    object of it takes 2 us, a third of a small call."""
    if stream is None:
        raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(device.index)
    return _stream_handle(stream, device).value or 0


class _Prepared:
    """What prepared calls share.  A subclass sets `out`, the call's tensors and the C function with its
    arguments up to the stream."""

    def _settle(self, device, out, tensors, fn, args):
        self.out, self.device = out, device
        self._keep = [t for t in tensors if t is not None]
        self._fn, self._args = fn, args
        self._streams = {_handle(None, device)}

    def __call__(self, stream=None):
        handle = _handle(stream, self.device)
        if handle not in self._streams:
            self._used_on(handle)
        status = self._fn(*self._args, handle)
        if status:
            _check(status)
        return self.out

    def _used_on(self, handle):
        """The allocator is told, once, that a further stream uses the tensors: memory freed while a call is in
        flight there is not handed out before it ends.  A captured call is none that can be waited for."""
        torch = _torch()
        stream = torch.cuda.ExternalStream(handle, device=self.device)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        for t in self._keep:
            t.record_stream(stream)
        self._streams.add(handle)


def _workspace(size, given, device):
    torch = _torch()
    if given is None:
        return torch.empty(max(size, 1), dtype=torch.uint8, device=device)
    if given.device != device:
        raise ValueError(f"the workspace is on {given.device}, not on {device}")
    if given.numel() * given.element_size() < size or not given.is_contiguous():
        raise ValueError(f"the workspace needs {size} contiguous bytes")
    return given


class LoraMatmul(_Prepared):
    """Prepared call of :func:`lora_matmul` (the same arguments); ``call(stream=None)`` enqueues
    the kernels on `stream` (default: torch's current stream) and returns ``out``."""

    def __init__(self, x1, a, b, indices, scale=None, *, ranks=None, x3=None, out=None, workspace=None):
        torch = _torch()
        device = x1.device
        if out is None:
            out = torch.empty(tuple(x1.shape[:-1]) + (b.shape[1] if b.dim() > 1 else 0,), dtype=x1.dtype, device=device)
        tensors = dict(x1=x1, a=a, b=b, indices=indices, scale=scale, ranks=ranks, x3=x3, out=out)
        _same_device(tensors, device)
        self._descs = [_desc(t) for t in tensors.values()]
        L = lib()
        ws = ctypes.c_uint64(0)
        _check(L.wq_lora_matmul_get_workspace_size(*map(_ref, self._descs), ctypes.byref(ws)))
        self.workspace_size = int(ws.value)
        self.workspace = _workspace(self.workspace_size, workspace, device)
        self._settle(device, out, [*tensors.values(), self.workspace], L.wq_lora_matmul,
                     (*map(_ref, self._descs), ctypes.c_void_p(self.workspace.data_ptr()),
                      ctypes.c_uint64(self.workspace.numel() * self.workspace.element_size())))


def lora_matmul(x1, a, b, indices, scale=None, *, ranks=None, x3=None, out=None, workspace=None, stream=None):
    """out[t] = x3[t] + scale[i] * ((x1[t] @ a[i]^T) @ b[i]^T) with i = indices[t].

    x1: fp16/bf16 (m, k) or (b, s, k), rows possibly strided; a: (L, r, k); b: (L, n, r); indices:
    int32 (m), a token whose index is outside [0, L) having no adapter; scale: fp32 (L), absent 1;
    ranks: int32 (L), each adapter's rank up to r, absent r; x3: the shared projection's result,
    absent 0, and possibly ``out`` itself.  The output and the workspace, unless given, are allocated
    on the stream the call runs on.  Returns the output."""
    with _alloc_on(stream, x1.device) as s:
        return LoraMatmul(x1, a, b, indices, scale, ranks=ranks, x3=x3, out=out, workspace=workspace)(s)


class Rope(_Prepared):
    """Prepared call of :func:`rope` (the same arguments); ``call(stream=None)`` enqueues the kernel
    and returns ``(q_out, k_out, v_out)``."""

    def __init__(self, q, k, v, positions, inv_freq, *, slots=None, interleaved=False, attention_factor=1.0,
                 q_out=None, k_out=None, v_out=None):
        torch = _torch()
        device = q.device
        like = lambda t: torch.empty(tuple(t.shape), dtype=t.dtype, device=device)
        q_out = like(q) if q_out is None else q_out
        if k is not None and k_out is None and slots is None:
            k_out = like(k)
        if v is not None and v_out is None and slots is None:
            v_out = like(v)
        tensors = dict(q=q, k=k, v=v, positions=positions, inv_freq=inv_freq, slots=slots)
        outs = dict(q_out=q_out, k_out=k_out, v_out=v_out)
        _same_device({**tensors, **outs}, device)
        self._ins = [_desc(t) for t in tensors.values()]
        self._outs = [_desc(t) for t in outs.values()]
        layout = WQ_ROPE_INTERLEAVED if interleaved else WQ_ROPE_HALF
        self._settle(device, (q_out, k_out, v_out), [*tensors.values(), *outs.values()], lib().wq_rope,
                     (*map(_ref, self._ins), layout, float(attention_factor), *map(_ref, self._outs)))


def rope(q, k, v, positions, inv_freq, *, slots=None, interleaved=False, attention_factor=1.0, q_out=None, k_out=None,
         v_out=None, stream=None):
    """Rotary positions of q (T, hq, d) and k (T, hkv, d), which may be views of one projection.

    positions: int32 (T); inv_freq: fp32 (rot/2) radians per position (:func:`rope_frequencies`), rot
    <= d elements of each head turning; interleaved: element 2j turns with 2j + 1, otherwise j with j
    + rot/2; attention_factor multiplies the cosines and sines.  v, if given, is copied to v_out.  With
    slots (int32 (T)), k_out and v_out are caches (S, hkv, d) and token t's k and v go to their
    row slots[t] (outside [0, S): nowhere).  k and v may be None.  Outputs not given are allocated on
    the stream the call runs on; q_out may be q, and without slots k_out may be k.  Returns
    (q_out, k_out, v_out)."""
    with _alloc_on(stream, q.device) as s:
        return Rope(q, k, v, positions, inv_freq, slots=slots, interleaved=interleaved,
                    attention_factor=attention_factor, q_out=q_out, k_out=k_out, v_out=v_out)(s)


def rope_frequencies(rot, base=10000.0, *, scaling="none", factor=1.0, original_length=None, beta_fast=32.0,
                     beta_slow=1.0, device=None):
    """(inv_freq, attention_factor) for :func:`rope`: inv_freq fp32 (rot/2), computed in fp64.

    scaling: "none"; "linear" (positions divided by factor); "base" (the base raised so that the
    lowest frequency is divided by factor and the highest is kept); "ramp" (frequencies that turn at
    least beta_fast times in original_length are kept, those that turn at most beta_slow times
    are divided by factor, between them a linear blend over the pair's index, whose end may lie past the
    last pair, at index rot - 1 at most; attention_factor = 0.1 ln(factor) + 1)."""
    torch = _torch()
    if rot < 2 or rot % 2 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("rot must be a positive even number, base above 1 and factor at least 1")
    pairs = rot // 2
    j = torch.arange(pairs, dtype=torch.float64)
    if scaling == "base" and pairs > 1:
        base = base * factor ** (pairs / (pairs - 1))
    freq, attention = base ** (-j / pairs), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ramp":
        if not original_length or original_length < 1 or not beta_fast > beta_slow > 0:
            raise ValueError("ramp scaling needs original_length and beta_fast > beta_slow > 0")
        # the (real) pair index whose frequency turns `turns` times in the original length
        at = lambda turns: pairs * math.log(original_length / (2 * math.pi * turns)) / math.log(base)
        lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot - 1)
        slow = ((j - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - slow) + freq / factor * slow
        attention = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(torch.float32).to(device or "cpu"), attention


class TreeAttention(_Prepared):
    """Prepared call of :func:`tree_attention` (the same arguments); ``call(stream=None)`` enqueues
    the kernels and returns ``out``."""

    def __init__(self, q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask=None, *, page_size,
                 scale=None, out=None, workspace=None):
        torch = _torch()
        device = q.device
        if out is None:
            out = torch.empty(tuple(q.shape), dtype=q.dtype, device=device)
        tensors = dict(q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, context_lens=context_lens,
                       q_starts=q_starts, tree_mask=tree_mask)
        _same_device({**tensors, "out": out}, device)
        self._descs = [_desc(t) for t in tensors.values()]
        self._out = _desc(out)
        scale = float(q.shape[-1]) ** -0.5 if scale is None else float(scale)
        L = lib()
        ws = ctypes.c_uint64(0)
        _check(L.wq_tree_attention_get_workspace_size(*map(_ref, self._descs), int(page_size), _ref(self._out),
                                                      ctypes.byref(ws)))
        self.workspace_size = int(ws.value)
        self.workspace = _workspace(self.workspace_size, workspace, device)
        self._settle(device, out, [*tensors.values(), out, self.workspace], L.wq_tree_attention,
                     (*map(_ref, self._descs), int(page_size), scale, _ref(self._out),
                      ctypes.c_void_p(self.workspace.data_ptr()),
                      ctypes.c_uint64(self.workspace.numel() * self.workspace.element_size())))


def tree_attention(q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask=None, *, page_size, scale=None,
                   out=None, workspace=None, stream=None):
    """Attention of each sequence's newest tokens over its pages of a cache that holds them.

    q: fp16/bf16 (N, hq, d), d in {64, 128, 256}, the rows q_starts[b] .. q_starts[b+1] being sequence b's T_b
    tokens; k_cache, v_cache: (S, hkv, d), key j of sequence b in row block_table[b, j // page_size]
    * page_size + j % page_size; context_lens: int32 (B) keys before the T_b tokens' own; tree_mask:
    int32 (N, words) as :func:`tree_mask_from_parents` makes it, None for a chain (each token sees those
    before it and itself; T_b = 1 is plain decoding); scale: default d ** -0.5.  A token that sees no
    key gives zeros.  The output and the workspace, unless given, are allocated on the stream the
    call runs on.  Returns the output."""
    with _alloc_on(stream, q.device) as s:
        return TreeAttention(q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask, page_size=page_size,
                             scale=scale, out=out, workspace=workspace)(s)


def tree_mask_from_parents(parents, q_starts, device=None):
    """The int32 (N, words) mask of trees given by parents: parents[i] is the index, within its
    sequence, of token i's parent (-1: its parent is the context's last token), an earlier token of
    that sequence.  A token sees its ancestors and itself.  Both arguments are read on the host."""
    torch = _torch()
    parents = [int(p) for p in parents]
    starts = [int(s) for s in q_starts]
    if not starts or starts[0] != 0 or starts[-1] != len(parents) or any(a > b for a, b in zip(starts, starts[1:])):
        raise ValueError("q_starts must ascend from 0 to the number of parents")
    words = max(1, -(-max((b - a for a, b in zip(starts, starts[1:])), default=0) // 32))
    rows = []
    for lo, hi in zip(starts, starts[1:]):
        sees = []
        for j in range(hi - lo):
            p = parents[lo + j]
            if not -1 <= p < j:
                raise ValueError(f"token {j} of a sequence has parent {p}: it must be -1 or an earlier token")
            sees.append((sees[p] if p >= 0 else 0) | 1 << j)
        for v in sees:
            w = [(v >> 32 * i) & 0xffffffff for i in range(words)]
            rows.append([x - (1 << 32) if x >> 31 else x for x in w])
    return torch.tensor(rows, dtype=torch.int32).reshape(len(rows), words).to(device or "cpu")
