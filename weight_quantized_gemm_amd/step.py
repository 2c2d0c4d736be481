"""The serving operators around a step's attention (``include/wqserve.h``): the paged layout of a step from
the requests' lengths, norms of the heads with rotary positions, attention behind a prefix that
sequences share, and the verification of drafted tokens.

Prepared calls (classes) and one-shot functions of the same arguments, as in ``serve.py``.
"""
from __future__ import annotations

import collections
import ctypes

from . import (_alloc_on, _check, _desc, _ref, _torch, lib)
from .serve import WQ_ROPE_HALF, WQ_ROPE_INTERLEAVED, _Prepared, _same_device, _workspace

StepTables = collections.namedtuple("StepTables", "q_starts requests positions slots tree_mask free_left")


class StepLayout(_Prepared):
    """Prepared call of :func:`step_layout` (the same arguments); ``call(stream=None)`` enqueues the kernel
    and returns the :class:`StepTables`."""

    def __init__(self, context_lens, new_lens, block_table, free_pages, free_count, *, tokens, page_size,
                 position_offsets=None, parents=None, mask_words=None, q_starts=None, requests=None, positions=None,
                 slots=None, tree_mask=None, free_left=None):
        torch = _torch()
        device = block_table.device
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)
        q_starts = new(block_table.shape[0] + 1) if q_starts is None else q_starts
        requests = new(tokens) if requests is None else requests
        positions = new(tokens) if positions is None else positions
        slots = new(tokens) if slots is None else slots
        free_left = new(1) if free_left is None else free_left
        if parents is not None and tree_mask is None:
            if mask_words is None:
                raise ValueError("with parents the mask's words are needed: ceil(most tokens of a request / 32)")
            tree_mask = new(tokens, mask_words)
        ins = dict(context_lens=context_lens, new_lens=new_lens, block_table=block_table, free_pages=free_pages,
                   free_count=free_count, position_offsets=position_offsets, parents=parents)
        outs = dict(q_starts=q_starts, requests=requests, positions=positions, slots=slots, tree_mask=tree_mask,
                    free_left=free_left)
        _same_device({**ins, **outs}, device)
        if slots.dim() != 1 or slots.shape[0] != tokens:
            raise ValueError(f"slots must hold {tokens} tokens")
        self._ins = [_desc(t) for t in ins.values()]
        self._outs = [_desc(t) for t in outs.values()]
        self._settle(device, StepTables(**outs), [*ins.values(), *outs.values()], lib().wq_step_layout,
                     (*map(_ref, self._ins), int(page_size), *map(_ref, self._outs)))


def step_layout(context_lens, new_lens, block_table, free_pages, free_count, *, tokens, page_size, position_offsets=None,
                parents=None, mask_words=None, q_starts=None, requests=None, positions=None, slots=None, tree_mask=None,
                free_left=None, stream=None):
    """The index tensors of a step, from the requests' lengths, on the GPU.

    Request b has context_lens[b] keys in the pages of its row of block_table and brings new_lens[b] tokens (all
    tensors int32).  The pages it needs beyond are taken from the top of the stack free_pages[0 : free_count] and
    written to its row of the table, in place.  tokens: the room for tokens N, of which those past the
    last request's get request -1, slot -1 and position 0 (so a captured step may be longer than its tokens).

    position_offsets: int32 (B), added to the positions (a shared prefix's length); parents: int32 (N), the
    index within its request of each token's parent (-1: none), for positions by depth and the mask of
    :func:`tree_attention`, of mask_words words.  Returns StepTables(q_starts (B + 1), requests (N), positions (N),
    slots (N), tree_mask (N, words) or None, free_left (1): pages left on the stack, negative if so many were
    missing).  Tensors given for these are written; the others are allocated on the stream the call runs
    on.  The caller copies free_left to free_count before the next step."""
    with _alloc_on(stream, block_table.device) as s:
        return StepLayout(context_lens, new_lens, block_table, free_pages, free_count, tokens=tokens, page_size=page_size,
                          position_offsets=position_offsets, parents=parents, mask_words=mask_words, q_starts=q_starts,
                          requests=requests, positions=positions, slots=slots, tree_mask=tree_mask, free_left=free_left)(s)


class NormRope(_Prepared):
    """Prepared call of :func:`norm_rope` (the same arguments); ``call(stream=None)`` enqueues the kernel
    and returns ``(q_out, k_out, v_out)``."""

    def __init__(self, q, k, v, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6, axes=None, slots=None,
                 interleaved=False, attention_factor=1.0, q_out=None, k_out=None, v_out=None):
        torch = _torch()
        device = q.device
        like = lambda t: torch.empty(tuple(t.shape), dtype=t.dtype, device=device)
        q_out = like(q) if q_out is None else q_out
        if k is not None and k_out is None and slots is None:
            k_out = like(k)
        if v is not None and v_out is None and slots is None:
            v_out = like(v)
        ins = dict(q=q, k=k, v=v, positions=positions, inv_freq=inv_freq, axes=axes, q_weight=q_weight, k_weight=k_weight)
        outs = dict(q_out=q_out, k_out=k_out, v_out=v_out)
        _same_device({**ins, "slots": slots, **outs}, device)
        self._ins = [_desc(t) for t in ins.values()]
        self._slots = _desc(slots)
        self._outs = [_desc(t) for t in outs.values()]
        layout = WQ_ROPE_INTERLEAVED if interleaved else WQ_ROPE_HALF
        self._settle(device, (q_out, k_out, v_out), [*ins.values(), slots, *outs.values()], lib().wq_norm_rope,
                     (*map(_ref, self._ins), float(eps), _ref(self._slots), layout, float(attention_factor),
                      *map(_ref, self._outs)))


def norm_rope(q, k, v, positions, inv_freq, *, q_weight=None, k_weight=None, eps=1e-6, axes=None, slots=None,
              interleaved=False, attention_factor=1.0, q_out=None, k_out=None, v_out=None, stream=None):
    """:func:`rope` with norms of the heads and positions of several axes, in the same pass and with one rounding.

    q_weight, k_weight: (d), of q's type or fp32, 16-byte aligned: each head x of q (of k) is first x / sqrt(mean(x^2) + eps) *
    weight; None: q (k) is not normed.  positions: int32 (T), or (A, T) with axes, int32 (rot/2), the axis of each pair
    of elements (:func:`rope_axes`); a pair whose axis is none of the A does not turn.  The other arguments and
    the result are those of :func:`rope`."""
    with _alloc_on(stream, q.device) as s:
        return NormRope(q, k, v, positions, inv_freq, q_weight=q_weight, k_weight=k_weight, eps=eps, axes=axes, slots=slots,
                        interleaved=interleaved, attention_factor=attention_factor, q_out=q_out, k_out=k_out,
                        v_out=v_out)(s)


def rope_axes(sections, *, mixed=False, device=None):
    """The axis of each pair for :func:`norm_rope`: int32 (sum(sections)), sections[i] pairs of axis i.  In
    blocks, or mixed: the axes in turn, pair by pair, each until its pairs are used up."""
    torch = _torch()
    left = [int(n) for n in sections]
    if not left or any(n < 0 for n in left) or not sum(left):
        raise ValueError("sections must be the numbers of pairs of the axes")
    axes = []
    if mixed:
        while any(left):
            for i, n in enumerate(left):
                if n:
                    axes.append(i)
                    left[i] -= 1
    else:
        axes = [i for i, n in enumerate(left) for _ in range(n)]
    return torch.tensor(axes, dtype=torch.int32).to(device or "cpu")


class PrefixAttention(_Prepared):
    """Prepared call of :func:`prefix_attention` (the same arguments); ``call(stream=None)`` enqueues
    the kernels and returns ``out``."""

    def __init__(self, q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, block_table, context_lens, q_starts,
                 tree_mask=None, *, page_size, scale=None, out=None, workspace=None):
        torch = _torch()
        device = q.device
        if out is None:
            out = torch.empty(tuple(q.shape), dtype=q.dtype, device=device)
        tensors = dict(q=q, k_cache=k_cache, v_cache=v_cache, prefix_table=prefix_table, prefix_lens=prefix_lens,
                       prefix_starts=prefix_starts, block_table=block_table, context_lens=context_lens, q_starts=q_starts,
                       tree_mask=tree_mask)
        _same_device({**tensors, "out": out}, device)
        self._descs = [_desc(t) for t in tensors.values()]
        self._out = _desc(out)
        scale = float(q.shape[-1]) ** -0.5 if scale is None else float(scale)
        L = lib()
        ws = ctypes.c_uint64(0)
        _check(L.wq_prefix_attention_get_workspace_size(*map(_ref, self._descs), int(page_size), _ref(self._out),
                                                        ctypes.byref(ws)))
        self.workspace_size = int(ws.value)
        self.workspace = _workspace(self.workspace_size, workspace, device)
        self._settle(device, out, [*tensors.values(), out, self.workspace], L.wq_prefix_attention,
                     (*map(_ref, self._descs), int(page_size), scale, _ref(self._out),
                      ctypes.c_void_p(self.workspace.data_ptr()),
                      ctypes.c_uint64(self.workspace.numel() * self.workspace.element_size())))


def prefix_attention(q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, block_table, context_lens, q_starts,
                     tree_mask=None, *, page_size, scale=None, out=None, workspace=None, stream=None):
    """:func:`tree_attention` of a batch whose sequences share long prefixes, each of which is read by rows of all
    its sequences together: once for 16, 32, 64, 128 or 256 rows (tokens times the query heads of a cached head) by the mean
    over the prefixes, with heads of 256 once for 16.

    The sequences prefix_starts[g] .. prefix_starts[g+1] (int32 (G + 1)) see, before their own keys, the
    prefix_lens[g] keys (int32 (G)) of prefix g, key j in row prefix_table[g, j // page_size] * page_size + j % page_size
    of the caches (int32 (G, Wp)).  block_table and context_lens are of a sequence's own keys, behind the prefix; the
    other arguments and the result are those of :func:`tree_attention`."""
    with _alloc_on(stream, q.device) as s:
        return PrefixAttention(q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, block_table, context_lens,
                               q_starts, tree_mask, page_size=page_size, scale=scale, out=out, workspace=workspace)(s)


class VerifyDrafts(_Prepared):
    """Prepared call of :func:`verify_drafts` (the same arguments); ``call(stream=None)`` enqueues the
    kernels and returns ``(accepted, counts, next_tokens)``."""

    def __init__(self, target, tokens, q_starts, accept_random, sample_random, *, depth, draft=None, parents=None,
                 accepted=None, counts=None, next_tokens=None, workspace=None):
        torch = _torch()
        device = target.device
        seqs = q_starts.shape[0] - 1 if q_starts.dim() == 1 else 0
        new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)
        accepted = new(max(seqs, 0), int(depth)) if accepted is None else accepted
        counts = new(max(seqs, 0)) if counts is None else counts
        next_tokens = new(max(seqs, 0)) if next_tokens is None else next_tokens
        if accepted.dim() != 2 or accepted.shape[1] != depth:
            raise ValueError(f"accepted must have {depth} columns")
        ins = dict(target=target, draft=draft, tokens=tokens, parents=parents, q_starts=q_starts,
                   accept_random=accept_random, sample_random=sample_random)
        outs = dict(accepted=accepted, counts=counts, next_tokens=next_tokens)
        _same_device({**ins, **outs}, device)
        self._descs = [_desc(t) for t in (*ins.values(), *outs.values())]
        L = lib()
        ws = ctypes.c_uint64(0)
        _check(L.wq_verify_drafts_get_workspace_size(*map(_ref, self._descs), ctypes.byref(ws)))
        self.workspace_size = int(ws.value)
        self.workspace = _workspace(self.workspace_size, workspace, device)
        self._settle(device, tuple(outs.values()), [*ins.values(), *outs.values(), self.workspace], L.wq_verify_drafts,
                     (*map(_ref, self._descs), ctypes.c_void_p(self.workspace.data_ptr()),
                      ctypes.c_uint64(self.workspace.numel() * self.workspace.element_size())))


def verify_drafts(target, tokens, q_starts, accept_random, sample_random, *, depth, draft=None, parents=None, accepted=None,
                  counts=None, next_tokens=None, workspace=None, stream=None):
    """Which drafted tokens the target accepts, and the token that follows, from given random numbers.

    Request b's rows q_starts[b] .. q_starts[b+1] are its last decided token and its drafted ones.  target: (N, V) fp32,
    fp16 or bf16 probabilities after each token; tokens: int32 (N); draft: (N, V), the probabilities that the children
    of each token were drawn from, None for drafts without (a draft's best tokens); parents: int32 (N), the
    index within its request of each token's parent, None for a chain; accept_random: fp32 (N), the number that each
    drafted token is tested with; sample_random: fp32 (B); depth: the most tokens to accept.

    The children x of the last accepted token are tried in their order: x is accepted if u draft[x] < r[x] (without
    draft: u (1 - what the refused ones had) < r[x]), r being the target's row; a refusal leaves max(r - draft, 0)
    scaled to 1 (without: r without x).  The next token is drawn from what is left at the last accepted token.
    So the tokens are distributed as the target's own.  Returns (accepted (B, depth): indices within the
    request, then -1; counts (B); next_tokens (B)), int32."""
    with _alloc_on(stream, target.device) as s:
        return VerifyDrafts(target, tokens, q_starts, accept_random, sample_random, depth=depth, draft=draft,
                            parents=parents, accepted=accepted, counts=counts, next_tokens=next_tokens,
                            workspace=workspace)(s)
