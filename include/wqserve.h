/*
 * wqserve -- what stands beside and between the weight-quantised projections of a serving
 * step, for AMD Instinct MI355X (gfx950): low-rank adapters of many requests, rotary
 * positions with the append to a paged cache, and attention for a tree of drafted tokens
 * over that cache.
 *
 * C ABI, part of the same library as wqgemm.h and under the same conventions: wq_tensor
 * descriptors, a size query that touches no device before each call that needs a workspace
 * (device memory owned by the caller, 256-byte aligned, no contents expected), asynchronous
 * launches on the caller's stream, stateless and repeatable calls, status codes only, and
 * checks in the order null pointers, dtypes, attributes, shapes.  No call allocates.
 *
 * Layout.  Where a rule below says "rows", the innermost axis is contiguous, every other
 * stride is a multiple of 8 elements (not read for an extent of 1), and the first element is
 * 16-byte aligned: slices of a wider tensor along its last axis are taken as they are.
 * Every other tensor is row-major contiguous.  An output's elements must not overlap each other,
 * and it spans at most 2^40 of them.
 *
 * Index tensors (adapter indices, cache slots, block tables, lengths, query starts) live on
 * the device and are bounds-checked by the kernels; what an index out of range means is said
 * at each call.
 */
#ifndef WQSERVE_H
#define WQSERVE_H

#include "wqgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Low-rank adapters of many requests beside a shared projection:
 *
 *   output[t] = x3[t] + scale[i] * ((x1[t] @ a[i]^T) @ b[i]^T),   i = indices[t]
 *
 *   x1       required; WQ_F16 or WQ_BF16; rows (m, k) or (b, s, k), in the 3-D form with
 *            stride[0] == s * stride[1]; m in [0, 2^28]; k in [8, 65535], a multiple of 8.
 *   a        required; x1's dtype; (L, r, k), contiguous; L in [1, 65535]; r in [8, 256], a
 *            multiple of 8.
 *   b        required; x1's dtype; (L, n, r), contiguous; n in [8, 2^22], a multiple of 8.
 *   indices  required; WQ_I32; (m).  A token whose index is outside [0, L) has no adapter:
 *            output[t] = x3[t].  Tokens of one adapter need not stand together.
 *   scale    optional; WQ_F32; (L).  Absent means 1.
 *   ranks    optional; WQ_I32; (L): the rank of each adapter, clamped to [0, r]; rows of a and
 *            columns of b past it are not part of the adapter, whatever they hold.  Absent
 *            means r.
 *   x3       optional; x1's dtype; rows, the output's shape (the shared projection's result).
 *            Absent means 0.  It may be the output itself (same address and strides).
 *   output   required; x1's dtype; rows (m, n) or (b, s, n) following x1.
 * m == 0 is a call with nothing to do.  Both products are summed in fp32; the first enters the
 * second to 2^-16 (bf16) or 2^-22 (fp16) of each number, in fp16 2^-39 of a token's largest; the
 * result is rounded once.  A token's result takes nothing from the other tokens' values,
 * and equal calls give equal bits.
 */
int wq_lora_matmul_get_workspace_size(const wq_tensor* x1, const wq_tensor* a, const wq_tensor* b,
                                      const wq_tensor* indices, const wq_tensor* scale,
                                      const wq_tensor* ranks, const wq_tensor* x3,
                                      const wq_tensor* output, uint64_t* workspace_size);
int wq_lora_matmul(const wq_tensor* x1, const wq_tensor* a, const wq_tensor* b,
                   const wq_tensor* indices, const wq_tensor* scale, const wq_tensor* ranks,
                   const wq_tensor* x3, const wq_tensor* output, void* workspace,
                   uint64_t workspace_size, void* stream);

/* Which elements of a head turn together (rot = 2 * the number of frequencies). */
#define WQ_ROPE_HALF 0        /* element j with element j + rot/2 */
#define WQ_ROPE_INTERLEAVED 1 /* element 2j with element 2j + 1 */

/*
 * Rotary positions, with the append to a cache.  For pair j of a token at position p, with
 * w = p * inv_freq[j] (taken modulo a turn in 64 bits):
 *
 *   (u, v) -> attention_factor * (u cos w - v sin w, v cos w + u sin w)
 *
 * Elements of a head past the first rot are copied.
 *
 *   q          required; WQ_F16 or WQ_BF16; rows (T, hq, d); d in [8, 256], a multiple of 8.
 *   k          optional; q's dtype; rows (T, hkv, d): rotated like q.
 *   v          optional (only with k); q's dtype; rows (T, hkv, d): copied to v_out.
 *   positions  required; WQ_I32; (T).
 *   inv_freq   required; WQ_F32; (rot/2), radians per position; 1 <= rot/2 <= d/2.
 *   slots      optional (only with k); WQ_I32; (T): the row of k_out and v_out that token t's
 *              k and v are written to.  A slot outside [0, S) drops that token's k and v; equal
 *              slots leave either token's values.  Absent means row t.
 *   layout     WQ_ROPE_HALF or WQ_ROPE_INTERLEAVED; attention_factor is finite.
 *   q_out      required; q's dtype; rows (T, hq, d).  It may be q itself.
 *   k_out      required with k; q's dtype; rows (S, hkv, d): S = T without slots, otherwise the
 *              rows of the cache.  Without slots it may be k itself.
 *   v_out      required with v; like k_out, of the same S.
 * Outputs must not overlap inputs otherwise.  T == 0 is a call with nothing to do.  No workspace.
 */
int wq_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
            const wq_tensor* inv_freq, const wq_tensor* slots, int32_t layout, float attention_factor,
            const wq_tensor* q_out, const wq_tensor* k_out, const wq_tensor* v_out, void* stream);

/*
 * Attention of each sequence's newest tokens -- one token, a chain, or a tree of drafted
 * tokens -- over its pages of a key / value cache that already holds them:
 *
 *   output[i, h] = sum_j p_ij v[j, h / G],   p_i = softmax_j(scale * q[i, h] . k[j, h / G])
 *
 * over the keys j that token i sees, G = hq / hkv.  Sequence b has the query rows
 * [q_starts[b], q_starts[b+1]), T_b of them, and the keys 0 .. context_lens[b] + T_b - 1; its
 * token i sees every key of the context and, of its own T_b tokens, those that its row of
 * tree_mask names.  Key j is row block_table[b, j / page_size] * page_size + j % page_size of
 * the caches.  A token that sees no key, or none whose score is above -inf, gives zeros.  What a
 * token does not see has no part in its result, NaN and infinities included; what it sees has the part
 * that the formula gives it, as far as its weight is above 0 in fp32.
 *
 *   q             required; WQ_F16 or WQ_BF16; rows (N, hq, d); d in {64, 128, 256}; N at most
 *                 2^24 and N * hq at most 2^30.
 *   k_cache       required; q's dtype; rows (S, hkv, d); S a multiple of page_size, at most
 *                 2^31-1; its row stride at most 2^30; hq a multiple of hkv.
 *   v_cache       required; q's dtype; rows (S, hkv, d), like k_cache.
 *   block_table   required; WQ_I32; (B, W), contiguous; W * page_size at most 2^31-2^16.  Keys past
 *                 its width, and keys on a page outside [0, S / page_size), are not seen.
 *   context_lens  required; WQ_I32; (B); a negative length counts as 0.
 *   q_starts      required; WQ_I32; (B + 1), ascending, clamped to [0, N].  Rows of output that
 *                 no sequence has are not written (nor, if starts do not ascend, need others be).
 *   tree_mask     optional; WQ_I32; (N, words): bit j % 32 of word j / 32 of a token's row says
 *                 whether it sees token j of its sequence; tokens past 32 * words are not seen.
 *                 Absent: each token sees the tokens of its sequence up to itself.
 *   page_size     in [1, 2^20].
 *   scale         in [-2^127, 2^127].
 *   output        required; q's dtype; rows (N, hq, d), not overlapping an input.
 * N == 0 or B == 0 is a call with nothing to do.  Scores, the softmax and the sums are fp32;
 * the weights p go into the product with v as the sum of two numbers of q's dtype (in fp16 to 2^-32 of
 * the largest), and the result is rounded once.
 */
int wq_tree_attention_get_workspace_size(const wq_tensor* q, const wq_tensor* k_cache,
                                         const wq_tensor* v_cache, const wq_tensor* block_table,
                                         const wq_tensor* context_lens, const wq_tensor* q_starts,
                                         const wq_tensor* tree_mask, int64_t page_size,
                                         const wq_tensor* output, uint64_t* workspace_size);
int wq_tree_attention(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                      const wq_tensor* block_table, const wq_tensor* context_lens,
                      const wq_tensor* q_starts, const wq_tensor* tree_mask, int64_t page_size,
                      float scale, const wq_tensor* output, void* workspace,
                      uint64_t workspace_size, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQSERVE_H */
