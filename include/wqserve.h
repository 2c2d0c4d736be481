/*
 * wqserve -- what stands beside and between the weight-quantised projections of a serving
 * step, for AMD Instinct MI355X (gfx950): the paged layout of a step, low-rank adapters of many
 * requests, rotary positions (with norms of the heads) and the append to a paged cache, attention
 * for a tree of drafted tokens over that cache, also behind a prefix that requests share, and the
 * verification of the drafts.
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

/*
 * Norms of the heads of q and k, then rotary positions of one or several axes, with the append to a
 * cache; one rounding at the end.  With a weight, a head x first becomes
 *
 *   x / sqrt(mean(x^2) + eps) * weight
 *
 * and then, or without one, its pairs turn as in wq_rope, pair j of token t by the position
 * positions[axes[j], t].
 *
 *   q, k, v, inv_freq, slots, layout, attention_factor, q_out, k_out, v_out   as in wq_rope.
 *   positions  required; WQ_I32; (T), or (A, T) with axes; A in [1, 16].
 *   axes       optional; WQ_I32; (rot/2): the axis of each pair.  A pair whose axis is outside [0, A) does
 *              not turn (its position is 0).  Required with positions of two dimensions.
 *   q_weight   optional; q's dtype or WQ_F32; (d), its first element 16-byte aligned.  Absent: q is not normed.
 *   k_weight   optional (only with k); the same for k.
 *   eps        finite and at least 2^-126.
 * Sums are fp32 and do not overflow: a head whose squares pass fp32 is taken with a factor.
 */
int wq_norm_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
                 const wq_tensor* inv_freq, const wq_tensor* axes, const wq_tensor* q_weight, const wq_tensor* k_weight,
                 float eps, const wq_tensor* slots, int32_t layout, float attention_factor, const wq_tensor* q_out,
                 const wq_tensor* k_out, const wq_tensor* v_out, void* stream);

/*
 * The paged layout of a step: from the requests' lengths, what the calls of the step take as index
 * tensors.  Request b has context_lens[b] keys in its pages and brings new_lens[b] tokens (negative
 * numbers count as 0), whose keys follow.  With T_b of them among the N there is room for:
 *
 *   q_starts     (B + 1): q_starts[b] = min(T_0 + .. + T_(b-1), N); tokens past the N-th are dropped.
 *   requests     (N): the request of each token.
 *   slots        (N): block_table[b, p / page_size] * page_size + p % page_size, p = context_lens[b] + j for token
 *                j of request b; -1 where its page is negative, past the table's width, or the product
 *                passes 2^31 - 1.
 *   positions    (N): position_offsets[b] + context_lens[b] + the token's depth, which is j, or with parents the
 *                number of its ancestors (at most 2^31 - 1).
 *   tree_mask    (N, words), with parents: bit i % 32 of word i / 32 says that the token is i or that i is one
 *                of its ancestors (wq_tree_attention's mask); tokens past 32 * words leave no bit.
 *   block_table  the pages that a request needs beyond ceil(context_lens[b] / page_size) are written to its row; the
 *                others stay.  They come from the top of a stack, free_pages[0 .. free_count), in the
 *                order of the requests and their pages; when it is empty, -1.
 *   free_left    (1): free_count less the pages that were needed; negative: so many were missing.
 * Tokens past the last request's: request -1, slot -1, position 0, mask 0.  With parents a token takes a step for each
 * of its ancestors, one after the other.
 *
 *   context_lens, new_lens  required; (B); B at most 65535.
 *   block_table             required; (B, W), contiguous; W * page_size at most 2^31-2^16; written in place.
 *   free_pages              required; (F); free_count required; (1), clamped to [0, F].
 *   position_offsets        optional; (B).  Absent means 0.
 *   parents                 optional; (N): the index, within its request, of each token's parent, an earlier
 *                           token of it; anything else means none.  Absent: a chain, depth j.
 *   page_size               in [1, 2^20].
 *   q_starts, slots, positions, free_left  required; N at most 2^24.
 *   requests                optional; tree_mask: required with parents, absent without; words in [0, 2^20].
 * All are WQ_I32 and contiguous; no output overlaps another tensor (free_left is not free_count).  No
 * workspace.
 */
int wq_step_layout(const wq_tensor* context_lens, const wq_tensor* new_lens, const wq_tensor* block_table,
                   const wq_tensor* free_pages, const wq_tensor* free_count, const wq_tensor* position_offsets,
                   const wq_tensor* parents, int64_t page_size, const wq_tensor* q_starts, const wq_tensor* requests,
                   const wq_tensor* positions, const wq_tensor* slots, const wq_tensor* tree_mask,
                   const wq_tensor* free_left, void* stream);

/*
 * Attention of a batch whose sequences share long prefixes, each prefix read by rows of all its
 * sequences together (once for a tile of up to 256 rows, a token's hq / hkv query heads being rows; the tile
 * follows from N, G and hq / hkv, the rows of the mean prefix; 16 with d = 256): as wq_tree_attention, but a token of sequence b, prefix_starts[g] <= b <
 * prefix_starts[g + 1], sees the prefix_lens[g] keys of prefix g besides, in one softmax with its
 * own.  Key j of prefix g is row prefix_table[g, j / page_size] * page_size + j % page_size of the caches.
 *
 *   prefix_table   required; WQ_I32; (G, Wp), contiguous; G at most 65535; Wp * page_size at most 2^31-2^16.
 *   prefix_lens    required; WQ_I32; (G); a negative length counts as 0.
 *   prefix_starts  required; WQ_I32; (G + 1), ascending, clamped to [0, B]: sequences of one prefix stand
 *                  together; those outside all prefixes have their own keys only.
 *   the others     as in wq_tree_attention; context_lens and block_table are of a sequence's own keys, which
 *                  follow the prefix.
 * Rows of output that no sequence has are not written.
 */
int wq_prefix_attention_get_workspace_size(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                                           const wq_tensor* prefix_table, const wq_tensor* prefix_lens,
                                           const wq_tensor* prefix_starts, const wq_tensor* block_table,
                                           const wq_tensor* context_lens, const wq_tensor* q_starts,
                                           const wq_tensor* tree_mask, int64_t page_size, const wq_tensor* output,
                                           uint64_t* workspace_size);
int wq_prefix_attention(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                        const wq_tensor* prefix_table, const wq_tensor* prefix_lens, const wq_tensor* prefix_starts,
                        const wq_tensor* block_table, const wq_tensor* context_lens, const wq_tensor* q_starts,
                        const wq_tensor* tree_mask, int64_t page_size, float scale, const wq_tensor* output,
                        void* workspace, uint64_t workspace_size, void* stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given random numbers.
 * Request b has the rows [q_starts[b], q_starts[b + 1]): its last decided token, then its drafted ones, each
 * the child of an earlier one.  Starting at the first, with r = target[its row]: the children x of the
 * last accepted token are tried in their order, and the first with
 *
 *   accept_random * draft[x] < r[x]                    (draft: of the last accepted token's row)
 *   accept_random * (1 - sum of the refused ones' r) < r[x]       (without draft)
 *
 * is accepted.  A refusal leaves max(r - draft, 0), divided by its sum, or, without draft, r with r[x] = 0.
 * When no child is left (or depth tokens have been accepted), the next token is the smallest x with
 *
 *   r[0] + .. + r[x] > max(sample_random, 0) * (r[0] + .. + r[V-1])
 *
 * (no such x, for a random number of 1 or NaN: the largest with r[x] > 0); where nothing is left of r, the target's
 * row stands for it, and where that holds nothing above 0, the token is -1.  Probabilities that are negative
 * or NaN count as 0.  What is compared or summed is fp64.
 * With draft and parents, a refusal that is followed by another child of the same token takes a pass over the
 * two rows, one after the other within a request.
 *
 *   target         required; WQ_F32, WQ_F16 or WQ_BF16; (N, V): row i, the probabilities after token i; V in
 *                  [1, 2^24], N at most 2^24.  The last axis is contiguous, the row stride at least V.
 *   draft          optional; target's dtype; (N, V): row i, those that the children of token i were drawn
 *                  from.  Absent: the drafts are given ones, without probabilities.
 *   tokens         required; WQ_I32; (N); a drafted token outside [0, V) has probability 0.
 *   parents        optional; WQ_I32; (N): the index, within its request, of each token's parent; a token whose
 *                  parent is no earlier token is nobody's child.  Absent: a chain.
 *   q_starts       required; WQ_I32; (B + 1), ascending, clamped to [0, N]; B at most 65535.  The first 1024 tokens
 *                  of a request are looked at.
 *   accept_random  required; WQ_F32; (N).  sample_random  required; WQ_F32; (B).
 *   accepted       required; WQ_I32; (B, depth), contiguous, depth in [0, 2^20]: the indices, within the request,
 *                  of the accepted tokens in their order, then -1.
 *   counts         required; WQ_I32; (B): how many.
 *   next_tokens    required; WQ_I32; (B): the next token, -1 for a request without tokens.
 */
int wq_verify_drafts_get_workspace_size(const wq_tensor* target, const wq_tensor* draft, const wq_tensor* tokens,
                                        const wq_tensor* parents, const wq_tensor* q_starts,
                                        const wq_tensor* accept_random, const wq_tensor* sample_random,
                                        const wq_tensor* accepted, const wq_tensor* counts,
                                        const wq_tensor* next_tokens, uint64_t* workspace_size);
int wq_verify_drafts(const wq_tensor* target, const wq_tensor* draft, const wq_tensor* tokens, const wq_tensor* parents,
                     const wq_tensor* q_starts, const wq_tensor* accept_random, const wq_tensor* sample_random,
                     const wq_tensor* accepted, const wq_tensor* counts, const wq_tensor* next_tokens, void* workspace,
                     uint64_t workspace_size, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQSERVE_H */
