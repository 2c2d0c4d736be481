// Argument checks of the serving operators around a step's attention, in the library's order (null
// pointers, dtypes, attributes, shapes and layout), and their size queries.  Pure host C++; no device
// is touched.
#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "serve_check.h"
#include "serve_step.h"

namespace wq {
namespace {

// Whether an output of `n` tensors (bits of `outputs`) starts where another one does.
bool shared_start(const wq_tensor* const* all, int n, uint32_t outputs) {
  for (int o = 0; o < n; ++o) {
    if (!((outputs >> o) & 1) || !all[o] || empty(all[o])) continue;
    for (int i = 0; i < n; ++i)
      if (i != o && all[i] && !empty(all[i]) && starts_at(all[i], all[o]->data)) return true;
  }
  return false;
}

}  // namespace

int validate_norm_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
                       const wq_tensor* inv_freq, const wq_tensor* axes, const wq_tensor* q_weight,
                       const wq_tensor* k_weight, float eps, const wq_tensor* slots, int32_t layout, float factor,
                       const wq_tensor* q_out, const wq_tensor* k_out, const wq_tensor* v_out, NormRopeProblem* p) {
  if (!q || !positions || !inv_freq || !q_out || (k && !k_out) || (v && !v_out)) return WQ_ERR_PARAM_NULLPTR;
  for (const wq_tensor* t : {q, k, v, positions, inv_freq, axes, q_weight, k_weight, slots, q_out, k_out, v_out})
    if (t && !data_ok(t)) return WQ_ERR_PARAM_NULLPTR;

  if (axes && axes->dtype != WQ_I32) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {q_weight, k_weight})
    if (t && t->dtype != q->dtype && t->dtype != WQ_F32) return WQ_ERR_PARAM_INVALID;
  if (!std::isfinite(eps) || !(eps >= FLT_MIN) || (k_weight && !k)) return WQ_ERR_PARAM_INVALID;

  if (!dims_ok(positions, 1, 2)) return WQ_ERR_PARAM_INVALID;
  if (positions->ndim == 2 && (!axes || positions->shape[0] < 1 || positions->shape[0] > 16 || !contiguous(positions)))
    return WQ_ERR_PARAM_INVALID;
  wq_tensor first = *positions;  // of the first axis
  if (positions->ndim == 2) {
    first.ndim = 1;
    first.shape[0] = positions->shape[1];
    first.stride[0] = 1;
  }
  NormRopeProblem r;
  const int st = validate_rope(q, k, v, &first, inv_freq, slots, layout, factor, q_out, k_out, v_out, &r.rope);
  if (st != WQ_OK) return st;

  const int64_t d = q->shape[2];
  if (axes && (!dims_ok(axes, 1, 1) || axes->shape[0] != inv_freq->shape[0] || !index_ok(axes))) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {q_weight, k_weight})
    if (t && (!dims_ok(t, 1, 1) || t->shape[0] != d || !contiguous(t) || ((uintptr_t)t->data & 15u) != 0))
      return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* o : {q_out, k_out, v_out})
    if (o && !empty(o))
      for (const wq_tensor* t : {axes, q_weight, k_weight})
        if (starts_at(t, o->data)) return WQ_ERR_PARAM_INVALID;

  if (p) {
    *p = r;
    p->axes = positions->ndim == 2 ? (int32_t)positions->shape[0] : 1;
    p->eps = eps;
    p->axis_of = axes ? (const int32_t*)axes->data : nullptr;
    if (q_weight) p->q_weight = q_weight->data, p->q_weight32 = q_weight->dtype == WQ_F32;
    if (k_weight) p->k_weight = k_weight->data, p->k_weight32 = k_weight->dtype == WQ_F32;
  }
  return WQ_OK;
}

int validate_layout(const wq_tensor* context_lens, const wq_tensor* new_lens, const wq_tensor* block_table,
                    const wq_tensor* free_pages, const wq_tensor* free_count, const wq_tensor* position_offsets,
                    const wq_tensor* parents, int64_t page_size, const wq_tensor* q_starts, const wq_tensor* requests,
                    const wq_tensor* positions, const wq_tensor* slots, const wq_tensor* tree_mask,
                    const wq_tensor* free_left, LayoutProblem* p) {
  if (!context_lens || !new_lens || !block_table || !free_pages || !free_count || !q_starts || !positions || !slots ||
      !free_left || (parents && !tree_mask))
    return WQ_ERR_PARAM_NULLPTR;
  const wq_tensor* all[] = {context_lens, new_lens, block_table, free_pages, free_count, position_offsets, parents,
                            q_starts, requests, positions, slots, tree_mask, free_left};
  for (const wq_tensor* t : all)
    if (t && !data_ok(t)) return WQ_ERR_PARAM_NULLPTR;
  for (const wq_tensor* t : all)
    if (t && t->dtype != WQ_I32) return WQ_ERR_PARAM_INVALID;
  if (page_size < 1 || page_size > (1 << 20) || (tree_mask && !parents)) return WQ_ERR_PARAM_INVALID;

  for (const wq_tensor* t : all)
    if (t && (!dims_ok(t, t == block_table || t == tree_mask ? 2 : 1, t == block_table || t == tree_mask ? 2 : 1) ||
              !index_ok(t)))
      return WQ_ERR_PARAM_INVALID;
  const int64_t B = block_table->shape[0], W = block_table->shape[1], N = slots->shape[0];
  if (B > 65535 || N > (1 << 24) || W * page_size > kMaxExtent - 65535) return WQ_ERR_PARAM_INVALID;
  if (context_lens->shape[0] != B || new_lens->shape[0] != B || q_starts->shape[0] != B + 1 || positions->shape[0] != N ||
      free_count->shape[0] != 1 || free_left->shape[0] != 1)
    return WQ_ERR_PARAM_INVALID;
  if ((position_offsets && position_offsets->shape[0] != B) || (requests && requests->shape[0] != N) ||
      (parents && parents->shape[0] != N))
    return WQ_ERR_PARAM_INVALID;
  if (tree_mask && (tree_mask->shape[0] != N || tree_mask->shape[1] > (1 << 20))) return WQ_ERR_PARAM_INVALID;
  if (shared_start(all, 13, 0x1f84u)) return WQ_ERR_PARAM_INVALID;

  if (p) {
    p->B = B; p->N = N; p->F = free_pages->shape[0]; p->width = W; p->page = page_size;
    p->words = tree_mask ? tree_mask->shape[1] : 0;
    p->context = (const int32_t*)context_lens->data; p->fresh = (const int32_t*)new_lens->data;
    p->table = (int32_t*)block_table->data;
    p->free_pages = (const int32_t*)free_pages->data; p->free_count = (const int32_t*)free_count->data;
    p->offsets = position_offsets ? (const int32_t*)position_offsets->data : nullptr;
    p->parents = parents ? (const int32_t*)parents->data : nullptr;
    p->starts = (int32_t*)q_starts->data;
    p->requests = requests ? (int32_t*)requests->data : nullptr;
    p->positions = (int32_t*)positions->data; p->slots = (int32_t*)slots->data;
    p->mask = tree_mask ? (uint32_t*)tree_mask->data : nullptr;
    p->free_left = (int32_t*)free_left->data;
  }
  return WQ_OK;
}

int validate_prefix(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache, const wq_tensor* prefix_table,
                    const wq_tensor* prefix_lens, const wq_tensor* prefix_starts, const wq_tensor* block_table,
                    const wq_tensor* context_lens, const wq_tensor* q_starts, const wq_tensor* tree_mask,
                    int64_t page_size, const wq_tensor* output, PrefixProblem* p) {
  if (!prefix_table || !prefix_lens || !prefix_starts) return WQ_ERR_PARAM_NULLPTR;
  for (const wq_tensor* t : {prefix_table, prefix_lens, prefix_starts})
    if (!data_ok(t)) return WQ_ERR_PARAM_NULLPTR;
  PrefixProblem r;
  const int st = validate_tree(q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask, page_size, output,
                               &r.own);
  if (st != WQ_OK) return st;
  for (const wq_tensor* t : {prefix_table, prefix_lens, prefix_starts})
    if (t->dtype != WQ_I32) return WQ_ERR_PARAM_INVALID;
  if (!dims_ok(prefix_table, 2, 2) || !dims_ok(prefix_lens, 1, 1) || !dims_ok(prefix_starts, 1, 1))
    return WQ_ERR_PARAM_INVALID;
  const int64_t G = prefix_table->shape[0], width = prefix_table->shape[1];
  if (G > 65535 || width * page_size > kMaxExtent - 65535) return WQ_ERR_PARAM_INVALID;
  if (prefix_lens->shape[0] != G || prefix_starts->shape[0] != G + 1) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {prefix_table, prefix_lens, prefix_starts})
    if (!index_ok(t) || (!empty(output) && starts_at(t, output->data))) return WQ_ERR_PARAM_INVALID;

  if (p) {
    *p = r;
    p->shared = r.own;
    p->shared.B = G;
    p->shared.width = (int32_t)width;
    p->shared.table = (const int32_t*)prefix_table->data;
    p->shared.context = (const int32_t*)prefix_lens->data;
    p->shared.has_mask = false;
    p->shared.words = 0;
    p->shared.mask = nullptr;
    p->group_starts = (const int32_t*)prefix_starts->data;
  }
  return WQ_OK;
}

int validate_verify(const wq_tensor* target, const wq_tensor* draft, const wq_tensor* tokens, const wq_tensor* parents,
                    const wq_tensor* q_starts, const wq_tensor* accept_random, const wq_tensor* sample_random,
                    const wq_tensor* accepted, const wq_tensor* counts, const wq_tensor* next_tokens, VerifyProblem* p) {
  if (!target || !tokens || !q_starts || !accept_random || !sample_random || !accepted || !counts || !next_tokens)
    return WQ_ERR_PARAM_NULLPTR;
  const wq_tensor* all[] = {target, draft, tokens, parents, q_starts, accept_random, sample_random, accepted, counts,
                            next_tokens};
  for (const wq_tensor* t : all)
    if (t && !data_ok(t)) return WQ_ERR_PARAM_NULLPTR;

  if ((target->dtype != WQ_F32 && !is16(target->dtype)) || (draft && draft->dtype != target->dtype))
    return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {tokens, parents, q_starts, accepted, counts, next_tokens})
    if (t && t->dtype != WQ_I32) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {accept_random, sample_random})
    if (t->dtype != WQ_F32) return WQ_ERR_PARAM_INVALID;

  for (const wq_tensor* t : {target, draft, accepted})
    if (t && !dims_ok(t, 2, 2)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {tokens, parents, q_starts, accept_random, sample_random, counts, next_tokens})
    if (t && (!dims_ok(t, 1, 1) || !index_ok(t))) return WQ_ERR_PARAM_INVALID;
  const int64_t N = target->shape[0], V = target->shape[1], B = counts->shape[0];
  if (V < 1 || V > (1 << 24) || N > (1 << 24) || B > 65535 || accepted->shape[1] > (1 << 20)) return WQ_ERR_PARAM_INVALID;
  if (draft && !same_shape(target, draft)) return WQ_ERR_PARAM_INVALID;
  if (tokens->shape[0] != N || (parents && parents->shape[0] != N) || accept_random->shape[0] != N ||
      sample_random->shape[0] != B || q_starts->shape[0] != B + 1 || accepted->shape[0] != B || next_tokens->shape[0] != B)
    return WQ_ERR_PARAM_INVALID;

  const uintptr_t size = target->dtype == WQ_F32 ? 4 : 2;
  for (const wq_tensor* t : {target, draft})
    if (t && !empty(t)) {
      if ((V > 1 && t->stride[1] != 1) || ((uintptr_t)t->data & (size - 1)) != 0) return WQ_ERR_PARAM_INVALID;
      if (N > 1 && (t->stride[0] < V || t->stride[0] > kMaxStride)) return WQ_ERR_PARAM_INVALID;
    }
  if (!index_ok(accepted)) return WQ_ERR_PARAM_INVALID;
  if (shared_start(all, 10, 0x380u)) return WQ_ERR_PARAM_INVALID;

  if (p) {
    p->N = N; p->B = B; p->V = V; p->depth = accepted->shape[1]; p->dtype = target->dtype;
    p->t_row = stride_of(target, 0); p->d_row = draft ? stride_of(draft, 0) : 0;
    p->target = target->data; p->draft = draft ? draft->data : nullptr;
    p->tokens = (const int32_t*)tokens->data; p->parents = parents ? (const int32_t*)parents->data : nullptr;
    p->starts = (const int32_t*)q_starts->data;
    p->accept = (const float*)accept_random->data; p->sample = (const float*)sample_random->data;
    p->accepted = (int32_t*)accepted->data; p->counts = (int32_t*)counts->data; p->next = (int32_t*)next_tokens->data;
  }
  return WQ_OK;
}

}  // namespace wq

extern "C" {

int wq_prefix_attention_get_workspace_size(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                                           const wq_tensor* prefix_table, const wq_tensor* prefix_lens,
                                           const wq_tensor* prefix_starts, const wq_tensor* block_table,
                                           const wq_tensor* context_lens, const wq_tensor* q_starts,
                                           const wq_tensor* tree_mask, int64_t page_size, const wq_tensor* output,
                                           uint64_t* workspace_size) {
  if (!workspace_size) return WQ_ERR_PARAM_NULLPTR;
  wq::PrefixProblem p;
  const int st = wq::validate_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, block_table,
                                     context_lens, q_starts, tree_mask, page_size, output, &p);
  if (st == WQ_OK) *workspace_size = (uint64_t)wq::plan_prefix(p).workspace;
  return st;
}

int wq_verify_drafts_get_workspace_size(const wq_tensor* target, const wq_tensor* draft, const wq_tensor* tokens,
                                        const wq_tensor* parents, const wq_tensor* q_starts,
                                        const wq_tensor* accept_random, const wq_tensor* sample_random,
                                        const wq_tensor* accepted, const wq_tensor* counts,
                                        const wq_tensor* next_tokens, uint64_t* workspace_size) {
  if (!workspace_size) return WQ_ERR_PARAM_NULLPTR;
  wq::VerifyProblem p;
  const int st = wq::validate_verify(target, draft, tokens, parents, q_starts, accept_random, sample_random, accepted,
                                     counts, next_tokens, &p);
  if (st == WQ_OK) *workspace_size = (uint64_t)wq::plan_verify(p).workspace;
  return st;
}

}  // extern "C"
