// Argument checks of the serving operators, in the library's order (null pointers, dtypes,
// attributes, shapes and layout), and their size queries.  Pure host C++; no device is touched.
#include <cmath>
#include <initializer_list>

#include "serve_check.h"

namespace wq {

FastDiv fast_div(uint32_t d) {
  FastDiv f;
  f.d = d;
  if (d <= 1) return f;
  uint32_t s = 0;
  while ((2ull << s) < d) ++s;  // 2^(s+1) >= d
  f.shift = s;
  f.mul = (uint32_t)(((1ull << (32 + s)) + d - 1) / d);
  return f;
}

int validate_lora(const wq_tensor* x1, const wq_tensor* a, const wq_tensor* b, const wq_tensor* indices,
                  const wq_tensor* scale, const wq_tensor* ranks, const wq_tensor* x3,
                  const wq_tensor* output, LoraProblem* p) {
  if (!x1 || !a || !b || !indices || !output) return WQ_ERR_PARAM_NULLPTR;
  for (const wq_tensor* t : {x1, a, b, indices, scale, ranks, x3, output})
    if (t && !data_ok(t)) return WQ_ERR_PARAM_NULLPTR;

  const int32_t act = x1->dtype;
  if (!is16(act)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {a, b, x3, output})
    if (t && t->dtype != act) return WQ_ERR_PARAM_INVALID;
  if (indices->dtype != WQ_I32 || (scale && scale->dtype != WQ_F32) || (ranks && ranks->dtype != WQ_I32))
    return WQ_ERR_PARAM_INVALID;

  if (!dims_ok(x1, 2, 3) || !dims_ok(a, 3, 3) || !dims_ok(b, 3, 3) || !dims_ok(indices, 1, 1) ||
      !dims_ok(output, 2, 3))
    return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {scale, ranks})
    if (t && !dims_ok(t, 1, 1)) return WQ_ERR_PARAM_INVALID;
  if (x3 && !dims_ok(x3, 2, 3)) return WQ_ERR_PARAM_INVALID;
  const int64_t k = x1->shape[x1->ndim - 1];
  int64_t m = 1;
  for (int i = 0; i < x1->ndim - 1; ++i) m *= x1->shape[i];  // two extents below 2^31
  if (m > (1 << 28)) return WQ_ERR_PARAM_INVALID;
  const int64_t L = a->shape[0], r = a->shape[1], n = b->shape[1];
  if (k < 8 || k > 65535 || k % 8 != 0) return WQ_ERR_PARAM_INVALID;
  if (L < 1 || L > 65535 || r < 8 || r > 256 || r % 8 != 0) return WQ_ERR_PARAM_INVALID;
  if (n < 8 || n > (1 << 22) || n % 8 != 0) return WQ_ERR_PARAM_INVALID;
  if (a->shape[2] != k || b->shape[0] != L || b->shape[2] != r) return WQ_ERR_PARAM_INVALID;
  if (indices->shape[0] != m) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {scale, ranks})
    if (t && t->shape[0] != L) return WQ_ERR_PARAM_INVALID;
  if (output->ndim != x1->ndim || output->shape[output->ndim - 1] != n) return WQ_ERR_PARAM_INVALID;
  for (int i = 0; i < x1->ndim - 1; ++i)
    if (output->shape[i] != x1->shape[i]) return WQ_ERR_PARAM_INVALID;
  if (x3 && !same_shape(x3, output)) return WQ_ERR_PARAM_INVALID;

  int64_t sx = 0, s3 = 0, so = 0;
  if (!rows_ok(x1) || !rows_ok(output) || !disjoint(output) || !fold_rows(x1, &sx) || !fold_rows(output, &so))
    return WQ_ERR_PARAM_INVALID;
  if (x3 && (!rows_ok(x3) || !fold_rows(x3, &s3))) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {a, b})
    if (!contiguous(t) || ((uintptr_t)t->data & 15u) != 0) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {indices, scale, ranks})
    if (t && !index_ok(t)) return WQ_ERR_PARAM_INVALID;
  if (x3 && starts_at(x3, output->data) && !same_place(x3, output)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {x1, a, b, indices, scale, ranks})
    if (starts_at(t, output->data)) return WQ_ERR_PARAM_INVALID;

  if (p) {
    p->m = m; p->n = n; p->L = L; p->k = (int32_t)k; p->r = (int32_t)r; p->act = act;
    p->sx = sx; p->s3 = s3; p->so = so;
    p->x1 = x1->data; p->a = a->data; p->b = b->data;
    p->indices = (const int32_t*)indices->data;
    p->scale = scale ? (const float*)scale->data : nullptr;
    p->ranks = ranks ? (const int32_t*)ranks->data : nullptr;
    p->x3 = x3 ? x3->data : nullptr;
    p->out = output->data;
  }
  return WQ_OK;
}

int validate_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
                  const wq_tensor* inv_freq, const wq_tensor* slots, int32_t layout, float factor,
                  const wq_tensor* q_out, const wq_tensor* k_out, const wq_tensor* v_out, RopeProblem* p) {
  if (!q || !positions || !inv_freq || !q_out || (k && !k_out) || (v && !v_out)) return WQ_ERR_PARAM_NULLPTR;
  for (const wq_tensor* t : {q, k, v, positions, inv_freq, slots, q_out, k_out, v_out})
    if (t && !data_ok(t)) return WQ_ERR_PARAM_NULLPTR;

  const int32_t act = q->dtype;
  if (!is16(act)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {k, v, q_out, k_out, v_out})
    if (t && t->dtype != act) return WQ_ERR_PARAM_INVALID;
  if (positions->dtype != WQ_I32 || inv_freq->dtype != WQ_F32 || (slots && slots->dtype != WQ_I32))
    return WQ_ERR_PARAM_INVALID;

  if (layout != WQ_ROPE_HALF && layout != WQ_ROPE_INTERLEAVED) return WQ_ERR_PARAM_INVALID;
  if (!std::isfinite(factor)) return WQ_ERR_PARAM_INVALID;
  if ((!k && (v || slots || k_out)) || (!v && v_out)) return WQ_ERR_PARAM_INVALID;

  for (const wq_tensor* t : {q, k, v, q_out, k_out, v_out})
    if (t && !dims_ok(t, 3, 3)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {positions, inv_freq, slots})
    if (t && !dims_ok(t, 1, 1)) return WQ_ERR_PARAM_INVALID;
  const int64_t T = q->shape[0], hq = q->shape[1], d = q->shape[2], half = inv_freq->shape[0];
  if (hq < 1 || hq > 65535 || d < 8 || d > 256 || d % 8 != 0) return WQ_ERR_PARAM_INVALID;
  if (half < 1 || half > d / 2) return WQ_ERR_PARAM_INVALID;
  if (positions->shape[0] != T || !same_shape(q, q_out)) return WQ_ERR_PARAM_INVALID;
  const int64_t hkv = k ? k->shape[1] : 0;
  if (k && (k->shape[0] != T || hkv < 1 || hkv > 65535 || k->shape[2] != d)) return WQ_ERR_PARAM_INVALID;
  if (v && !same_shape(k, v)) return WQ_ERR_PARAM_INVALID;
  if (slots && slots->shape[0] != T) return WQ_ERR_PARAM_INVALID;
  int64_t S = T;
  if (k) {
    S = k_out->shape[0];
    if ((!slots && S != T) || k_out->shape[1] != hkv || k_out->shape[2] != d) return WQ_ERR_PARAM_INVALID;
    if (v && !same_shape(k_out, v_out)) return WQ_ERR_PARAM_INVALID;
  }

  for (const wq_tensor* t : {q, k, v, q_out, k_out, v_out})
    if (t && !rows_ok(t)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {q_out, k_out, v_out})
    if (t && !disjoint(t)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {positions, inv_freq, slots})
    if (t && !index_ok(t)) return WQ_ERR_PARAM_INVALID;
  // in place: q_out may be q, and without slots k_out may be k; no other output starts at
  // another tensor
  struct { const wq_tensor* out; const wq_tensor* in; } pairs[] = {
      {q_out, q}, {k_out, slots ? nullptr : k}, {v_out, nullptr}};
  for (const auto& o : pairs) {
    if (!o.out || empty(o.out)) continue;
    for (const wq_tensor* t : {q, k, v, positions, inv_freq, slots})
      if (starts_at(t, o.out->data) && !(t == o.in && same_place(t, o.out))) return WQ_ERR_PARAM_INVALID;
    for (const wq_tensor* t : {q_out, k_out, v_out})
      if (t != o.out && starts_at(t, o.out->data)) return WQ_ERR_PARAM_INVALID;
  }

  if (p) {
    p->T = T; p->S = S; p->hq = (int32_t)hq; p->hkv = (int32_t)hkv; p->d = (int32_t)d; p->half = (int32_t)half;
    p->act = act; p->interleaved = layout == WQ_ROPE_INTERLEAVED; p->factor = factor;
    p->q = q->data; p->q_t = stride_of(q, 0); p->q_h = stride_of(q, 1);
    p->qo = q_out->data; p->qo_t = stride_of(q_out, 0); p->qo_h = stride_of(q_out, 1);
    if (k) {
      p->k = k->data; p->k_t = stride_of(k, 0); p->k_h = stride_of(k, 1);
      p->ko = k_out->data; p->ko_t = stride_of(k_out, 0); p->ko_h = stride_of(k_out, 1);
    }
    if (v) {
      p->v = v->data; p->v_t = stride_of(v, 0); p->v_h = stride_of(v, 1);
      p->vo = v_out->data; p->vo_t = stride_of(v_out, 0); p->vo_h = stride_of(v_out, 1);
    }
    p->positions = (const int32_t*)positions->data;
    p->inv_freq = (const float*)inv_freq->data;
    p->slots = slots ? (const int32_t*)slots->data : nullptr;
  }
  return WQ_OK;
}

int validate_tree(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                  const wq_tensor* block_table, const wq_tensor* context_lens, const wq_tensor* q_starts,
                  const wq_tensor* tree_mask, int64_t page_size, const wq_tensor* output, TreeProblem* p) {
  if (!q || !k_cache || !v_cache || !block_table || !context_lens || !q_starts || !output)
    return WQ_ERR_PARAM_NULLPTR;
  for (const wq_tensor* t : {q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask, output})
    if (t && !data_ok(t)) return WQ_ERR_PARAM_NULLPTR;

  const int32_t act = q->dtype;
  if (!is16(act)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {k_cache, v_cache, output})
    if (t->dtype != act) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {block_table, context_lens, q_starts, tree_mask})
    if (t && t->dtype != WQ_I32) return WQ_ERR_PARAM_INVALID;

  if (page_size < 1 || page_size > (1 << 20)) return WQ_ERR_PARAM_INVALID;

  for (const wq_tensor* t : {q, k_cache, v_cache, output})
    if (!dims_ok(t, 3, 3)) return WQ_ERR_PARAM_INVALID;
  if (!dims_ok(block_table, 2, 2) || !dims_ok(context_lens, 1, 1) || !dims_ok(q_starts, 1, 1) ||
      (tree_mask && !dims_ok(tree_mask, 2, 2)))
    return WQ_ERR_PARAM_INVALID;
  const int64_t N = q->shape[0], hq = q->shape[1], d = q->shape[2], S = k_cache->shape[0], hkv = k_cache->shape[1];
  const int64_t B = block_table->shape[0], width = block_table->shape[1];
  if (d != 64 && d != 128 && d != 256) return WQ_ERR_PARAM_INVALID;
  if (hq < 1 || hq > 65535 || hkv < 1 || hkv > hq || hq % hkv != 0) return WQ_ERR_PARAM_INVALID;
  if (N > (1 << 24) || N * hq > (1 << 30) || B > 65535) return WQ_ERR_PARAM_INVALID;
  if (k_cache->shape[2] != d || S % page_size != 0 || !same_shape(k_cache, v_cache) || !same_shape(q, output))
    return WQ_ERR_PARAM_INVALID;
  // keys past the last by a tile, a unit or the slots that stand in LDS are still 32-bit numbers
  if (width * page_size > kMaxExtent - 65535) return WQ_ERR_PARAM_INVALID;
  if (context_lens->shape[0] != B || q_starts->shape[0] != B + 1) return WQ_ERR_PARAM_INVALID;
  if (tree_mask && (tree_mask->shape[0] != N || tree_mask->shape[1] > (1 << 20))) return WQ_ERR_PARAM_INVALID;

  for (const wq_tensor* t : {q, k_cache, v_cache, output})
    if (!rows_ok(t)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {k_cache, v_cache})
    if (!empty(t) && stride_of(t, 0) > (1 << 30)) return WQ_ERR_PARAM_INVALID;
  if (!disjoint(output)) return WQ_ERR_PARAM_INVALID;
  for (const wq_tensor* t : {block_table, context_lens, q_starts, tree_mask})
    if (t && !index_ok(t)) return WQ_ERR_PARAM_INVALID;
  if (!empty(output))
    for (const wq_tensor* t : {q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask})
      if (starts_at(t, output->data)) return WQ_ERR_PARAM_INVALID;

  if (p) {
    p->N = N; p->B = B; p->pages = S / page_size;
    p->hq = (int32_t)hq; p->hkv = (int32_t)hkv; p->group = (int32_t)(hq / hkv); p->d = (int32_t)d;
    p->width = (int32_t)width; p->page = (int32_t)page_size; p->act = act;
    p->q = q->data; p->q_t = stride_of(q, 0); p->q_h = stride_of(q, 1);
    p->k = k_cache->data; p->k_t = stride_of(k_cache, 0); p->k_h = stride_of(k_cache, 1);
    p->v = v_cache->data; p->v_t = stride_of(v_cache, 0); p->v_h = stride_of(v_cache, 1);
    p->out = output->data; p->o_t = stride_of(output, 0); p->o_h = stride_of(output, 1);
    p->table = (const int32_t*)block_table->data;
    p->context = (const int32_t*)context_lens->data;
    p->starts = (const int32_t*)q_starts->data;
    p->has_mask = tree_mask != nullptr;
    p->words = tree_mask ? (int32_t)tree_mask->shape[1] : 0;
    p->mask = tree_mask ? (const uint32_t*)tree_mask->data : nullptr;
  }
  return WQ_OK;
}

}  // namespace wq

extern "C" {

int wq_lora_matmul_get_workspace_size(const wq_tensor* x1, const wq_tensor* a, const wq_tensor* b,
                                      const wq_tensor* indices, const wq_tensor* scale, const wq_tensor* ranks,
                                      const wq_tensor* x3, const wq_tensor* output, uint64_t* workspace_size) {
  if (!workspace_size) return WQ_ERR_PARAM_NULLPTR;
  wq::LoraProblem p;
  const int st = wq::validate_lora(x1, a, b, indices, scale, ranks, x3, output, &p);
  if (st == WQ_OK) *workspace_size = (uint64_t)wq::plan_lora(p).workspace;
  return st;
}

int wq_tree_attention_get_workspace_size(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                                         const wq_tensor* block_table, const wq_tensor* context_lens,
                                         const wq_tensor* q_starts, const wq_tensor* tree_mask, int64_t page_size,
                                         const wq_tensor* output, uint64_t* workspace_size) {
  if (!workspace_size) return WQ_ERR_PARAM_NULLPTR;
  wq::TreeProblem p;
  const int st = wq::validate_tree(q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask, page_size,
                                   output, &p);
  if (st == WQ_OK) *workspace_size = (uint64_t)wq::plan_tree(p).workspace;
  return st;
}

}  // extern "C"
