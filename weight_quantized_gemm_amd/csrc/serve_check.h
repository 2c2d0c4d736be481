// Checks of descriptors that the serving operators' validation shares.  Pure host C++.
#pragma once
#include <climits>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "serve_problem.h"

namespace wq {

constexpr int64_t kMaxExtent = INT32_MAX;
constexpr int64_t kMaxStride = (int64_t)1 << 40;  // element strides: products stay far inside int64

inline bool dims_ok(const wq_tensor* t, int lo, int hi) {
  if (t->ndim < lo || t->ndim > hi) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] < 0 || t->shape[i] > kMaxExtent) return false;
  return true;
}

inline bool empty(const wq_tensor* t) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] == 0) return true;
  return false;
}

// data may be NULL only for an empty tensor
inline bool data_ok(const wq_tensor* t) {
  return t->data != nullptr || (t->ndim >= 1 && t->ndim <= 3 && empty(t));
}

inline bool contiguous(const wq_tensor* t) {
  if (empty(t)) return true;
  // extents are at most 2^31 - 1, so the running product is compared before it can overflow
  int64_t expect = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] > 1 && t->stride[i] != expect) return false;
    if (expect > kMaxStride) return false;
    expect *= t->shape[i];
  }
  return true;
}

// "rows": contiguous innermost axis, other strides non-negative multiples of 8, 16-byte aligned
inline bool rows_ok(const wq_tensor* t) {
  if (empty(t)) return true;
  if (t->shape[t->ndim - 1] > 1 && t->stride[t->ndim - 1] != 1) return false;
  for (int i = 0; i < t->ndim - 1; ++i)
    if (t->shape[i] > 1 && (t->stride[i] < 0 || t->stride[i] > kMaxStride || t->stride[i] % 8 != 0)) return false;
  return ((uintptr_t)t->data & 15u) == 0;
}

inline bool index_ok(const wq_tensor* t) { return contiguous(t) && ((uintptr_t)t->data & 3u) == 0; }

// No two elements of a rows-tensor share an address: of its axes in ascending order of stride,
// each steps over everything the ones before it reach.
inline bool disjoint(const wq_tensor* t) {
  if (empty(t)) return true;
  int axis[2] = {-1, -1}, n = 0;
  for (int i = 0; i < t->ndim - 1; ++i)
    if (t->shape[i] > 1) axis[n++] = i;
  if (n == 2 && t->stride[axis[0]] < t->stride[axis[1]]) std::swap(axis[0], axis[1]);
  int64_t reach = t->shape[t->ndim - 1];
  for (int j = n - 1; j >= 0; --j) {
    if (t->stride[axis[j]] < reach) return false;
    if (t->shape[axis[j]] > kMaxStride / t->stride[axis[j]]) return false;  // the extent would pass 2^40 elements
    reach += t->stride[axis[j]] * (t->shape[axis[j]] - 1);
  }
  return true;
}

// the stride of an axis, 0 where its extent does not read it
inline int64_t stride_of(const wq_tensor* t, int i) { return t->shape[i] > 1 ? t->stride[i] : 0; }

inline bool same_shape(const wq_tensor* a, const wq_tensor* b) {
  if (a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

inline bool same_place(const wq_tensor* a, const wq_tensor* b) {
  if (a->data != b->data) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] > 1 && a->stride[i] != b->stride[i]) return false;
  return true;
}

inline bool is16(int32_t dt) { return dt == WQ_F16 || dt == WQ_BF16; }

inline bool starts_at(const wq_tensor* t, const void* p) { return t && t->data && t->data == p; }

// the row stride of a 2-D or 3-D rows-tensor read as (m, cols); false where the two leading
// axes of a 3-D one do not fold into one
inline bool fold_rows(const wq_tensor* t, int64_t* stride) {
  if (t->ndim == 2) { *stride = stride_of(t, 0); return true; }
  if (t->shape[0] > 1 && t->shape[1] > 1 && t->stride[0] != t->shape[1] * t->stride[1]) return false;
  *stride = t->shape[1] > 1 ? t->stride[1] : stride_of(t, 0);
  return true;
}

}  // namespace wq
