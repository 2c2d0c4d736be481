// Resolved problems, validation and planning of the serving operators (wqserve.h).
// Host-only C++ (no HIP types), so that it builds and runs without a GPU.
#pragma once
#include <cstdint>

#include "wqserve.h"

namespace wq {

// Division of 0 <= x < 2^31 by a fixed d in [1, 2^31): x / d = (x * mul) >> (32 + shift).
// shift is the smallest s with 2^(s + 1) >= d and mul = ceil(2^(32 + s) / d), which fits 32
// bits.  mul * d exceeds 2^(32 + s) by e < d <= 2^(s + 1), so the quotient is too large by
// x e / (d 2^(32 + s)) < 1 / d, which never reaches the next integer.
struct FastDiv {
  uint32_t mul = 0;  // 0: d == 1
  uint32_t shift = 0;
  uint32_t d = 1;
};
FastDiv fast_div(uint32_t d);

struct LoraProblem {
  int64_t m = 0, n = 0, L = 0;
  int32_t k = 0, r = 0;
  int32_t act = WQ_F16;
  int64_t sx = 0, s3 = 0, so = 0;  // row strides of x1, x3, output in elements
  const void* x1 = nullptr;
  const void* a = nullptr;
  const void* b = nullptr;
  const int32_t* indices = nullptr;
  const float* scale = nullptr;     // may be null
  const int32_t* ranks = nullptr;   // may be null
  const void* x3 = nullptr;         // may be null
  void* out = nullptr;
};

struct LoraPlan {
  int window = 16;         // token rows of a work item (16 or 64)
  int64_t windows = 0;
  int slots = 1;           // 16-row windows: work items of one that run side by side
  int splits = 1;          // k splits of the first product
  int kchunk = 0;          // k per split, a multiple of 64
  int rank_tiles = 4;      // 16-rank tiles of a workgroup of the first product, and blocks of them
  int rank_blocks = 1;
  int cols = 128;          // columns of a workgroup of the second product, and blocks of them
  int col_blocks = 1;
  int64_t shrink_blocks = 0, expand_blocks = 0;  // workgroups of the two products
  int64_t list_bytes = 0;  // 64-row windows: the list of work items and its length
  int64_t workspace = 0;   // the list, then fp32 partials of x1 @ a^T, [splits][m][r]
};

struct RopeProblem {
  int64_t T = 0, S = 0;
  int32_t hq = 0, hkv = 0, d = 0, half = 0;  // half = rot / 2
  int32_t act = WQ_F16;
  bool interleaved = false;
  float factor = 1.f;
  // token (row) and head strides in elements
  int64_t q_t = 0, q_h = 0, k_t = 0, k_h = 0, v_t = 0, v_h = 0;
  int64_t qo_t = 0, qo_h = 0, ko_t = 0, ko_h = 0, vo_t = 0, vo_h = 0;
  const void* q = nullptr;
  const void* k = nullptr;  // may be null
  const void* v = nullptr;  // may be null
  const int32_t* positions = nullptr;
  const float* inv_freq = nullptr;
  const int32_t* slots = nullptr;  // may be null
  void* qo = nullptr;
  void* ko = nullptr;
  void* vo = nullptr;
};

struct TreeProblem {
  int64_t N = 0, B = 0, pages = 0;
  int32_t hq = 0, hkv = 0, group = 0, d = 0, width = 0, words = 0, page = 0;
  int32_t act = WQ_F16;
  int64_t q_t = 0, q_h = 0, k_t = 0, k_h = 0, v_t = 0, v_h = 0, o_t = 0, o_h = 0;
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  const int32_t* table = nullptr;
  const int32_t* context = nullptr;
  const int32_t* starts = nullptr;
  bool has_mask = false;           // (a mask of no words is one that shows no drafted token)
  const uint32_t* mask = nullptr;
  void* out = nullptr;
};

struct TreePlan {
  bool split_rows = false;  // a workgroup's waves split the rows of a tile (else its keys)
  int waves = 4;
  int rows = 16;            // of a tile: tokens x query heads of a cached head
  int unit = 128;           // keys, the unit of the work that workgroups share
  int64_t blocks = 0;       // workgroups (an upper bound of the shares)
  int64_t tiles = 0;        // an upper bound of the tiles
  int64_t notes_bytes = 0;  // the tiles' notes
  int64_t workspace = 0;    // the notes, then two partial tiles for each workgroup
};

int validate_lora(const wq_tensor* x1, const wq_tensor* a, const wq_tensor* b, const wq_tensor* indices,
                  const wq_tensor* scale, const wq_tensor* ranks, const wq_tensor* x3,
                  const wq_tensor* output, LoraProblem* p);
int validate_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
                  const wq_tensor* inv_freq, const wq_tensor* slots, int32_t layout, float factor,
                  const wq_tensor* q_out, const wq_tensor* k_out, const wq_tensor* v_out, RopeProblem* p);
int validate_tree(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                  const wq_tensor* block_table, const wq_tensor* context_lens, const wq_tensor* q_starts,
                  const wq_tensor* tree_mask, int64_t page_size, const wq_tensor* output, TreeProblem* p);

// The plans depend on the arguments' shapes alone (the size queries touch no device).
LoraPlan plan_lora(const LoraProblem& p);
TreePlan plan_tree(const TreeProblem& p);

}  // namespace wq
