// Resolved problems, validation and planning of the serving operators around a step's attention
// (wqserve.h): layout, head norms with rotary positions, shared prefixes, verification.  Host-only
// C++ (no HIP types).
#pragma once
#include <cstdint>

#include "serve_problem.h"

namespace wq {

struct NormRopeProblem {
  RopeProblem rope;                 // positions: of the first axis
  int32_t axes = 1;                 // rows of positions
  float eps = 0.f;
  const int32_t* axis_of = nullptr;  // of each pair; may be null
  const void* q_weight = nullptr;   // may be null
  const void* k_weight = nullptr;
  bool q_weight32 = false, k_weight32 = false;  // fp32, not the activations' type
};

struct LayoutProblem {
  int64_t B = 0, N = 0, F = 0, width = 0, page = 1, words = 0;
  const int32_t* context = nullptr;
  const int32_t* fresh = nullptr;
  int32_t* table = nullptr;
  const int32_t* free_pages = nullptr;
  const int32_t* free_count = nullptr;
  const int32_t* offsets = nullptr;   // may be null
  const int32_t* parents = nullptr;   // may be null
  int32_t* starts = nullptr;
  int32_t* requests = nullptr;        // may be null
  int32_t* positions = nullptr;
  int32_t* slots = nullptr;
  uint32_t* mask = nullptr;           // may be null
  int32_t* free_left = nullptr;
};

// Attention of tokens over a prefix of their group and over keys of their sequence: two problems whose
// rows are the same tokens.
struct PrefixProblem {
  TreeProblem own, shared;  // shared: B groups, context their lengths, no mask
  const int32_t* group_starts = nullptr;
};

struct PrefixPlan {
  TreePlan own, shared;
  bool split_join = false;  // whether four waves share the parts of a row
  // offsets in bytes; parts: two of each workgroup, then one for each tile
  int64_t shared_notes = 0, own_notes = 0, groups = 0, shared_parts = 0, own_parts = 0;
  int64_t workspace = 0;
};

struct VerifyProblem {
  int64_t N = 0, B = 0, V = 0, depth = 0;
  int32_t dtype = WQ_F32;
  int64_t t_row = 0, d_row = 0;      // row strides in elements
  const void* target = nullptr;
  const void* draft = nullptr;       // may be null
  const int32_t* tokens = nullptr;
  const int32_t* parents = nullptr;  // may be null
  const int32_t* starts = nullptr;
  const float* accept = nullptr;
  const float* sample = nullptr;
  int32_t* accepted = nullptr;
  int32_t* counts = nullptr;
  int32_t* next = nullptr;
};

struct VerifyPlan {
  int64_t unit = 0, units = 0;    // probabilities of a sum, and sums of a row
  int64_t chunk = 0, chunks = 0;  // units of a workgroup, and workgroups of a row
  int64_t sums = 0, refused = 0;  // offsets in bytes: the units' sums; the refused tokens (without draft)
  int64_t workspace = 0;          // states first
};
constexpr int kVerifyStateBytes = 16;
constexpr int kVerifyTokens = 1024;  // of a request

int validate_norm_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
                       const wq_tensor* inv_freq, const wq_tensor* axes, const wq_tensor* q_weight,
                       const wq_tensor* k_weight, float eps, const wq_tensor* slots, int32_t layout, float factor,
                       const wq_tensor* q_out, const wq_tensor* k_out, const wq_tensor* v_out, NormRopeProblem* p);
int validate_layout(const wq_tensor* context_lens, const wq_tensor* new_lens, const wq_tensor* block_table,
                    const wq_tensor* free_pages, const wq_tensor* free_count, const wq_tensor* position_offsets,
                    const wq_tensor* parents, int64_t page_size, const wq_tensor* q_starts, const wq_tensor* requests,
                    const wq_tensor* positions, const wq_tensor* slots, const wq_tensor* tree_mask,
                    const wq_tensor* free_left, LayoutProblem* p);
int validate_prefix(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache, const wq_tensor* prefix_table,
                    const wq_tensor* prefix_lens, const wq_tensor* prefix_starts, const wq_tensor* block_table,
                    const wq_tensor* context_lens, const wq_tensor* q_starts, const wq_tensor* tree_mask,
                    int64_t page_size, const wq_tensor* output, PrefixProblem* p);
int validate_verify(const wq_tensor* target, const wq_tensor* draft, const wq_tensor* tokens, const wq_tensor* parents,
                    const wq_tensor* q_starts, const wq_tensor* accept_random, const wq_tensor* sample_random,
                    const wq_tensor* accepted, const wq_tensor* counts, const wq_tensor* next_tokens, VerifyProblem* p);

PrefixPlan plan_prefix(const PrefixProblem& p);
VerifyPlan plan_verify(const VerifyProblem& p);

}  // namespace wq
