// Run entry points of the serving operators around a step's attention (wqserve.h): validate, plan, launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "serve_step_kernels.h"

namespace {

int check_workspace(const void* workspace, uint64_t size, int64_t need) {
  if (size < (uint64_t)need) return WQ_ERR_PARAM_INVALID;
  if (need > 0 && !workspace) return WQ_ERR_PARAM_NULLPTR;
  if (need > 0 && ((uintptr_t)workspace & 255u) != 0) return WQ_ERR_PARAM_INVALID;
  return WQ_OK;
}

int status(hipError_t e) { return e == hipSuccess ? WQ_OK : WQ_ERR_RUNTIME; }

}  // namespace

extern "C" {

int wq_norm_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
                 const wq_tensor* inv_freq, const wq_tensor* axes, const wq_tensor* q_weight, const wq_tensor* k_weight,
                 float eps, const wq_tensor* slots, int32_t layout, float attention_factor, const wq_tensor* q_out,
                 const wq_tensor* k_out, const wq_tensor* v_out, void* stream) {
  wq::NormRopeProblem p;
  const int st = wq::validate_norm_rope(q, k, v, positions, inv_freq, axes, q_weight, k_weight, eps, slots, layout,
                                        attention_factor, q_out, k_out, v_out, &p);
  if (st != WQ_OK) return st;
  if (p.rope.T == 0) return WQ_OK;
  return status(wq::launch_norm_rope(p, (hipStream_t)stream));
}

int wq_step_layout(const wq_tensor* context_lens, const wq_tensor* new_lens, const wq_tensor* block_table,
                   const wq_tensor* free_pages, const wq_tensor* free_count, const wq_tensor* position_offsets,
                   const wq_tensor* parents, int64_t page_size, const wq_tensor* q_starts, const wq_tensor* requests,
                   const wq_tensor* positions, const wq_tensor* slots, const wq_tensor* tree_mask,
                   const wq_tensor* free_left, void* stream) {
  wq::LayoutProblem p;
  const int st = wq::validate_layout(context_lens, new_lens, block_table, free_pages, free_count, position_offsets,
                                     parents, page_size, q_starts, requests, positions, slots, tree_mask, free_left, &p);
  if (st != WQ_OK) return st;
  return status(wq::launch_layout(p, (hipStream_t)stream));
}

int wq_prefix_attention(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                        const wq_tensor* prefix_table, const wq_tensor* prefix_lens, const wq_tensor* prefix_starts,
                        const wq_tensor* block_table, const wq_tensor* context_lens, const wq_tensor* q_starts,
                        const wq_tensor* tree_mask, int64_t page_size, float scale, const wq_tensor* output,
                        void* workspace, uint64_t workspace_size, void* stream) {
  wq::PrefixProblem p;
  int st = wq::validate_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, prefix_starts, block_table, context_lens,
                               q_starts, tree_mask, page_size, output, &p);
  if (st != WQ_OK) return st;
  if (!(std::fabs(scale) <= 0x1p127f)) return WQ_ERR_PARAM_INVALID;  // its product with log2(e) is finite
  const wq::PrefixPlan pl = wq::plan_prefix(p);
  if ((st = check_workspace(workspace, workspace_size, pl.workspace)) != WQ_OK) return st;
  if (p.own.N == 0 || p.own.B == 0) return WQ_OK;
  return status(wq::launch_prefix(p, pl, scale, workspace, (hipStream_t)stream));
}

int wq_verify_drafts(const wq_tensor* target, const wq_tensor* draft, const wq_tensor* tokens, const wq_tensor* parents,
                     const wq_tensor* q_starts, const wq_tensor* accept_random, const wq_tensor* sample_random,
                     const wq_tensor* accepted, const wq_tensor* counts, const wq_tensor* next_tokens, void* workspace,
                     uint64_t workspace_size, void* stream) {
  wq::VerifyProblem p;
  int st = wq::validate_verify(target, draft, tokens, parents, q_starts, accept_random, sample_random, accepted, counts,
                               next_tokens, &p);
  if (st != WQ_OK) return st;
  const wq::VerifyPlan pl = wq::plan_verify(p);
  if ((st = check_workspace(workspace, workspace_size, pl.workspace)) != WQ_OK) return st;
  if (p.B == 0) return WQ_OK;
  return status(wq::launch_verify(p, pl, workspace, (hipStream_t)stream));
}

}  // extern "C"
