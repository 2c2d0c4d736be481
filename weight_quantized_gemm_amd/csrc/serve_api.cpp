// Run entry points of the serving operators (wqserve.h): validate, plan, launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "serve_kernels.h"

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

int wq_lora_matmul(const wq_tensor* x1, const wq_tensor* a, const wq_tensor* b, const wq_tensor* indices,
                   const wq_tensor* scale, const wq_tensor* ranks, const wq_tensor* x3, const wq_tensor* output,
                   void* workspace, uint64_t workspace_size, void* stream) {
  wq::LoraProblem p;
  int st = wq::validate_lora(x1, a, b, indices, scale, ranks, x3, output, &p);
  if (st != WQ_OK) return st;
  const wq::LoraPlan pl = wq::plan_lora(p);
  if ((st = check_workspace(workspace, workspace_size, pl.workspace)) != WQ_OK) return st;
  if (p.m == 0) return WQ_OK;
  return status(wq::launch_lora(p, pl, workspace, (hipStream_t)stream));
}

int wq_rope(const wq_tensor* q, const wq_tensor* k, const wq_tensor* v, const wq_tensor* positions,
            const wq_tensor* inv_freq, const wq_tensor* slots, int32_t layout, float attention_factor,
            const wq_tensor* q_out, const wq_tensor* k_out, const wq_tensor* v_out, void* stream) {
  wq::RopeProblem p;
  const int st = wq::validate_rope(q, k, v, positions, inv_freq, slots, layout, attention_factor, q_out, k_out,
                                   v_out, &p);
  if (st != WQ_OK) return st;
  if (p.T == 0) return WQ_OK;
  return status(wq::launch_rope(p, (hipStream_t)stream));
}

int wq_tree_attention(const wq_tensor* q, const wq_tensor* k_cache, const wq_tensor* v_cache,
                      const wq_tensor* block_table, const wq_tensor* context_lens, const wq_tensor* q_starts,
                      const wq_tensor* tree_mask, int64_t page_size, float scale, const wq_tensor* output,
                      void* workspace, uint64_t workspace_size, void* stream) {
  wq::TreeProblem p;
  int st = wq::validate_tree(q, k_cache, v_cache, block_table, context_lens, q_starts, tree_mask, page_size, output,
                             &p);
  if (st != WQ_OK) return st;
  if (!(std::fabs(scale) <= 0x1p127f)) return WQ_ERR_PARAM_INVALID;  // its product with log2(e) is finite
  const wq::TreePlan pl = wq::plan_tree(p);
  if ((st = check_workspace(workspace, workspace_size, pl.workspace)) != WQ_OK) return st;
  if (p.N == 0 || p.B == 0) return WQ_OK;
  return status(wq::launch_tree(p, pl, scale, workspace, (hipStream_t)stream));
}

}  // extern "C"
