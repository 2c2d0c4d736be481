// Launchers of the serving operators (host side of their HIP translation units).
#pragma once
#include <hip/hip_runtime.h>

#include "serve_problem.h"

namespace wq {

hipError_t launch_lora(const LoraProblem& p, const LoraPlan& pl, void* workspace, hipStream_t stream);
hipError_t launch_rope(const RopeProblem& p, hipStream_t stream);
hipError_t launch_tree(const TreeProblem& p, const TreePlan& pl, float scale, void* workspace, hipStream_t stream);

}  // namespace wq
