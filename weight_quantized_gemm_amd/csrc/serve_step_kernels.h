// Launchers of the serving operators around a step's attention (host side of their HIP translation units).
#pragma once
#include <hip/hip_runtime.h>

#include "serve_step.h"

namespace wq {

hipError_t launch_norm_rope(const NormRopeProblem& p, hipStream_t stream);
hipError_t launch_layout(const LayoutProblem& p, hipStream_t stream);
hipError_t launch_prefix(const PrefixProblem& p, const PrefixPlan& pl, float scale, void* workspace, hipStream_t stream);
hipError_t launch_verify(const VerifyProblem& p, const VerifyPlan& pl, void* workspace, hipStream_t stream);

}  // namespace wq
