// The kernel families of the group norm (host code only): the general path
// (group_norm_scalar.cu).
#pragma once

#include "ops.h"

namespace rmsn {

size_t gn_scalar_workspace(bool bwd, const GroupNormArgs& a);
cudaError_t gn_scalar_launch(int dtype, bool bwd, const GroupNormArgs& a, void* ws, cudaStream_t s);

}  // namespace rmsn
