// Group norm kernels of bf16 tensors.
#include "group_norm_kernels.cuh"

namespace rmsn {

SlabFn gn_kernel_bf16(bool bwd, int act, SlabKind k) { return slab_kernel_of<__nv_bfloat16>(bwd, act, k); }

}  // namespace rmsn
