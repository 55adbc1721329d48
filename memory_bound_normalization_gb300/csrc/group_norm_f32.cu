// Group norm kernels of f32 tensors.
#include "group_norm_kernels.cuh"

namespace rmsn {

SlabFn gn_kernel_f32(bool bwd, int act, SlabKind k) { return slab_kernel_of<float>(bwd, act, k); }

}  // namespace rmsn
