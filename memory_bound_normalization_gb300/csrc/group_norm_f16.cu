// Group norm kernels of f16 tensors.
#include "group_norm_kernels.cuh"

namespace rmsn {

SlabFn gn_kernel_f16(bool bwd, int act, SlabKind k) { return slab_kernel_of<__half>(bwd, act, k); }

}  // namespace rmsn
