// Rotary kernels of bf16 tensors.
#include "rope_kernels.cuh"

namespace rmsn {

RopeFn rope_kernel_bf16(int e, int units, int lanes, bool bwd, bool adjacent, bool norm) {
    return kernel_for_type<__nv_bfloat16>(e, units, lanes, bwd, adjacent, norm);
}

}  // namespace rmsn
