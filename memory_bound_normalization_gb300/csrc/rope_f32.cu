// Rotary kernels of f32 tensors.
#include "rope_kernels.cuh"

namespace rmsn {

RopeFn rope_kernel_f32(int e, int units, int lanes, bool bwd, bool adjacent, bool norm) {
    return kernel_for_type<float>(e, units, lanes, bwd, adjacent, norm);
}

}  // namespace rmsn
