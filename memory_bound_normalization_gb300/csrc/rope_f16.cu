// Rotary kernels of f16 tensors.
#include "rope_kernels.cuh"

namespace rmsn {

RopeFn rope_kernel_f16(int e, int units, int lanes, bool bwd, bool adjacent, bool norm) {
    return kernel_for_type<__half>(e, units, lanes, bwd, adjacent, norm);
}

}  // namespace rmsn
