// Device helpers of the group norm kernels: the activations and their
// derivatives.
#pragma once

#include "common.cuh"
#include "rmsnorm.h"

namespace rmsn {

// silu(z) = z / (1 + e^-z). For z below -88 the power is infinite and the
// quotient a zero, the fp32 limit.
__device__ __forceinline__ float act_value(float z, int act) {
    if (act == RMSNORM_ACT_SILU) return z / (1.f + expf(-z));
    if (act == RMSNORM_ACT_GELU) return z * normcdff(z);
    return z;
}
// d silu = s (1 + z (1 - s)), s = 1 / (1 + e^-z); d gelu = Phi(z) + z phi(z).
__device__ __forceinline__ float act_slope(float z, int act) {
    if (act == RMSNORM_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        return s * fmaf(z, 1.f - s, 1.f);
    }
    if (act == RMSNORM_ACT_GELU)
        return fmaf(z * 0.3989422804014327f, expf(-0.5f * z * z), normcdff(z));
    return 1.f;
}

// One element rounded once, to nearest even.
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_f32(__half* p, float v) { *p = __float2half_rn(v); }

}  // namespace rmsn
