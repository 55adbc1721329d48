// Column sums of dw partial rows for two outputs at once (the weight
// gradients of queries and keys; dw and db of a group norm), in a fixed
// order: thread row q of a block adds rows q, q + R, q + 2R, ... in ascending
// order, then a pairwise tree adds the R sums of a column. The same bits on
// every run for given sizes. A few hundred rows of a few hundred columns: the
// time is one trip to L2 and the launch, so columns are spread over as many
// blocks as keep 16-byte row pieces.
#include "common.cuh"
#include "ops.h"

namespace rmsn {
namespace {

template <int C>
__global__ void __launch_bounds__(1024) pair_sum_kernel(const __grid_constant__ PairSum a) {
    constexpr int R = 1024 / C;
    __shared__ float part[R][C + 1];
    const int cx = threadIdx.x % C, q = threadIdx.x / C;
    const int which = blockIdx.y;
    const int col = blockIdx.x * C + cx;
    wait_for_prerequisite_grid();  // partial rows complete and visible
    allow_dependent_launch();
    const float* src = a.part[which];
    float* out = a.out[which];
    float s = 0.f;
    if (col < a.n && out != nullptr) {
#pragma unroll 4
        for (int p = q; p < a.rows[which]; p += R) s += src[static_cast<int64_t>(p) * a.stride + col];
    }
    part[q][cx] = s;
    __syncthreads();
#pragma unroll
    for (int h = R / 2; h > 0; h >>= 1) {
        if (q < h) part[q][cx] += part[q + h][cx];
        __syncthreads();
    }
    if (q == 0 && col < a.n && out != nullptr &&
        RMSN_OK(span_in(out + col, 4, out, static_cast<int64_t>(a.n) * 4), a.status))
        out[col] = part[0][cx];
}

}  // namespace

cudaError_t pair_sum_launch(const PairSum& a, cudaStream_t s) {
    const int c = a.n >= 1024 ? 32 : a.n >= 256 ? 8 : 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cdiv(a.n, c)), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_allowed();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (c == 32) return cudaLaunchKernelEx(&cfg, pair_sum_kernel<32>, a);
    if (c == 8) return cudaLaunchKernelEx(&cfg, pair_sum_kernel<8>, a);
    return cudaLaunchKernelEx(&cfg, pair_sum_kernel<4>, a);
}

}  // namespace rmsn
