// Column sums of dw partial rows for two outputs at once (the weight gradients
// of queries and keys; dw and db of a group norm), in a fixed order: a block of
// eight warps takes W neighbouring columns, thread t adds rows t, t + 256, ...
// in ascending order (in runs of 64, and the runs: a chain of a million samples' rows
// was 645 roundings off), a butterfly adds a warp's lanes and thread 0 the warps.
// The same bits on every run for given sizes. A few hundred rows of a few
// hundred columns: the time is the launch and one trip to L2 (some 3 us of 304
// rows of 128), so every row has a thread of its own where there are no more than
// 256, and one barrier is all.
#include "common.cuh"
#include "ops.h"

namespace rmsn {
namespace {

constexpr unsigned kRun = 64;

template <int W>
struct Columns;
template <>
struct Columns<4> {
    using V = float4;
    __device__ static void add(float (&s)[4], const float4& v) {
        s[0] += v.x;
        s[1] += v.y;
        s[2] += v.z;
        s[3] += v.w;
    }
};
template <>
struct Columns<2> {
    using V = float2;
    __device__ static void add(float (&s)[2], const float2& v) {
        s[0] += v.x;
        s[1] += v.y;
    }
};
template <>
struct Columns<1> {
    using V = float;
    __device__ static void add(float (&s)[1], const float& v) { s[0] += v; }
};

template <int W>
__global__ void __launch_bounds__(kItemThreads) pair_sum_kernel(const __grid_constant__ PairSum a) {
    using V = typename Columns<W>::V;
    __shared__ float part[kItemThreads / 32][W];
    const int which = blockIdx.y, col = blockIdx.x * W;
    const unsigned rows = a.rows[which];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    wait_for_prerequisite_grid();  // partial rows complete and visible
    allow_dependent_launch();
    float* out = a.out[which];
    if (out == nullptr) return;
    const float* src = a.part[which] + col;
    float s[W] = {};
    for (unsigned p = threadIdx.x; p < rows;) {
        const unsigned end = min(rows, p + kRun * kItemThreads);
        float run[W] = {};
#pragma unroll 4
        for (; p < end; p = next_item(p)) Columns<W>::add(run, *reinterpret_cast<const V*>(src + p * a.stride));
#pragma unroll
        for (int i = 0; i < W; ++i) s[i] += run[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = group_allreduce<32>(s[i]);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < W; ++i) part[warp][i] = s[i];
    }
    __syncthreads();
    if (threadIdx.x < W && RMSN_OK(span_in(out + col + threadIdx.x, 4, out, static_cast<int64_t>(a.n) * 4), a.status)) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kItemThreads / 32; ++w) t += part[w][threadIdx.x];
        out[col + threadIdx.x] = t;
    }
}

}  // namespace

cudaError_t pair_sum_launch(const PairSum& a, cudaStream_t s) {
    auto fits = [&](int w) {
        if (a.n % w || a.stride % w) return false;
        for (const float* p : a.part)
            if (reinterpret_cast<uintptr_t>(p) % (4 * w)) return false;
        return true;
    };
    const int w = fits(4) ? 4 : fits(2) ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n / w), 2);
    cfg.blockDim = dim3(kItemThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_allowed();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (w == 4) return cudaLaunchKernelEx(&cfg, pair_sum_kernel<4>, a);
    if (w == 2) return cudaLaunchKernelEx(&cfg, pair_sum_kernel<2>, a);
    return cudaLaunchKernelEx(&cfg, pair_sum_kernel<1>, a);
}

}  // namespace rmsn
