// Group norm with an activation, channels last, for any channel count and
// alignment: two kernels and, in the backward, a column sum.
//   statistics   chunks of a (sample, group) slab: each block takes the mean
//                of its chunk and then the deviations from it and their squares
//                (a second read that L1 and L2 serve); the deviations' mean puts
//                right what rounding left out of the first, so a mean far from
//                zero costs no digits; chunks are combined by the distances of
//                their means from the first one's and by
//                sum M2_k + n_k (m_k - mean)^2
//   apply        y = act(xhat w + b)
//   backward     per-channel sums of dz and dz xhat over chunks of positions,
//                then dx = rstd (dz w - A - xhat B); the channel sums of all
//                chunks add up to db and dw
// A thread adds in runs of 64, and the runs: a chain of all its values would lose
// digits where their number is large and they have one sign (12 million values that
// differ little: the mean was 115 roundings off).
// The path of shapes that 16-byte vectors do not fit: element by element.
#include <algorithm>

#include "group_norm.cuh"
#include "ops.h"
#include "group_norm.h"

namespace rmsn {
namespace {

constexpr int kThreads = kItemThreads;

// Sum over the block, the same bits in every thread.
__device__ __forceinline__ float block_sum(float v, float* scratch) {
    v = group_allreduce<32>(v);
    __syncthreads();  // the scratch's last readers are done
    if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += scratch[i];
    return s;
}

// term(i, sums) for i = first, first + step, ... below n: adds to N sums, which are
// those of runs of kRun terms; `total` is the sum of the runs.
constexpr int kRun = 64;
template <int N, typename Term>
__device__ __forceinline__ void sum_in_runs(float (&total)[N], int64_t first, int64_t n, int step, Term term) {
#pragma unroll
    for (float& t : total) t = 0.f;
    for (int64_t i = first; i < n;) {
        const int64_t end = min(n, i + static_cast<int64_t>(kRun) * step);
        float run[N] = {};
        for (; i < end; i += step) term(i, run);
#pragma unroll
        for (int k = 0; k < N; ++k) total[k] += run[k];
    }
}

template <typename T>
__device__ __forceinline__ float weight_at(const void* w, int c, int w_f32, const T*) {
    return w_f32 ? static_cast<const float*>(w)[c] : to_f32(static_cast<const T*>(w)[c]);
}

struct Chunk {
    int64_t b, s0, s1;
    int g, k;
};
__device__ __forceinline__ Chunk chunk_of(const GroupNormArgs& a, int chunks) {
    Chunk c;
    int64_t i = blockIdx.x;
    c.k = static_cast<int>(i % chunks);
    i /= chunks;
    c.g = static_cast<int>(i % a.G);
    c.b = i / a.G;
    c.s0 = a.S * c.k / chunks;
    c.s1 = a.S * (c.k + 1) / chunks;
    return c;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_scalar_stats_kernel(const __grid_constant__ GroupNormArgs a,
                                                                   float2* parts, int chunks) {
    __shared__ float scratch[kThreads / 32];
    const Chunk c = chunk_of(a, chunks);
    const int D = a.C / a.G;
    const T* x = static_cast<const T*>(a.x) + (c.b * a.S + c.s0) * a.C + c.g * D;
    const int64_t n = (c.s1 - c.s0) * D;
    wait_for_prerequisite_grid();
    auto value = [&](int64_t i) { return to_f32(x[i / D * a.C + i % D]); };
    const float count = fmaxf(static_cast<float>(n), 1.f);
    float s[1], t[2];
    sum_in_runs(s, threadIdx.x, n, kThreads, [&](int64_t i, float (&r)[1]) { r[0] += value(i); });
    const float near = block_sum(s[0], scratch) / count;
    sum_in_runs(t, threadIdx.x, n, kThreads, [&](int64_t i, float (&r)[2]) {
        const float d = value(i) - near;
        r[0] += d;
        r[1] = fmaf(d, d, r[1]);
    });
    const float off = block_sum(t[0], scratch), squares = block_sum(t[1], scratch), shift = off / count;
    if (threadIdx.x == 0) parts[blockIdx.x] = make_float2(near + shift, fmaxf(fmaf(-off, shift, squares), 0.f));
    allow_dependent_launch();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_scalar_fwd_kernel(const __grid_constant__ GroupNormArgs a,
                                                                 const float2* parts, int chunks) {
    const Chunk c = chunk_of(a, chunks);
    const int D = a.C / a.G;
    wait_for_prerequisite_grid();  // the statistics are complete
    const float2* mine = parts + (c.b * a.G + c.g) * chunks;
    const float first = mine[0].x;
    float sum = 0.f;
    for (int k = 1; k < chunks; ++k)
        sum = fmaf(mine[k].x - first, static_cast<float>((a.S * (k + 1) / chunks - a.S * k / chunks) * D), sum);
    const float count = static_cast<float>(a.S * D);
    const float mean = first + sum / count;
    float m2 = 0.f;
    for (int k = 0; k < chunks; ++k) {
        const float d = mine[k].x - mean;
        m2 += fmaf(d * d, static_cast<float>((a.S * (k + 1) / chunks - a.S * k / chunks) * D), mine[k].y);
    }
    const float rstd = rsqrtf(m2 / count + a.eps);
    if (c.k == 0 && threadIdx.x == 0) {
        a.mean[c.b * a.G + c.g] = mean;
        a.rstd[c.b * a.G + c.g] = rstd;
    }
    const int64_t base = (c.b * a.S + c.s0) * a.C + c.g * D;
    const T* x = static_cast<const T*>(a.x) + base;
    T* y = static_cast<T*>(a.out) + base;
    const int64_t n = (c.s1 - c.s0) * D;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int64_t at = i / D * a.C + i % D;
        const int ch = c.g * D + static_cast<int>(i % D);
        float z = (to_f32(x[at]) - mean) * rstd;
        if (a.w != nullptr)
            z = fmaf(z, weight_at(a.w, ch, a.w_f32, x), weight_at(a.b, ch, a.w_f32, x));
        const float v = act_value(z, a.act);
        if (RMSN_OK(span_in(y + at, sizeof(T), a.out, a.B * a.S * a.C * static_cast<int64_t>(sizeof(T))),
                    a.status))
            store_f32(y + at, v);
    }
    allow_dependent_launch();
}

// dz of one element
template <typename T>
__device__ __forceinline__ float dz_at(const GroupNormArgs& a, int64_t at, int ch, float mean,
                                       float rstd, float& xhat) {
    const T* x = static_cast<const T*>(a.x);
    xhat = (to_f32(x[at]) - mean) * rstd;
    float z = xhat;
    if (a.w != nullptr) z = fmaf(xhat, weight_at(a.w, ch, a.w_f32, x), weight_at(a.b, ch, a.w_f32, x));
    return to_f32(static_cast<const T*>(a.dy)[at]) * act_slope(z, a.act);
}

// Block (32 channels, 8 rows of threads) of (sample, chunk): the chunk's sums
// of dz (columns 0..C-1 of the partial row) and of dz xhat (C..2C-1).
template <typename T>
__global__ void __launch_bounds__(kThreads) gn_scalar_sums_kernel(const __grid_constant__ GroupNormArgs a,
                                                                  float* parts, int chunks) {
    __shared__ float sp[8][33], sq[8][33];
    const int cx = threadIdx.x % 32, ry = threadIdx.x / 32;
    const int ctiles = channel_tiles(a.C);
    const int64_t row = blockIdx.x / ctiles;  // sample * chunks + chunk
    const int ch = static_cast<int>(blockIdx.x % ctiles) * 32 + cx;
    const int64_t b = row / chunks, k = row % chunks;
    const int64_t s1 = a.S * (k + 1) / chunks;
    wait_for_prerequisite_grid();
    float t[2] = {};
    if (ch < a.C) {
        const int g = ch / (a.C / a.G);
        const float mean = a.mean[b * a.G + g], rstd = a.rstd[b * a.G + g];
        sum_in_runs(t, a.S * k / chunks + ry, s1, 8, [&](int64_t s, float (&r)[2]) {
            float xhat;
            const float dz = dz_at<T>(a, (b * a.S + s) * a.C + ch, ch, mean, rstd, xhat);
            r[0] += dz;
            r[1] = fmaf(dz, xhat, r[1]);
        });
    }
    float p = t[0], q = t[1];
    sp[ry][cx] = p;
    sq[ry][cx] = q;
    __syncthreads();
    if (ry == 0 && ch < a.C) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            p += sp[i][cx];
            q += sq[i][cx];
        }
        parts[row * 2 * a.C + ch] = p;
        parts[row * 2 * a.C + a.C + ch] = q;
    }
    allow_dependent_launch();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_scalar_bwd_kernel(const __grid_constant__ GroupNormArgs a,
                                                                 const float* parts, int chunks) {
    __shared__ float scratch[kThreads / 32];
    const Chunk c = chunk_of(a, chunks);
    const int D = a.C / a.G;
    const T* x = static_cast<const T*>(a.x);
    T* dx = static_cast<T*>(a.out);
    wait_for_prerequisite_grid();  // the channel sums are complete
    float t[2];
    sum_in_runs(t, threadIdx.x, static_cast<int64_t>(chunks) * D, kThreads, [&](int64_t i, float (&r)[2]) {
        const unsigned at = static_cast<unsigned>(i);  // below 2^31
        const int ch = c.g * D + static_cast<int>(at % D);
        const float w = a.w != nullptr ? weight_at(a.w, ch, a.w_f32, x) : 1.f;
        const float* row = parts + (c.b * chunks + at / D) * 2 * a.C + ch;
        r[0] = fmaf(w, row[0], r[0]);
        r[1] = fmaf(w, row[a.C], r[1]);
    });
    const float inv = 1.f / static_cast<float>(a.S * D);
    const float A = block_sum(t[0], scratch) * inv, Bq = block_sum(t[1], scratch) * inv;
    const float mean = a.mean[c.b * a.G + c.g], rstd = a.rstd[c.b * a.G + c.g];
    const int64_t base = (c.b * a.S + c.s0) * a.C + c.g * D;
    const int64_t n = (c.s1 - c.s0) * D;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const int64_t at = base + i / D * a.C + i % D;
        const int ch = c.g * D + static_cast<int>(i % D);
        float xhat;
        const float dz = dz_at<T>(a, at, ch, mean, rstd, xhat);
        const float w = a.w != nullptr ? weight_at(a.w, ch, a.w_f32, x) : 1.f;
        const float v = rstd * (dz * w - A - xhat * Bq);
        if (RMSN_OK(span_in(dx + at, sizeof(T), a.out, a.B * a.S * a.C * static_cast<int64_t>(sizeof(T))),
                    a.status))
            store_f32(dx + at, v);
    }
    allow_dependent_launch();
}

// Chunks of a sample: blocks of about 64 positions, at most 64 of them.
int scalar_chunks(const GroupNormArgs& a) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, a.S / 64)));
}

template <typename T>
cudaError_t launch_typed(bool bwd, const GroupNormArgs& a, void* ws, cudaStream_t s) {
    const int chunks = scalar_chunks(a);
    const int64_t slabs = a.B * a.G * chunks, rows = a.B * chunks, ctiles = channel_tiles(a.C);
    if (!bwd) {
        float2* parts = static_cast<float2*>(ws);
        cudaError_t err = launch_pdl(&gn_scalar_stats_kernel<T>, static_cast<int>(slabs), kThreads,
                                     0, 1, s, a, parts, chunks);
        if (err != cudaSuccess) return err;
        return launch_pdl(&gn_scalar_fwd_kernel<T>, static_cast<int>(slabs), kThreads, 0, 1, s, a,
                          static_cast<const float2*>(parts), chunks);
    }
    float* parts = static_cast<float*>(ws);
    cudaError_t err = launch_pdl(&gn_scalar_sums_kernel<T>, static_cast<int>(rows * ctiles), kThreads,
                                 0, 1, s, a, parts, chunks);
    if (err != cudaSuccess) return err;
    err = launch_pdl(&gn_scalar_bwd_kernel<T>, static_cast<int>(slabs), kThreads, 0, 1, s, a,
                     static_cast<const float*>(parts), chunks);
    if (err != cudaSuccess || a.dw == nullptr) return err;
    PairSum p{};
    p.part[0] = parts + a.C;
    p.part[1] = parts;
    p.out[0] = a.dw;
    p.out[1] = a.db;
    p.rows[0] = p.rows[1] = static_cast<int>(rows);
    p.n = a.C;
    p.stride = 2 * static_cast<int64_t>(a.C);
    p.status = a.status;
    return pair_sum_launch(p, s);
}

}  // namespace

bool gn_scalar_fits(const GroupNormArgs& a) {
    const int64_t wide = std::max<int64_t>(a.G, channel_tiles(a.C));  // blocks of a chunk
    return a.B <= INT32_MAX / (wide * scalar_chunks(a));
}

size_t gn_scalar_workspace(bool bwd, const GroupNormArgs& a) {
    const size_t rows = static_cast<size_t>(a.B) * scalar_chunks(a);
    return bwd ? rows * 2 * a.C * 4 : rows * a.G * 8;
}

cudaError_t gn_scalar_launch(int dtype, bool bwd, const GroupNormArgs& a, void* ws, cudaStream_t s) {
    switch (dtype) {
        case RMSNORM_F32: return launch_typed<float>(bwd, a, ws, s);
        case RMSNORM_BF16:
        case RMSNORM_BF16_W_F32: return launch_typed<__nv_bfloat16>(bwd, a, ws, s);
        default: return launch_typed<__half>(bwd, a, ws, s);
    }
}

}  // namespace rmsn
