// Group norm with an activation, channels last, for any channel count and
// alignment: two kernels and, in the backward, a column sum.
//   statistics   chunks of a (sample, group) slab: each block takes the mean
//                of its chunk and then the squares about that mean (a second
//                read that L1 and L2 serve), so a mean far from zero costs no
//                digits; chunks are combined by sum n_k m_k and
//                sum M2_k + n_k (m_k - mean)^2
//   apply        y = act(xhat w + b)
//   backward     per-channel sums of dz and dz xhat over chunks of positions,
//                then dx = rstd (dz w - A - xhat B); the channel sums of all
//                chunks add up to db and dw
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
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) s += to_f32(x[i / D * a.C + i % D]);
    const float mean = n > 0 ? block_sum(s, scratch) / static_cast<float>(n) : 0.f;
    float m2 = 0.f;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const float d = to_f32(x[i / D * a.C + i % D]) - mean;
        m2 = fmaf(d, d, m2);
    }
    m2 = block_sum(m2, scratch);
    if (threadIdx.x == 0) parts[blockIdx.x] = make_float2(mean, m2);
    allow_dependent_launch();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gn_scalar_fwd_kernel(const __grid_constant__ GroupNormArgs a,
                                                                 const float2* parts, int chunks) {
    const Chunk c = chunk_of(a, chunks);
    const int D = a.C / a.G;
    wait_for_prerequisite_grid();  // the statistics are complete
    const float2* mine = parts + (c.b * a.G + c.g) * chunks;
    float sum = 0.f;
    for (int k = 0; k < chunks; ++k)
        sum = fmaf(mine[k].x, static_cast<float>((a.S * (k + 1) / chunks - a.S * k / chunks) * D), sum);
    const float count = static_cast<float>(a.S * D);
    const float mean = sum / count;
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
    float p = 0.f, q = 0.f;
    if (ch < a.C) {
        const int g = ch / (a.C / a.G);
        const float mean = a.mean[b * a.G + g], rstd = a.rstd[b * a.G + g];
        for (int64_t s = a.S * k / chunks + ry; s < s1; s += 8) {
            float xhat;
            const float dz = dz_at<T>(a, (b * a.S + s) * a.C + ch, ch, mean, rstd, xhat);
            p += dz;
            q = fmaf(dz, xhat, q);
        }
    }
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
    float p = 0.f, q = 0.f;
    for (unsigned i = threadIdx.x; i < static_cast<unsigned>(chunks * D); i = next_item(i)) {
        const int ch = c.g * D + static_cast<int>(i % D);
        const float w = a.w != nullptr ? weight_at(a.w, ch, a.w_f32, x) : 1.f;
        const float* r = parts + (c.b * chunks + i / D) * 2 * a.C + ch;
        p = fmaf(w, r[0], p);
        q = fmaf(w, r[a.C], q);
    }
    const float inv = 1.f / static_cast<float>(a.S * D);
    const float A = block_sum(p, scratch) * inv, Bq = block_sum(q, scratch) * inv;
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
