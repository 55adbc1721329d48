// Group norm with an activation, channels last, by 16-byte vectors.
//
// A slab is one sample's positions by a run of whole groups of channels. A
// block takes a contiguous range of its positions; each thread owns one
// 16-byte vector of channels and strides over positions, so its channels'
// constants and sums stay in registers, whatever the group width (a vector may
// span groups: sums are kept per channel and joined per group afterwards).
//
// Forward statistics. A thread sums d = x - p and d^2 about its own first
// value p of each channel, which turns into (count, mean, M2); these are joined
// over the block, the cluster and the slab by
//   mean = sum n_i m_i / n,   M2 = sum M2_i + n_i (m_i - mean)^2
// so neither a mean far from zero nor one wild first value costs digits (a wild
// p spoils only the few hundred values of one thread, and then only relative to
// its own square, which is part of M2).
// Backward sums. Per channel P = sum dz, Q = sum dz xhat: they give the slab's
// means (sum_c w P, sum_c w Q) and, added over samples, db and dw.
//
// Bound by DRAM: x once in and y once out (x, dy, dx). Between the sums and the
// second pass the slab has to be kept near. Two families:
//   resident  the slab fits the shared memory of a cluster of at most 16
//             blocks: one kernel, each thread keeps what it read in its own
//             shared-memory slots, the blocks' sums meet in distributed shared
//             memory. One read of x.
//   stream    larger slabs: a kernel for the sums (clusters join their blocks'
//             sums, so few partial results are written) and one that applies
//             them, in the opposite order so that it starts with what L2 still
//             holds; samples go in batches that L2 holds.
#include <algorithm>
#include <mutex>

#include "group_norm.cuh"
#include "group_norm.h"

namespace rmsn {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxSmem = 227 * 1024;

struct SlabArgs {
    GroupNormArgs a;
    int nvec;      // 16-byte vectors of a slab's row
    int lanes;     // positions a block takes at once
    int splits;    // slabs of a sample (runs of channels)
    int cw, gw;    // channels and groups of a slab
    int D;         // channels of a group
    int cluster;   // blocks that join their sums
    int chunks;    // clusters of a slab
    int64_t sample0;
    float2* stats; // stream: [slab][chunk][gw], (mean, M2) or (sum w P, sum w Q)
    float* rows;   // backward: partial rows [sample * chunks + chunk][2 C] (Q, then P)
};

// Where a block works.
struct Place {
    int64_t sample;
    int split, chunk, rank, slab;
    int64_t r0, r1;  // its positions
};
__device__ __forceinline__ int64_t part_begin(int64_t S, int64_t p, int64_t parts) {
    return S * p / parts;  // S * parts < 2^31 * 2^12
}
__device__ __forceinline__ Place place_of(const SlabArgs& g) {
    Place p;
    const int cl = static_cast<int>(blockIdx.x) / g.cluster;
    p.rank = static_cast<int>(blockIdx.x) - cl * g.cluster;
    p.slab = cl / g.chunks;
    p.chunk = cl - p.slab * g.chunks;
    const int s = p.slab / g.splits;
    p.split = p.slab - s * g.splits;
    p.sample = g.sample0 + s;
    const int64_t parts = static_cast<int64_t>(g.chunks) * g.cluster;
    const int64_t part = static_cast<int64_t>(p.chunk) * g.cluster + p.rank;
    p.r0 = part_begin(g.a.S, part, parts);
    p.r1 = part_begin(g.a.S, part + 1, parts);
    return p;
}

// i / d for 0 <= i < 2^20 and d >= 1, by the reciprocal in fp32: (i + 1/2) / d
// is at least 1/(2d) from an integer, more than its rounding.
__device__ __forceinline__ int quotient(int i, float inv_d) {
    return static_cast<int>((static_cast<float>(i) + 0.5f) * inv_d);
}

__device__ __forceinline__ float2 ld_cluster_f32x2(const float2* local, uint32_t rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(cluster_map(local, rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(const float* local, uint32_t rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                 : "=f"(v)
                 : "r"(cluster_map(local, rank))
                 : "memory");
    return v;
}

// A thread's channels: scale and offset of the affine map.
template <typename T>
__device__ __forceinline__ void load_channels(const SlabArgs& g, const void* p, int64_t c, float one,
                                              float2 (&f)[Pack<T>::PAIRS]) {
    constexpr int PAIRS = Pack<T>::PAIRS;
    if (p == nullptr) {
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) f[e] = f2_splat(one);
    } else if (g.a.w_f32) {
        // weights need only their own alignment
        const float* w = static_cast<const float*>(p) + c;
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) f[e] = make_float2(w[2 * e], w[2 * e + 1]);
    } else {
        const T* w = static_cast<const T*>(p) + c;
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) f[e] = make_float2(to_f32(w[2 * e]), to_f32(w[2 * e + 1]));
    }
}

// Constants of a thread's channels from per-group values in shared or global
// memory: v[group of the channel].
template <typename T, typename F>
__device__ __forceinline__ void per_channel(const SlabArgs& g, int c, float inv_d, F value,
                                            float2 (&f)[Pack<T>::PAIRS]) {
#pragma unroll
    for (int e = 0; e < Pack<T>::PAIRS; ++e)
        f[e] = make_float2(value(quotient(c + 2 * e, inv_d)), value(quotient(c + 2 * e + 1, inv_d)));
}

__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    return __fadd2_rn(a, make_float2(-b.x, -b.y));
}

__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// A read of memory that this thread may overwrite later in the kernel.
__device__ __forceinline__ uint4 ld_global_16_own(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// 16-bit outputs take the fast exponential and reciprocal (off by some 2^-21,
// far inside half a step of 2^-12); fp32 outputs the accurate ones.
template <typename T>
__device__ __forceinline__ float act_of(float z, int act) {
    if constexpr (sizeof(T) == 2)
        if (act == RMSNORM_ACT_SILU) return z * rcp_fast(1.f + __expf(-z));
    return act_value(z, act);
}
template <typename T>
__device__ __forceinline__ float slope_of(float z, int act) {
    if constexpr (sizeof(T) == 2) {
        if (act == RMSNORM_ACT_SILU) {
            const float s = rcp_fast(1.f + __expf(-z));
            return s * fmaf(z, 1.f - s, 1.f);
        }
    }
    return act_slope(z, act);
}

// The constants and sums of a thread's channels, and the two passes' steps.
template <typename T, bool BWD>
struct Columns;

template <typename T>
struct Columns<T, false> {
    static constexpr int PAIRS = Pack<T>::PAIRS;
    float2 pivot[PAIRS], s1[PAIRS], s2[PAIRS];
    float2 mean[PAIRS], scale[PAIRS], shift[PAIRS];

    __device__ __forceinline__ void start(const uint4& first) {
        Pack<T>::unpack2(first, pivot);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) s1[e] = s2[e] = make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ void add(const uint4& v) {
        float2 f[PAIRS];
        Pack<T>::unpack2(v, f);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            const float2 d = sub2(f[e], pivot[e]);
            s1[e] = __fadd2_rn(s1[e], d);
            s2[e] = __ffma2_rn(d, d, s2[e]);
        }
    }
    // y = act((x - mean) * scale + shift), rounded once
    __device__ __forceinline__ uint4 apply(const uint4& v, int act) const {
        float2 f[PAIRS];
        Pack<T>::unpack2(v, f);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            f[e] = __ffma2_rn(sub2(f[e], mean[e]), scale[e], shift[e]);
            if (act != RMSNORM_ACT_NONE) {
                f[e].x = act_of<T>(f[e].x, act);
                f[e].y = act_of<T>(f[e].y, act);
            }
        }
        return Pack<T>::pack2(f);
    }
};

template <typename T>
struct Columns<T, true> {
    static constexpr int PAIRS = Pack<T>::PAIRS;
    float2 mean[PAIRS], rstd[PAIRS], w[PAIRS], b[PAIRS];
    float2 p[PAIRS], q[PAIRS];
    float2 A[PAIRS], B[PAIRS];  // the slab's means, times rstd

    __device__ __forceinline__ void dz(const uint4& x, const uint4& dy, int act,
                                       float2 (&xhat)[PAIRS], float2 (&d)[PAIRS]) const {
        Pack<T>::unpack2(x, xhat);
        Pack<T>::unpack2(dy, d);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            xhat[e] = __fmul2_rn(sub2(xhat[e], mean[e]), rstd[e]);
            if (act != RMSNORM_ACT_NONE) {
                const float2 z = __ffma2_rn(xhat[e], w[e], b[e]);
                d[e].x *= slope_of<T>(z.x, act);
                d[e].y *= slope_of<T>(z.y, act);
            }
        }
    }
    __device__ __forceinline__ void add(const uint4& x, const uint4& dy, int act) {
        float2 xhat[PAIRS], d[PAIRS];
        dz(x, dy, act, xhat, d);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            p[e] = __fadd2_rn(p[e], d[e]);
            q[e] = __ffma2_rn(d[e], xhat[e], q[e]);
        }
    }
    // dx = rstd (dz w - mean(dz w) - xhat mean(dz w xhat)), rounded once
    __device__ __forceinline__ uint4 apply(const uint4& x, const uint4& dy, int act) const {
        float2 xhat[PAIRS], d[PAIRS];
        dz(x, dy, act, xhat, d);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            const float2 g = __fmul2_rn(d[e], w[e]);
            const float2 t = __ffma2_rn(xhat[e], make_float2(-B[e].x, -B[e].y), sub2(g, A[e]));
            d[e] = __fmul2_rn(t, rstd[e]);
        }
        return Pack<T>::pack2(d);
    }
};

// Shared memory besides the resident slab: the threads' sums [2][lanes][cw]
// and two values a group, twice (the block's and the slab's).
__host__ __device__ __forceinline__ int sums_floats(int lanes, int cw) { return 2 * lanes * cw; }
int fixed_smem(int lanes, int cw, int gw) {
    return (sums_floats(lanes, cw) + 4 * gw) * 4;
}

// Joins the block's sums: (mean, M2) per group into `mine`.
template <typename T>
__device__ __forceinline__ void join_block(const SlabArgs& g, const Columns<T, false>& col,
                                           float* sums, float2* mine, int64_t rows, int lane,
                                           int vec, float inv_d) {
    constexpr int PAIRS = Pack<T>::PAIRS, VEC = Pack<T>::VEC;
    float* means = sums;
    float* m2s = sums + g.lanes * g.cw;
    if (lane < g.lanes) {
        const int n = static_cast<int>(rows > lane ? (rows - lane + g.lanes - 1) / g.lanes : 0);
        const float inv_n = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            const int at = lane * g.cw + vec * VEC + 2 * e;
            // the mean's distance from the pivot, and the squares about the mean
            const float2 d = n > 0 ? __fmul2_rn(col.s1[e], f2_splat(inv_n)) : make_float2(0.f, 0.f);
            const float2 m2 = n > 0 ? sub2(col.s2[e], __fmul2_rn(col.s1[e], d)) : make_float2(0.f, 0.f);
            const float2 m = n > 0 ? __fadd2_rn(col.pivot[e], d) : make_float2(0.f, 0.f);
            *reinterpret_cast<float2*>(means + at) = m;
            *reinterpret_cast<float2*>(m2s + at) = m2;
        }
    }
    __syncthreads();
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, l = threadIdx.x % 32;
    const int entries = g.lanes * g.D;
    const float count = static_cast<float>(rows) * static_cast<float>(g.D);
    for (int k = warp; k < g.gw; k += warps) {
        float s = 0.f;
        for (int i = l; i < entries; i += 32) {
            const int r = quotient(i, inv_d);
            const int n = static_cast<int>(rows > r ? (rows - r + g.lanes - 1) / g.lanes : 0);
            s = fmaf(static_cast<float>(n), means[r * g.cw + k * g.D + (i - r * g.D)], s);
        }
        s = group_allreduce<32>(s);
        const float mean = count > 0.f ? s / count : 0.f;
        float m2 = 0.f;
        for (int i = l; i < entries; i += 32) {
            const int r = quotient(i, inv_d);
            const int n = static_cast<int>(rows > r ? (rows - r + g.lanes - 1) / g.lanes : 0);
            const int at = r * g.cw + k * g.D + (i - r * g.D);
            const float d = means[at] - mean;
            m2 += n > 0 ? fmaf(static_cast<float>(n) * d, d, m2s[at]) : 0.f;
        }
        m2 = group_allreduce<32>(m2);
        if (l == 0) mine[k] = make_float2(mean, m2);
    }
}

// Joins the block's sums: per channel over its lanes (in place, into the first
// lane's row of `sums`: P, and Q behind it), then (sum w P, sum w Q) per group
// into `mine`.
template <typename T>
__device__ __forceinline__ void join_block(const SlabArgs& g, const Columns<T, true>& col,
                                           float* sums, float2* mine, int lane, int vec,
                                           int64_t c0) {
    constexpr int PAIRS = Pack<T>::PAIRS, VEC = Pack<T>::VEC;
    float* ps = sums;
    float* qs = sums + g.lanes * g.cw;
    if (lane < g.lanes) {
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            const int at = lane * g.cw + vec * VEC + 2 * e;
            *reinterpret_cast<float2*>(ps + at) = col.p[e];
            *reinterpret_cast<float2*>(qs + at) = col.q[e];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * g.cw; c += blockDim.x) {
        float* at = c < g.cw ? ps + c : qs + (c - g.cw);
        float s = 0.f;
        for (int r = 0; r < g.lanes; ++r) s += at[r * g.cw];
        at[0] = s;
    }
    __syncthreads();
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, l = threadIdx.x % 32;
    for (int k = warp; k < g.gw; k += warps) {
        float sp = 0.f, sq = 0.f;
        for (int i = l; i < g.D; i += 32) {
            const int c = k * g.D + i;
            float w = 1.f;
            if (g.a.w != nullptr)
                w = g.a.w_f32 ? static_cast<const float*>(g.a.w)[c0 + c]
                              : to_f32(static_cast<const T*>(g.a.w)[c0 + c]);
            sp = fmaf(w, ps[c], sp);
            sq = fmaf(w, qs[c], sq);
        }
        sp = group_allreduce<32>(sp);
        sq = group_allreduce<32>(sq);
        if (l == 0) mine[k] = make_float2(sp, sq);
    }
}

// The statistics of (mean, M2) results with their counts, in rank order.
struct Joined {
    float mean, m2;
};
template <typename Get, typename Count>
__device__ __forceinline__ Joined join_means(int n, float total, Get get, Count count) {
    float s = 0.f;
    for (int k = 0; k < n; ++k) s = fmaf(count(k), get(k).x, s);
    const float mean = s / total;
    float m2 = 0.f;
    for (int k = 0; k < n; ++k) {
        const float2 v = get(k);
        const float d = v.x - mean;
        m2 += fmaf(count(k) * d, d, v.y);
    }
    return {mean, m2};
}

// The sums of a slab (stream), or both passes over it (resident).
template <typename T, bool BWD, bool RESIDENT>
__global__ void __launch_bounds__(kMaxThreads) gn_slab_kernel(const __grid_constant__ SlabArgs g) {
    constexpr int VEC = Pack<T>::VEC, PAIRS = Pack<T>::PAIRS, U = BWD ? 4 : 8;
    const Place at = place_of(g);
    const int lane = static_cast<int>(threadIdx.x) / g.nvec;
    const int vec = static_cast<int>(threadIdx.x) - lane * g.nvec;
    const bool active = lane < g.lanes;
    const float inv_d = 1.f / static_cast<float>(g.D);
    float* sums = reinterpret_cast<float*>(rmsn_dynamic_smem);
    float2* mine = reinterpret_cast<float2*>(sums + sums_floats(g.lanes, g.cw));
    float2* slab = mine + g.gw;
    uint4* keep = reinterpret_cast<uint4*>(slab + g.gw);
    const int slots = g.lanes * g.nvec;  // a pass of the block over `lanes` positions
    const int64_t rows = at.r1 - at.r0;
    const int64_t c0 = static_cast<int64_t>(at.split) * g.cw;
    const int64_t base = (at.sample * g.a.S + at.r0) * g.a.C + c0 + static_cast<int64_t>(vec) * VEC;
    const int64_t step = static_cast<int64_t>(g.lanes) * g.a.C;
    const T* x = static_cast<const T*>(g.a.x) + base;
    [[maybe_unused]] const T* dy = BWD ? static_cast<const T*>(g.a.dy) + base : nullptr;
    const int n = active && rows > lane ? static_cast<int>((rows - lane + g.lanes - 1) / g.lanes) : 0;
    const int act = g.a.act;
    Columns<T, BWD> col;
    wait_for_prerequisite_grid();  // no global access before this

    if constexpr (BWD) {
        const float* ms = g.a.mean + at.sample * g.a.G + at.split * g.gw;
        const float* rs = g.a.rstd + at.sample * g.a.G + at.split * g.gw;
        if (active) {
            const int c = vec * VEC;
            per_channel<T>(g, c, inv_d, [&](int k) { return ms[k]; }, col.mean);
            per_channel<T>(g, c, inv_d, [&](int k) { return rs[k]; }, col.rstd);
            load_channels<T>(g, g.a.w, c0 + c, 1.f, col.w);
            load_channels<T>(g, g.a.b, c0 + c, 0.f, col.b);
        }
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) col.p[e] = col.q[e] = make_float2(0.f, 0.f);
    } else {
        col.start(n > 0 ? ld_global_16_stream(x + lane * g.a.C) : make_uint4(0, 0, 0, 0));
    }

    // first pass: U positions in flight
    {
        const T* px = x + static_cast<int64_t>(lane) * g.a.C;
        [[maybe_unused]] const T* pd = BWD ? dy + static_cast<int64_t>(lane) * g.a.C : nullptr;
        uint4* slot = keep + threadIdx.x;
        int i = 0;
        for (; i + U <= n; i += U) {
            uint4 xv[U], dv[BWD ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                xv[u] = ld_global_16_stream(px + u * step);
                if constexpr (BWD) dv[u] = ld_global_16_stream(pd + u * step);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (RESIDENT) {
                    if (RMSN_OK(smem_span_in(slot, 16), g.a.status)) slot[0] = xv[u];
                    if constexpr (BWD)
                        if (RMSN_OK(smem_span_in(slot + slots, 16), g.a.status)) slot[slots] = dv[u];
                    slot += BWD ? 2 * slots : slots;
                }
                if constexpr (BWD) col.add(xv[u], dv[u], act);
                else col.add(xv[u]);
            }
            px += U * step;
            if constexpr (BWD) pd += U * step;
        }
        for (; i < n; ++i) {
            const uint4 xv = ld_global_16_stream(px);
            uint4 dv = make_uint4(0, 0, 0, 0);
            if constexpr (BWD) dv = ld_global_16_stream(pd);
            if constexpr (RESIDENT) {
                if (RMSN_OK(smem_span_in(slot, 16), g.a.status)) slot[0] = xv;
                if constexpr (BWD)
                    if (RMSN_OK(smem_span_in(slot + slots, 16), g.a.status)) slot[slots] = dv;
                slot += BWD ? 2 * slots : slots;
            }
            if constexpr (BWD) col.add(xv, dv, act);
            else col.add(xv);
            px += step;
            if constexpr (BWD) pd += step;
        }
    }
    if constexpr (BWD) join_block<T>(g, col, sums, mine, lane, vec, c0);
    else join_block<T>(g, col, sums, mine, rows, lane, vec, inv_d);

    // the cluster's blocks meet
    __syncwarp();
    if (g.cluster > 1) cluster_sync_all();
    else __syncthreads();
    const int64_t parts = static_cast<int64_t>(g.chunks) * g.cluster;
    const int64_t part0 = static_cast<int64_t>(at.chunk) * g.cluster;
    for (int k = threadIdx.x; k < g.gw; k += blockDim.x) {
        if (!RESIDENT && at.rank != 0) break;
        float2 v = make_float2(0.f, 0.f);
        if constexpr (BWD) {
            for (int r = 0; r < g.cluster; ++r) {
                const float2 t = g.cluster > 1 ? ld_cluster_f32x2(mine + k, r) : mine[k];
                v = __fadd2_rn(v, t);
            }
        } else {
            const float total =
                static_cast<float>(part_begin(g.a.S, part0 + g.cluster, parts) -
                                   part_begin(g.a.S, part0, parts)) * static_cast<float>(g.D);
            const Joined j = join_means(
                g.cluster, total,
                [&](int r) { return g.cluster > 1 ? ld_cluster_f32x2(mine + k, r) : mine[k]; },
                [&](int r) {
                    return static_cast<float>(part_begin(g.a.S, part0 + r + 1, parts) -
                                              part_begin(g.a.S, part0 + r, parts)) *
                           static_cast<float>(g.D);
                });
            v = make_float2(j.mean, j.m2);
        }
        if constexpr (RESIDENT) {
            const float inv = 1.f / (static_cast<float>(g.a.S) * static_cast<float>(g.D));
            if constexpr (BWD) {
                slab[k] = make_float2(v.x * inv, v.y * inv);
            } else {
                v.y = rsqrtf(v.y * inv + g.a.eps);
                slab[k] = v;
                if (at.rank == 0) {
                    const int64_t o = at.sample * g.a.G + at.split * g.gw + k;
                    g.a.mean[o] = v.x;
                    g.a.rstd[o] = v.y;
                }
            }
        } else {
            g.stats[(static_cast<int64_t>(at.slab) * g.chunks + at.chunk) * g.gw + k] = v;
        }
    }
    if constexpr (BWD) {
        // each block adds its share of the cluster's channel sums
        if (g.a.dw != nullptr) {
            const int lo = static_cast<int>(static_cast<int64_t>(2 * g.cw) * at.rank / g.cluster);
            const int hi = static_cast<int>(static_cast<int64_t>(2 * g.cw) * (at.rank + 1) / g.cluster);
            for (int i = lo + threadIdx.x; i < hi; i += blockDim.x) {
                const bool q = i >= g.cw;
                const int c = q ? i - g.cw : i;
                const float* src = sums + (q ? g.lanes * g.cw : 0) + c;
                float s = 0.f;
                for (int r = 0; r < g.cluster; ++r) s += g.cluster > 1 ? ld_cluster_f32(src, r) : *src;
                float* d;
                if (g.rows == nullptr) d = (q ? g.a.dw : g.a.db) + c0 + c;
                else
                    d = g.rows + (at.sample * g.chunks + at.chunk) * 2 * g.a.C + (q ? 0 : g.a.C) + c0 + c;
                *d = s;
            }
        }
    }
    __syncwarp();
    if (g.cluster > 1) cluster_arrive_relaxed();  // this block is done reading its peers
    allow_dependent_launch();

    if constexpr (RESIDENT) {
        __syncthreads();
        if (active) {
            const int c = vec * VEC;
            if constexpr (BWD) {
                per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].x; }, col.A);
                per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].y; }, col.B);
            } else {
                float2 w[PAIRS];
                load_channels<T>(g, g.a.w, c0 + c, 1.f, w);
                load_channels<T>(g, g.a.b, c0 + c, 0.f, col.shift);
                per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].x; }, col.mean);
                per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].y; }, col.scale);
#pragma unroll
                for (int e = 0; e < PAIRS; ++e) col.scale[e] = __fmul2_rn(col.scale[e], w[e]);
            }
            T* out = static_cast<T*>(g.a.out) + base + static_cast<int64_t>(lane) * g.a.C;
            [[maybe_unused]] const int64_t bytes = g.a.B * g.a.S * g.a.C * static_cast<int64_t>(sizeof(T));
            const uint4* slot = keep + threadIdx.x;
#pragma unroll 2
            for (int i = 0; i < n; ++i) {
                uint4 v;
                if constexpr (BWD) {
                    v = col.apply(slot[0], slot[slots], act);
                    slot += 2 * slots;
                } else {
                    v = col.apply(slot[0], act);
                    slot += slots;
                }
                if (RMSN_OK(span_in(out, 16, g.a.out, bytes), g.a.status)) st_global_16(out, v);
                out += step;
            }
        }
    }
    __syncwarp();
    if (g.cluster > 1) cluster_wait();  // no block leaves while a peer reads it
}

// Stream: the second pass, over the same ranges of positions from their ends.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kMaxThreads) gn_apply_kernel(const __grid_constant__ SlabArgs g) {
    constexpr int VEC = Pack<T>::VEC, PAIRS = Pack<T>::PAIRS, U = 4;
    const Place at = place_of(g);
    const int lane = static_cast<int>(threadIdx.x) / g.nvec;
    const int vec = static_cast<int>(threadIdx.x) - lane * g.nvec;
    const bool active = lane < g.lanes;
    const float inv_d = 1.f / static_cast<float>(g.D);
    float2* slab = reinterpret_cast<float2*>(rmsn_dynamic_smem);
    const int64_t rows = at.r1 - at.r0;
    const int64_t c0 = static_cast<int64_t>(at.split) * g.cw;
    const int64_t step = static_cast<int64_t>(g.lanes) * g.a.C;
    const int n = active && rows > lane ? static_cast<int>((rows - lane + g.lanes - 1) / g.lanes) : 0;
    const int act = g.a.act;
    wait_for_prerequisite_grid();  // the partial results are complete
    {
        const int warps = blockDim.x / 32, warp = threadIdx.x / 32, l = threadIdx.x % 32;
        const float inv = 1.f / (static_cast<float>(g.a.S) * static_cast<float>(g.D));
        const float2* stats = g.stats + static_cast<int64_t>(at.slab) * g.chunks * g.gw;
        for (int k = warp; k < g.gw; k += warps) {
            float2 v = make_float2(0.f, 0.f);
            if constexpr (BWD) {
                for (int i = l; i < g.chunks; i += 32)
                    v = __fadd2_rn(v, stats[static_cast<int64_t>(i) * g.gw + k]);
                v.x = group_allreduce<32>(v.x) * inv;
                v.y = group_allreduce<32>(v.y) * inv;
            } else {
                const int64_t parts = static_cast<int64_t>(g.chunks) * g.cluster;
                auto count = [&](int i) {
                    return static_cast<float>(
                               part_begin(g.a.S, static_cast<int64_t>(i + 1) * g.cluster, parts) -
                               part_begin(g.a.S, static_cast<int64_t>(i) * g.cluster, parts)) *
                           static_cast<float>(g.D);
                };
                float s = 0.f;
                for (int i = l; i < g.chunks; i += 32)
                    s = fmaf(count(i), stats[static_cast<int64_t>(i) * g.gw + k].x, s);
                const float mean = group_allreduce<32>(s) * inv;
                float m2 = 0.f;
                for (int i = l; i < g.chunks; i += 32) {
                    const float2 t = stats[static_cast<int64_t>(i) * g.gw + k];
                    const float d = t.x - mean;
                    m2 += fmaf(count(i) * d, d, t.y);
                }
                v = make_float2(mean, rsqrtf(group_allreduce<32>(m2) * inv + g.a.eps));
                if (at.chunk == 0 && at.rank == 0 && l == 0) {
                    const int64_t o = at.sample * g.a.G + at.split * g.gw + k;
                    g.a.mean[o] = v.x;
                    g.a.rstd[o] = v.y;
                }
            }
            if (l == 0) slab[k] = v;
        }
    }
    __syncthreads();
    allow_dependent_launch();
    if (n == 0) return;
    Columns<T, BWD> col;
    const int c = vec * VEC;
    if constexpr (BWD) {
        const float* ms = g.a.mean + at.sample * g.a.G + at.split * g.gw;
        const float* rs = g.a.rstd + at.sample * g.a.G + at.split * g.gw;
        per_channel<T>(g, c, inv_d, [&](int k) { return ms[k]; }, col.mean);
        per_channel<T>(g, c, inv_d, [&](int k) { return rs[k]; }, col.rstd);
        load_channels<T>(g, g.a.w, c0 + c, 1.f, col.w);
        load_channels<T>(g, g.a.b, c0 + c, 0.f, col.b);
        per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].x; }, col.A);
        per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].y; }, col.B);
    } else {
        float2 w[PAIRS];
        load_channels<T>(g, g.a.w, c0 + c, 1.f, w);
        load_channels<T>(g, g.a.b, c0 + c, 0.f, col.shift);
        per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].x; }, col.mean);
        per_channel<T>(g, c, inv_d, [&](int k) { return slab[k].y; }, col.scale);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) col.scale[e] = __fmul2_rn(col.scale[e], w[e]);
    }
    const int64_t last = (at.sample * g.a.S + at.r0 + lane) * g.a.C + c0 + c +
                         static_cast<int64_t>(n - 1) * step;
    const T* x = static_cast<const T*>(g.a.x) + last;
    // dx may be the dy buffer: each element is read before this thread writes it
    const T* dy = BWD ? static_cast<const T*>(g.a.dy) + last : nullptr;
    T* out = static_cast<T*>(g.a.out) + last;
    [[maybe_unused]] const int64_t bytes = g.a.B * g.a.S * g.a.C * static_cast<int64_t>(sizeof(T));
    int i = 0;
    for (; i + U <= n; i += U) {
        uint4 xv[U], dv[BWD ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xv[u] = ld_global_16_stream(x - u * step);
            if constexpr (BWD) dv[u] = ld_global_16_own(dy - u * step);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint4 v;
            if constexpr (BWD) v = col.apply(xv[u], dv[u], act);
            else v = col.apply(xv[u], act);
            if (RMSN_OK(span_in(out - u * step, 16, g.a.out, bytes), g.a.status))
                st_global_16(out - u * step, v);
        }
        x -= U * step;
        if constexpr (BWD) dy -= U * step;
        out -= U * step;
    }
    for (; i < n; ++i) {
        uint4 v;
        if constexpr (BWD) v = col.apply(ld_global_16_stream(x), ld_global_16_own(dy), act);
        else v = col.apply(ld_global_16_stream(x), act);
        if (RMSN_OK(span_in(out, 16, g.a.out, bytes), g.a.status)) st_global_16(out, v);
        x -= step;
        if constexpr (BWD) dy -= step;
        out -= step;
    }
}

// ---------------------------------------------------------------- host side
using SlabFn = void (*)(const SlabArgs);
enum Kind { kResident, kSums, kApply };

template <typename T, bool BWD>
SlabFn kernel_of(Kind k) {
    if (k == kResident) return &gn_slab_kernel<T, BWD, true>;
    if (k == kSums) return &gn_slab_kernel<T, BWD, false>;
    return &gn_apply_kernel<T, BWD>;
}
SlabFn kernel_for(int dtype, bool bwd, Kind k) {
    switch (dtype) {
        case RMSNORM_F32: return bwd ? kernel_of<float, true>(k) : kernel_of<float, false>(k);
        case RMSNORM_BF16:
        case RMSNORM_BF16_W_F32:
            return bwd ? kernel_of<__nv_bfloat16, true>(k) : kernel_of<__nv_bfloat16, false>(k);
        default: return bwd ? kernel_of<__half, true>(k) : kernel_of<__half, false>(k);
    }
}

// Clusters of a kernel that the device runs at once (0: it refuses the size);
// the answer is kept, so that a shape's grid is the same on every call.
struct OccEntry {
    int device;
    SlabFn fn;
    int threads, smem, cluster, clusters;
};
std::mutex g_occ_mu;
OccEntry g_occ[256];
int g_occ_n = 0;

int resident_clusters(const DeviceInfo& dev, SlabFn fn, int threads, int smem, int cluster) {
    std::lock_guard<std::mutex> lk(g_occ_mu);
    for (int i = 0; i < g_occ_n; ++i) {
        const OccEntry& e = g_occ[i];
        if (e.device == dev.device && e.fn == fn && e.threads == threads && e.smem == smem &&
            e.cluster == cluster)
            return e.clusters;
    }
    const void* f = reinterpret_cast<const void*>(fn);
    int n = 0;
    cudaError_t err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (err == cudaSuccess && cluster > 8)
        err = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cluster * dev.sm_count));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        err = cudaOccupancyMaxActiveClusters(&n, f, &cfg);
    }
    if (err != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    if (g_occ_n < 256) g_occ[g_occ_n++] = {dev.device, fn, threads, smem, cluster, n};
    return n;
}

struct Plan {
    bool ok = false, resident = false;
    int splits = 1, cluster = 1, chunks = 1, lanes = 1, threads = 32, smem = 0, nvec = 0;
    int64_t samples = 1;  // stream: samples of a batch
};

void geometry(Plan* p, int nvec) {
    p->nvec = nvec;
    p->lanes = std::max(1, kMaxThreads / nvec);
    p->threads = round_up(p->lanes * nvec, 32);
}

// Bytes of x (and dy) that a batch of the stream family may hold: what L2
// keeps besides the output written meanwhile.
constexpr int64_t kBatchBytes = 64ll << 20;

Plan make_plan(const DeviceInfo& dev, int dtype, bool bwd, const GroupNormArgs& a) {
    Plan best;
    const int size = dtype_size(dtype), tensors = bwd ? 2 : 1;
    const int64_t row_bytes = static_cast<int64_t>(a.C) * size;
    double best_cost = 0;
    // resident: microseconds a wave of blocks needs, by the slice a block keeps
    // (44 KB/us is an SM's share of the DRAM rate, in and out), the blocks'
    // meeting, and a fixed start; rows are split no finer than 128 bytes
    for (int splits = 1; splits <= a.G; splits *= 2) {
        if (a.G % splits) break;
        const int64_t wide = row_bytes / splits;
        if (row_bytes % splits || wide % 16 || (splits > 1 && wide < 128)) break;
        if (wide / 16 > kMaxThreads) continue;
        Plan p;
        p.splits = splits;
        geometry(&p, static_cast<int>(wide / 16));
        const int fixed = round_up(fixed_smem(p.lanes, a.C / splits, a.G / splits), 16);
        for (int cluster = 1; cluster <= 16; cluster *= 2) {
            const int64_t rows = cdiv(a.S, cluster);
            const int64_t slice = cdiv(rows, p.lanes) * p.lanes * wide * tensors;
            if (fixed + slice > kMaxSmem) continue;
            if (cluster > 1 && rows < p.lanes) break;
            const int64_t blocks = a.B * splits * cluster;
            if (blocks > INT32_MAX) break;
            const double waves = static_cast<double>(cdiv(blocks, dev.sm_count));
            const double cost = waves * (1.5 + (cluster > 8 ? 1.5 : cluster > 1 ? 1.0 : 0.0) +
                                         slice * (bwd ? 1.5 : 2.0) / 44e3);
            if (best.ok && cost >= best_cost) continue;
            const int smem = static_cast<int>(fixed + slice);
            if (resident_clusters(dev, kernel_for(dtype, bwd, kResident), p.threads, kMaxSmem, cluster) < 1)
                continue;
            p.ok = p.resident = true;
            p.cluster = cluster;
            p.smem = smem;
            best = p;
            best_cost = cost;
        }
    }
    // stream: all SMs on two launches
    Plan p;
    while (p.splits <= a.G && row_bytes / p.splits / 16 > kMaxThreads) p.splits *= 2;
    if (p.splits > a.G || a.G % p.splits || row_bytes % (16ll * p.splits)) return best;
    geometry(&p, static_cast<int>(row_bytes / p.splits / 16));
    p.smem = fixed_smem(p.lanes, a.C / p.splits, a.G / p.splits);
    if (p.smem > kMaxSmem) return best;
    const double total = static_cast<double>(a.B) * a.S * row_bytes * tensors;
    const double cost = 6.0 + total * (bwd ? 2.0 : 2.5) / (44e3 * dev.sm_count);
    if (best.ok && best_cost <= cost) return best;
    p.cluster = 8;
    int clusters = resident_clusters(dev, kernel_for(dtype, bwd, kSums), p.threads, p.smem, p.cluster);
    if (clusters < 1) {
        p.cluster = 1;
        clusters = resident_clusters(dev, kernel_for(dtype, bwd, kSums), p.threads, p.smem, 1);
        if (clusters < 1) return best;
    }
    p.samples = std::max<int64_t>(
        1, std::min<int64_t>(a.B, kBatchBytes / (a.S * row_bytes * tensors)));
    const int64_t slabs = p.samples * p.splits;
    p.chunks = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(clusters / slabs, a.S / (p.cluster * p.lanes))));
    if (slabs * p.chunks * p.cluster > INT32_MAX || a.B * p.chunks > INT32_MAX) return best;
    p.ok = true;
    p.resident = false;
    return p;
}

// The last plans by shape: making one asks the occupancy tables some twenty
// times, a few microseconds of a call that may run for as many on the GPU.
struct PlanEntry {
    int device, dtype, bwd, C, G;
    int64_t B, S;
    Plan plan;
};
std::mutex g_plan_mu;
PlanEntry g_plans[64];
int g_plan_n = 0, g_plan_next = 0;

Plan plan_of(const DeviceInfo& dev, int dtype, bool vec, bool bwd, const GroupNormArgs& a) {
    if (!vec) return Plan{};
    {
        std::lock_guard<std::mutex> lk(g_plan_mu);
        for (int i = 0; i < g_plan_n; ++i) {
            const PlanEntry& e = g_plans[i];
            if (e.S == a.S && e.B == a.B && e.C == a.C && e.G == a.G && e.dtype == dtype &&
                e.bwd == (bwd ? 1 : 0) && e.device == dev.device)
                return e.plan;
        }
    }
    const Plan p = make_plan(dev, dtype, bwd, a);
    std::lock_guard<std::mutex> lk(g_plan_mu);
    g_plans[g_plan_next] = {dev.device, dtype, bwd ? 1 : 0, a.C, a.G, a.B, a.S, p};
    g_plan_next = (g_plan_next + 1) % 64;
    g_plan_n = std::min(64, g_plan_n + 1);
    return p;
}

SlabArgs args_of(const Plan& p, const GroupNormArgs& a) {
    SlabArgs g{};
    g.a = a;
    g.nvec = p.nvec;
    g.lanes = p.lanes;
    g.splits = p.splits;
    g.cw = a.C / p.splits;
    g.gw = a.G / p.splits;
    g.D = a.C / a.G;
    g.cluster = p.cluster;
    g.chunks = p.chunks;
    return g;
}

size_t stats_bytes(const Plan& p, const GroupNormArgs& a) {
    return p.resident ? 0
                      : (static_cast<size_t>(p.samples) * p.chunks * a.G * 8 + 255) / 256 * 256;
}
// Rows of dw partial sums, 0 where the kernel writes dw and db itself.
int64_t partial_rows(const Plan& p, bool bwd, const GroupNormArgs& a) {
    const int64_t rows = a.B * p.chunks;
    return bwd && a.dw != nullptr && rows > 1 ? rows : 0;
}

}  // namespace

size_t group_norm_workspace(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                            const GroupNormArgs& a) {
    const Plan p = plan_of(dev, dtype, vec, bwd, a);
    if (!p.ok) return gn_scalar_workspace(bwd, a);
    return stats_bytes(p, a) + static_cast<size_t>(partial_rows(p, bwd, a)) * 2 * a.C * 4;
}

cudaError_t group_norm_launch(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                              const GroupNormArgs& a, void* workspace, cudaStream_t s) {
    const Plan p = plan_of(dev, dtype, vec, bwd, a);
    if (!p.ok) return gn_scalar_launch(dtype, bwd, a, workspace, s);
    SlabArgs g = args_of(p, a);
    const int64_t rows = partial_rows(p, bwd, a);
    g.stats = static_cast<float2*>(workspace);
    if (rows > 0) g.rows = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(p, a));
    cudaError_t err = cudaSuccess;
    if (p.resident) {
        err = launch_pdl(kernel_for(dtype, bwd, kResident),
                         static_cast<int>(a.B * p.splits * p.cluster), p.threads, p.smem, p.cluster, s, g);
    } else {
        for (int64_t b = 0; b < a.B && err == cudaSuccess; b += p.samples) {
            g.sample0 = b;
            const int64_t n = std::min<int64_t>(p.samples, a.B - b);
            const int grid = static_cast<int>(n * p.splits * p.chunks * p.cluster);
            err = launch_pdl(kernel_for(dtype, bwd, kSums), grid, p.threads, p.smem, p.cluster, s, g);
            if (err == cudaSuccess)
                err = launch_pdl(kernel_for(dtype, bwd, kApply), grid, p.threads,
                                 static_cast<size_t>(g.gw) * 8, 1, s, g);
        }
    }
    if (err != cudaSuccess || rows == 0) return err;
    PairSum sum{};
    sum.part[0] = g.rows;
    sum.part[1] = g.rows + a.C;
    sum.out[0] = a.dw;
    sum.out[1] = a.db;
    sum.rows[0] = sum.rows[1] = static_cast<int>(rows);
    sum.n = a.C;
    sum.stride = 2 * a.C;
    sum.status = a.status;
    return pair_sum_launch(sum, s);
}

}  // namespace rmsn
