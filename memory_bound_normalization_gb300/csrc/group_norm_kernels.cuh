// Group norm with an activation, channels last, by 16-byte vectors.
//
// A slab is one sample's positions by a run of whole groups of channels. A
// block takes a contiguous range of its positions; each thread owns one
// 16-byte vector of channels and strides over positions, so its channels'
// constants and sums stay in registers, whatever the group width (a vector may
// span groups: sums are kept per channel and joined per group afterwards).
//
// Forward statistics. A block sums d = x - p and d^2 for each channel about p,
// the median of the channel's values at three of the block's positions, which
// gives (count, mean, M2); these are joined over channels, blocks and the slab by
//   mean = sum n_i m_i / n,   M2 = sum M2_i + n_i (m_i - mean)^2
// so a mean far from zero costs no digits, as long as p lies among the values:
// the sum of squares is rounded at 2^-24 of n_i (p - m_i)^2. The median of three
// positions a quarter of the block apart leaves out a border of zeros.
// Backward sums. Per channel P = sum dz, Q = sum dz xhat: they give the slab's
// means (sum_c w P, sum_c w Q) and, added over samples, db and dw.
//
// Bound by DRAM: x once in and y once out (x, dy, dx). Between the sums and the
// second pass the slab has to be kept near. Two families:
//   resident  the slab fits the shared memory of a cluster of at most 16
//             blocks: one kernel, each thread keeps what it read in its own
//             shared-memory slots, the blocks' sums meet in distributed shared
//             memory. One read of x. Bound by its steps' latency (launch, first
//             bytes, two joins): 4 samples of 4096 positions of 320 f16 channels
//             take 10.4 us forward (21 MB, a floor of 3.1), 8 of 1024 of 640 bf16
//             backward 13.9 (31 MB, 4.7), 2 of 64 of 1280 forward 3.8.
//   stream    larger slabs: persistent blocks of one cooperative launch sum a
//             slab and apply it in the opposite order, so that the second pass
//             starts with what L2 still holds. Bound by the two passes, whose
//             second is served by L2 for some six tenths of its bytes (DRAM read
//             1.4 times x for slabs of 67 MB), and by the meeting between them
//             (some 5 us a round): 1048576 positions of 128 bf16 channels forward
//             (537 MB) take 125 us (4.3 TB/s of x and y), 2 samples of 262144 of
//             256 backward (805 MB) 204 (3.9 TB/s).
#pragma once

#include "group_norm.cuh"
#include "group_norm.h"
#include "own_copy.cuh"

namespace rmsn {
namespace {

// First position of a block's range: S split as evenly as it goes.
__device__ __forceinline__ int64_t part_begin(const SlabArgs& g, int part) {
    return static_cast<int64_t>(part) * g.part_rows + min(part, g.part_more);
}

// Where a block works.
struct Place {
    int64_t sample, r0;  // its first position
    int split, rank, rows;
};
__device__ __forceinline__ Place place_of(const SlabArgs& g) {
    Place p;
    const int slab = static_cast<int>(blockIdx.x) / g.cluster;
    p.rank = static_cast<int>(blockIdx.x) - slab * g.cluster;
    p.sample = slab / g.splits;
    p.split = slab - static_cast<int>(p.sample) * g.splits;
    p.r0 = part_begin(g, p.rank);
    p.rows = g.part_rows + (p.rank < g.part_more ? 1 : 0);
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

// A channel's weight or bias.
template <typename T>
__device__ __forceinline__ float channel(const SlabArgs& g, const void* p, int c, float none) {
    if (p == nullptr) return none;
    return g.a.w_f32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const T*>(p)[c]);
}
// A thread's channels of a row of floats in shared memory (16-byte aligned).
template <typename T>
__device__ __forceinline__ void read_channels(const float* row, float2 (&f)[Pack<T>::PAIRS]) {
#pragma unroll
    for (int e = 0; e < Pack<T>::PAIRS; e += 2) {
        const float4 v = *reinterpret_cast<const float4*>(row + 2 * e);
        f[e] = make_float2(v.x, v.y);
        f[e + 1] = make_float2(v.z, v.w);
    }
}
template <typename T>
__device__ __forceinline__ void write_channels(float* row, const float2 (&f)[Pack<T>::PAIRS]) {
#pragma unroll
    for (int e = 0; e < Pack<T>::PAIRS; e += 2)
        *reinterpret_cast<float4*>(row + 2 * e) = make_float4(f[e].x, f[e].y, f[e + 1].x, f[e + 1].y);
}

__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    return __fadd2_rn(a, make_float2(-b.x, -b.y));
}

__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// v, or the bound (positive) with v's sign where |v| is larger.
__device__ __forceinline__ float held_to(float v, float bound) {
    float r;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(bound));
    return r;
}
__device__ __forceinline__ float2 exp2_pair(float2 v) {
    return make_float2(exp2_fast(v.x), exp2_fast(v.y));
}
__device__ __forceinline__ float2 rcp_pair(float2 v) {
    return make_float2(rcp_fast(v.x), rcp_fast(v.y));
}

// The normal distribution function of z and e^(-z^2/2).
// 16-bit outputs: the form of Hastings, Approximations for Digital Computers
// (1955): with y = |z|, t = 1 / (1 + p y),
//   Phi(-y) = (a1 t + ... + a5 t^5) e^(-y^2/2),
// fitted over y up to 13 (least squares, reweighted until the largest errors agree).
// What is rounded to 16 bits takes p and five terms for the relative error, nine times
// looser past y = 4.7: off by 1.4e-5 of the value up to y = 4.5, where normal f16
// values end (half a step is 2.4e-4), and 1.1e-4 behind (half a bf16 step is 2e-3).
// What is summed (SUMMED) in 32 bits takes p and six terms for the absolute error, as
// long as the relative one stays below 5e-5: 2e-7 in fp32 arithmetic. (The sums with
// five terms for the relative error were 1e-5 off; a fit to the absolute error alone,
// as that of erf, is steps of the output off in the tail.)
// fp32 outputs: the form of Shepherd and Laframboise, Mathematics of Computation
// 36 (1981): (1 + 2 x) e^(x^2) erfc(x) is a polynomial in (x - k) / (x + k) to any
// accuracy; here with y = |z|, half of (1 + sqrt 2 y) e^(y^2/2) erfc(y / sqrt 2) in
// t = (y - 3) / (y + 3), of degree 9 by least squares at Chebyshev points up to
// y = 20, behind which the bell is 0: off by 3.1e-7 of its value in fp32
// arithmetic. One reciprocal serves both quotients. (The bell's argument is rounded
// twice, which leaves some z^2 2^-24 of the tail; to put that back, as silu does,
// makes a backward 12% slower, 166 -> 186 us of 6 samples of 7456 positions of 1024
// channels, and a form by 1 + erf is off by far more there.)
template <typename T, bool SUMMED>
__device__ __forceinline__ void normal_pair(float2 z, float2& phi, float2& bell) {
    float2 x = make_float2(fabsf(z.x), fabsf(z.y));
    float2 q;
    if constexpr (sizeof(T) == 4) {
        x = make_float2(fminf(x.x, 20.f), fminf(x.y, 20.f));
        const float2 a = __fadd2_rn(x, f2_splat(3.f)), b = __ffma2_rn(x, f2_splat(1.41421356f), f2_splat(1.f));
        const float2 r = rcp_pair(__fmul2_rn(a, b));
        const float2 t = __fmul2_rn(__fadd2_rn(x, f2_splat(-3.f)), __fmul2_rn(b, r));
        bell = exp2_pair(__fmul2_rn(__fmul2_rn(x, x), f2_splat(-0.72134752f)));
        q = __ffma2_rn(t, f2_splat(-8.372210141e-05f), f2_splat(-6.254466134e-04f));
        q = __ffma2_rn(q, t, f2_splat(-2.296439488e-04f));
        q = __ffma2_rn(q, t, f2_splat(4.599653184e-03f));
        q = __ffma2_rn(q, t, f2_splat(3.787202295e-04f));
        q = __ffma2_rn(q, t, f2_splat(-3.467372805e-02f));
        q = __ffma2_rn(q, t, f2_splat(8.302349597e-02f));
        q = __ffma2_rn(q, t, f2_splat(-7.428076863e-02f));
        q = __ffma2_rn(q, t, f2_splat(-5.101513118e-02f));
        q = __ffma2_rn(q, t, f2_splat(6.370539665e-01f));
        q = __fmul2_rn(__fmul2_rn(q, __fmul2_rn(a, r)), bell);
    } else {
        const float2 t = rcp_pair(__ffma2_rn(x, f2_splat(SUMMED ? 0.29133f : 0.36571f), f2_splat(1.f)));
        // e^(-z^2/2) = 2^(-z^2 log2(e) / 2)
        bell = exp2_pair(__fmul2_rn(__fmul2_rn(z, z), f2_splat(-0.72134752f)));
        if constexpr (SUMMED) {
            q = __ffma2_rn(t, f2_splat(-8.762242645e-02f), f2_splat(2.761290669e-01f));
            q = __ffma2_rn(q, t, f2_splat(-8.285358548e-02f));
            q = __ffma2_rn(q, t, f2_splat(1.744683087e-01f));
            q = __ffma2_rn(q, t, f2_splat(1.025927290e-01f));
            q = __ffma2_rn(q, t, f2_splat(1.172858700e-01f));
        } else {
            q = __ffma2_rn(t, f2_splat(-9.361262619e-02f), f2_splat(2.265792787e-01f));
            q = __ffma2_rn(q, t, f2_splat(6.293377280e-02f));
            q = __ffma2_rn(q, t, f2_splat(1.592284888e-01f));
            q = __ffma2_rn(q, t, f2_splat(1.448649615e-01f));
        }
        q = __fmul2_rn(__fmul2_rn(q, t), bell);
    }
    phi = make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
}

// 1 + e^-z, to infinity, by the hardware's power 2^t, which is off by 2^-22 of its
// value and by what rounding t = -z log2(e) leaves out, some |z| 2^-24 of it. In 32
// bits the latter is put back: e^-z = 2^t e^-r, r = z + t ln 2, which is small where
// z is held to what the power's range takes. Silu by it and the hardware's reciprocal
// is within 6 2^-24 of its value for z > -20 (0.7 on average; 3.5 and 0.6 by expf and
// a division), 8 behind, at the cost of the power alone but for resident slabs (8
// samples of 1024 positions of 640 fp32 channels backward 23.6 -> 25.0 us). By expf
// and a division 6 samples of 7456 positions of 1024 fp32 channels backward take 171
// us, by these 134, as without an activation. 16-bit outputs, whose half step is
// 2^-12 of a value, need no more than 2^t: the accurate functions cost the
// backward's first pass 18 instructions an element, where DRAM leaves room for 22.
template <typename T>
__device__ __forceinline__ float2 one_plus_exp(float2 z) {
    if constexpr (sizeof(T) == 2) {
        return __fadd2_rn(exp2_pair(__fmul2_rn(z, f2_splat(-1.44269504f))), f2_splat(1.f));
    } else {
        const float2 c = make_float2(held_to(z.x, 128.f), held_to(z.y, 128.f));
        const float2 t = __fmul2_rn(c, f2_splat(-1.44269504f));
        const float2 r = __ffma2_rn(t, f2_splat(0.69314718f), c);
        return __ffma2_rn(exp2_pair(t), __ffma2_rn(r, f2_splat(-1.f), f2_splat(1.f)), f2_splat(1.f));
    }
}

template <typename T, int ACT>
__device__ __forceinline__ float2 act_pair(float2 z) {
    if constexpr (ACT == RMSNORM_ACT_NONE) {
        return z;
    } else if constexpr (ACT == RMSNORM_ACT_SILU) {
        return __fmul2_rn(z, rcp_pair(one_plus_exp<T>(z)));
    } else {
        float2 phi, bell;
        normal_pair<T, false>(z, phi, bell);
        return __fmul2_rn(z, phi);
    }
}
template <typename T, int ACT, bool SUMMED>
__device__ __forceinline__ float2 slope_pair(float2 z) {
    if constexpr (ACT == RMSNORM_ACT_SILU) {
        // s (1 + z (1 - s)) = s + (z s) (1 - s)
        const float2 s = rcp_pair(one_plus_exp<T>(z));
        const float2 r = __ffma2_rn(s, f2_splat(-1.f), f2_splat(1.f));
        return __fmul2_rn(s, __ffma2_rn(z, r, f2_splat(1.f)));
    } else {
        float2 phi, bell;
        normal_pair<T, SUMMED>(z, phi, bell);
        return __ffma2_rn(__fmul2_rn(z, f2_splat(0.39894228f)), bell, phi);
    }
}

// The constants and sums of a thread's channels, and the two passes' steps.
// Products with the mean are folded into constants: their rounding is of the
// size of the mean's own.
template <typename T, bool BWD, int ACT>
struct Columns;

template <typename T, int ACT>
struct Columns<T, false, ACT> {
    static constexpr int PAIRS = Pack<T>::PAIRS;
    float2 pivot[PAIRS], s1[PAIRS], s2[PAIRS];
    float2 scale[PAIRS], shift[PAIRS];  // rstd w and b - mean rstd w

    __device__ __forceinline__ void start(const uint4 (&three)[3]) {
        float2 b[PAIRS], c[PAIRS];
        Pack<T>::unpack2(three[0], pivot);
        Pack<T>::unpack2(three[1], b);
        Pack<T>::unpack2(three[2], c);
        auto median = [](float p, float q, float r) { return fmaxf(fminf(p, q), fminf(fmaxf(p, q), r)); };
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            pivot[e] = make_float2(median(pivot[e].x, b[e].x, c[e].x), median(pivot[e].y, b[e].y, c[e].y));
            s1[e] = s2[e] = make_float2(0.f, 0.f);
        }
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
    // act(x scale + shift), rounded once
    __device__ __forceinline__ uint4 apply(const uint4& v) const {
        float2 f[PAIRS];
        Pack<T>::unpack2(v, f);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) f[e] = act_pair<T, ACT>(__ffma2_rn(f[e], scale[e], shift[e]));
        return Pack<T>::pack2(f);
    }
};

template <typename T, int ACT>
struct Columns<T, true, ACT> {
    static constexpr int PAIRS = Pack<T>::PAIRS;
    // First pass: x - mean, z = (x - mean) k1 + b with k1 = rstd w, and the sums
    // of dz and dz (x - mean). Second: z = x k1 + k2, dx = dz k1 + (x k3 + k4)
    // with k2 = b - mean k1, k3 = -rstd^2 B, k4 = -rstd A - mean k3.
    float2 mean[PAIRS], k1[PAIRS], b[PAIRS];
    float2 p[PAIRS], q[PAIRS];
    float2 k2[PAIRS], k3[PAIRS], k4[PAIRS];

    __device__ __forceinline__ void add(const uint4& x, const uint4& dy) {
        float2 c[PAIRS], d[PAIRS];
        Pack<T>::unpack2(x, c);
        Pack<T>::unpack2(dy, d);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            c[e] = __fadd2_rn(c[e], mean[e]);
            if constexpr (ACT != RMSNORM_ACT_NONE)
                d[e] = __fmul2_rn(d[e], slope_pair<T, ACT, true>(__ffma2_rn(c[e], k1[e], b[e])));
            p[e] = __fadd2_rn(p[e], d[e]);
            q[e] = __ffma2_rn(d[e], c[e], q[e]);
        }
    }
    // dx = rstd (dz w - A - xhat B), rounded once
    __device__ __forceinline__ uint4 apply(const uint4& xv, const uint4& dy) const {
        float2 x[PAIRS], d[PAIRS];
        Pack<T>::unpack2(xv, x);
        Pack<T>::unpack2(dy, d);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
            if constexpr (ACT != RMSNORM_ACT_NONE)
                d[e] = __fmul2_rn(d[e], slope_pair<T, ACT, false>(__ffma2_rn(x[e], k1[e], k2[e])));
            d[e] = __ffma2_rn(d[e], k1[e], __ffma2_rn(x[e], k3[e], k4[e]));
        }
        return Pack<T>::pack2(d);
    }
};

// Sums of a block's channels over its lanes: two values a channel in `sums`
// ([2][lanes][cw]), added into the first lane's rows. A thread adds four
// neighbouring values of every g.join-th lane from lane j on into lane j's row,
// then the first threads add the g.join rows.
__device__ __forceinline__ void sum_lanes(const SlabArgs& g, float* sums) {
    const int quads = g.cw / 2, half = g.cw / 4;  // of both values, and of one
    auto at = [&](int q, int lane) {
        return reinterpret_cast<float4*>(sums + ((q < half ? 0 : g.lanes) + lane) * g.cw + (q < half ? q : q - half) * 4);
    };
    auto add = [](float4& s, const float4& v) {
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    };
    __syncthreads();
    for (int i = threadIdx.x; i < quads * g.join; i += blockDim.x) {
        const int j = i / quads, q = i - j * quads;
        float4 s = *at(q, j);
#pragma unroll 4
        for (int r = j + g.join; r < g.lanes; r += g.join) add(s, *at(q, r));
        *at(q, j) = s;
    }
    __syncthreads();
    if (g.join > 1) {
        for (int q = threadIdx.x; q < quads; q += blockDim.x) {
            float4 s = *at(q, 0);
#pragma unroll 4
            for (int j = 1; j < g.join; ++j) add(s, *at(q, j));
            *at(q, 0) = s;
        }
        __syncthreads();
    }
}

// A thread's place in its block, the same in both families.
struct Seat {
    int lane, vec, c;   // its lane of positions, its vector, its first channel
    bool active;
    int warps, warp, l;
    float inv_d;
    __device__ __forceinline__ Seat(const SlabArgs& g, int vec_elems) {
        lane = static_cast<int>(threadIdx.x) / g.nvec;
        vec = static_cast<int>(threadIdx.x) - lane * g.nvec;
        c = vec * vec_elems;
        active = lane < g.lanes;
        warps = blockDim.x / 32;
        warp = threadIdx.x / 32;
        l = threadIdx.x % 32;
        inv_d = 1.f / static_cast<float>(g.D);
    }
    __device__ __forceinline__ int positions(const SlabArgs& g, int rows) const {
        return active && rows > lane ? (rows - lane - 1) / g.lanes + 1 : 0;
    }
};

// A slab's channels in shared memory ([4][cw]): -mean, rstd w, b and rstd, or w
// in the second row and b in the third. Thread i keeps channel i.
template <typename T, bool BWD>
__device__ __forceinline__ void load_channels(const SlabArgs& g, const Seat& s, float* chan, int c0,
                                              int64_t group0) {
    for (int i = threadIdx.x; i < g.cw; i += blockDim.x) {
        const float w = channel<T>(g, g.a.w, c0 + i, 1.f), b = channel<T>(g, g.a.b, c0 + i, 0.f);
        if constexpr (BWD) {
            const int k = quotient(i, s.inv_d);
            const float r = g.a.rstd[group0 + k], m = g.a.mean[group0 + k];
            chan[i] = -m;
            chan[g.cw + i] = r * w;
            chan[3 * g.cw + i] = r;
        } else {
            chan[g.cw + i] = w;
        }
        chan[2 * g.cw + i] = b;
    }
}

// A thread's channels at three of the block's positions, a quarter of it apart;
// `p` points to them at its first position, `pitch` bytes before the next.
__device__ __forceinline__ void load_three(uint4 (&three)[3], const void* p, int rows, int64_t pitch) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
        three[i] = ld_global_16_stream(static_cast<const char*>(p) + (static_cast<int64_t>(rows) * (i + 1) / 4) * pitch);
}

// The first pass's constants of a thread's channels, and its sums. `three`:
// positions of the block to take the pivots from (forward).
template <typename T, int ACT>
__device__ __forceinline__ void start(Columns<T, false, ACT>& col, const SlabArgs&, const Seat&, const float*,
                                      const uint4 (&three)[3]) {
    col.start(three);
}
template <typename T, int ACT>
__device__ __forceinline__ void start(Columns<T, true, ACT>& col, const SlabArgs& g, const Seat& s,
                                      const float* chan, const uint4 (&)[3]) {
    if (s.active) {
        read_channels<T>(chan + s.c, col.mean);
        read_channels<T>(chan + g.cw + s.c, col.k1);
        read_channels<T>(chan + 2 * g.cw + s.c, col.b);
    }
#pragma unroll
    for (int e = 0; e < Pack<T>::PAIRS; ++e) col.p[e] = col.q[e] = make_float2(0.f, 0.f);
}

// Sum over the `width` neighbouring lanes (a power of two) that v belongs to.
__device__ __forceinline__ float lanes_sum(float v, int width) {
#pragma unroll
    for (int off = 16; off >= 1; off /= 2)
        if (off < width) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Joins the block's first pass: emit(k, (mean, M2)) for each group of channels,
// from each channel's sums about its pivot. 2^g.seg_log lanes take a group.
template <typename T, int ACT, typename Emit>
__device__ __forceinline__ void join(const Columns<T, false, ACT>& col, const SlabArgs& g, const Seat& s,
                                     float* sums, float* chan, int rows, Emit emit) {
    if (s.active) {
        write_channels<T>(sums + s.lane * g.cw + s.c, col.s1);
        write_channels<T>(sums + (g.lanes + s.lane) * g.cw + s.c, col.s2);
        if (s.lane == 0) write_channels<T>(chan + s.c, col.pivot);
    }
    sum_lanes(g, sums);
    const float* squares = sums + g.lanes * g.cw;
    const float frows = static_cast<float>(rows), inv_rows = 1.f / fmaxf(frows, 1.f);
    const int seg = 1 << g.seg_log, at_once = 32 >> g.seg_log, sl = s.l & (seg - 1);
    for (int k0 = s.warp * at_once; k0 < g.gw; k0 += s.warps * at_once) {
        const int k = k0 + (s.l >> g.seg_log), end = k < g.gw ? (k + 1) * g.D : 0;
        float t = 0.f;
        for (int i = k * g.D + sl; i < end; i += seg) t += fmaf(sums[i], inv_rows, chan[i]);
        const float m = lanes_sum(t, seg) * s.inv_d;
        float m2 = 0.f;
        for (int i = k * g.D + sl; i < end; i += seg) {
            // squares about the channel's mean, and its mean's distance from the group's
            const float off = sums[i] * inv_rows, d = chan[i] + off - m;
            m2 += fmaf(frows * d, d, fmaf(-sums[i], off, squares[i]));
        }
        m2 = lanes_sum(m2, seg);
        if (sl == 0 && k < g.gw) emit(k, make_float2(m, m2));
    }
}
// The backward's: emit(k, (rstd sum w dz, sum w dz xhat)), which sums of P and
// of Q = sum dz (x - mean) weighted by k1 = rstd w are. The channels' sums stay
// in the first lane's rows of `sums`: P, and Q behind all lanes of P.
template <typename T, int ACT, typename Emit>
__device__ __forceinline__ void join(const Columns<T, true, ACT>& col, const SlabArgs& g, const Seat& s,
                                     float* sums, float* chan, int, Emit emit) {
    if (s.active) {
        write_channels<T>(sums + s.lane * g.cw + s.c, col.p);
        write_channels<T>(sums + (g.lanes + s.lane) * g.cw + s.c, col.q);
    }
    sum_lanes(g, sums);
    const float* ps = sums;
    const float* qs = sums + g.lanes * g.cw;
    const int seg = 1 << g.seg_log, at_once = 32 >> g.seg_log, sl = s.l & (seg - 1);
    for (int k0 = s.warp * at_once; k0 < g.gw; k0 += s.warps * at_once) {
        const int k = k0 + (s.l >> g.seg_log), end = k < g.gw ? (k + 1) * g.D : 0;
        float sp = 0.f, sq = 0.f;
        for (int i = k * g.D + sl; i < end; i += seg) {
            const float k1 = chan[g.cw + i];
            sp = fmaf(k1, ps[i], sp);
            sq = fmaf(k1, qs[i], sq);
        }
        sp = lanes_sum(sp, seg);
        sq = lanes_sum(sq, seg);
        if (sl == 0 && k < g.gw) emit(k, make_float2(sp, sq));
    }
}

// The slab's result of a group from NP results a lane of `width` lanes with
// their counts of values (0: none there), by a fixed tree: (mean, rstd), or the
// backward's two sums as means.
template <bool BWD, int NP>
__device__ __forceinline__ float2 combine(const float2 (&t)[NP], const float (&count)[NP], float inv_count,
                                          float eps, int width) {
    float2 v = make_float2(0.f, 0.f);
    if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < NP; ++i) v = __fadd2_rn(v, t[i]);
        v.x = lanes_sum(v.x, width) * inv_count;
        v.y = lanes_sum(v.y, width) * inv_count;
    } else {
        // mean = sum n m / n, M2 = sum M2 + n (m - mean)^2
#pragma unroll
        for (int i = 0; i < NP; ++i) v.x = fmaf(count[i], t[i].x, v.x);
        v.x = lanes_sum(v.x, width) * inv_count;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float d = t[i].x - v.x;
            v.y += fmaf(count[i] * d, d, t[i].y);
        }
        v.y = rsqrtf(lanes_sum(v.y, width) * inv_count + eps);
    }
    return v;
}

// The second pass's constants from the slab's results, in the channels' place,
// and a thread's own. Every thread has written `slab` and is done with `chan`.
template <typename T, bool BWD, int ACT>
__device__ __forceinline__ void finish(Columns<T, BWD, ACT>& col, const SlabArgs& g, const Seat& s,
                                       float* chan, const float2* slab) {
    __syncthreads();
    for (int i = threadIdx.x; i < g.cw; i += blockDim.x) {
        const float2 v = slab[quotient(i, s.inv_d)];
        if constexpr (BWD) {
            const float m = chan[i], r = chan[3 * g.cw + i];
            const float k3 = -v.y * r * r;
            chan[2 * g.cw + i] = fmaf(m, chan[g.cw + i], chan[2 * g.cw + i]);
            chan[i] = k3;
            chan[3 * g.cw + i] = fmaf(m, k3, -v.x);
        } else {
            const float scale = v.y * chan[g.cw + i];
            chan[g.cw + i] = scale;
            chan[2 * g.cw + i] = fmaf(-v.x, scale, chan[2 * g.cw + i]);
        }
    }
    __syncthreads();
    if (!s.active) return;
    if constexpr (BWD) {
        read_channels<T>(chan + s.c, col.k3);
        read_channels<T>(chan + g.cw + s.c, col.k1);
        read_channels<T>(chan + 2 * g.cw + s.c, col.k2);
        read_channels<T>(chan + 3 * g.cw + s.c, col.k4);
    } else {
        read_channels<T>(chan + g.cw + s.c, col.scale);
        read_channels<T>(chan + 2 * g.cw + s.c, col.shift);
    }
}

// Resident: a thread's way through its positions. Copies run kDepth positions
// ahead, in groups of kGroup, into the thread's own slots, a slot for every
// position, which stays there for the second pass.
template <typename T, bool BWD>
struct Feed {
    const T* x;      // the next position to copy
    const T* dy;
    int64_t step;    // elements from a position to the thread's next
    uint32_t slots;  // this thread's first slot (a shared-memory address)
    uint32_t pitch;  // bytes from a tensor's slot to the next one's
    int n;
    static constexpr uint32_t TENSORS = BWD ? 2 : 1;

    __device__ __forceinline__ void issue(uint32_t slot, int left, int* status) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            if (u < left) {
                copy_own(slot + u * TENSORS * pitch, x, status);
                if constexpr (BWD) copy_own(slot + (u * TENSORS + 1) * pitch, dy, status);
            }
            x += step;
            if constexpr (BWD) dy += step;
        }
        copies_commit();
    }
    // the first kDepth positions' copies
    __device__ __forceinline__ void prepare(int* status) {
#pragma unroll
        for (int i = 0; i < kDepth; i += kGroup) issue(slots + i * TENSORS * pitch, n - i, status);
    }
    // visit(i, x vector, dy vector) for every position in order
    template <typename Visit>
    __device__ __forceinline__ void run(int* status, Visit visit) {
        const uint32_t group = kGroup * TENSORS * pitch;
        uint32_t at = slots, ahead = slots + kDepth * TENSORS * pitch;
#pragma unroll 1
        for (int i = 0; i < n; i += kGroup) {
            copies_wait<kDepth / kGroup - 1>();
            uint4 xv[kGroup], dv[kGroup];
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                if (i + u < n) {
                    xv[u] = ld_slot(at + u * TENSORS * pitch);
                    if constexpr (BWD) dv[u] = ld_slot(at + (u * TENSORS + 1) * pitch);
                }
            }
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
                if (i + u < n) visit(i + u, xv[u], dv[u]);
            issue(ahead, n - i - kDepth, status);
            at += group;
            ahead += group;
        }
        copies_wait<0>();
    }
};

// ----------------------------------------------------------------- resident
// Both passes over a slab that its cluster keeps.
template <typename T, bool BWD, int ACT>
__global__ void __launch_bounds__(kMaxThreads) gn_resident_kernel(const __grid_constant__ SlabArgs g) {
    const Place at = place_of(g);
    const Seat s(g, Pack<T>::VEC);
    // shared memory: the threads' sums [2][lanes][cw], the channels' constants
    // [4][cw], the block's and the slab's results of each group, the slots
    float* sums = reinterpret_cast<float*>(rmsn_dynamic_smem);
    float* chan = sums + 2 * g.lanes * g.cw;
    float2* mine = reinterpret_cast<float2*>(chan + 4 * g.cw);
    float2* slab = mine + g.gw;
    uint4* keep = reinterpret_cast<uint4*>(slab + g.gw);
    const int c0 = at.split * g.cw, n = s.positions(g, at.rows);
    const int64_t base = (at.sample * g.a.S + at.r0 + s.lane) * g.a.C + c0 + s.c;
    const int64_t group0 = at.sample * g.a.G + at.split * g.gw;
    Feed<T, BWD> feed;
    feed.x = static_cast<const T*>(g.a.x) + base;
    feed.dy = BWD ? static_cast<const T*>(g.a.dy) + base : nullptr;
    feed.step = static_cast<int64_t>(g.lanes) * g.a.C;
    feed.slots = smem_u32(keep + threadIdx.x);
    feed.pitch = static_cast<uint32_t>(g.lanes * g.nvec) * 16u;
    feed.n = n;
    Columns<T, BWD, ACT> col;
    wait_for_prerequisite_grid();  // no global access before this

    feed.prepare(g.a.status);
    uint4 three[3] = {};
    if (!BWD && s.active && at.rows > 0)
        load_three(three, static_cast<const T*>(g.a.x) + base - static_cast<int64_t>(s.lane) * g.a.C, at.rows,
                   g.a.C * static_cast<int64_t>(sizeof(T)));
    load_channels<T, BWD>(g, s, chan, c0, group0);
    __syncthreads();
    start(col, g, s, chan, three);
    feed.run(g.a.status, [&](int, const uint4& x, const uint4& dy) {
        if constexpr (BWD) col.add(x, dy);
        else col.add(x);
    });
    join(col, g, s, sums, chan, at.rows, [&](int k, float2 v) { mine[k] = v; });

    // the cluster's blocks meet and read one another's results
    __syncwarp();
    if (g.cluster > 1) cluster_sync_all();
    else __syncthreads();
    const float inv_count = 1.f / (static_cast<float>(g.a.S) * static_cast<float>(g.D));
    // as many lanes a group as there are blocks
    const int log = __ffs(g.cluster) - 1, peer = s.l & (g.cluster - 1), at_once = 32 >> log;
    const float count[1] = {static_cast<float>(g.part_rows + (peer < g.part_more ? 1 : 0)) * static_cast<float>(g.D)};
    for (int k0 = s.warp * at_once; k0 < g.gw; k0 += s.warps * at_once) {
        const int k = k0 + (s.l >> log);
        float2 t[1] = {make_float2(0.f, 0.f)};
        if (k < g.gw) t[0] = g.cluster > 1 ? ld_cluster_f32x2(mine + k, peer) : mine[k];
        __syncwarp();
        const float2 v = combine<BWD>(t, count, inv_count, g.a.eps, g.cluster);
        if (peer == 0 && k < g.gw) {
            slab[k] = v;
            if (!BWD && at.rank == 0) {
                g.a.mean[group0 + k] = v.x;
                g.a.rstd[group0 + k] = v.y;
            }
        }
    }
    if constexpr (BWD) {
        // each block adds its share of the cluster's channel sums
        if (g.a.dw != nullptr) {
            const int lo = 2 * g.cw * at.rank / g.cluster, hi = 2 * g.cw * (at.rank + 1) / g.cluster;
            for (int i = lo + threadIdx.x; i < hi; i += blockDim.x) {
                const bool q = i >= g.cw;
                const int c = q ? i - g.cw : i;
                const float* src = sums + (q ? g.lanes * g.cw : 0) + c;
                float t = 0.f;
#pragma unroll 4
                for (int r = 0; r < g.cluster; ++r) t += g.cluster > 1 ? ld_cluster_f32(src, r) : *src;
                if (q) t *= chan[3 * g.cw + c];
                float* d = g.rows == nullptr ? (q ? g.a.dw : g.a.db)
                                             : g.rows + at.sample * 2 * g.a.C + (q ? 0 : g.a.C);
                d[c0 + c] = t;
            }
        }
    }
    __syncwarp();
    if (g.cluster > 1) cluster_arrive_relaxed();  // this block is done reading its peers
    allow_dependent_launch();

    finish(col, g, s, chan, slab);
    T* out = static_cast<T*>(g.a.out) + base;
    [[maybe_unused]] const int64_t bytes = g.a.B * g.a.S * g.a.C * static_cast<int64_t>(sizeof(T));
    uint32_t slot = feed.slots;
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
        uint4 v;
        if constexpr (BWD) v = col.apply(ld_slot(slot), ld_slot(slot + feed.pitch));
        else v = col.apply(ld_slot(slot));
        slot += feed.pitch * Feed<T, BWD>::TENSORS;
        if (RMSN_OK(span_in(out, 16, g.a.out, bytes), g.a.status)) st_global_16(out, v);
        out += feed.step;
    }
    __syncwarp();
    if (g.cluster > 1) cluster_wait();  // no block leaves while a peer reads it
}

// ------------------------------------------------------------------- stream
// One cooperative launch for slabs that no cluster holds: persistent blocks
// take the slabs in rounds of as many as L2 keeps (g.together, g.parts blocks a
// slab). In a round a block sums its positions, publishes its groups' results
// and counts itself in; while the others arrive, its copies of the second pass,
// which goes from its last position back to the first, are under way. Copies
// run some positions ahead across passes and rounds, so that DRAM stays busy
// while sums are joined. The wait for the others is bounded in time.
template <typename T, bool BWD>
struct Copies {
    static constexpr int TENSORS = BWD ? 2 : 1;
    static constexpr uint32_t PITCH = kStreamThreads * 16, GROUP = TENSORS * PITCH;
    static constexpr int DEPTH = BWD ? stream_depth(true) : stream_depth(false);
    // a pass: where its copies come from and how many positions it has
    struct Pass {
        const char* x;
        const char* dy;
        uint32_t off, step;  // bytes of this thread's next position, and to the one after
        int n;
        bool last_use;       // read for the last time: L2 need not keep it
    };
    uint32_t first, slot;  // shared-memory addresses of this thread's ring and its next group
    uint64_t drop;         // L2 policies
    int* status;

    __device__ __forceinline__ void copy(uint32_t to, const char* from, bool last_use) const {
        if (!RMSN_OK(slot_in<16>(to), status)) return;
        if (last_use)
            asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "l"(drop) : "memory");
        else
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    // copies a pass's next position, if it has one
    __device__ __forceinline__ void issue(Pass& p, bool has) const {
        if (has) {
            copy(slot, p.x + p.off, p.last_use);
            if constexpr (BWD) copy(slot + PITCH, p.dy + p.off, p.last_use);
            p.off += p.step;
        }
        copies_commit();
    }
    __device__ __forceinline__ void advance() { slot = slot + GROUP == first + DEPTH * GROUP ? first : slot + GROUP; }
    // A pass whose first DEPTH copies are under way: visits its positions in
    // order, and starts the next pass's copies as its own run out. `p` is the
    // pass's next position to copy, and the next pass's in the end.
    template <typename Next, typename Visit>
    __device__ __forceinline__ void run(Pass& p, Next next_pass, Visit visit) {
        int i = 0;
#pragma unroll 1
        for (; i < p.n - DEPTH; ++i) {
            copies_wait<DEPTH - 1>();
            const uint4 x = ld_slot(slot);
            uint4 dy = x;
            if constexpr (BWD) dy = ld_slot(slot + PITCH);
            visit(x, dy);
            issue(p, true);
            advance();
        }
        Pass next = next_pass();
        const int end = max(p.n, DEPTH);
        int ahead = 0;  // positions of the next pass under way
#pragma unroll 1
        for (; i < end; ++i) {
            copies_wait<DEPTH - 1>();
            if (i < p.n) {
                const uint4 x = ld_slot(slot);
                uint4 dy = x;
                if constexpr (BWD) dy = ld_slot(slot + PITCH);
                visit(x, dy);
            }
            issue(next, ahead++ < next.n);
            advance();
        }
        p = next;
    }
};

// Waits until every block of a slab has published its results, for a limited
// time; a wait that runs out is reported.
__device__ __forceinline__ bool all_arrived(const SlabArgs& g, int64_t slab) {
    const uint64_t t0 = global_timer_ns();
    while (true) {
        unsigned seen;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(g.arrived + slab) : "memory");
        if (seen >= static_cast<unsigned>(g.parts)) return true;
        if (global_timer_ns() - t0 > g.a.wait_limit_ns) {
            report_status(g.a.status, kStatusTimeout);
            return false;
        }
    }
}

template <typename T, bool BWD, int ACT>
__global__ void __launch_bounds__(kStreamThreads, 2) gn_stream_kernel(const __grid_constant__ SlabArgs g) {
    constexpr int SIZE = sizeof(T);
    using Ring = Copies<T, BWD>;
    using Pass = typename Ring::Pass;
    const Seat s(g, Pack<T>::VEC);
    const float fd = static_cast<float>(g.D), inv_count = 1.f / (static_cast<float>(g.a.S) * fd);
    const int team = static_cast<int>(blockIdx.x) / g.parts;
    const int part = static_cast<int>(blockIdx.x) - team * g.parts;
    const int64_t r0 = part_begin(g, part);
    const int rows = g.part_rows + (part < g.part_more ? 1 : 0);
    const int n_all = s.positions(g, rows);
    // shared memory: the ring, the threads' sums [2][lanes][cw], the channels'
    // constants [4][cw], the groups' results
    float* sums = reinterpret_cast<float*>(rmsn_dynamic_smem + Ring::DEPTH * Ring::GROUP);
    float* chan = sums + 2 * g.lanes * g.cw;
    float2* slab = reinterpret_cast<float2*>(chan + 4 * g.cw);

    Ring ring;
    ring.first = ring.slot = smem_u32(rmsn_dynamic_smem) + threadIdx.x * 16;
    ring.drop = l2_policy_evict_first();
    ring.status = g.a.status;
    const uint32_t pitch = static_cast<uint32_t>(g.a.C) * SIZE;  // bytes of a position
    const uint32_t own = pitch * s.lane + s.c * SIZE;
    auto pass_of = [&](int round, bool second) {
        Pass p{};
        const int64_t i = static_cast<int64_t>(round) * g.together + team;
        const int64_t sample = i / g.splits;
        if (round >= g.rounds || sample >= g.a.B) return p;
        const int64_t at =
            ((sample * g.a.S + r0) * g.a.C + (i - sample * g.splits) * g.cw) * static_cast<int64_t>(SIZE);
        p.x = static_cast<const char*>(g.a.x) + at;
        if constexpr (BWD) p.dy = static_cast<const char*>(g.a.dy) + at;
        p.n = n_all;
        p.step = pitch * g.lanes;
        p.off = own;
        if (second) {
            p.off += p.step * static_cast<uint32_t>(n_all > 0 ? n_all - 1 : 0);
            p.step = 0u - p.step;
        }
        p.last_use = second && g.drop;
        return p;
    };
    // The kernel before this one lets it start when all earlier work is done, and
    // sets the arrival counters: nothing else has to wait for it.
    bool failed = false;  // thread 0's: a wait ran out
    Pass pass = pass_of(0, false);
#pragma unroll
    for (int i = 0; i < Ring::DEPTH; ++i) {
        ring.issue(pass, i < pass.n);
        ring.advance();
    }

    // Two teams: the second starts when the first has its sums, so that one
    // reads while the other, and its wait, leave DRAM to it.
    if (g.together == 2 && team == 1 && g.rounds > 1) {
        if (threadIdx.x == 0) {
            wait_for_prerequisite_grid();
            failed = !all_arrived(g, 0);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int round = 0; round < g.rounds; ++round) {
        const int64_t slab_i = static_cast<int64_t>(round) * g.together + team;
        const int64_t sample = slab_i / g.splits;
        const int split = static_cast<int>(slab_i - sample * g.splits);
        const bool live = sample < g.a.B;
        const int n = live ? n_all : 0, c0 = split * g.cw;
        const int64_t group0 = sample * g.a.G + split * g.gw;
        uint4 three[3] = {};
        if (!BWD && live && s.active && rows > 0)
            load_three(three, static_cast<const char*>(g.a.x) + s.c * SIZE +
                                  ((sample * g.a.S + r0) * g.a.C + c0) * static_cast<int64_t>(SIZE),
                       rows, pitch);
        if (live) load_channels<T, BWD>(g, s, chan, c0, group0);
        __syncthreads();
        Columns<T, BWD, ACT> col;
        start(col, g, s, chan, three);
        ring.run(pass, [&] { return pass_of(round, true); }, [&](const uint4& x, const uint4& dy) {
            if constexpr (BWD) col.add(x, dy);
            else col.add(x);
        });
        join(col, g, s, sums, chan, rows, [&](int k, float2 v) {
            if (live) g.stats[(slab_i * g.gw + k) * g.parts + part] = v;
        });
        if constexpr (BWD) {
            if (g.rows != nullptr && live) {
                float* row = g.rows + (sample * g.parts + part) * 2 * g.a.C + c0;
                for (int i = threadIdx.x; i < g.cw; i += blockDim.x) {
                    row[i] = sums[g.lanes * g.cw + i] * chan[3 * g.cw + i];
                    row[g.a.C + i] = sums[i];
                }
            }
        }
        // count this block in, then wait for the slab's others
        __syncthreads();
        if (live && threadIdx.x == 0) {
            wait_for_prerequisite_grid();
            if (blockIdx.x != 0 || slab_i != g.drop_unit)  // failure injection: not counted in
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(g.arrived + slab_i) : "memory");
            if (!failed) failed = !all_arrived(g, slab_i);  // later waits are not made
        }
        __syncthreads();
        // the slab's results, two groups a warp; all that a lane adds are read at once
        for (int k0 = live ? s.warp : g.gw; k0 < g.gw; k0 += 2 * s.warps) {
            constexpr int NP = kStreamMaxParts / 32;
            float2 t[2][NP];
            float count[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int j = s.l + 32 * i;
                count[i] = j < g.parts ? static_cast<float>(g.part_rows + (j < g.part_more ? 1 : 0)) * fd : 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int k = k0 + u * s.warps;
                    t[u][i] = j < g.parts && k < g.gw ? __ldcg(g.stats + (slab_i * g.gw + k) * g.parts + j)
                                                      : make_float2(0.f, 0.f);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k = k0 + u * s.warps;
                const float2 v = combine<BWD>(t[u], count, inv_count, g.a.eps, 32);
                if (s.l == 0 && k < g.gw) {
                    slab[k] = v;
                    if (!BWD && part == 0) {
                        g.a.mean[group0 + k] = v.x;
                        g.a.rstd[group0 + k] = v.y;
                    }
                }
            }
        }
        finish(col, g, s, chan, slab);
        if (round == g.rounds - 1) allow_dependent_launch();
        // The second pass. dx may be the dy buffer: a position's copies are
        // waited for before this thread, and no other, writes it.
        const int64_t back = static_cast<int64_t>(pitch) * g.lanes;
        char* out = static_cast<char*>(g.a.out) +
                    ((sample * g.a.S + r0) * g.a.C + c0) * static_cast<int64_t>(SIZE) + own + back * (n - 1);
        [[maybe_unused]] const int64_t bytes = g.a.B * g.a.S * g.a.C * static_cast<int64_t>(SIZE);
        const bool drop = g.drop;
        ring.run(pass, [&] { return pass_of(round + 1, false); }, [&](const uint4& x, const uint4& dy) {
            uint4 v;
            if constexpr (BWD) v = col.apply(x, dy);
            else v = col.apply(x);
            if (RMSN_OK(span_in(out, 16, g.a.out, bytes), g.a.status)) {
                if (drop) st_global_16_hint(out, v, ring.drop);
                else st_global_16(out, v);
            }
            out -= back;
        });
        __syncthreads();  // the constants' readers are done
    }
    copies_wait<0>();
}

template <typename T, bool BWD, int ACT>
SlabFn slab_kernel(SlabKind k) {
    if (k == SlabKind::kResident) return &gn_resident_kernel<T, BWD, ACT>;
    return &gn_stream_kernel<T, BWD, ACT>;
}
template <typename T>
SlabFn slab_kernel_of(bool bwd, int act, SlabKind k) {
    if (act == RMSNORM_ACT_SILU)
        return bwd ? slab_kernel<T, true, RMSNORM_ACT_SILU>(k) : slab_kernel<T, false, RMSNORM_ACT_SILU>(k);
    if (act == RMSNORM_ACT_GELU)
        return bwd ? slab_kernel<T, true, RMSNORM_ACT_GELU>(k) : slab_kernel<T, false, RMSNORM_ACT_GELU>(k);
    return bwd ? slab_kernel<T, true, RMSNORM_ACT_NONE>(k) : slab_kernel<T, false, RMSNORM_ACT_NONE>(k);
}

}  // namespace
}  // namespace rmsn
