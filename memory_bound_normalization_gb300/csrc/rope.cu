// Rotary positions of several axes for queries and keys, with the RMSNorm of
// their heads (the QK-norm) fused in front, forward and backward.
//
// A head of D elements holds rot/2 rotated pairs (a, b) and D - rot elements
// that pass. With theta = position[axis(p)] * inv_freq[p]:
//   forward   n = x * rstd * w (n = x without weights)
//             y_a = n_a cos - n_b sin,  y_b = n_b cos + n_a sin
//   backward  g = dy turned back by theta,  h = g * w,  xhat = x * rstd
//             dx = rstd * (h - xhat * mean(h * xhat)),  dw = sum g * xhat
// The backward recomputes rstd: the row is in registers for the second sum
// anyway, and one saved value per 128-element row would cost 1.6% of traffic.
//
// Everything is bound by DRAM: a row is read once into registers and written
// once. A group of `lanes` lanes shares a row and each lane owns whole pairs
// (both halves), so the rotation needs no exchange between lanes and the row
// sum is one butterfly. The elements that pass are pairs of a zero angle.
//
// Angles: one turn is 2^64, so the product of an integer position and the
// frequency in turns wraps exactly where the circle does, however far the
// position; an fp32 product at position 2^20 would be off by 0.06 radians.
#include <algorithm>
#include <mutex>
#include <map>
#include <tuple>

#include "common.cuh"
#include "ops.h"

namespace rmsn {
namespace {

// E elements of T as floats, by one load or store of E * sizeof(T) bytes.
template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };

template <typename T, int E>
struct Elems {
    using W = typename Word<E * static_cast<int>(sizeof(T))>::type;
    union U {
        W w;
        T e[E];
        __device__ U() {}
    };
    __device__ __forceinline__ static W load(const T* p) {
        W v;
        if constexpr (sizeof(W) == 16)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
        else
            v = *reinterpret_cast<const W*>(p);
        return v;
    }
    __device__ __forceinline__ static void unpack(const W& w, float* f) {
        if constexpr (sizeof(W) == 16) {
            float2 p[E / 2];
            Pack<T>::unpack2(w, p);
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = i % 2 ? p[i / 2].y : p[i / 2].x;
        } else {
            U u;
            u.w = w;
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = to_f32(u.e[i]);
        }
    }
    // each element rounded once, to nearest even
    __device__ __forceinline__ static W pack(const float* f) {
        if constexpr (sizeof(W) == 16) {
            float2 p[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) p[i] = make_float2(f[2 * i], f[2 * i + 1]);
            return Pack<T>::pack2(p);
        } else {
            U u;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if constexpr (std::is_same<T, float>::value) u.e[i] = f[i];
                else u.e[i] = Pack<T>::from_float(f[i]);
            }
            return u.w;
        }
    }
};

// inv_freq / 2 pi in units of 2^-64 turns: the 24-bit mantissa times 2^66/2pi,
// shifted by the exponent. Off by at most one unit for |inv_freq| < 2^25.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max(1, static_cast<int>((bits >> 23) & 255));
    const uint32_t m = (bits & 0x7fffffu) | ((bits & 0x7f800000u) ? 0x800000u : 0u);
    constexpr uint64_t kTwo66OverTwoPi = 0xA2F9836E4E441529ull;
    const unsigned __int128 prod = static_cast<unsigned __int128>(kTwo66OverTwoPi) * m;
    const int shift = 152 - e;
    uint64_t v;
    if (shift >= 128) v = 0;
    else if (shift >= 0) v = static_cast<uint64_t>(prod >> shift);
    else v = shift > -64 ? static_cast<uint64_t>(prod) << -shift : 0;
    return (bits >> 31) ? 0ull - v : v;
}

__device__ __forceinline__ float2 cos_sin(int64_t pos, float f, float sign) {
    const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * turns_per_position(f));
    // 2^-63: half turns
    float s, c;
    sincospif(__ll2float_rn(turn) * 1.0842021724855044e-19f, &s, &c);
    if (!isfinite(f)) s = c = f - f;  // NaN, as the product of an infinity would give
    return make_float2(c, sign * s);
}

template <int E>
struct Layout {
    static constexpr int CH = E >= 2 ? 2 : 1;  // pairs in a 16-byte word of the tables
    // Float offset of pair e of unit u: lanes of a group read consecutive
    // 16-byte words (8-byte ones when E is 1), so the reads do not conflict.
    __device__ __forceinline__ static int at(int units, int u, int e) {
        return ((e / CH) * units + u) * (2 * CH) + (e % CH) * 2;
    }
};

// The two E-element pieces of unit u: its first elements and its second.
template <int E, bool ADJ>
__device__ __forceinline__ void unit_offsets(const RopeArgs& a, int u, int& lo, int& hi) {
    const int p = u * E;
    if constexpr (ADJ) {
        lo = 2 * p;
        hi = 2 * p + E;
    } else {
        const int half = a.rot / 2;
        if (p < half) {
            lo = p;
            hi = p + half;
        } else {
            lo = a.rot + (p - half);
            hi = lo + (a.head_dim - a.rot) / 2;
        }
    }
}
// Element index of the members of pair p.
template <bool ADJ>
__device__ __forceinline__ void pair_members(const RopeArgs& a, int p, int& i, int& j) {
    const int half = a.rot / 2;
    if (ADJ) {
        i = 2 * p;
        j = i + 1;
    } else if (p < half) {
        i = p;
        j = p + half;
    } else {
        i = a.rot + (p - half);
        j = i + (a.head_dim - a.rot) / 2;
    }
}
// (first members, second members) of the unit's pairs from its two pieces.
template <int E, bool ADJ>
__device__ __forceinline__ void split_pairs(const float (&v)[2 * E], float (&f)[E], float (&s)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
        f[e] = ADJ ? v[2 * e] : v[e];
        s[e] = ADJ ? v[2 * e + 1] : v[E + e];
    }
}
template <int E, bool ADJ>
__device__ __forceinline__ void join_pairs(const float (&f)[E], const float (&s)[E], float (&v)[2 * E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
        v[ADJ ? 2 * e : e] = f[e];
        v[ADJ ? 2 * e + 1 : E + e] = s[e];
    }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
    for (int off = 16; off >= 1; off /= 2)
        if (off < lanes) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ int64_t position_of(const RopeArgs& a, int axis, int64_t batch,
                                               int64_t token) {
    const int64_t at = axis * a.ps[0] + batch * a.ps[1] + token * a.ps[2];
    return a.pos64 ? static_cast<const int64_t*>(a.pos)[at]
                   : static_cast<int64_t>(static_cast<const int32_t*>(a.pos)[at]);
}

// cos/sin of every pair of the tile's tokens into `tab` (D floats a token).
template <int E, bool ADJ>
__device__ __forceinline__ void fill_angles(const RopeArgs& a, float* tab, int64_t first,
                                            int tokens) {
    const int pairs = a.head_dim / 2, half = a.rot / 2;
    for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
        const int t = i / pairs, p = i - t * pairs;
        float2 cs = make_float2(1.f, 0.f);
        if (p < half) {
            const int64_t tok = first + t;
            const int64_t b = tok / a.length;
            cs = cos_sin(position_of(a, a.axis[p], b, tok - b * a.length), a.inv_freq[p], a.sign);
        }
        float* d = tab + t * a.head_dim + Layout<E>::at(a.units, p / E, p % E);
        d[0] = cs.x;
        d[1] = cs.y;
    }
}

// Weights of one tensor as fp32, in the order of the angle tables.
template <typename T, int E, bool ADJ>
__device__ __forceinline__ void fill_weights(const RopeArgs& a, const void* w, float* tab) {
    for (int p = threadIdx.x; p < a.head_dim / 2; p += blockDim.x) {
        int i, j;
        pair_members<ADJ>(a, p, i, j);
        float* d = tab + Layout<E>::at(a.units, p / E, p % E);
        d[0] = a.w_f32 ? static_cast<const float*>(w)[i] : to_f32(static_cast<const T*>(w)[i]);
        d[1] = a.w_f32 ? static_cast<const float*>(w)[j] : to_f32(static_cast<const T*>(w)[j]);
    }
}

template <int E>
__device__ __forceinline__ void read_table(const float* tab, int units, int u, float (&f)[E],
                                           float (&s)[E]) {
    if constexpr (E >= 2) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float4 v = *reinterpret_cast<const float4*>(tab + Layout<E>::at(units, u, e));
            f[e] = v.x;
            s[e] = v.y;
            f[e + 1] = v.z;
            s[e + 1] = v.w;
        }
    } else {
        const float2 v = *reinterpret_cast<const float2*>(tab + Layout<E>::at(units, u, 0));
        f[0] = v.x;
        s[0] = v.y;
    }
}

// One past the last element of a tensor that the call may touch (strides
// are not negative), for the checked build.
[[maybe_unused]] __device__ __forceinline__ int64_t extent_bytes(const RopeArgs& a, const RopeTensor& t,
                                                const int64_t (&s)[3], int size) {
    const int64_t batch = a.tokens / a.length;
    return ((batch - 1) * s[0] + (a.length - 1) * s[1] + (t.heads - 1) * s[2] + a.head_dim) * size;
}

constexpr int kRopeThreads = 256;

// Units a lane owns at most: head_dim / 2 pairs over 32 lanes.
template <int E> constexpr int kUnitsPerLane = E >= 4 ? 1 : kRopeMaxPairs / 32 / E;

// ------------------------------------------------------------------ forward
// A block takes `tile` tokens (or a share of the heads of one, when there are
// few tokens): the angles go to shared memory once for all heads, then each
// group of lanes takes rows (token, head).
template <typename T, int E, bool ADJ, bool NORM>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int NU = kUnitsPerLane<E>;
    using X = Elems<T, E>;
    float* tab = reinterpret_cast<float*>(rmsn_dynamic_smem);
    float* wtab = tab + a.tile * a.head_dim;  // [2][D] when NORM
    const int lane = threadIdx.x % a.lanes, group = threadIdx.x / a.lanes;
    const int groups = kRopeThreads / a.lanes;
    const int64_t first = static_cast<int64_t>(blockIdx.x / a.splits) * a.tile;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tile), a.tokens - first));
    const int heads = a.t[0].heads + a.t[1].heads;
    const int split = blockIdx.x % a.splits;
    // rows of this block: heads [h0, h1) of each of its tokens
    const int h0 = static_cast<int>(static_cast<int64_t>(heads) * split / a.splits);
    const int h1 = static_cast<int>(static_cast<int64_t>(heads) * (split + 1) / a.splits);
    const int rows = tokens * (h1 - h0);
    wait_for_prerequisite_grid();  // no global access before this
    fill_angles<E, ADJ>(a, tab, first, tokens);
    if constexpr (NORM) {
        fill_weights<T, E, ADJ>(a, a.t[0].w, wtab);
        if (a.t[1].heads > 0) fill_weights<T, E, ADJ>(a, a.t[1].w, wtab + a.head_dim);
    }
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += groups) {
        const int r = r0 + group;
        const bool live = r < rows;
        const int t = live ? r / (h1 - h0) : 0;
        int head = live ? h0 + r - t * (h1 - h0) : 0;
        const int which = head >= a.t[0].heads ? 1 : 0;
        const RopeTensor& x = a.t[which];
        if (which) head -= a.t[0].heads;
        const int64_t tok = first + t, b = tok / a.length, l = tok - b * a.length;
        const T* src = static_cast<const T*>(x.x) + b * x.xs[0] + l * x.xs[1] + head * x.xs[2];
        T* dst = static_cast<T*>(x.out) + b * x.os[0] + l * x.os[1] + head * x.os[2];
        typename X::W lo[NU], hi[NU];
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int u = lane + i * a.lanes;
            if (live && u < a.units) {
                int ol, oh;
                unit_offsets<E, ADJ>(a, u, ol, oh);
                lo[i] = X::load(src + ol);
                hi[i] = X::load(src + oh);
            }
        }
        float rs = 1.f;
        if constexpr (NORM) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (live && lane + i * a.lanes < a.units) {
                    float v[2 * E];
                    X::unpack(lo[i], v);
                    X::unpack(hi[i], v + E);
#pragma unroll
                    for (int e = 0; e < 2 * E; ++e) ss = fmaf(v[e], v[e], ss);
                }
            }
            rs = rsqrtf(lanes_sum(ss, a.lanes) / static_cast<float>(a.head_dim) + a.eps);
        }
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int u = lane + i * a.lanes;
            if (!live || u >= a.units) continue;
            float v[2 * E], f[E], s[E], c[E], n[E];
            X::unpack(lo[i], v);
            X::unpack(hi[i], v + E);
            split_pairs<E, ADJ>(v, f, s);
            if constexpr (NORM) {
                float wf[E], ws[E];
                read_table<E>(wtab + which * a.head_dim, a.units, u, wf, ws);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    f[e] = f[e] * rs * wf[e];
                    s[e] = s[e] * rs * ws[e];
                }
            }
            read_table<E>(tab + t * a.head_dim, a.units, u, c, n);
            float yf[E], ys[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                yf[e] = f[e] * c[e] - s[e] * n[e];
                ys[e] = s[e] * c[e] + f[e] * n[e];
            }
            join_pairs<E, ADJ>(yf, ys, v);
            int ol, oh;
            unit_offsets<E, ADJ>(a, u, ol, oh);
            using W = typename X::W;
            if (RMSN_OK(span_in(dst + ol, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))) &&
                            span_in(dst + oh, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))),
                        a.status)) {
                *reinterpret_cast<W*>(dst + ol) = X::pack(v);
                *reinterpret_cast<W*>(dst + oh) = X::pack(v + E);
            }
        }
    }
    allow_dependent_launch();
}

// ----------------------------------------------------------------- backward
// Persistent blocks, the first blocks0 of them on the queries and the others
// on the keys, each striding over tiles of tokens with its lanes' shares of
// dw in registers; at the end the groups' shares are added in a fixed order
// into the block's partial row. No floating-point atomics.
template <typename T, int E, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int NU = kUnitsPerLane<E>;
    using X = Elems<T, E>;
    using W = typename X::W;
    float* wtab = reinterpret_cast<float*>(rmsn_dynamic_smem);
    float* tab = wtab + a.head_dim;
    const int lane = threadIdx.x % a.lanes, group = threadIdx.x / a.lanes;
    const int groups = kRopeThreads / a.lanes;
    const int which = static_cast<int>(blockIdx.x) >= a.blocks0 ? 1 : 0;
    const RopeTensor& x = a.t[which];
    const int block = static_cast<int>(blockIdx.x) - which * a.blocks0;
    const int blocks = which ? static_cast<int>(gridDim.x) - a.blocks0 : a.blocks0;
    const int64_t tiles = (a.tokens + a.tile - 1) / a.tile;
    const float inv_d = 1.f / static_cast<float>(a.head_dim);
    float dwf[NU][E], dws[NU][E];
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) dwf[i][e] = dws[i][e] = 0.f;
    wait_for_prerequisite_grid();  // no global access before this
    fill_weights<T, E, ADJ>(a, x.w, wtab);
    for (int64_t tile = block; tile < tiles; tile += blocks) {
        const int64_t first = tile * a.tile;
        const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tile), a.tokens - first));
        const int rows = tokens * x.heads;
        __syncthreads();  // the last tile's readers are done
        fill_angles<E, ADJ>(a, tab, first, tokens);
        __syncthreads();
        for (int r0 = 0; r0 < rows; r0 += groups) {
            const int r = r0 + group;
            const bool live = r < rows;
            const int t = live ? r / x.heads : 0;
            const int head = live ? r - t * x.heads : 0;
            const int64_t tok = first + t, b = tok / a.length, l = tok - b * a.length;
            const T* src = static_cast<const T*>(x.x) + b * x.xs[0] + l * x.xs[1] + head * x.xs[2];
            const T* dys = static_cast<const T*>(x.dy) + b * x.dys[0] + l * x.dys[1] + head * x.dys[2];
            T* dst = static_cast<T*>(x.out) + b * x.os[0] + l * x.os[1] + head * x.os[2];
            W lo[NU], hi[NU], glo[NU], ghi[NU];
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const int u = lane + i * a.lanes;
                if (live && u < a.units) {
                    int ol, oh;
                    unit_offsets<E, ADJ>(a, u, ol, oh);
                    lo[i] = X::load(src + ol);
                    hi[i] = X::load(src + oh);
                    glo[i] = X::load(dys + ol);
                    ghi[i] = X::load(dys + oh);
                }
            }
            float ss = 0.f, hx = 0.f;
            float gf[NU][E], gs[NU][E];  // the gradient turned back
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const int u = lane + i * a.lanes;
                if (!live || u >= a.units) continue;
                float v[2 * E], f[E], s[E], c[E], n[E], df[E], ds[E], wf[E], ws[E];
                X::unpack(lo[i], v);
                X::unpack(hi[i], v + E);
                split_pairs<E, ADJ>(v, f, s);
                X::unpack(glo[i], v);
                X::unpack(ghi[i], v + E);
                split_pairs<E, ADJ>(v, df, ds);
                read_table<E>(tab + t * a.head_dim, a.units, u, c, n);
                read_table<E>(wtab, a.units, u, wf, ws);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    gf[i][e] = df[e] * c[e] - ds[e] * n[e];
                    gs[i][e] = ds[e] * c[e] + df[e] * n[e];
                    ss = fmaf(f[e], f[e], fmaf(s[e], s[e], ss));
                    hx = fmaf(gf[i][e] * wf[e], f[e], fmaf(gs[i][e] * ws[e], s[e], hx));
                }
            }
            ss = lanes_sum(ss, a.lanes);
            hx = lanes_sum(hx, a.lanes);
            const float rs = rsqrtf(ss * inv_d + a.eps);
            const float coef = rs * rs * (hx * inv_d);  // times x: xhat * mean(h * xhat)
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                const int u = lane + i * a.lanes;
                if (!live || u >= a.units) continue;
                float v[2 * E], f[E], s[E], wf[E], ws[E], of[E], os[E];
                X::unpack(lo[i], v);
                X::unpack(hi[i], v + E);
                split_pairs<E, ADJ>(v, f, s);
                read_table<E>(wtab, a.units, u, wf, ws);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    dwf[i][e] = fmaf(gf[i][e], f[e] * rs, dwf[i][e]);
                    dws[i][e] = fmaf(gs[i][e], s[e] * rs, dws[i][e]);
                    of[e] = rs * (gf[i][e] * wf[e] - f[e] * coef);
                    os[e] = rs * (gs[i][e] * ws[e] - s[e] * coef);
                }
                join_pairs<E, ADJ>(of, os, v);
                int ol, oh;
                unit_offsets<E, ADJ>(a, u, ol, oh);
                if (RMSN_OK(span_in(dst + ol, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))) &&
                                span_in(dst + oh, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))),
                            a.status)) {
                    *reinterpret_cast<W*>(dst + ol) = X::pack(v);
                    *reinterpret_cast<W*>(dst + oh) = X::pack(v + E);
                }
            }
        }
    }
    // the groups' shares, a half of the block's groups at a time to bound the
    // scratch (the angle table's space), added in ascending group order
    allow_dependent_launch();
    float* part = tab;  // [groups][D]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int u = lane + i * a.lanes;
        if (u >= a.units) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            int p, q;
            pair_members<ADJ>(a, u * E + e, p, q);
            part[group * a.head_dim + p] = dwf[i][e];
            part[group * a.head_dim + q] = dws[i][e];
        }
    }
    __syncthreads();
    float* row = a.partial + static_cast<int64_t>(blockIdx.x) * a.head_dim;
    for (int d = threadIdx.x; d < a.head_dim; d += kRopeThreads) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g) s += part[g * a.head_dim + d];
        if (RMSN_OK(span_in(row + d, 4, a.partial,
                            static_cast<int64_t>(gridDim.x) * a.head_dim * 4), a.status))
            row[d] = s;
    }
}

// ---------------------------------------------------------------- host side
// Widest piece (elements of one access) that every offset of the call allows.
bool fits(const void* p, const int64_t (&s)[3], int bytes, int size) {
    if (p == nullptr) return true;
    if (reinterpret_cast<uintptr_t>(p) % bytes) return false;
    for (int64_t v : s)
        if (v * size % bytes) return false;
    return true;
}
int piece_of(const RopeArgs& a, int dtype, bool adjacent) {
    const int size = dtype_size(dtype);
    for (int e : {16 / size, 8 / size, 4}) {
        if (e > 16 / size || e < 4) continue;
        bool ok = adjacent ? a.head_dim % (2 * e) == 0
                           : a.rot / 2 % e == 0 && (a.head_dim - a.rot) / 2 % e == 0;
        // an adjacent unit must not mix rotated and passing pairs' tables: it
        // does not, the tables hold every pair; only the pieces have to align
        for (const RopeTensor& t : a.t) {
            if (t.heads == 0) continue;
            ok = ok && fits(t.x, t.xs, e * size, size) && fits(t.dy, t.dys, e * size, size) &&
                 fits(t.out, t.os, e * size, size);
        }
        if (ok) return e;
    }
    return 1;
}

using KernelFn = void (*)(const RopeArgs);
template <typename T, int E>
KernelFn fwd_of(bool adjacent, bool norm) {
    if (adjacent) return norm ? &rope_fwd_kernel<T, E, true, true> : &rope_fwd_kernel<T, E, true, false>;
    return norm ? &rope_fwd_kernel<T, E, false, true> : &rope_fwd_kernel<T, E, false, false>;
}
template <typename T, int E>
KernelFn bwd_of(bool adjacent) {
    return adjacent ? &rope_bwd_kernel<T, E, true> : &rope_bwd_kernel<T, E, false>;
}
template <typename T>
KernelFn kernel_for_type(int e, bool bwd, bool adjacent, bool norm) {
    if constexpr (sizeof(T) == 2)
        if (e == 8) return bwd ? bwd_of<T, 8>(adjacent) : fwd_of<T, 8>(adjacent, norm);
    if (e == 4) return bwd ? bwd_of<T, 4>(adjacent) : fwd_of<T, 4>(adjacent, norm);
    return bwd ? bwd_of<T, 1>(adjacent) : fwd_of<T, 1>(adjacent, norm);
}
KernelFn kernel_for(int dtype, int e, bool bwd, bool adjacent, bool norm) {
    switch (dtype) {
        case RMSNORM_F32: return kernel_for_type<float>(e, bwd, adjacent, norm);
        case RMSNORM_BF16:
        case RMSNORM_BF16_W_F32: return kernel_for_type<__nv_bfloat16>(e, bwd, adjacent, norm);
        default: return kernel_for_type<__half>(e, bwd, adjacent, norm);
    }
}

void shape_of(RopeArgs* a, int e) {
    a->units = a->head_dim / 2 / e;
    a->lanes = 4;
    while (a->lanes < 32 && a->lanes < a->units) a->lanes *= 2;
}

// Shared memory of the backward: weights, then the larger of the angle table
// and the groups' shares of dw.
int bwd_smem(const RopeArgs& a) {
    return a.head_dim * 4 * (1 + std::max(a.tile, kRopeThreads / a.lanes));
}

int bwd_tile(const RopeArgs& a) {
    const int groups = kRopeThreads / a.lanes;
    int heads = 1;
    for (const RopeTensor& t : a.t)
        if (t.heads > 0) heads = std::max(heads, t.heads);
    return std::max(1, std::min(16, 4 * groups / heads));
}

}  // namespace

cudaError_t rope_fwd_launch(const DeviceInfo& dev, int dtype, bool adjacent, RopeArgs a,
                            cudaStream_t s) {
    const int e = piece_of(a, dtype, adjacent);
    shape_of(&a, e);
    const bool norm = a.t[0].w != nullptr;
    const int heads = a.t[0].heads + a.t[1].heads;
    const int groups = kRopeThreads / a.lanes;
    // about four passes of the block's groups over its rows, and no more
    // tokens than leave every SM a block; few tokens share their heads out
    a.tile = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>({16, cdiv(4 * groups, heads), a.tokens / (2 * dev.sm_count)})));
    a.splits = 1;
    const int64_t tiles = cdiv(a.tokens, a.tile);
    if (a.tile == 1)
        a.splits = static_cast<int>(std::max<int64_t>(
            1, std::min<int64_t>(cdiv(heads, groups), 2 * dev.sm_count / tiles)));
    if (tiles * a.splits > INT32_MAX) return cudaErrorInvalidValue;
    const int smem = a.head_dim * 4 * (a.tile + (norm ? 2 : 0));
    return launch_pdl(kernel_for(dtype, e, false, adjacent, norm),
                      static_cast<int>(tiles * a.splits), kRopeThreads, smem, 1, s, a);
}

int rope_bwd_max_rows(const DeviceInfo& dev) { return 3 * dev.sm_count + 2; }

cudaError_t rope_bwd_rows(const DeviceInfo& dev, int dtype, bool adjacent, const RopeArgs& in,
                          int rows[2]) {
    RopeArgs a = in;
    shape_of(&a, piece_of(a, dtype, adjacent));
    a.tile = bwd_tile(a);
    const int64_t tiles = cdiv(a.tokens, a.tile);
    // three blocks an SM, shared out by the heads of the two tensors
    const int64_t total = rope_bwd_max_rows(dev) - 2;
    const int64_t heads = a.t[0].heads + a.t[1].heads;
    rows[0] = static_cast<int>(std::max<int64_t>(1, std::min(tiles, total * a.t[0].heads / heads)));
    rows[1] = a.t[1].heads == 0
                  ? 0
                  : static_cast<int>(std::max<int64_t>(1, std::min(tiles, total * a.t[1].heads / heads)));
    return cudaSuccess;
}

cudaError_t rope_bwd_launch(const DeviceInfo& dev, int dtype, bool adjacent, RopeArgs a,
                            const int rows[2], cudaStream_t s) {
    (void)dev;
    const int e = piece_of(a, dtype, adjacent);
    shape_of(&a, e);
    a.tile = bwd_tile(a);
    a.blocks0 = rows[0];
    cudaError_t err = launch_pdl(kernel_for(dtype, e, true, adjacent, true), rows[0] + rows[1],
                                 kRopeThreads, bwd_smem(a), 1, s, a);
    if (err != cudaSuccess) return err;
    PairSum p{};
    for (int i = 0; i < 2; ++i) {
        p.part[i] = a.partial + static_cast<int64_t>(i ? rows[0] : 0) * a.head_dim;
        p.out[i] = a.t[i].dw;
        p.rows[i] = rows[i];
    }
    p.n = p.stride = a.head_dim;
    p.status = a.status;
    return pair_sum_launch(p, s);
}

}  // namespace rmsn
