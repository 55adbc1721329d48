// Device helpers of the operators that move rows by an index: pieces of a row
// (E elements that a thread moves by one access of up to 16 bytes), and items
// read through strides.
#pragma once

#include "common.cuh"
#include "rows.h"

namespace rmsn {

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using type = uint4;
};
template <>
struct Word<8> {
    using type = uint2;
};
template <>
struct Word<4> {
    using type = uint32_t;
};
template <>
struct Word<2> {
    using type = uint16_t;
};

__device__ __forceinline__ uint4 ld_stream(const uint4* p) { return ld_global_16_stream(p); }
template <typename W>
__device__ __forceinline__ W ld_stream(const W* p) {
    return *p;
}

template <typename T, int E>
struct Piece {
    static constexpr int BYTES = E * static_cast<int>(sizeof(T));
    static constexpr int WORDS = BYTES > 16 ? BYTES / 16 : 1;
    using W = typename Word<(BYTES > 16 ? 16 : BYTES)>::type;
    W w[WORDS];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = W{};
    }
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = ld_stream(reinterpret_cast<const W*>(p) + i);
    }
    // in order with this thread's other accesses (what it reads may be written)
    __device__ __forceinline__ void load_plain(const T* p) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = reinterpret_cast<const W*>(p)[i];
    }
    // through L1: others of the SM read the same
    __device__ __forceinline__ void load_shared_row(const T* p) {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                W& o = w[i];
                asm volatile("ld.global.ca.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                             : "l"(reinterpret_cast<const W*>(p) + i));
            }
        } else {
            load(p);
        }
    }
    // issued here, whatever becomes of it
    __device__ __forceinline__ void load_now(const T* p) {
        if constexpr (BYTES >= 16) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                W& o = w[i];
                asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                             : "l"(reinterpret_cast<const W*>(p) + i));
            }
        } else {
            load_plain(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) reinterpret_cast<W*>(p)[i] = w[i];
    }
    // not to be kept in L2
    __device__ __forceinline__ void store_streamed(T* p) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) __stcs(reinterpret_cast<W*>(p) + i, w[i]);
    }
    __device__ __forceinline__ void unpack(float (&f)[E]) const {
        if constexpr (sizeof(T) == 2 && E % 2 == 0) {
            uint32_t u[E / 2];
            memcpy(u, w, BYTES);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 v = Pack<T>::word_to_f2(u[i]);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        } else {
            T t[E];
            memcpy(t, w, BYTES);
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = to_f32(t[i]);
        }
    }
    __device__ __forceinline__ void pack(const float (&f)[E]) {
        if constexpr (sizeof(T) == 2 && E % 2 == 0) {
            uint32_t u[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) u[i] = Pack<T>::pack2(f[2 * i], f[2 * i + 1]);
            memcpy(w, u, BYTES);
        } else if constexpr (sizeof(T) == 2) {
            T t = Pack<T>::from_float(f[0]);
            memcpy(w, &t, BYTES);
        } else {
            memcpy(w, f, BYTES);
        }
    }
};

// The number at item i.
__device__ __forceinline__ int64_t id_at(const KeySource& k, unsigned i) {
    int64_t at;
    if (k.inner >= k.n) {
        at = i * k.stride_inner;
    } else {
        const unsigned o = i / k.inner;
        at = o * k.stride_outer + (i - o * k.inner) * k.stride_inner;
    }
    return k.ids_64 ? static_cast<const int64_t*>(k.ids)[at] : static_cast<const int32_t*>(k.ids)[at];
}
__device__ __forceinline__ uint32_t key_at(const KeySource& k, unsigned i) {
    const int64_t id = id_at(k, i);
    return id >= 0 && id < k.limit && id != k.skip ? static_cast<uint32_t>(id) : static_cast<uint32_t>(k.limit);
}

// Bytes from the first to behind the last of n rows.
__device__ __forceinline__ int64_t rows_bytes(int64_t n, int64_t stride, int64_t width, int size) {
    return ((n - 1) * stride + width) * size;
}

// Zeroes `bytes` bytes from p (aligned to 2) by `threads` threads: 16 bytes a store
// between the first and the last boundary.
__device__ __forceinline__ void zero_span(char* p, int64_t bytes, int thread, int threads, const void* base,
                                          int64_t extent, int* status) {
    if (!RMSN_OK(span_in(p, bytes, base, extent), status)) return;
    const int64_t head = min(static_cast<int64_t>(-reinterpret_cast<uintptr_t>(p) & 15), bytes);
    const int64_t words = (bytes - head) / 16, tail = head + words * 16;
    for (int64_t i = 2 * thread; i < head; i += 2 * threads) *reinterpret_cast<uint16_t*>(p + i) = 0;
    for (int64_t i = thread; i < words; i += threads)
        *reinterpret_cast<uint4*>(p + head + i * 16) = make_uint4(0, 0, 0, 0);
    for (int64_t i = tail + 2 * thread; i < bytes; i += 2 * threads) *reinterpret_cast<uint16_t*>(p + i) = 0;
}

// The first run of neighbouring bits that are set: where it starts, and how long;
// cleared in `bits`.
__device__ __forceinline__ int take_run(unsigned& bits, int* length) {
    const int from = __ffs(bits) - 1;
    const unsigned rest = bits >> from;
    *length = rest == 0xffffffffu ? 32 : __ffs(~rest) - 1;
    bits &= *length == 32 ? 0u : ~(((1u << *length) - 1) << from);
    return from;
}

// The group of lanes a thread of a block of THREADS belongs to, counted over the grid
// from its first_block on.
template <int THREADS>
__device__ __forceinline__ unsigned group_index(int lanes, unsigned first_block = 0) {
    return (blockIdx.x - first_block) * (THREADS / lanes) + threadIdx.x / lanes;
}

// ------------------------------------------------------------ host geometry
// Groups of lanes (a power of two, up to a warp) that move a row's pieces, up to U
// pieces a lane and chunk.
struct RowShape {
    int pieces;  // of a row
    int lanes;   // of a group
    int chunks;  // of a row
};
// Few lanes with many pieces each move more at a time, but only once there are warps
// enough to fill the device: 5835 rows of 51 pieces take 6.6 us by 32 lanes and 10.0 by
// 8, 33660 rows of 32 pieces 6.8 and 5.7.
constexpr int64_t kFullWarps = kSms * 48;
inline RowShape row_shape(int pieces, int u, int64_t rows) {
    RowShape r{pieces, 1, 1};
    while (r.lanes < 32 && r.lanes < pieces && (r.lanes * u < pieces || rows * r.lanes / 32 < kFullWarps)) r.lanes *= 2;
    r.chunks = static_cast<int>(cdiv(pieces, static_cast<int64_t>(r.lanes) * u));
    return r;
}
// Calls fn with the group's lanes: a constant where they are a whole warp, whose
// pieces then lie at constant offsets.
template <typename F>
cudaError_t with_lanes(int lanes, F fn) {
    return lanes == 32 ? fn(std::integral_constant<int, 32>()) : fn(std::integral_constant<int, 0>());
}
// Whether rows of `bytes` pieces can be moved from p.
inline bool piece_fits(const void* p, int64_t stride, int size, int e) {
    const int bytes = e * size > 16 ? 16 : e * size;
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * size % bytes == 0);
}

}  // namespace rmsn
