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
// Everything is bound by DRAM: a row is read once and written once (16384 tokens
// of 40 bf16 heads of 128 forward, 336 MB, in 56 us: 6.0 TB/s; 32768 backward,
// 1 GB, in 152 us: 6.6 TB/s; one token of 8 sequences in 3.4 us, the launch and
// three trips to memory). A group of `lanes` lanes shares a row and each lane owns whole pairs
// (both halves), so the rotation needs no exchange between lanes and the row
// sum is one butterfly. The elements that pass are pairs too, whose values are
// taken past the rotation (a turn by zero would give the partner of an infinity
// inf * 0).
//
// Angles: one turn is 2^64, so the product of an integer position and the
// frequency in turns wraps exactly where the circle does, off by what the
// frequency's last place makes of it, |position| 2^-63 turns; an fp32 product at
// position 2^20 would be off by 0.06 radians.
#pragma once

#include "common.cuh"
#include "own_copy.cuh"
#include "rope.h"

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
    static constexpr int P = (E + 1) / 2;  // float2 values; one element leaves .y zero
    using W = typename Word<E * static_cast<int>(sizeof(T))>::type;
    union U {
        W w;
        T e[E];
        __device__ U() {}
    };
    // coherent: the output may be the input's buffer (wider words are copied ahead)
    __device__ __forceinline__ static W load(const T* p) {
        static_assert(sizeof(W) <= 4, "a single element");
        return *reinterpret_cast<const W*>(p);
    }
    __device__ __forceinline__ static void unpack(const W& w, float2 (&f)[P]) {
        if constexpr (sizeof(W) == 16) {
            Pack<T>::unpack2(w, f);
        } else {
            U u;
            u.w = w;
#pragma unroll
            for (int i = 0; i < P; ++i)
                f[i] = make_float2(to_f32(u.e[2 * i]), 2 * i + 1 < E ? to_f32(u.e[(2 * i + 1) % E]) : 0.f);
        }
    }
    // each element rounded once, to nearest even
    __device__ __forceinline__ static W pack(const float2 (&f)[P]) {
        if constexpr (sizeof(W) == 16) {
            return Pack<T>::pack2(f);
        } else {
            U u;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float v = i % 2 ? f[i / 2].y : f[i / 2].x;
                if constexpr (std::is_same<T, float>::value) u.e[i] = v;
                else u.e[i] = Pack<T>::from_float(v);
            }
            return u.w;
        }
    }
};

// inv_freq / 2 pi in units of 2^-64 turns: the 24-bit mantissa times 2^66/2pi (to 96
// bits: with 64 a frequency of 10^4 was off by 2^12 units), shifted by the exponent.
// Off by less than two units for |inv_freq| < 2^25.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max(1, static_cast<int>((bits >> 23) & 255));
    const uint32_t m = (bits & 0x7fffffu) | ((bits & 0x7f800000u) ? 0x800000u : 0u);
    constexpr uint64_t kTwo66OverTwoPi = 0xA2F9836E4E441529ull;
    constexpr uint32_t kNext = 0xFC2757D1u;  // its next 32 bits
    const uint64_t more = static_cast<uint64_t>(kNext) * m >> 32;
    const uint64_t lo = kTwo66OverTwoPi * m + more;
    const uint64_t hi = __umul64hi(kTwo66OverTwoPi, m) + (lo < more ? 1 : 0);
    const int shift = 152 - e;  // of hi:lo to the right
    uint64_t v;
    if (shift >= 64) v = shift < 128 ? hi >> (shift - 64) : 0;
    else if (shift > 0) v = (lo >> shift) | (hi << (64 - shift));
    else v = shift > -64 ? lo << -shift : 0;
    return (bits >> 31) ? 0ull - v : v;
}

// cos and sin of pos * turns, with 2^64 turns a circle. 16-bit outputs take the
// fast functions (off by 2^-20, half a step of fp16 is 2^-12).
template <typename T>
__device__ __forceinline__ float2 cos_sin(int64_t pos, uint64_t turns) {
    const int64_t at = static_cast<int64_t>(static_cast<uint64_t>(pos) * turns);
    float s, c;
    if constexpr (sizeof(T) == 2) {
        // the top 32 bits of the angle, in radians
        __sincosf(static_cast<float>(static_cast<int32_t>(at >> 32)) * 1.46291807926715968e-9f, &s, &c);
    } else {
        sincospif(__ll2float_rn(at) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    }
    return make_float2(c, s);
}

// The tables (cos and sin of a token's pairs; the weights of a pair's members)
// hold D floats: two pairs a 16-byte word, firsts before seconds, so that they
// load as the float2 values they multiply; lanes of a group read consecutive
// words and do not conflict.
// LANES, where it is positive, is the number of lanes of a group, one for each
// unit of a head; where it is below -1, minus that number, of which some may have
// no unit: lane masks, the row sum's steps and (positive) table offsets are then
// constants. (Left to run time, they and the kernel parameters reloaded for them
// made up half of the forward's instructions.) -1: any number up to 32. 0: a lane
// may own several units (single elements).
// The lanes of a group are the power of two at or above the units, or as many as
// the units where a warp then holds more groups: 5 units leave 6 groups instead of
// 4 (24489 tokens of 24 bf16 heads of 80 forward: 50.8 -> 40.0 us).
//
// A unit is the E pairs that a lane takes at once, from two pieces of E elements:
// the pairs' first elements and their second ones; where pairs are neighbours,
// each piece holds E/2 whole pairs, one piece from either half of the head. (Two
// neighbouring pieces a lane instead take half a sector with each access: 65
// against 42 us for the backward of 3760 tokens of 80 bf16 heads of 128.)
template <int E, bool ADJ>
__device__ __forceinline__ int table_at(int units, int p) {
    if constexpr (E == 1) return 2 * p;
    int u = p / E, e = p % E;
    if constexpr (ADJ && E > 1) {
        const int half = units * (E / 2), upper = p >= half;
        const int at = p - (upper ? half : 0);
        u = at / (E / 2);
        e = at % (E / 2) + (upper ? E / 2 : 0);
    }
    return ((e / 2) * units + u) * 4 + e % 2;
}
// Pair e of unit u.
template <int E, bool ADJ>
__device__ __forceinline__ int pair_at(int units, int u, int e) {
    if constexpr (ADJ && E > 1) return (u + (e < E / 2 ? 0 : units)) * (E / 2) + e % (E / 2);
    return u * E + e;
}
template <int LANES>
constexpr bool kPowerOfTwo = LANES != 0 && (LANES & (LANES - 1)) == 0;
template <int E>
constexpr int kSecond = E == 1 ? 1 : 2;  // floats from a pair's first value to its second

// The two E-element pieces of unit u.
template <int E, bool ADJ>
__device__ __forceinline__ void unit_offsets(const RopeArgs& a, int u, int& lo, int& hi) {
    const int p = u * E;
    if constexpr (ADJ) {
        lo = E == 1 ? 2 * p : p;
        hi = E == 1 ? lo + 1 : p + a.head_dim / 2;
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
// (first members, second members) of the unit's pairs from its two pieces, and
// back.
template <int E, bool ADJ>
__device__ __forceinline__ void split_pairs(const float2 (&lo)[(E + 1) / 2], const float2 (&hi)[(E + 1) / 2],
                                            float2 (&f)[(E + 1) / 2], float2 (&s)[(E + 1) / 2]) {
    constexpr int P = (E + 1) / 2;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if constexpr (ADJ && E > 1) {
            const float2 v = 2 * i < P ? lo[(2 * i) % P] : hi[(2 * i) % P];
            const float2 w = 2 * i + 1 < P ? lo[(2 * i + 1) % P] : hi[(2 * i + 1) % P];
            f[i] = make_float2(v.x, w.x);
            s[i] = make_float2(v.y, w.y);
        } else {
            f[i] = lo[i];
            s[i] = hi[i];
        }
    }
}
template <int E, bool ADJ>
__device__ __forceinline__ void join_pairs(const float2 (&f)[(E + 1) / 2], const float2 (&s)[(E + 1) / 2],
                                           float2 (&lo)[(E + 1) / 2], float2 (&hi)[(E + 1) / 2]) {
    constexpr int P = (E + 1) / 2;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if constexpr (ADJ && E > 1) {
            const float2 v = make_float2(f[i].x, s[i].x), w = make_float2(f[i].y, s[i].y);
            if (2 * i < P) lo[(2 * i) % P] = v;
            else hi[(2 * i) % P] = v;
            if (2 * i + 1 < P) lo[(2 * i + 1) % P] = w;
            else hi[(2 * i + 1) % P] = w;
        } else {
            lo[i] = f[i];
            hi[i] = s[i];
        }
    }
}

// Sum over a group's lanes, of which the caller is number `lane`.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v, int some_lanes, int lane) {
    constexpr int N = LANES > 0 ? LANES : LANES < -1 ? -LANES : 0;
    const int lanes = N > 0 ? N : some_lanes;
    if constexpr (kPowerOfTwo<N>) {
        return group_allreduce<N>(v);
    } else if (LANES == 0 || (N == 0 && (lanes & (lanes - 1)) == 0)) {
#pragma unroll
        for (int off = 16; off >= 1; off /= 2)
            if (off < lanes) v += __shfl_xor_sync(0xffffffffu, v, off);
        return v;
    } else {
        // lane i < off takes what lane i + off has, which is complete for all of
        // its residue modulo 2 off
#pragma unroll
        for (int off = 16; off >= 1; off /= 2)
            if (off < lanes) {
                const float u = __shfl_down_sync(0xffffffffu, v, off);
                if (lane + off < lanes) v += u;
            }
        return __shfl_sync(0xffffffffu, v, static_cast<int>(threadIdx.x % 32) - lane);
    }
}

// A thread's place: its group of lanes and its number in it. `on` is false for
// lanes that no group or no unit has.
struct Lane {
    int lane, group, groups;
    bool on;
};
template <int LANES>
__device__ __forceinline__ Lane lane_of(const RopeArgs& a) {
    constexpr int N = LANES > 0 ? LANES : LANES < -1 ? -LANES : 0;
    Lane p;
    const int l = threadIdx.x % 32;
    int in_warp, per_warp, lanes;
    if constexpr (N > 0) {
        in_warp = l / N;
        per_warp = 32 / N;
        lanes = N;
    } else {
        in_warp = l * a.inv_lanes >> 16;  // exact for l below 32
        per_warp = a.per_warp;
        lanes = a.lanes;
    }
    p.lane = l - in_warp * lanes;
    p.group = static_cast<int>(threadIdx.x / 32) * per_warp + in_warp;
    p.groups = kRopeThreads / 32 * per_warp;
    p.on = (kPowerOfTwo<N> || in_warp < per_warp) && (LANES >= 0 || p.lane < a.units);
    return p;
}

__device__ __forceinline__ int64_t position_at(const RopeArgs& a, int64_t at) {
    return a.pos64 ? static_cast<const int64_t*>(a.pos)[at]
                   : static_cast<int64_t>(static_cast<const int32_t*>(a.pos)[at]);
}

// Element offset of a token in a tensor with these (batch, token) strides.
__device__ __forceinline__ int64_t token_offset(const RopeArgs& a, int64_t batch, int64_t token,
                                                int64_t tok) {
    const unsigned b = static_cast<unsigned>(tok) / static_cast<unsigned>(a.length);
    return b * batch + (tok - static_cast<int64_t>(b) * a.length) * token;
}

// What a block knows of a tile of tokens: the tokens' addresses in up to four
// tensors and their positions. Two more of them than rows ahead: while the
// block's slowest warp still reads those of a tile and of the tiles of its rows
// ahead, the one after is written.
constexpr int kTensors = 4;
struct TileInfo {
    int64_t addr[kTensors][kRopeMaxTile];
    int64_t pos[RMSNORM_ROPE_MAX_AXES][kRopeMaxTile];
};
static_assert((kTensors + RMSNORM_ROPE_MAX_AXES) * kRopeMaxTile <= kRopeThreads,
              "a thread for each value");

// A block's range of tokens, split evenly, in tiles of at most a.tile tokens.
struct TileRange {
    int64_t first;
    int tokens, tile, tiles;
    __device__ __forceinline__ TileRange(const RopeArgs& a, int part, int parts) {
        first = a.tokens * part / parts;
        tokens = static_cast<int>(a.tokens * (part + 1) / parts - first);
        tiles = (tokens + a.tile - 1) / a.tile;
        tile = tiles > 0 ? (tokens + tiles - 1) / tiles : 1;
    }
    __device__ __forceinline__ int count(int i) const { return min(tile, tokens - i * tile); }
};
// A tensor's base address and its strides over (batch, token), in bytes.
struct TokenBase {
    int64_t base, batch, token;
};
__device__ __forceinline__ TokenBase token_base(const void* p, const int64_t (&s)[3], int size) {
    return {reinterpret_cast<int64_t>(p), s[0] * size, s[1] * size};
}
// This thread's value of a tile's info, to be stored once it is needed: a
// position's load is then long back. `mine`: the tensor whose tokens it does.
__device__ __forceinline__ int64_t fetch_info(const RopeArgs& a, const TileRange& range, int tile,
                                              const TokenBase& mine) {
    const int i = threadIdx.x / kRopeMaxTile, t = threadIdx.x % kRopeMaxTile;
    if (i >= kTensors + a.axes || tile >= range.tiles || t >= range.count(tile)) return 0;
    const int64_t tok = range.first + tile * range.tile + t;
    if (i < kTensors) return mine.base + token_offset(a, mine.batch, mine.token, tok);
    return position_at(a, (i - kTensors) * a.ps[0] + token_offset(a, a.ps[1], a.ps[2], tok));
}
__device__ __forceinline__ void store_info(const RopeArgs& a, TileInfo& info, int64_t v) {
    const int i = threadIdx.x / kRopeMaxTile, t = threadIdx.x % kRopeMaxTile;
    if (i < kTensors) info.addr[i][t] = v;
    else if (i < kTensors + a.axes) info.pos[i - kTensors][t] = v;
}

// A thread's pair: which one, and what turns it. Threads beyond a whole number
// of tokens' pairs have none.
struct PairOf {
    uint64_t turns;
    int pair, token, stride, axis;  // its first token of a tile, and the step
    bool has, turned, bad;
};
__device__ __forceinline__ PairOf pair_of(const RopeArgs& a) {
    PairOf p;
    const int pairs = a.head_dim / 2;
    p.stride = kRopeThreads / pairs;  // at least 2
    p.token = threadIdx.x / pairs;
    p.pair = threadIdx.x - p.token * pairs;
    p.has = p.token < p.stride;
    p.turned = p.has && p.pair < a.rot / 2;
    p.axis = p.turned ? a.axis[p.pair] : 0;
    const float f = p.turned ? a.inv_freq[p.pair] : 0.f;
    p.turns = turns_per_position(f);
    p.bad = !isfinite(f);
    return p;
}
// cos/sin of every pair of a tile's tokens into `tab` (D floats a token).
template <typename T, int E, bool ADJ>
__device__ __forceinline__ void fill_angles(const RopeArgs& a, const PairOf& p, float* tab,
                                            const TileInfo& info, int tokens) {
    if (!p.has) return;
    float* d = tab + table_at<E, ADJ>(a.units, p.pair);
#pragma unroll 2
    for (int t = p.token; t < tokens; t += p.stride) {
        float2 cs = make_float2(1.f, 0.f);
        if (p.turned) cs = cos_sin<T>(info.pos[p.axis][t], p.turns);
        if (p.bad) cs.x = cs.y = __int_as_float(0x7fc00000);  // NaN
        d[t * a.head_dim] = cs.x;
        d[t * a.head_dim + kSecond<E>] = a.sign * cs.y;
    }
}

// Weights of one tensor as fp32, in the order of the angle tables.
template <typename T, int E, bool ADJ>
__device__ __forceinline__ void fill_weights(const RopeArgs& a, const void* w, float* tab) {
    for (int p = threadIdx.x; p < a.head_dim / 2; p += kRopeThreads) {
        int i, j;
        pair_members<ADJ>(a, p, i, j);
        float* d = tab + table_at<E, ADJ>(a.units, p);
        d[0] = a.w_f32 ? static_cast<const float*>(w)[i] : to_f32(static_cast<const T*>(w)[i]);
        d[kSecond<E>] = a.w_f32 ? static_cast<const float*>(w)[j] : to_f32(static_cast<const T*>(w)[j]);
    }
}

template <int E, int LANES>
__device__ __forceinline__ void read_table(const float* tab, int some_units, int u,
                                           float2 (&f)[(E + 1) / 2], float2 (&s)[(E + 1) / 2]) {
    const int units = LANES > 0 ? LANES : some_units;
    if constexpr (E == 1) {
        const float2 v = *reinterpret_cast<const float2*>(tab + 2 * u);
        f[0] = make_float2(v.x, 0.f);
        s[0] = make_float2(v.y, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(tab + (i * units + u) * 4);
            f[i] = make_float2(v.x, v.y);
            s[i] = make_float2(v.z, v.w);
        }
    }
}

template <typename W>
__device__ __forceinline__ W slot_word(uint32_t slot) {
    if constexpr (sizeof(W) == 16) return ld_slot(slot);
    else return ld_slot_8(slot);
}

// x * c - y * s and y * c + x * s. (The negation rides on scalar multiply-adds:
// the packed form has none, and two sign flips a pair cost more.)
__device__ __forceinline__ void turn(float2 x, float2 y, float2 c, float2 s, float2& ox, float2& oy) {
    const float2 xc = __fmul2_rn(x, c), xs = __fmul2_rn(x, s);
    ox = make_float2(fmaf(-y.x, s.x, xc.x), fmaf(-y.y, s.y, xc.y));
    oy = __ffma2_rn(y, c, xs);
}

// Turns a unit's pairs; in a head that is turned in part (`some`) but those that pass:
// `passes` has a bit for each of them where pairs are neighbours, and says it of the
// whole unit of halves.
template <int E, bool ADJ>
__device__ __forceinline__ void turn_unit(bool some, unsigned passes, float2 (&f)[(E + 1) / 2],
                                          float2 (&s)[(E + 1) / 2], const float2 (&c)[(E + 1) / 2],
                                          const float2 (&n)[(E + 1) / 2]) {
    auto stays = [&](int e) { return some && (ADJ && E > 1 ? (passes >> e & 1) != 0 : passes != 0); };
#pragma unroll
    for (int i = 0; i < (E + 1) / 2; ++i) {
        float2 tf, ts;
        turn(f[i], s[i], c[i], n[i], tf, ts);
        if (!stays(2 * i)) f[i].x = tf.x, s[i].x = ts.x;
        if (!stays(2 * i + 1)) f[i].y = tf.y, s[i].y = ts.y;
    }
}

// One past the last element of a tensor that the call may touch (strides
// are not negative), for the checked build.
[[maybe_unused]] __device__ __forceinline__ int64_t extent_bytes(const RopeArgs& a, const RopeTensor& t,
                                                const int64_t (&s)[3], int size) {
    const int64_t batch = a.tokens / a.length;
    return ((batch - 1) * s[0] + (a.length - 1) * s[1] + (t.heads - 1) * s[2] + a.head_dim) * size;
}

// Units a lane owns at most: head_dim / 2 pairs over 32 lanes.
template <int E> constexpr int kUnitsPerLane = E >= 4 ? 1 : kRopeMaxPairs / 32 / E;

// Byte offsets of a lane's pieces in a head: the first one's, and the second's
// distance from it; and which of the unit's pairs pass.
template <typename T, int E, bool ADJ, int LANES>
struct Pieces {
    static constexpr int NU = LANES != 0 ? 1 : kUnitsPerLane<E>;
    int lo[NU], gap[NU];
    unsigned passes[NU];
    __device__ __forceinline__ void start(const RopeArgs& a, int lane, int lanes) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            int l, h;
            unit_offsets<E, ADJ>(a, lane + i * lanes, l, h);
            lo[i] = l * static_cast<int>(sizeof(T));
            gap[i] = (h - l) * static_cast<int>(sizeof(T));
        }
    }
    // called once the first copies are under way
    __device__ __forceinline__ void find_passing(const RopeArgs& a, int lane, int lanes) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            passes[i] = 0;
            if constexpr (ADJ && E > 1) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    passes[i] |= pair_at<E, ADJ>(a.units, lane + i * lanes, e) >= a.rot / 2 ? 1u << e : 0u;
            } else {
                passes[i] = (lane + i * lanes) * E >= a.rot / 2;
            }
        }
    }
    __device__ __forceinline__ int hop(int i) const {
        if constexpr (ADJ && LANES > 0) return E * LANES * static_cast<int>(sizeof(T));
        return gap[i];
    }
};
// Address of a head's row: strides of heads are below 2^32 bytes.
__device__ __forceinline__ uint64_t row_address(int64_t token, int head, uint32_t step) {
    return static_cast<uint64_t>(token) + static_cast<uint64_t>(static_cast<uint32_t>(head)) * step;
}

// A group's way through the rows (token, head) of a tile, groups apart.
struct RowCursor {
    int t, head;
    __device__ __forceinline__ void start(int group, int heads) {
        t = group / heads;
        head = group - t * heads;
    }
    __device__ __forceinline__ void advance(int dt, int dh, int heads) {
        t += dt;
        head += dh;
        if (head >= heads) {
            head -= heads;
            ++t;
        }
    }
};

// Both kernels are persistent: a block strides over tiles of tokens. The
// angles of the next tile are filled into the other of two tables before this
// tile's rows are worked on, so one barrier a tile is enough; each group of
// lanes takes rows (token, head). Pieces of 16 or 8 bytes are copied some rows
// ahead, across tiles, into the thread's own slots of shared memory: the next
// rows alone, in registers, do not fill DRAM's latency, and more of them would
// cost warps. With two blocks an SM, 48 KB on the way an SM (three rows of the
// forward) and 64 KB (two of the backward) did best, and more is worse again:
// 16384 tokens of 40 bf16 heads of 128 forward (336 MB) take 58 us with one row
// (four blocks an SM), 56 with three and 60 with four; the backward of 32768
// (1 GB) takes 194 us with one, 157 with two, 167 with three, 179 with four.
// A row ahead may lie as many tiles ahead, whose addresses are kept for it.

// ------------------------------------------------------------------ forward
// A token's rows are the heads of q, then those of k. With few tokens the blocks
// of a tile share out its heads.
template <typename T, int E, bool ADJ, bool NORM, int LANES>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_fwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int NU = LANES != 0 ? 1 : kUnitsPerLane<E>, P = (E + 1) / 2;
    const int lanes = LANES > 0 ? LANES : LANES < -1 ? -LANES : a.lanes, D = LANES > 0 ? 2 * E * LANES : a.head_dim;
    using X = Elems<T, E>;
    using W = typename X::W;
    constexpr bool RING = E >= 4;
    constexpr int AHEAD = RING ? kRopeFwdAhead : 1, SLOTS = AHEAD + 2;
    constexpr int RING_BYTES = RING ? kRopeFwdWords * static_cast<int>(sizeof(W)) : 0;
    __shared__ TileInfo info[SLOTS];
    float* wtab = reinterpret_cast<float*>(rmsn_dynamic_smem + RING_BYTES);  // [2][D] when NORM
    float* tabs = wtab + (NORM ? 2 * D : 0);                                 // [2][tile][D]
    const Lane me = lane_of<LANES>(a);
    const int lane = me.lane, group = me.group, groups = me.groups;

    const int part = static_cast<int>(blockIdx.x) / a.splits;
    const int split = static_cast<int>(blockIdx.x) - part * a.splits;
    const TileRange range(a, part, static_cast<int>(gridDim.x) / a.splits);
    if (range.tiles == 0) return;
    const TokenBase mine = [&] {
        const int i = threadIdx.x / kRopeMaxTile;
        const RopeTensor& x = a.t[i >= 2 ? 1 : 0];
        return i % 2 ? token_base(x.out, x.os, sizeof(T)) : token_base(x.x, x.xs, sizeof(T));
    }();
    // heads [h0, h0 + heads) of each token of either tensor
    const int qh0 = a.t[0].heads * split / a.splits, kh0 = a.t[1].heads * split / a.splits;
    const int qheads = a.t[0].heads * (split + 1) / a.splits - qh0;
    const int heads = qheads + a.t[1].heads * (split + 1) / a.splits - kh0;
    const int dt = groups / heads, dh = groups - dt * heads;
    Pieces<T, E, ADJ, LANES> at;
    at.start(a, lane, lanes);
    const float inv_d = 1.f / static_cast<float>(D);
    wait_for_prerequisite_grid();  // no global access before this

    int64_t fetched[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetched[i] = fetch_info(a, range, i, mine);
    const PairOf pair = pair_of(a);
    if constexpr (NORM) {
        fill_weights<T, E, ADJ>(a, a.t[0].w, wtab);
        if (a.t[1].heads > 0) fill_weights<T, E, ADJ>(a, a.t[1].w, wtab + D);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) store_info(a, info[i], fetched[i]);
    int64_t next_info = fetch_info(a, range, AHEAD, mine);
    __syncthreads();
    auto passes_of = [&](int tile) { return (range.count(tile) * heads + groups - 1) / groups; };
    auto info_after = [](int slot) { return slot == SLOTS - 1 ? 0 : slot + 1; };
    // The row to fetch next: of which tile, and how many passes that still has.
    RowCursor row;
    row.start(group, heads);
    int row_tile = 0, row_slot = 0, row_passes = passes_of(0);
    W lo[NU], hi[NU];
    const uint32_t ring_first = smem_u32(rmsn_dynamic_smem) + threadIdx.x * static_cast<uint32_t>(sizeof(W));
    constexpr uint32_t kPiece = kRopeThreads * sizeof(W), kRow = 2 * kPiece;
    uint32_t ring_at = ring_first;  // this pass's slots, and those of the row AHEAD of it
    auto fetch = [&](uint32_t to) {
        if (row_passes > 0) {
            if (me.on && row.t < range.count(row_tile)) {
                const bool second = row.head >= qheads;
                const uint64_t src =
                    row_address(info[row_slot].addr[second ? 2 : 0][row.t], row.head + (second ? kh0 - qheads : qh0),
                                static_cast<uint32_t>((second ? a.t[1].xs[2] : a.t[0].xs[2]) * sizeof(T)));
#pragma unroll
                for (int i = 0; i < NU; ++i)
                    if (LANES != 0 || lane + i * lanes < a.units) {
                        const uint64_t p = src + at.lo[i], p2 = p + at.hop(i);
                        if constexpr (RING) {
                            copy_own<sizeof(W)>(to, reinterpret_cast<const void*>(p), a.status);
                            copy_own<sizeof(W)>(to + kPiece, reinterpret_cast<const void*>(p2), a.status);
                        } else {
                            lo[i] = X::load(reinterpret_cast<const T*>(p));
                            hi[i] = X::load(reinterpret_cast<const T*>(p2));
                        }
                    }
            }
            row.advance(dt, dh, heads);
            if (--row_passes == 0 && ++row_tile < range.tiles) {
                row.start(group, heads);
                row_slot = info_after(row_slot);
                row_passes = passes_of(row_tile);
            }
        }
        if constexpr (RING) copies_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(ring_first + i * kRow);
    at.find_passing(a, lane, lanes);
    fill_angles<T, E, ADJ>(a, pair, tabs, info[0], range.count(0));
    int buf = 0, slot = 0, fill = AHEAD;
#pragma unroll 1
    for (int tile = 0; tile < range.tiles; ++tile, buf ^= 1) {
        const int tokens = range.count(tile);
        const float* tab = tabs + buf * a.tile * D;
        if (tile + AHEAD < range.tiles) {
            store_info(a, info[fill], next_info);
            next_info = fetch_info(a, range, tile + AHEAD + 1, mine);
            fill = info_after(fill);
        }
        __syncthreads();  // this tile's table is filled; the other one's readers are done
        if (tile + 1 < range.tiles)
            fill_angles<T, E, ADJ>(a, pair, tabs + (buf ^ 1) * a.tile * D, info[info_after(slot)],
                                   range.count(tile + 1));
        const int passes = passes_of(tile);
        RowCursor cur;
        cur.start(group, heads);
#pragma unroll 1
        for (int pass = 0; pass < passes; ++pass, cur.advance(dt, dh, heads)) {
            const bool live = me.on && cur.t < tokens, second = cur.head >= qheads;
            if constexpr (RING) {
                copies_wait<AHEAD - 1>();
                lo[0] = slot_word<W>(ring_at);
                hi[0] = slot_word<W>(ring_at + kPiece);
            }
            float2 f[NU][P], s[NU][P];
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float2 l[P], h[P];
                X::unpack(lo[i], l);
                X::unpack(hi[i], h);
                split_pairs<E, ADJ>(l, h, f[i], s[i]);
            }
            fetch(ring_at);
            if constexpr (RING) ring_at = ring_at == ring_first + (AHEAD - 1) * kRow ? ring_first : ring_at + kRow;
            if constexpr (NORM) {
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < NU; ++i)
                    if (live && (LANES != 0 || lane + i * lanes < a.units)) {
#pragma unroll
                        for (int e = 0; e < P; ++e)
                            ss = __ffma2_rn(f[i][e], f[i][e], __ffma2_rn(s[i][e], s[i][e], ss));
                    }
                const float2 rs = f2_splat(rsqrtf(lanes_sum<LANES>(ss.x + ss.y, lanes, lane) * inv_d + a.eps));
#pragma unroll
                for (int i = 0; i < NU; ++i)
                    if (live && (LANES != 0 || lane + i * lanes < a.units)) {
                        float2 wf[P], ws[P];
                        read_table<E, LANES>(wtab + (second ? D : 0), a.units, lane + i * lanes, wf, ws);
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            f[i][e] = __fmul2_rn(__fmul2_rn(f[i][e], rs), wf[e]);
                            s[i][e] = __fmul2_rn(__fmul2_rn(s[i][e], rs), ws[e]);
                        }
                    }
            }
            if (!live) continue;
            const uint64_t dst =
                row_address(info[slot].addr[second ? 3 : 1][cur.t], cur.head + (second ? kh0 - qheads : qh0),
                            static_cast<uint32_t>((second ? a.t[1].os[2] : a.t[0].os[2]) * sizeof(T)));
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (LANES == 0 && lane + i * lanes >= a.units) continue;
                auto put = [&] {
                    float2 yl[P], yh[P];
                    join_pairs<E, ADJ>(f[i], s[i], yl, yh);
                    W* dl = reinterpret_cast<W*>(dst + at.lo[i]);
                    W* dhi = reinterpret_cast<W*>(dst + at.lo[i] + at.hop(i));
                    [[maybe_unused]] const RopeTensor& x = a.t[second ? 1 : 0];
                    if (RMSN_OK(span_in(dl, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))) &&
                                    span_in(dhi, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))),
                                a.status)) {
                        *dl = X::pack(yl);
                        *dhi = X::pack(yh);
                    }
                };
                float2 c[P], n[P];
                read_table<E, LANES>(tab + cur.t * D, a.units, lane + i * lanes, c, n);
                // either kind of head down to its stores: with them behind the branch,
                // arithmetic and stores do not overlap
                if (a.rot == D) {
                    turn_unit<E, ADJ>(false, 0, f[i], s[i], c, n);
                    put();
                } else {
                    turn_unit<E, ADJ>(true, at.passes[i], f[i], s[i], c, n);
                    put();
                }
            }
        }
        slot = info_after(slot);
    }
    if constexpr (RING) copies_wait<0>();
    allow_dependent_launch();
}

// ----------------------------------------------------------------- backward
// The first blocks0 blocks take the queries and the others the keys, with
// their lanes' shares of dw in registers; at the end the groups' shares are
// added in a fixed order into the block's partial row. No floating-point
// atomics.
template <typename T, int E, bool ADJ, int LANES>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    rope_bwd_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int NU = LANES != 0 ? 1 : kUnitsPerLane<E>, P = (E + 1) / 2;
    const int lanes = LANES > 0 ? LANES : LANES < -1 ? -LANES : a.lanes, D = LANES > 0 ? 2 * E * LANES : a.head_dim;
    using X = Elems<T, E>;
    using W = typename X::W;
    constexpr bool RING = E >= 4;
    constexpr int AHEAD = RING ? kRopeBwdAhead : 1, SLOTS = AHEAD + 2;
    constexpr int RING_BYTES = RING ? kRopeBwdWords * static_cast<int>(sizeof(W)) : 0;
    __shared__ TileInfo info[SLOTS];
    float* wtab = reinterpret_cast<float*>(rmsn_dynamic_smem + RING_BYTES);
    float* tabs = wtab + D;  // [2][tile][D]
    const Lane me = lane_of<LANES>(a);
    const int lane = me.lane, group = me.group, groups = me.groups;

    const int which = static_cast<int>(blockIdx.x) >= a.blocks0 ? 1 : 0;
    const RopeTensor& x = a.t[which];
    const TileRange range(a, static_cast<int>(blockIdx.x) - which * a.blocks0,
                          which ? static_cast<int>(gridDim.x) - a.blocks0 : a.blocks0);
    const int heads = x.heads;
    const TokenBase mine = [&] {
        const int i = threadIdx.x / kRopeMaxTile;
        if (i == 0) return token_base(x.x, x.xs, sizeof(T));
        return i == 1 ? token_base(x.dy, x.dys, sizeof(T)) : token_base(x.out, x.os, sizeof(T));
    }();
    const float inv_d = 1.f / static_cast<float>(D);
    const int dt = groups / heads, dh = groups - dt * heads;
    const uint32_t x_step = static_cast<uint32_t>(x.xs[2] * sizeof(T));
    const uint32_t dy_step = static_cast<uint32_t>(x.dys[2] * sizeof(T));
    const uint32_t out_step = static_cast<uint32_t>(x.os[2] * sizeof(T));
    Pieces<T, E, ADJ, LANES> at;
    at.start(a, lane, lanes);
    float2 dwf[NU][P], dws[NU][P];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
        for (int e = 0; e < P; ++e) dwf[i][e] = dws[i][e] = make_float2(0.f, 0.f);
    }
    wait_for_prerequisite_grid();  // no global access before this

    int64_t fetched[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetched[i] = fetch_info(a, range, i, mine);
    const PairOf pair = pair_of(a);
    fill_weights<T, E, ADJ>(a, x.w, wtab);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) store_info(a, info[i], fetched[i]);
    int64_t next_info = fetch_info(a, range, AHEAD, mine);
    __syncthreads();
    // The row to fetch next: of which tile, and how many passes that still has.
    auto passes_of = [&](int tile) { return (range.count(tile) * heads + groups - 1) / groups; };
    auto info_after = [](int slot) { return slot == SLOTS - 1 ? 0 : slot + 1; };
    RowCursor row;
    row.start(group, heads);
    int row_tile = 0, row_slot = 0, row_tokens = range.tiles > 0 ? range.count(0) : 0;
    int row_passes = range.tiles > 0 ? passes_of(0) : 0;
    W lo[NU], hi[NU], glo[NU], ghi[NU];
    const uint32_t ring_first = smem_u32(rmsn_dynamic_smem) + threadIdx.x * static_cast<uint32_t>(sizeof(W));
    constexpr uint32_t kPiece = kRopeThreads * sizeof(W), kRow = 4 * kPiece;
    uint32_t ring_at = ring_first;  // this pass's slots, and those of the row AHEAD of it
    auto fetch = [&](uint32_t to) {
        if (row_passes > 0) {
            if (me.on && row.t < row_tokens) {
                const uint64_t src = row_address(info[row_slot].addr[0][row.t], row.head, x_step);
                const uint64_t dys = row_address(info[row_slot].addr[1][row.t], row.head, dy_step);
#pragma unroll
                for (int i = 0; i < NU; ++i)
                    if (LANES != 0 || lane + i * lanes < a.units) {
                        const T* p = reinterpret_cast<const T*>(src + at.lo[i]);
                        const T* q = reinterpret_cast<const T*>(dys + at.lo[i]);
                        const T* p2 = reinterpret_cast<const T*>(src + at.lo[i] + at.hop(i));
                        const T* q2 = reinterpret_cast<const T*>(dys + at.lo[i] + at.hop(i));
                        if constexpr (RING) {
                            copy_own<sizeof(W)>(to, p, a.status);
                            copy_own<sizeof(W)>(to + kPiece, p2, a.status);
                            copy_own<sizeof(W)>(to + 2 * kPiece, q, a.status);
                            copy_own<sizeof(W)>(to + 3 * kPiece, q2, a.status);
                        } else {
                            lo[i] = X::load(p);
                            hi[i] = X::load(p2);
                            glo[i] = X::load(q);
                            ghi[i] = X::load(q2);
                        }
                    }
            }
            row.advance(dt, dh, heads);
            if (--row_passes == 0 && ++row_tile < range.tiles) {
                row.start(group, heads);
                row_slot = info_after(row_slot);
                row_tokens = range.count(row_tile);
                row_passes = passes_of(row_tile);
            }
        }
        if constexpr (RING) copies_commit();
    };
    // the pass's row, once it is there
    auto take = [&](uint32_t from) {
        if constexpr (RING) {
            copies_wait<AHEAD - 1>();
            lo[0] = slot_word<W>(from);
            hi[0] = slot_word<W>(from + kPiece);
            glo[0] = slot_word<W>(from + 2 * kPiece);
            ghi[0] = slot_word<W>(from + 3 * kPiece);
        }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(ring_first + i * kRow);
    at.find_passing(a, lane, lanes);
    // fill_weights is complete: this lane's weights, in registers
    float2 wf[NU][P], ws[NU][P];
#pragma unroll
    for (int i = 0; i < NU; ++i)
        if (LANES != 0 || lane + i * lanes < a.units)
            read_table<E, LANES>(wtab, a.units, lane + i * lanes, wf[i], ws[i]);
    if (range.tiles > 0) fill_angles<T, E, ADJ>(a, pair, tabs, info[0], range.count(0));
    int buf = 0, slot = 0, fill = AHEAD;
#pragma unroll 1
    for (int tile = 0; tile < range.tiles; ++tile, buf ^= 1) {
        const int tokens = range.count(tile);
        const bool more = tile + 1 < range.tiles;
        const float* tab = tabs + buf * a.tile * D;
        if (tile + AHEAD < range.tiles) {
            store_info(a, info[fill], next_info);
            next_info = fetch_info(a, range, tile + AHEAD + 1, mine);
            fill = info_after(fill);
        }
        __syncthreads();  // this tile's table is filled; the other one's readers are done
        if (more)
            fill_angles<T, E, ADJ>(a, pair, tabs + (buf ^ 1) * a.tile * D, info[info_after(slot)], range.count(tile + 1));
        const int passes = passes_of(tile);
        RowCursor cur;
        cur.start(group, heads);
#pragma unroll 1
        for (int pass = 0; pass < passes; ++pass, cur.advance(dt, dh, heads)) {
            const bool live = me.on && cur.t < tokens;
            take(ring_at);
            W xl[NU], xh[NU];
            float2 gf[NU][P], gs[NU][P];
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                float2 l[P], h[P];
                xl[i] = lo[i];
                xh[i] = hi[i];
                X::unpack(glo[i], l);
                X::unpack(ghi[i], h);
                split_pairs<E, ADJ>(l, h, gf[i], gs[i]);
            }
            fetch(ring_at);
            if constexpr (RING) ring_at = ring_at == ring_first + (AHEAD - 1) * kRow ? ring_first : ring_at + kRow;
            float2 ss = make_float2(0.f, 0.f), hx = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (!live || (LANES == 0 && lane + i * lanes >= a.units)) continue;
                float2 l[P], h[P], f[P], s[P], c[P], n[P];
                X::unpack(xl[i], l);
                X::unpack(xh[i], h);
                split_pairs<E, ADJ>(l, h, f, s);
                read_table<E, LANES>(tab + cur.t * D, a.units, lane + i * lanes, c, n);
                if constexpr (ADJ && E > 1) {
                    if (a.rot == D) turn_unit<E, ADJ>(false, 0, gf[i], gs[i], c, n);
                    else turn_unit<E, ADJ>(true, at.passes[i], gf[i], gs[i], c, n);
                } else if (at.passes[i] == 0) {
                    // by lane, unlike the forward: 32768 tokens of 40 bf16 heads of 128
                    // take 152 us so and 154 by the kind of head
                    turn_unit<E, ADJ>(false, 0, gf[i], gs[i], c, n);
                }
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    ss = __ffma2_rn(f[e], f[e], __ffma2_rn(s[e], s[e], ss));
                    hx = __ffma2_rn(__fmul2_rn(gf[i][e], wf[i][e]), f[e],
                                    __ffma2_rn(__fmul2_rn(gs[i][e], ws[i][e]), s[e], hx));
                }
            }
            const float sum = lanes_sum<LANES>(ss.x + ss.y, lanes, lane), dot = lanes_sum<LANES>(hx.x + hx.y, lanes, lane);
            const float rs = rsqrtf(sum * inv_d + a.eps);
            const float2 rs2 = f2_splat(rs);
            // rs (h - xhat mean(h xhat)) = (g rs) w + x coef
            const float2 coef = f2_splat(-rs * rs * rs * (dot * inv_d));
            if (!live) continue;
            const uint64_t dst = row_address(info[slot].addr[2][cur.t], cur.head, out_step);
#pragma unroll
            for (int i = 0; i < NU; ++i) {
                if (LANES == 0 && lane + i * lanes >= a.units) continue;
                float2 l[P], h[P], f[P], s[P];
                X::unpack(xl[i], l);
                X::unpack(xh[i], h);
                split_pairs<E, ADJ>(l, h, f, s);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const float2 gfr = __fmul2_rn(gf[i][e], rs2), gsr = __fmul2_rn(gs[i][e], rs2);
                    dwf[i][e] = __ffma2_rn(gfr, f[e], dwf[i][e]);
                    dws[i][e] = __ffma2_rn(gsr, s[e], dws[i][e]);
                    f[e] = __ffma2_rn(gfr, wf[i][e], __fmul2_rn(f[e], coef));
                    s[e] = __ffma2_rn(gsr, ws[i][e], __fmul2_rn(s[e], coef));
                }
                join_pairs<E, ADJ>(f, s, l, h);
                W* dl = reinterpret_cast<W*>(dst + at.lo[i]);
                W* dhi = reinterpret_cast<W*>(dst + at.lo[i] + at.hop(i));
                if (RMSN_OK(span_in(dl, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))) &&
                                span_in(dhi, sizeof(W), x.out, extent_bytes(a, x, x.os, sizeof(T))),
                            a.status)) {
                    *dl = X::pack(l);
                    *dhi = X::pack(h);
                }
            }
        }
        slot = info_after(slot);
    }
    // the groups' shares, in the tables' space, added in ascending group order
    if constexpr (RING) copies_wait<0>();
    allow_dependent_launch();
    float* part = tabs;  // [groups][D]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NU; ++i) {
        const int u = lane + i * lanes;
        if (!me.on || (LANES == 0 && u >= a.units)) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            int p, q;
            pair_members<ADJ>(a, pair_at<E, ADJ>(a.units, u, e), p, q);
            part[group * D + p] = e % 2 ? dwf[i][e / 2].y : dwf[i][e / 2].x;
            part[group * D + q] = e % 2 ? dws[i][e / 2].y : dws[i][e / 2].x;
        }
    }
    __syncthreads();
    float* sums = a.partial + static_cast<int64_t>(blockIdx.x) * D;
    for (int d = threadIdx.x; d < D; d += kRopeThreads) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g) s += part[g * D + d];
        if (RMSN_OK(span_in(sums + d, 4, a.partial,
                            static_cast<int64_t>(gridDim.x) * D * 4), a.status))
            sums[d] = s;
    }
}

template <typename T, int E, int LANES>
RopeFn kernel_of(bool bwd, bool adjacent, bool norm) {
    if (bwd) return adjacent ? &rope_bwd_kernel<T, E, true, LANES> : &rope_bwd_kernel<T, E, false, LANES>;
    if (adjacent)
        return norm ? &rope_fwd_kernel<T, E, true, true, LANES> : &rope_fwd_kernel<T, E, true, false, LANES>;
    return norm ? &rope_fwd_kernel<T, E, false, true, LANES> : &rope_fwd_kernel<T, E, false, false, LANES>;
}
template <typename T>
RopeFn kernel_for_type(int e, int units, int lanes, bool bwd, bool adjacent, bool norm) {
    // constant geometry for 16-byte pieces of heads of 64, 80, 96, 128 and 256, a
    // constant number of lanes for those in between
    constexpr int E = 16 / sizeof(T), U = 32 / E;
    if (e == E) {
        if (units == U) return kernel_of<T, E, U>(bwd, adjacent, norm);
        if (units == 2 * U) return kernel_of<T, E, 2 * U>(bwd, adjacent, norm);
        if (units == 4 * U) return kernel_of<T, E, 4 * U>(bwd, adjacent, norm);
        if (lanes == 40 / E) return kernel_of<T, E, 40 / E>(bwd, adjacent, norm);
        if constexpr (E == 8)
            if (lanes == 6) return kernel_of<T, E, 6>(bwd, adjacent, norm);
        if (lanes == 2 * U) return kernel_of<T, E, -2 * U>(bwd, adjacent, norm);
        return kernel_of<T, E, -1>(bwd, adjacent, norm);
    }
    if constexpr (E != 4)
        if (e == 4) return kernel_of<T, 4, -1>(bwd, adjacent, norm);
    return kernel_of<T, 1, 0>(bwd, adjacent, norm);
}
}  // namespace
}  // namespace rmsn
