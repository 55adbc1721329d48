// Rows of a mixture of experts: tokens' rows sent to the rows of their experts,
// sorted by expert, and weighted sums back, with the gradients.
//
// A row of a token has `choices` rows of its own in the sorted order, anywhere, or
// none. Each kernel goes by token, so that the token's row is moved once and the
// sorted rows once:
//   scatter     out[p_tk] = x_t                           (dispatch)
//   gather      y_t = x_t + sum_k w_tk in[p_tk]           (combine; dispatch backward without x and w)
//   gather_bwd  out[p_tk] = w_tk x_t, dw_tk = <x_t, in[p_tk]>   (combine backward, x the gradient)
// One to three operations a byte: bytes bound all three. The positions are
// what a row's loads wait for, so a thread has the pieces of several choices in
// flight. Sums are fp32 in the choices' order; a result is rounded once.
// Rows of the sorted order without a choice are zeroed by the first blocks, by
// `source` (by the last ones they were the tail of the call).
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "own_copy.cuh"
#include "rows.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
// Pieces of a lane: small ones need more of them in flight.
__host__ __device__ constexpr int scatter_pieces(int bytes) { return bytes == 16 ? 4 : 8; }
__host__ __device__ constexpr int gather_pieces(int bytes) { return bytes == 16 ? 2 : bytes == 8 ? 4 : 8; }
// by the choices taken together: 128 bytes of rows in flight
__host__ __device__ constexpr int bwd_pieces(int bytes, int kc) { return 8 / kc * (bytes >= 8 ? 16 / bytes : 4); }
constexpr int kChoices = 4;     // in flight

struct KernelArgs {
    ExpertArgs x;
    RowShape shape;
    unsigned zero_blocks;  // the first ones, which zero rows without a choice,
    int zero_runs;         // so many times 32 of them a block
    int zero_slices;       // blocks that share the same rows' bytes
    int team;               // threads of a token (gather_bwd)
    // ring: the first blocks' tokens are every main_blocks-th of main_tokens, the
    // others' `tail` each of the rest
    unsigned main_blocks;
    int64_t main_tokens;
    int tail;
};

// Zeroes those of 32 rows from row0 on that are in `todo`, by `threads` threads: where
// rows follow one another a run of them as one piece of memory (part `slice` of
// `slices`), else a warp each.
__device__ __forceinline__ void zero_found(const ExpertArgs& x, int64_t row0, unsigned todo, int size, int threads, int slice,
                                           int slices) {
    const int64_t bytes = static_cast<int64_t>(x.width) * size, stride = x.out_stride * size,
                  extent = rows_bytes(x.rows, x.out_stride, x.width, size);
    char* rows = static_cast<char*>(x.out) + row0 * stride;
    if (bytes == stride) {
        while (todo) {
            int length;
            const int from = take_run(todo, &length);
            const int64_t all = length * bytes, part = slices == 1 ? all : ceil_div(all, slices * 16) * 16,
                          at = min(part * slice, all);
            zero_span(rows + from * bytes + at, min(part, all - at), threadIdx.x, threads, x.out, extent, x.status);
        }
    } else if (slice == 0) {
        for (int i = 0; todo; todo &= todo - 1, ++i)
            if (i % (threads / 32) == static_cast<int>(threadIdx.x / 32))
                zero_span(rows + (__ffs(todo) - 1) * stride, bytes, threadIdx.x % 32, 32, x.out, extent, x.status);
    }
}

// Rows without a choice, of a block's share: all its warps look at the same 32.
__device__ __forceinline__ void zero_rows(const KernelArgs& a, int size) {
    const ExpertArgs& x = a.x;
    const int slice = blockIdx.x % a.zero_slices, block = blockIdx.x / a.zero_slices,
              blocks = a.zero_blocks / a.zero_slices;
    auto source_of = [&](int i) {  // of this lane in the block's i-th 32
        const int64_t row = (static_cast<int64_t>(i) * blocks + block) * 32 + threadIdx.x % 32;
        return i < a.zero_runs && row < x.rows ? x.source[row] : 0;
    };
    int32_t next = source_of(0);
    for (int i = 0; i < a.zero_runs; ++i) {
        const unsigned todo = __ballot_sync(0xffffffffu, next < 0);
        next = source_of(i + 1);
        if (todo) zero_found(x, (static_cast<int64_t>(i) * blocks + block) * 32, todo, size, kThreads, slice, a.zero_slices);
    }
}

template <typename T, int E, int LANES>
__global__ void __launch_bounds__(kThreads) expert_scatter_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kScatterPieces = scatter_pieces(E * sizeof(T));
    const ExpertArgs& x = a.x;
    const int lanes = LANES > 0 ? LANES : a.shape.lanes;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x < a.zero_blocks) {
        zero_rows(a, sizeof(T));
        return;
    }
    const unsigned group = group_index<kThreads>(lanes, a.zero_blocks);
    const unsigned token = group / a.shape.chunks;
    if (token >= x.tokens) return;
    const int first = (group - token * a.shape.chunks) * (lanes * kScatterPieces) + (threadIdx.x & (lanes - 1));
    const T* src = static_cast<const T*>(x.x) + token * x.x_stride + static_cast<int64_t>(first) * E;
    Piece<T, E> v[kScatterPieces];
#pragma unroll
    for (int u = 0; u < kScatterPieces; ++u) {
        v[u].zero();
        if (first + u * lanes < a.shape.pieces) v[u].load(src + u * lanes * E);
    }
    const int32_t* pos = x.position + static_cast<int64_t>(token) * x.choices;
    for (int k = 0; k < x.choices; ++k) {
        const int32_t row = pos[k];
        if (static_cast<uint32_t>(row) >= static_cast<uint32_t>(x.rows)) continue;
        T* to = static_cast<T*>(x.out) + row * x.out_stride + static_cast<int64_t>(first) * E;
#pragma unroll
        for (int u = 0; u < kScatterPieces; ++u) {
            if (first + u * lanes < a.shape.pieces &&
                RMSN_OK(span_in(to + u * lanes * E, E * sizeof(T), x.out,
                                rows_bytes(x.rows, x.out_stride, x.width, sizeof(T))),
                        x.status))
                v[u].store(to + u * lanes * E);
        }
    }
}

template <typename T, typename TW, int E, int LANES>
__global__ void __launch_bounds__(kThreads, E >= 4 ? 4 : 3) expert_gather_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kGatherPieces = gather_pieces(E * sizeof(T));
    const ExpertArgs& x = a.x;
    const int lanes = LANES > 0 ? LANES : a.shape.lanes;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const unsigned group = group_index<kThreads>(lanes);
    const unsigned token = group / a.shape.chunks;
    if (token >= x.tokens) return;
    const int first = (group - token * a.shape.chunks) * (lanes * kGatherPieces) + (threadIdx.x & (lanes - 1));
    const int64_t column = static_cast<int64_t>(first) * E;
    float sum[kGatherPieces][E];
    // whole: every piece of the lane is there, so that none has to be asked for
    auto gather = [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
        auto live = [&](int u) { return kWhole || first + u * lanes < a.shape.pieces; };
        const T* res = static_cast<const T*>(x.x) + token * x.x_stride + column;
#pragma unroll
        for (int u = 0; u < kGatherPieces; ++u) {
            Piece<T, E> v;
            v.zero();
            if (x.x != nullptr && live(u)) v.load(res + u * lanes * E);
            v.unpack(sum[u]);
        }
        const int32_t* pos = x.position + static_cast<int64_t>(token) * x.choices;
        const TW* wgt = static_cast<const TW*>(x.weights) + static_cast<int64_t>(token) * x.choices;
        for (unsigned k0 = 0; more_choices(k0, x.choices); k0 += kChoices) {
            Piece<T, E> v[kChoices][kGatherPieces];
            float w[kChoices];
            bool there[kChoices];
#pragma unroll
            for (int k = 0; k < kChoices; ++k) {
                const int32_t row = more_choices(k0 + k, x.choices) ? pos[k0 + k] : -1;
                there[k] = static_cast<uint32_t>(row) < static_cast<uint32_t>(x.rows);
                w[k] = there[k] && x.weights != nullptr ? to_f32(wgt[k0 + k]) : 1.f;
                const T* src = static_cast<const T*>(x.in) + row * x.in_stride + column;
#pragma unroll
                for (int u = 0; u < kGatherPieces; ++u) {
                    v[k][u].zero();
                    if (there[k] && live(u) &&
                        RMSN_OK(span_in(src + u * lanes * E, E * sizeof(T), x.in,
                                        rows_bytes(x.rows, x.in_stride, x.width, sizeof(T))),
                                x.status))
                        v[k][u].load(src + u * lanes * E);
                }
            }
#pragma unroll
            for (int k = 0; k < kChoices; ++k) {
                if (!there[k]) continue;  // also where its weight is infinite or NaN
#pragma unroll
                for (int u = 0; u < kGatherPieces; ++u) {
                    float f[E];
                    v[k][u].unpack(f);
#pragma unroll
                    for (int e = 0; e < E; ++e) sum[u][e] = fmaf(w[k], f[e], sum[u][e]);
                }
            }
        }
        T* to = static_cast<T*>(x.out) + token * x.out_stride + column;
#pragma unroll
        for (int u = 0; u < kGatherPieces; ++u) {
            Piece<T, E> out;
            out.pack(sum[u]);
            if (live(u) && RMSN_OK(span_in(to + u * lanes * E, E * sizeof(T), x.out,
                                           rows_bytes(x.tokens, x.out_stride, x.width, sizeof(T))),
                                   x.status))
                out.store(to + u * lanes * E);
        }
    };
    if (E * sizeof(T) < 8 && LANES > 0 && first - static_cast<int>(threadIdx.x & 31) <= a.shape.pieces - 32 * kGatherPieces)
        gather(std::true_type());
    else
        gather(std::false_type());
}

// A team of threads (a power of two, 4 to 256) takes a token and all its columns, KC
// choices at a time: a thread has U pieces of each in flight.
template <typename T, typename TW, int E, int U, int KC>
__global__ void __launch_bounds__(kThreads) expert_gather_bwd_kernel(const __grid_constant__ KernelArgs a) {
    __shared__ float part[kThreads / 32][KC];
    const ExpertArgs& x = a.x;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x < a.zero_blocks) {
        zero_rows(a, sizeof(T));
        return;
    }
    const int team = a.team, lane = threadIdx.x & (team - 1);
    const int64_t token = static_cast<int64_t>(blockIdx.x - a.zero_blocks) * (kThreads / team) + threadIdx.x / team;
    const bool live = token < x.tokens;  // the others keep the barriers company
    const T* dy = static_cast<const T*>(x.x) + token * x.x_stride;
    const int32_t* pos = x.position + token * x.choices;
    const TW* wgt = static_cast<const TW*>(x.weights) + token * x.choices;
    for (unsigned k0 = 0; more_choices(k0, x.choices); k0 += KC) {
        const int here = live ? min(KC, x.choices - static_cast<int>(k0)) : 0;
        int32_t row[KC];
        float w[KC], dot[KC];
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            row[k] = k < here ? pos[k0 + k] : -1;
            w[k] = k < here ? to_f32(wgt[k0 + k]) : 0.f;
            if (static_cast<uint32_t>(row[k]) >= static_cast<uint32_t>(x.rows)) row[k] = -1;
            dot[k] = 0.f;
        }
        const int step = team * E;
        // unsigned: behind the last of 2^31 - 1 pieces
        const unsigned pieces = live ? a.shape.pieces : 0;
        for (unsigned c = lane; c < pieces; c += team * U) {
            const int64_t column = static_cast<int64_t>(c) * E;
            const unsigned count = (pieces - c + team - 1) / team;  // of this thread's pieces
            Piece<T, E> g[U], v[KC][U];
            const T* src = dy + column;
#pragma unroll
            for (int u = 0; u < U; ++u, src += step) {
                g[u].zero();
                if (u < count) g[u].load(src);
            }
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                src = static_cast<const T*>(x.in) + row[k] * x.in_stride + column;
#pragma unroll
                for (int u = 0; u < U; ++u, src += step) {
                    v[k][u].zero();
                    if (row[k] >= 0 && u < count &&
                        RMSN_OK(span_in(src, E * sizeof(T), x.in, rows_bytes(x.rows, x.in_stride, x.width, sizeof(T))),
                                x.status))
                        v[k][u].load(src);
                }
            }
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                if (row[k] < 0) continue;
                T* to = static_cast<T*>(x.out) + row[k] * x.out_stride + column;
#pragma unroll
                for (int u = 0; u < U; ++u, to += step) {
                    float f[E], h[E];
                    g[u].unpack(h);
                    v[k][u].unpack(f);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        dot[k] = fmaf(f[e], h[e], dot[k]);
                        f[e] = w[k] * h[e];
                    }
                    Piece<T, E> out;
                    out.pack(f);
                    if (u < count &&
                        RMSN_OK(span_in(to, E * sizeof(T), x.out, rows_bytes(x.rows, x.out_stride, x.width, sizeof(T))),
                                x.status))
                        out.store(to);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < KC; ++k)
            for (int off = min(team, 32) / 2; off >= 1; off /= 2) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], off);
        float* to = x.dweights + token * x.choices + k0;
        if (team <= 32) {
#pragma unroll
            for (int k = 0; k < KC; ++k)
                if (lane == 0 && k < here && RMSN_OK(span_in(to + k, 4, x.dweights, 4 * x.tokens * x.choices), x.status))
                    to[k] = dot[k];
        } else {
            if (threadIdx.x % 32 == 0) {
#pragma unroll
                for (int k = 0; k < KC; ++k) part[threadIdx.x / 32][k] = dot[k];
            }
            __syncthreads();
            if (lane < here && RMSN_OK(span_in(to + lane, 4, x.dweights, 4 * x.tokens * x.choices), x.status)) {
                float sum = 0.f;
                for (int w = 0; w < team / 32; ++w) sum += part[threadIdx.x / 32 + w][lane];
                to[lane] = sum;
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- by a ring
// The same for rows that asynchronous copies can move (pieces of 16, 8 or 4 bytes): a
// token at a time, 16 bytes of each choice's row a thread. The pieces are copied into the thread's own slots of
// shared memory, D - 1 steps (a step: a token's KC choices of a block's columns) ahead,
// so no thread waits for another's copies. For more than four choices of some bytes:
// 16384 tokens of 8 rows of 2048 bf16 take 178 us, 221 with loads into registers (the
// kernel above), which of 4 rows take 102 as well, of 2 rows 58 instead of 67, and of
// 1000 tokens of 8 rows of 256 7 instead of 10.
struct Ring {
    static constexpr int kChoices = 8;
    static constexpr int kDepth = 3;
    static constexpr int kSlots = kChoices + 1;  // of a step: the choices, then dy
    static constexpr int kThreadBytes = kDepth * kSlots * 16;
};

constexpr int64_t kRingBytes = 8 << 20;  // of rows, from which on
constexpr int kRingMostChoices = RMSNORM_MAX_EXPERTS;

// Sums over a warp of KC values each lane has; lane l returns that of value
// l / (32 / KC).
template <int KC>
__device__ __forceinline__ float sum_of_lanes(float (&v)[KC]) {
    const unsigned lane = threadIdx.x % 32;
#pragma unroll
    for (int n = KC / 2, off = 16; n >= 1; n /= 2, off /= 2) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float give = upper ? v[k] : v[k + n], keep = upper ? v[k + n] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
    float s = v[0];
#pragma unroll
    for (int off = 16 / KC; off >= 1; off /= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

template <typename T, typename TW, int E>
__global__ void __launch_bounds__(kThreads) expert_ring_bwd_kernel(const __grid_constant__ KernelArgs a) {
    using R = Ring;
    constexpr int KC = R::kChoices, D = R::kDepth, kPiece = E * static_cast<int>(sizeof(T)), U = 16 / kPiece;  // a slot holds U pieces
    __shared__ float part[2][kThreads / 32][KC];
    const ExpertArgs& x = a.x;
    const int team = blockDim.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = team / 32;
    const uint32_t slots = smem_u32(rmsn_dynamic_smem) + threadIdx.x * 16;  // [D][slots][team]
    const int groups = (x.choices + KC - 1) / KC, chunks = static_cast<int>((static_cast<unsigned>(a.shape.pieces) + team * U - 1) / (team * U));
    wait_for_prerequisite_grid();
    allow_dependent_launch();

    // Step n of the block. A warp's lanes keep the rows (and weights) of kBatch steps at a
    // time, lane l those of choice l % KC in step l / KC, read two batches (one) ahead: a
    // step's own would be waited for, which was 1.8 us a step.
    constexpr int kBatch = 32 / KC;
    static_assert(D - 1 <= kBatch, "a step's copies are issued from this batch or the next");
    struct Step {
        int64_t token;
        int group, chunk;
    };
    const int per_token = groups * chunks;
    const bool main = blockIdx.x < a.main_blocks;
    const int64_t token0 = main ? blockIdx.x : a.main_tokens + static_cast<int64_t>(blockIdx.x - a.main_blocks) * a.tail,
                  stride = main ? a.main_blocks : 1,
                  end = main ? a.main_tokens : min(token0 + a.tail, x.tokens);
    auto step_at = [&](unsigned n) {
        const unsigned t = n / per_token, left = n - t * per_token, g = left / chunks;
        return Step{token0 + t * stride, static_cast<int>(g), static_cast<int>(left - g * chunks)};
    };
    auto next = [&](Step& s) {
        if (++s.chunk < chunks) return;
        s.chunk = 0;
        if (++s.group < groups) return;
        s.group = 0;
        s.token += stride;
    };
    auto choice_at = [&](unsigned batch) {  // of this lane; -1: none
        const Step s = step_at(batch * kBatch + lane / KC);
        const int k = s.group * KC + lane % KC;
        return s.token < end && k < x.choices ? s.token * x.choices + k : -1;
    };
    auto rows_of = [&](unsigned batch) {
        const int64_t c = choice_at(batch);
        int32_t row = -1;
        if (c >= 0) row = x.position[c];
        return row;
    };
    auto weights_of = [&](unsigned batch) {
        const int64_t c = choice_at(batch);
        TW w{};
        if (c >= 0) w = static_cast<const TW*>(x.weights)[c];
        return w;
    };
    auto valid = [&](int32_t row) { return static_cast<uint32_t>(row) < static_cast<uint32_t>(x.rows); };
    auto slot = [&](int at, int k) { return slots + (at * R::kSlots + k) * team * 16; };

    int32_t rows0 = rows_of(0), rows1 = rows_of(1), rows2 = -1;  // of this batch and the next ones
    TW weights0 = weights_of(0), weights1{};
    auto issue = [&](const Step& s, int in_batch, int at) {
        const int p0 = s.chunk * team * U + threadIdx.x;
        auto copy = [&](int k, const T* row, const void* base, int64_t rows, int64_t row_stride) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (p0 + u * team < a.shape.pieces &&
                    RMSN_OK(span_in(row + static_cast<int64_t>(p0 + u * team) * E, kPiece, base,
                                    rows_bytes(rows, row_stride, x.width, sizeof(T))),
                            x.status))
                    copy_own<kPiece>(slot(at, k) + u * kPiece, row + static_cast<int64_t>(p0 + u * team) * E, x.status);
        };
        const bool live = s.token < end;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const int32_t r = __shfl_sync(0xffffffffu, in_batch < kBatch ? rows0 : rows1, in_batch % kBatch * KC + k);
            if (live && valid(r)) copy(k, static_cast<const T*>(x.in) + r * x.in_stride, x.in, x.rows, x.in_stride);
        }
        if (live) copy(KC, static_cast<const T*>(x.x) + s.token * x.x_stride, x.x, x.tokens, x.x_stride);
        copies_commit();
    };

    Step here{token0, 0, 0}, copied = here;  // the step that is computed; the next one to be copied
#pragma unroll
    for (int j = 0; j < D - 1; ++j) {
        issue(copied, j, j);
        next(copied);
    }

    // Meanwhile the rows without a choice: a warp looks at 32, the team zeroes what
    // all of its warps found. Neighbouring runs of 32 are different blocks'.
    if (main) {
        __shared__ unsigned found[kThreads / 32];
        for (int64_t run0 = 0; (run0 * a.main_blocks + blockIdx.x) * 32 < x.rows; run0 += warps) {
            const int64_t row = ((run0 + warp) * a.main_blocks + blockIdx.x) * 32 + lane;
            const unsigned none = __ballot_sync(0xffffffffu, row < x.rows && x.source[row] < 0);
            if (lane == 0) found[warp] = none;
            __syncthreads();
            for (int w = 0; w < warps; ++w)
                zero_found(x, ((run0 + w) * a.main_blocks + blockIdx.x) * 32, found[w], sizeof(T), team, 0, 1);
            __syncthreads();
        }
    }

    float dot[KC] = {};
    int at = 0, parity = 0, in_batch = 0;
    unsigned batch = 0;
    while (here.token < end) {
        if (in_batch == 0) {
            rows2 = rows_of(batch + 2);
            weights1 = weights_of(batch + 1);
        }
        issue(copied, in_batch + D - 1, at == 0 ? D - 1 : at - 1);
        next(copied);
        copies_wait<D - 1>();
        const int p0 = here.chunk * team * U + threadIdx.x;
        const float weight = to_f32(weights0);
        // the U pieces of a slot together, as one of 16 bytes
        Piece<T, U * E> g;
        float h[U * E];
        g.w[0] = ld_slot(slot(at, KC));
        g.unpack(h);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (U > 1 && p0 + u * team >= a.shape.pieces) h[u * E + e] = 0.f;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const int32_t r = __shfl_sync(0xffffffffu, rows0, in_batch * KC + k);
            const float w = __shfl_sync(0xffffffffu, weight, in_batch * KC + k);
            if (!valid(r) || p0 >= a.shape.pieces) continue;
            Piece<T, U * E> v;
            float f[U * E];
            v.w[0] = ld_slot(slot(at, k));
            v.unpack(f);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool live = U == 1 || p0 + u * team < a.shape.pieces;
#pragma unroll
                for (int e = u * E; e < (u + 1) * E; ++e) {
                    if (live) dot[k] = fmaf(f[e], h[e], dot[k]);  // what no copy wrote may be anything
                    f[e] = w * h[e];
                }
            }
            v.pack(f);
            T* row = static_cast<T*>(x.out) + r * x.out_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                T* to = row + static_cast<int64_t>(p0 + u * team) * E;
                if (p0 + u * team < a.shape.pieces &&
                    RMSN_OK(span_in(to, kPiece, x.out, rows_bytes(x.rows, x.out_stride, x.width, sizeof(T))), x.status)) {
                    Piece<T, E> part;
                    memcpy(part.w, reinterpret_cast<const char*>(v.w) + u * kPiece, kPiece);
                    part.store(to);
                }
            }
        }
        if (here.chunk + 1 == chunks) {  // the columns are done: the team's sums
            const float s = sum_of_lanes<KC>(dot);
            if (lane % (32 / KC) == 0) part[parity][warp][lane / (32 / KC)] = s;
            __syncthreads();
            const int k = here.group * KC + threadIdx.x;
            float* to = x.dweights + here.token * x.choices + k;
            if (threadIdx.x < KC && k < x.choices &&
                RMSN_OK(span_in(to, 4, x.dweights, 4 * x.tokens * x.choices), x.status)) {
                float all = 0.f;
                for (int w = 0; w < warps; ++w) all += part[parity][w][threadIdx.x];
                *to = all;
            }
            parity ^= 1;  // written again behind the next barrier but one
#pragma unroll
            for (int i = 0; i < KC; ++i) dot[i] = 0.f;
        }
        next(here);
        at = at + 1 == D ? 0 : at + 1;
        if (++in_batch == kBatch) {
            in_batch = 0;
            ++batch;
            rows0 = rows1;
            rows1 = rows2;
            weights0 = weights1;
        }
    }
    copies_wait<0>();
}

int piece_of(const ExpertArgs& a, int dtype) {
    const int size = dtype_size(dtype);
    for (int e : {8, 4, 2}) {
        if (e * size > 16 || a.width % e) continue;
        if (piece_fits(a.x, a.x_stride, size, e) && piece_fits(a.in, a.in_stride, size, e) &&
            piece_fits(a.out, a.out_stride, size, e))
            return e;
    }
    return 1;
}

// Blocks that zero rows: 32 rows each, or as many as keep them at one wave; where rows
// are few and long, several for the same ones (some 64 KB each).
void zero_shape(const DeviceInfo& dev, int dtype, KernelArgs* a) {
    const int64_t runs = cdiv(a->x.rows, 32), most = dev.sm_count * 4;
    a->zero_runs = static_cast<int>(cdiv(runs, most));
    const int64_t blocks = a->zero_runs ? cdiv(runs, a->zero_runs) : 0,
                  slices = cdiv(static_cast<int64_t>(a->x.width) * dtype_size(dtype) * 32, 65536);
    a->zero_slices = static_cast<int>(std::max<int64_t>(1, std::min(slices, blocks ? most / blocks : 1)));
    a->zero_blocks = static_cast<unsigned>(blocks * a->zero_slices);
}

// fn(E) for the piece's width
template <typename T, typename F>
cudaError_t with_piece(int e, F fn) {
    if constexpr (sizeof(T) == 2) {
        if (e == 8) return fn(std::integral_constant<int, 8>());
    }
    if (e == 4) return fn(std::integral_constant<int, 4>());
    if (e == 2) return fn(std::integral_constant<int, 2>());
    return fn(std::integral_constant<int, 1>());
}
// fn(T, TW) for the types
template <typename F>
cudaError_t with_types(int dtype, F fn) {
    switch (dtype) {
        case RMSNORM_F32: return fn(float(), float());
        case RMSNORM_BF16: return fn(__nv_bfloat16(), __nv_bfloat16());
        case RMSNORM_F16: return fn(__half(), __half());
        case RMSNORM_BF16_W_F32: return fn(__nv_bfloat16(), float());
        default: return fn(__half(), float());
    }
}

// Lets a kernel have a ring's shared memory, once a device.
cudaError_t allow_smem(const DeviceInfo& dev, const void* fn, int bytes) {
    static std::mutex mu;
    static struct {
        int device;
        const void* fn;
    } done[1024];
    static int n = 0;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n; ++i)
        if (done[i].device == dev.device && done[i].fn == fn) return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && n < 1024) done[n++] = {dev.device, fn};
    return err;
}

template <typename T, typename TW, int E>
cudaError_t ring_launch(const DeviceInfo& dev, const KernelArgs& in, cudaStream_t s) {
    constexpr int U = 16 / (E * static_cast<int>(sizeof(T)));
    const int pieces = static_cast<int>(cdiv(in.shape.pieces, U)), team = pieces <= 32 ? 32 : pieces <= 64 ? 64 : pieces <= 128 ? 128 : kThreads;
    constexpr int kBytes = Ring::kThreadBytes;
    const auto fn = expert_ring_bwd_kernel<T, TW, E>;
    const cudaError_t err = allow_smem(dev, reinterpret_cast<const void*>(fn), kBytes * kThreads);
    if (err != cudaSuccess) return err;
    // Blocks of 256 threads two an SM, smaller ones as many more. SMs get up to 15% more
    // or less of the memory's rate than the mean: the blocks that fit at once share
    // 12/16 of the tokens out evenly, and the rest goes in small blocks to SMs as they
    // come free (16384 tokens of 8 rows of 2048 bf16: 205 us with all shared out evenly,
    // 178 so). Few tokens go in small blocks altogether (2048 of 8 rows: 39 us
    // shared out, 34 so); the first blocks then only zero rows.
    const int64_t resident = static_cast<int64_t>(dev.sm_count) * 2 * (kThreads / team);
    KernelArgs a = in;
    a.main_tokens = in.x.tokens >= 16 * resident ? in.x.tokens / 16 * 12 : 0;
    a.tail = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(2, in.x.tokens / resident)));
    a.main_blocks = static_cast<unsigned>(std::min(std::max<int64_t>(a.main_tokens, cdiv(in.x.rows, 32)), resident));
    const int grid = static_cast<int>(a.main_blocks + cdiv(in.x.tokens - a.main_tokens, a.tail));
    return launch_pdl(fn, grid, team, kBytes * team, 1, s, a);
}

}  // namespace

bool experts_fit(const ExpertArgs& a) {
    return a.tokens * cdiv(a.width, 32 * gather_pieces(2)) <= kMaxGrid;  // groups, element by element
}

cudaError_t expert_scatter_launch(const DeviceInfo& dev, int dtype, const ExpertArgs& in, cudaStream_t s) {
    KernelArgs a{in};
    const int e = piece_of(in, dtype);
    a.shape = row_shape(in.width / e, scatter_pieces(e * dtype_size(dtype)), in.tokens);
    zero_shape(dev, dtype, &a);
    const int grid = static_cast<int>(a.zero_blocks + cdiv(in.tokens * a.shape.chunks * a.shape.lanes, kThreads));
    auto go = [&](auto t) {
        using T = decltype(t);
        return with_piece<T>(e, [&](auto n) {
            return with_lanes(a.shape.lanes, [&](auto l) {
                return launch_pdl(expert_scatter_kernel<T, decltype(n)::value, decltype(l)::value>, grid, kThreads, 0, 1,
                                  s, a);
            });
        });
    };
    // a copy: the type's size alone counts
    return dtype_size(dtype) == 4 ? go(float()) : go(__nv_bfloat16());
}

cudaError_t expert_gather_launch(const DeviceInfo&, int dtype, const ExpertArgs& in, cudaStream_t s) {
    KernelArgs a{in};
    const int e = piece_of(in, dtype);
    a.shape = row_shape(in.width / e, gather_pieces(e * dtype_size(dtype)), in.tokens);
    const int grid = static_cast<int>(cdiv(in.tokens * a.shape.chunks * a.shape.lanes, kThreads));
    return with_types(dtype, [&](auto t, auto w) {
        using T = decltype(t);
        return with_piece<T>(e, [&](auto n) {
            return with_lanes(a.shape.lanes, [&](auto l) {
                return launch_pdl(expert_gather_kernel<T, decltype(w), decltype(n)::value, decltype(l)::value>, grid,
                                  kThreads, 0, 1, s, a);
            });
        });
    });
}

cudaError_t expert_gather_bwd_launch(const DeviceInfo& dev, int dtype, const ExpertArgs& in, cudaStream_t s) {
    KernelArgs a{in};
    const int e = piece_of(in, dtype);
    a.shape.pieces = in.width / e;
    const int64_t row_bytes = static_cast<int64_t>(in.width) * dtype_size(dtype);
    // a block's steps (groups of choices times chunks of columns times tokens) are counted in 32 bits
    if (in.choices > 4 && in.choices <= kRingMostChoices && e * dtype_size(dtype) >= 4 && row_bytes >= 512 &&
        in.rows * row_bytes >= kRingBytes) {
        return with_types(dtype, [&](auto t, auto w) {
            using T = decltype(t);
            return with_piece<T>(e, [&](auto n) {
                constexpr int E = decltype(n)::value;
                if constexpr (E * sizeof(T) >= 4) return ring_launch<T, decltype(w), E>(dev, a, s);
                else return cudaErrorInvalidValue;
            });
        });
    }
    zero_shape(dev, dtype, &a);
    return with_types(dtype, [&](auto t, auto w) {
        using T = decltype(t);
        return with_piece<T>(e, [&](auto n) {
            constexpr int E = decltype(n)::value;
            auto go = [&](auto kc) {
                constexpr int KC = decltype(kc)::value, U = bwd_pieces(E * sizeof(T), KC);
                a.shape = row_shape(in.width / E, U, 0);
                a.team = 4;
                while (a.team < kThreads && a.team * U < a.shape.pieces) a.team *= 2;
                const int grid = static_cast<int>(a.zero_blocks + cdiv(in.tokens, kThreads / a.team));
                return launch_pdl(expert_gather_bwd_kernel<T, decltype(w), E, U, KC>, grid, kThreads, 0, 1, s, a);
            };
            if (in.choices == 1) return go(std::integral_constant<int, 1>());
            if (in.choices == 2) return go(std::integral_constant<int, 2>());
            return go(std::integral_constant<int, 4>());
        });
    });
}

}  // namespace rmsn
