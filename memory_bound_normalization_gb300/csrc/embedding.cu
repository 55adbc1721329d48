// Embedding lookup with a scale, and its gradient by sorted tokens.
//
// Forward: y_i = scale * table[id_i], rows of zeros for ids outside the table. A
// group of lanes moves a piece of a row each; bytes alone (the rows that are hit,
// in; every token's, out).
//
// Backward: row v of the gradient is scale * the sum of dy_i over the tokens with
// id v, in fp32 and in an order that the sizes and the alignment alone fix. The tokens are sorted
// by id (sort.cu); the sorted list is cut in segments of a few tokens. A group of
// lanes adds up its columns of a segment, a block those of neighbouring segments. Runs
// of one id that lie in a segment are written to their row at once; a run over
// several is joined, in the segments' order, through shared memory, and one over
// several blocks through shares in the workspace, which embedding_join_kernel adds
// in the blocks' order. So a token that fills half of the batch is as much work for
// each group as any other, and nothing depends on which block is first.
// Bytes: dy once, the whole gradient once. Most of them are the rows without a token,
// which blocks of their own zero: the last rows beside the sort, whether they have a
// token or not, the others beside the sums, by the sort's marks.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 8;        // rows of dy in flight a lane
constexpr int kZeroBytes = 16384;  // of a warp
constexpr int kMaxSpan = 2048;     // sorted tokens of a block

struct FwdKernelArgs {
    KeySource k;
    const void* table;
    void* y;
    int64_t table_stride, y_stride;
    RowShape shape;
    float scale;
    int streamed;  // y is larger than L2 keeps until it is read
    int* status;
};

// Pieces of a lane: 8 where they are small or rows are many and end early in a second
// chunk of 4, else 4.
constexpr int kFwdPieces = 8;
bool fwd_by_four(int e, int pieces, int64_t rows) {
    const int64_t by4 = cdiv(pieces, 32 * 4), by8 = cdiv(pieces, 32 * 8);
    return e >= 4 && (2 * by8 > by4 || rows * by4 < kFullWarps);
}


template <typename TT, typename TA, int E, int U, int LANES>
__global__ void __launch_bounds__(kThreads) embedding_fwd_kernel(const __grid_constant__ FwdKernelArgs a) {
    const int lanes = LANES > 0 ? LANES : a.shape.lanes;
    const unsigned group = group_index<kThreads>(lanes);
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const unsigned item = group / a.shape.chunks;
    if (item >= a.k.n) return;
    const int first = (group - item * a.shape.chunks) * (lanes * U) + (threadIdx.x & (lanes - 1));
    const uint32_t row = key_at(a.k, item);
    const bool there = row < a.k.limit;
    const TT* src = static_cast<const TT*>(a.table) + row * a.table_stride + static_cast<int64_t>(first) * E;
    TA* dst = static_cast<TA*>(a.y) + item * a.y_stride + static_cast<int64_t>(first) * E;
    const float scale = there ? a.scale : 0.f;  // a row of zeros, also where the scale is infinite or NaN
    // whole: every piece of the lane is there, so that none has to be asked for
    auto look_up = [&](auto whole) {
        auto live = [&](int u) { return decltype(whole)::value || first + u * lanes < a.shape.pieces; };
        Piece<TT, E> in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            in[u].zero();
            // a frequent token's row is in many warps' hands: from L2 alone, 22400 tokens of 22
            // rows of 520 fp32 waited for the few lines that hold them (14.8 us)
            if (there && live(u) &&
                RMSN_OK(span_in(src + u * lanes * E, E * sizeof(TT), a.table,
                                rows_bytes(a.k.limit, a.table_stride, static_cast<int64_t>(a.shape.pieces) * E,
                                           sizeof(TT))),
                        a.status))
                in[u].load_shared_row(src + u * lanes * E);
        }
        asm volatile("" ::: "memory");  // every load before the first store
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[E];
            in[u].unpack(f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] *= scale;
            Piece<TA, E> out;
            out.pack(f);
            TA* to = dst + u * lanes * E;
            if (!live(u) || !RMSN_OK(span_in(to, E * sizeof(TA), a.y,
                                             rows_bytes(a.k.n, a.y_stride, static_cast<int64_t>(a.shape.pieces) * E,
                                                        sizeof(TA))),
                                     a.status))
                continue;
            if (a.streamed) out.store_streamed(to);
            else out.store(to);
        }
    };
    if (E < 4 && LANES > 0 && first - static_cast<int>(threadIdx.x & 31) <= a.shape.pieces - 32 * U)
        look_up(std::true_type());
    else
        look_up(std::false_type());
}

struct BwdKernelArgs {
    KeySource k;           // few tokens: sorted by every block
    const KeyItem* pairs;  // sorted
    const uint8_t* present;
    const void* dy;
    void* grad;
    float* partial;  // [spans][2][width]: of the run that comes in, of the one that goes out
    int64_t dy_stride, grad_stride;
    int64_t rows;  // of the table
    uint32_t n, limit;
    RowShape shape;
    unsigned spans;       // of the sorted tokens: a block's share
    unsigned sum_blocks;  // blocks that add; the others zero rows
    int segment;          // tokens of a group
    int span;             // tokens of a block
    int64_t zero_to;  // rows before it are zeroed beside the sums where they have no token
    int zero_rows, zero_slices;  // rows of a warp's share (whole 32s, if more), shares of a row
    int accumulate;
    float scale;
    int* status;
};

template <int E, int U>
struct Columns {
    float v[U][E];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
    }
    __device__ __forceinline__ void add(const Columns& o) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] += o.v[u][e];
    }
};

// Row v's columns: scale * sum, on top of what is there with accumulate.
template <typename TG, int E, int U>
__device__ __forceinline__ void put_row(const BwdKernelArgs& a, uint32_t v, int piece, const Columns<E, U>& sum) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = piece + u * a.shape.lanes;
        if (p >= a.shape.pieces) continue;
        TG* to = static_cast<TG*>(a.grad) + v * a.grad_stride + static_cast<int64_t>(p) * E;
        if (!RMSN_OK(span_in(to, E * sizeof(TG), a.grad,
                             rows_bytes(a.rows, a.grad_stride, static_cast<int64_t>(a.shape.pieces) * E, sizeof(TG))),
                     a.status))
            continue;
        Piece<TG, E> out;
        float f[E];
        if (a.accumulate) {
            out.load_plain(to);
            out.unpack(f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = fmaf(a.scale, sum.v[u][e], f[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = a.scale * sum.v[u][e];
        }
        out.pack(f);
        out.store(to);
    }
}

template <int E>
__device__ __forceinline__ float* partial_at(const BwdKernelArgs& a, unsigned span, int slot, int piece) {
    return a.partial + (static_cast<int64_t>(span) * 2 + slot) * a.shape.pieces * E + static_cast<int64_t>(piece) * E;
}
template <int E, int U>
__device__ __forceinline__ void put_partial(const BwdKernelArgs& a, unsigned span, int slot, int piece,
                                            const Columns<E, U>& sum) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = piece + u * a.shape.lanes;
        if (p >= a.shape.pieces) continue;
        float* to = partial_at<E>(a, span, slot, p);
        if (!RMSN_OK(span_in(to, E * 4, a.partial, static_cast<int64_t>(a.spans) * 8 * a.shape.pieces * E), a.status))
            continue;
        Piece<float, E> out;
        out.pack(sum.v[u]);
        out.store(to);
    }
}

// What a group's tokens leave for the block to join.
constexpr int kHead = 1;     // the sum of a run that began before them
constexpr int kTail = 2;     // the sum of a run that goes on behind them
constexpr int kThrough = 4;  // both: one run fills them (its sum is the head)

// The tokens of a span in shared memory: key [span + 2] (the token before, ours, the
// next), item [span].
struct Staged {
    uint32_t* key;
    int32_t* item;
    int count;
};
constexpr uint32_t kNoKey = 0xffffffffu;

__device__ __forceinline__ Staged stage(const BwdKernelArgs& a, unsigned span) {
    Staged t;
    t.key = reinterpret_cast<uint32_t*>(rmsn_dynamic_smem);
    t.item = reinterpret_cast<int32_t*>(t.key + a.span + 2);
    const uint32_t first = span * static_cast<uint32_t>(a.span);
    t.count = static_cast<int>(min(static_cast<uint32_t>(a.span), a.n - first));
    constexpr int kAhead = 4;  // of a thread's tokens, read together
    for (int i0 = threadIdx.x; i0 < t.count + 2; i0 += kAhead * kThreads) {
        uint2 pair[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            const int64_t at = static_cast<int64_t>(first) + i - 1;
            pair[j] = make_uint2(kNoKey, 0);
            if (i < t.count + 2 && at >= 0 && at < a.n) pair[j] = *reinterpret_cast<const uint2*>(a.pairs + at);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            if (i < t.count + 2) t.key[i] = pair[j].x;
            if (i > 0 && i <= t.count) t.item[i - 1] = static_cast<int32_t>(pair[j].y);
        }
    }
    __syncthreads();
    return t;
}

template <typename TA, typename TG, int E, int U>
__device__ __forceinline__ void add_tokens(const BwdKernelArgs& a, const Staged& t, unsigned span, int slice) {
    __shared__ float held[2][U * E][kThreads];  // heads and tails, a column a thread
    __shared__ bool state[kThreads];  // a group's: the scan's second part
    const uint32_t* key = t.key;
    const int32_t* item = t.item;
    const int count = t.count;
    const int lanes = a.shape.lanes, group = threadIdx.x / lanes, groups = kThreads / lanes;
    const int piece = slice * lanes * U + (threadIdx.x & (lanes - 1));
    const int from = group * a.segment, to = min(from + a.segment, count);
    Columns<E, U> sum;
    sum.clear();
    int left = 0;
    auto put = [&](int slot, const Columns<E, U>& c) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) held[slot][u * E + e][threadIdx.x] = c.v[u][e];
    };
    auto held_by = [&](int slot, int g) {
        Columns<E, U> c;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) c.v[u][e] = held[slot][u * E + e][threadIdx.x + (g - group) * lanes];
        return c;
    };
    if (from < to) {
        uint32_t run = key[from + 1];
        bool came_in = key[from] == run;
        const TA* dy = static_cast<const TA*>(a.dy);
        for (int i = from; i < to; i += kRun) {
            Piece<TA, E> in[kRun][U];
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const bool live = i + j < to && key[i + j + 1] < a.limit;
                const TA* row = dy + (live ? item[i + j] : 0) * a.dy_stride;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int p = piece + u * lanes;
                    in[j][u].zero();
                    if (live && p < a.shape.pieces &&
                        RMSN_OK(span_in(row + static_cast<int64_t>(p) * E, E * sizeof(TA), a.dy,
                                        rows_bytes(a.n, a.dy_stride, static_cast<int64_t>(a.shape.pieces) * E,
                                                   sizeof(TA))),
                                a.status))
                        in[j][u].load(row + static_cast<int64_t>(p) * E);
                }
            }
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                if (i + j >= to) break;
                const uint32_t k = key[i + j + 1];
                if (k != run) {
                    if (came_in) {
                        put(0, sum);
                        left |= kHead;
                    } else if (run < a.limit) {
                        put_row<TG, E, U>(a, run, piece, sum);
                    }
                    run = k;
                    came_in = false;
                    sum.clear();
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[E];
                    in[j][u].unpack(f);
#pragma unroll
                    for (int e = 0; e < E; ++e) sum.v[u][e] += f[e];
                }
            }
        }
        const bool goes_on = key[to + 1] == run;
        if (came_in) {
            put(0, sum);
            left |= goes_on ? kHead | kThrough : kHead;
        } else if (goes_on) {
            put(1, sum);
            left |= kTail;
        } else if (run < a.limit) {
            put_row<TG, E, U>(a, run, piece, sum);
        }
    }
    // A run over several groups belongs to the group where it begins (the one that came
    // into the block, to the first), which needs the heads of the groups behind as far
    // as the run goes: a scan from behind, sum and "goes on to the block's end".
    Columns<E, U> heads;  // from this group on
    bool on;
    {
        const int member = threadIdx.x & (lanes - 1);
        heads.clear();
        if (left & kHead) heads = held_by(0, group);
        on = (left & kThrough) != 0;
        if (member == 0) state[group] = on;
        if (__syncthreads_or(on)) {
            for (int d = 1; d < groups; d *= 2) {
                const bool more = on && group + d < groups;
                Columns<E, U> next;
                bool next_on = on;
                if (more) {
                    next = held_by(0, group + d);
                    next_on = state[group + d] != 0;
                }
                __syncthreads();
                if (more) {
                    heads.add(next);
                    on = next_on;
                    put(0, heads);
                    if (member == 0) state[group] = on;
                }
                __syncthreads();
            }
        }
    }
    if (group == 0 && (left & kHead) && key[1] < a.limit) put_partial<E, U>(a, span, 0, piece, heads);
    if ((left & kTail) && key[to] < a.limit) {
        Columns<E, U> all = held_by(1, group);
        bool goes_on = true;
        if (group + 1 < groups) {
            all.add(held_by(0, group + 1));
            goes_on = state[group + 1] != 0;
        }
        if (goes_on) put_partial<E, U>(a, span, 1, piece, all);
        else put_row<TG, E, U>(a, key[to], piece, all);
    }
}

// Zeroes rows without a token: a warp takes some 16 KB, rows or a part of a long one.
// absent(row0, rows): those of up to 32 rows from row0 on that have none, a bit each.
template <typename TG, int E, typename Absent>
__device__ __forceinline__ void zero_share(const BwdKernelArgs& a, Absent absent) {
    const int64_t unit = static_cast<int64_t>(blockIdx.x - a.sum_blocks) * (kThreads / 32) + threadIdx.x / 32;
    if (unit >= ceil_div(a.zero_to, a.zero_rows) * a.zero_slices) return;
    const int lane = threadIdx.x % 32;
    const int64_t part = a.zero_slices == 1 ? unit : unit / a.zero_slices;
    const int slice = static_cast<int>(unit - part * a.zero_slices);
    const int64_t width = static_cast<int64_t>(a.shape.pieces) * E, row_bytes = width * static_cast<int>(sizeof(TG)),
                  stride_bytes = a.grad_stride * static_cast<int>(sizeof(TG)),
                  extent = rows_bytes(a.rows, a.grad_stride, width, sizeof(TG));
    const bool dense = a.grad_stride == width && a.zero_slices == 1;  // neighbouring rows are one piece of memory
    const int64_t end = min((part + 1) * a.zero_rows, a.zero_to);
    for (int64_t row0 = part * a.zero_rows; row0 < end; row0 += 32) {
        unsigned todo = absent(row0, static_cast<int>(min(end - row0, static_cast<int64_t>(32))));
        char* rows = static_cast<char*>(a.grad) + row0 * stride_bytes;
        while (todo) {
            if (dense) {
                int length;
                const int from = take_run(todo, &length);
                zero_span(rows + from * row_bytes, length * row_bytes, lane, 32, a.grad, extent, a.status);
            } else {
                const int r = __ffs(todo) - 1;
                todo &= todo - 1;
                const int64_t from = static_cast<int64_t>(slice) * kZeroBytes;
                zero_span(rows + r * stride_bytes + from, min(static_cast<int64_t>(kZeroBytes), row_bytes - from), lane, 32,
                          a.grad, extent, a.status);
            }
        }
    }
}
__device__ __forceinline__ auto by_marks(const BwdKernelArgs& a) {
    return [&a](int64_t row0, int rows) {
        const int lane = threadIdx.x % 32;
        return __ballot_sync(0xffffffffu, lane < rows && a.present[row0 + lane] == 0);
    };
}

template <typename TA, typename TG, int E, int U>
__global__ void __launch_bounds__(kThreads, 3) embedding_sum_kernel(const __grid_constant__ BwdKernelArgs a) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x >= a.sum_blocks) {
        zero_share<TG, E>(a, by_marks(a));
        return;
    }
    const unsigned span = blockIdx.x / a.shape.chunks;
    add_tokens<TA, TG, E, U>(a, stage(a, span), span, static_cast<int>(blockIdx.x - span * a.shape.chunks));
}

// Up to kThreads tokens: all in one launch. Every block sorts them, a token a thread
// whose place is the count of those before it.
template <typename TA, typename TG, int E, int U>
__global__ void __launch_bounds__(kThreads, 3) embedding_few_kernel(const __grid_constant__ BwdKernelArgs a) {
    __shared__ uint32_t raw[kThreads];
    __shared__ uint32_t key[kThreads + 2];
    __shared__ int32_t item[kThreads];
    const int i = threadIdx.x, n = static_cast<int>(a.n);
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const uint32_t mine = i < n ? key_at(a.k, i) : kNoKey;
    raw[i] = mine;
    __syncthreads();
    if (blockIdx.x >= a.sum_blocks) {
        zero_share<TG, E>(a, [&](int64_t row0, int rows) {
            unsigned there = 0;
            for (int j = threadIdx.x % 32; j < n; j += 32) {
                const int64_t r = static_cast<int64_t>(raw[j]) - row0;
                if (r >= 0 && r < rows) there |= 1u << r;
            }
            return ~__reduce_or_sync(0xffffffffu, there) & (rows >= 32 ? 0xffffffffu : (1u << rows) - 1);
        });
        return;
    }
    int place = 0;
#pragma unroll 16
    for (int j = 0; j < n; ++j) place += raw[j] < mine + (j < i) ? 1 : 0;
    if (i < n) {
        key[place + 1] = mine;
        item[place] = i;
    }
    if (i == 0) key[0] = key[n + 1] = kNoKey;
    __syncthreads();
    add_tokens<TA, TG, E, U>(a, Staged{key, item, n}, 0, static_cast<int>(blockIdx.x));
}

// Runs that cross blocks: the group that takes the span where one begins adds the
// spans' shares in order, eight and eight.
template <typename TG, int E, int U>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const __grid_constant__ BwdKernelArgs a) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    constexpr int kAhead = 8;
    const unsigned group = group_index<kThreads>(a.shape.lanes);
    const unsigned span = group / a.shape.chunks;
    const int piece = (group - span * a.shape.chunks) * (a.shape.lanes * U) + (threadIdx.x & (a.shape.lanes - 1));
    if (span + 1 >= a.spans) return;
    const uint32_t first = span * static_cast<uint32_t>(a.span), next = first + a.span;
    // the first ids of the next spans, read before those of the last ones are looked at
    uint32_t begins[kAhead];
    auto read_begins = [&](unsigned s) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            begins[j] = s + j < a.spans ? a.pairs[(s + j) * static_cast<uint32_t>(a.span)].key : 0xffffffffu;
    };
    const uint32_t run = a.pairs[next - 1].key, begin = a.pairs[first].key,
                   before = first > 0 ? a.pairs[first - 1].key : 0xffffffffu;
    read_begins(span + 1);
    if (run >= a.limit || begins[0] != run || (begin == run && before == run)) return;  // ends here, or began before
    Columns<E, U> sum;
    auto load = [&](Columns<E, U>& c, unsigned s, int slot, bool live) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = piece + u * a.shape.lanes;
            Piece<float, E> in;
            in.zero();
            if (live && p < a.shape.pieces &&
                RMSN_OK(span_in(partial_at<E>(a, s, slot, p), E * 4, a.partial,
                                static_cast<int64_t>(a.spans) * 8 * a.shape.pieces * E),
                        a.status))
                in.load_now(partial_at<E>(a, s, slot, p));
            in.unpack(c.v[u]);
        }
    };
    load(sum, span, 1, true);
    for (unsigned s = span + 1;; s += kAhead) {
        // a span has a share where it starts with this id; what others hold is not used
        bool live[kAhead];
        Columns<E, U> in[kAhead], eight;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) live[j] = begins[j] == run;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) load(in[j], s + j, 0, s + j < a.spans);
        read_begins(s + kAhead);
        eight.clear();
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            // selected, not branched on: the loads stay together
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) eight.v[u][e] += live[j] ? in[j].v[u][e] : 0.f;
        }
        sum.add(eight);
        if (!live[kAhead - 1]) break;
    }
    put_row<TG, E, U>(a, run, piece, sum);
}

// Widest piece (elements) of rows of `width` of two types: 16 bytes of the wider one,
// so that a group's accesses are dense in both.
int piece_of(const void* p, int64_t ps, int size_p, const void* q, int64_t qs, int size_q, int width) {
    for (int e : {8, 4, 2}) {
        if (e * std::max(size_p, size_q) > 16 || width % e) continue;
        if (piece_fits(p, ps, size_p, e) && piece_fits(q, qs, size_q, e)) return e;
    }
    return 1;
}

template <typename TT, typename TA>
cudaError_t fwd_typed(int e, int width, FwdKernelArgs a, cudaStream_t s) {
    auto go = [&](auto n) {
        constexpr int E = decltype(n)::value;
        auto with_pieces = [&](auto u) {
            constexpr int U = decltype(u)::value;
            a.shape = row_shape(width / E, U, a.k.n);
            const int64_t blocks = cdiv(static_cast<int64_t>(a.k.n) * a.shape.chunks * a.shape.lanes, kThreads);
            return with_lanes(a.shape.lanes, [&](auto lanes) {
                return launch_pdl(embedding_fwd_kernel<TT, TA, E, U, decltype(lanes)::value>, static_cast<int>(blocks),
                                  kThreads, 0, 1, s, a);
            });
        };
        if constexpr (E >= 4) {
            if (fwd_by_four(E, width / E, a.k.n)) return with_pieces(std::integral_constant<int, 4>());
        }
        return with_pieces(std::integral_constant<int, kFwdPieces>());
    };
    if constexpr (sizeof(TT) == 2) {
        if (e == 8) return go(std::integral_constant<int, 8>());
    }
    if (e == 4) return go(std::integral_constant<int, 4>());
    if (e == 2) return go(std::integral_constant<int, 2>());
    return go(std::integral_constant<int, 1>());
}

// Bytes of rows that are zeroed beside a sort by one cluster, and beside each launch of
// another (the last rows); the others beside the sums. Beside the join they cost more
// than they saved (32001 rows of 1000 fp32: 38 us, 34 without).
constexpr int64_t kZeroBesideSort = 48 << 20, kZeroBesidePass = 12 << 20;

// Four times the warps that fit at once. With shares of 16 KB however short the rows, 253
// tokens' gradient of 5288 rows of 2 f16 was two warps' work (107 us, 6 so), that of 10^6
// rows of 1 bf16 took 120 (9 so); by as many warps as fit at once 3000017 rows of 9 fp32
// take 60 us, by four times as many 36.
constexpr int64_t kZeroWarps = kSms * 96;

int64_t zero_blocks(const BwdKernelArgs& a) {
    return cdiv(cdiv(a.zero_to, a.zero_rows) * a.zero_slices, kThreads / 32);
}

template <typename TA, typename TG, int E>
cudaError_t bwd_launches(BwdKernelArgs a, int64_t width, cudaStream_t s) {
    constexpr int U = E >= 4 ? 1 : 2;
    a.shape = row_shape(static_cast<int>(width / E), U, 0);
    if (a.n <= kThreads) {
        // narrower groups while that shortens a group's tokens to what it has in flight
        while (a.shape.lanes > 8 && cdiv(a.n, kThreads / a.shape.lanes) > kRun) a.shape.lanes /= 2;
        a.shape.chunks = static_cast<int>(cdiv(a.shape.pieces, a.shape.lanes * U));
        a.segment = static_cast<int>(cdiv(a.n, kThreads / a.shape.lanes));
        a.spans = 1;
        a.sum_blocks = static_cast<unsigned>(a.shape.chunks);
        return launch_pdl(embedding_few_kernel<TA, TG, E, U>, static_cast<int>(a.sum_blocks + zero_blocks(a)), kThreads, 0,
                          1, s, a);
    }
    a.segment = std::min(a.segment, kMaxSpan * a.shape.lanes / kThreads);
    a.span = a.segment * (kThreads / a.shape.lanes);
    a.spans = static_cast<unsigned>(cdiv(a.n, a.span));
    a.sum_blocks = a.spans * a.shape.chunks;
    cudaError_t err = launch_pdl(embedding_sum_kernel<TA, TG, E, U>, static_cast<int>(a.sum_blocks + zero_blocks(a)),
                                 kThreads, (a.span * 2 + 2) * 4, 1, s, a);
    if (err != cudaSuccess || a.spans == 1) return err;
    const int64_t groups = static_cast<int64_t>(a.spans) * a.shape.chunks;
    return launch_pdl(embedding_join_kernel<TG, E, U>, static_cast<int>(cdiv(groups * a.shape.lanes, kThreads)), kThreads,
                      0, 1, s, a);
}
template <typename TA, typename TG>
cudaError_t bwd_typed(int e, const BwdKernelArgs& a, int64_t width, cudaStream_t s) {
    if constexpr (sizeof(TG) == 2) {
        if (e == 8) return bwd_launches<TA, TG, 8>(a, width, s);
    }
    if (e == 4) return bwd_launches<TA, TG, 4>(a, width, s);
    if (e == 2) return bwd_launches<TA, TG, 2>(a, width, s);
    return bwd_launches<TA, TG, 1>(a, width, s);
}

// Tokens of a group: as many as 32, but groups enough for every SM to have
// some 16 warps. A block's: kMaxSpan at most.
constexpr int kMaxSegment = 32, kMinSegment = 8;
constexpr int64_t kFullGroups = kSms * 16;
int segment_of(int64_t n, int64_t width) {
    int seg = kMaxSegment;
    while (seg > kMinSegment && cdiv(n, seg) * cdiv(width, 256) < kFullGroups) seg /= 2;
    return seg;
}
// Spans of up to n tokens: a block takes a segment a warp at least. Shorter segments than
// the longest are taken while those twice as long are too few to fill the device, so that
// no fewer tokens than n have more spans than n is given room for.
int64_t most_spans(int64_t n, int64_t width) {
    constexpr int kGroups = kThreads / 32;
    const int64_t of_short = kFullGroups / cdiv(width, 256) * 2 / kGroups + 1;
    return std::min(cdiv(n, kMinSegment * kGroups), std::max(cdiv(n, kMaxSegment * kGroups), of_short));
}

struct BwdLayout {
    size_t pairs[2], present, counts, partial, bytes;
    BwdLayout(int64_t n, int64_t rows, int64_t width) {
        size_t at = 0;
        auto take = [&](size_t b) {
            const size_t here = at;
            at += (b + 255) / 256 * 256;
            return here;
        };
        for (int i = 0; i < 2; ++i) pairs[i] = take(n * sizeof(KeyItem));
        present = take(rows);
        counts = take(sort_counts_words(n, sort_max_bins(rows)) * 4);
        partial = take(static_cast<size_t>(most_spans(n, width)) * 2 * width * 4);
        bytes = at;
    }
};

}  // namespace

bool embedding_fits(int64_t n, int64_t width) {
    // element by element, which takes the most groups; they are counted in 32 bits
    return n * cdiv(width, 32 * kFwdPieces) <= kMaxGrid && most_spans(n, width) * cdiv(width, 128) <= kMaxGrid / 2;
}

cudaError_t embedding_fwd_launch(const DeviceInfo& dev, int dtype, const EmbeddingArgs& in, cudaStream_t s) {
    const int st = weight_size(dtype), sa = dtype_size(dtype);
    const int e = piece_of(in.src, in.src_stride, st, in.dst, in.dst_stride, sa, in.width);
    FwdKernelArgs a{in.k, in.src, in.dst, in.src_stride, in.dst_stride, {}, in.scale, 0, in.status};
    // streamed: 134 MB of rows in 31 us, 35 otherwise; 33 MB in 7.8, 7.5 otherwise
    a.streamed = static_cast<int64_t>(in.k.n) * in.width * sa > dev.l2_bytes / 2;
    switch (dtype) {
        case RMSNORM_F32: return fwd_typed<float, float>(e, in.width, a, s);
        case RMSNORM_BF16: return fwd_typed<__nv_bfloat16, __nv_bfloat16>(e, in.width, a, s);
        case RMSNORM_F16: return fwd_typed<__half, __half>(e, in.width, a, s);
        case RMSNORM_BF16_W_F32: return fwd_typed<float, __nv_bfloat16>(e, in.width, a, s);
        default: return fwd_typed<float, __half>(e, in.width, a, s);
    }
}

size_t embedding_bwd_workspace(int64_t n, int64_t rows, int64_t width) {
    return n <= kThreads ? 0 : BwdLayout(n, rows, width).bytes;
}

cudaError_t embedding_bwd_launch(const DeviceInfo& dev, int dtype, const EmbeddingArgs& in, bool accumulate,
                                 void* workspace, cudaStream_t s) {
    const int sg = weight_size(dtype), sa = dtype_size(dtype);
    const int e = piece_of(in.dst, in.dst_stride, sg, in.src, in.src_stride, sa, in.width);
    const int64_t n = in.k.n;
    const int64_t row_bytes = static_cast<int64_t>(in.width) * sg, stride_bytes = in.dst_stride * sg;
    int64_t zeroed = 0;  // rows, beside the sort
    BwdKernelArgs a{};
    a.k = in.k;
    if (n > kThreads) {
        const BwdLayout l(n, in.rows, in.width);
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        SortBuffers b{};
        for (int i = 0; i < 2; ++i) b.pairs[i] = reinterpret_cast<KeyItem*>(ws + l.pairs[i]);
        b.counts = reinterpret_cast<uint32_t*>(ws + l.counts);
        b.status = in.status;
        if (!accumulate) {
            const int launches = sort_launches(n, in.k.limit);
            zeroed = std::min(in.rows, cdiv(launches > 1 ? launches * kZeroBesidePass : kZeroBesideSort, row_bytes));
            char* at = static_cast<char*>(in.dst) + (in.rows - zeroed) * stride_bytes;
            const int64_t extent = (in.rows - 1) * stride_bytes + row_bytes;
            b.zero = stride_bytes == row_bytes ? ZeroJob{at, zeroed * row_bytes, 0, 1, in.dst, extent}
                                               : ZeroJob{at, row_bytes, stride_bytes, zeroed, in.dst, extent};
            if (zeroed < in.rows) b.present = ws + l.present;
        }
        const cudaError_t err = sort_launch(dev, in.k, b, s);
        if (err != cudaSuccess) return err;
        a.pairs = b.pairs[sort_result(sort_passes(in.k.limit))];
        a.present = b.present;
        a.partial = reinterpret_cast<float*>(ws + l.partial);
    }
    a.dy = in.src;
    a.grad = in.dst;
    a.dy_stride = in.src_stride;
    a.grad_stride = in.dst_stride;
    a.rows = in.rows;
    a.n = in.k.n;
    a.limit = static_cast<uint32_t>(in.k.limit);
    a.segment = segment_of(n, in.width);
    a.accumulate = accumulate;
    a.scale = in.scale;
    a.status = in.status;
    a.zero_to = accumulate ? 0 : in.rows - zeroed;
    // some 16 KB a warp: a few rows, or a part of a long one; of short rows at most an even
    // share of kZeroWarps, in whole 32s (a warp looks at 32 after 32)
    const int64_t of_bytes = kZeroBytes / row_bytes, of_warps = cdiv(cdiv(a.zero_to, kZeroWarps), 32) * 32;
    a.zero_rows = static_cast<int>(of_bytes <= 32 ? std::max<int64_t>(1, of_bytes)
                                                  : std::max<int64_t>(32, std::min(of_bytes / 32 * 32, of_warps)));
    a.zero_slices = static_cast<int>(cdiv(row_bytes, kZeroBytes));
    switch (dtype) {
        case RMSNORM_F32: return bwd_typed<float, float>(e, a, in.width, s);
        case RMSNORM_BF16: return bwd_typed<__nv_bfloat16, __nv_bfloat16>(e, a, in.width, s);
        case RMSNORM_F16: return bwd_typed<__half, __half>(e, a, in.width, s);
        case RMSNORM_BF16_W_F32: return bwd_typed<__nv_bfloat16, float>(e, a, in.width, s);
        default: return bwd_typed<__half, float>(e, a, in.width, s);
    }
}

}  // namespace rmsn
