// Embedding lookup with a scale, and its gradient by sorted tokens.
//
// Forward: y_i = scale * table[id_i], rows of zeros for ids outside the table. A
// group of lanes moves a piece of a row each; bytes alone (the rows that are hit,
// in; every token's, out).
//
// Backward: row v of the gradient is scale * the sum of dy_i over the tokens with
// id v, in fp32 and in an order that the sizes alone fix. The tokens are sorted
// by id (sort.cu); the sorted list is cut in segments of a few tokens. A group of
// lanes adds up its columns of a segment: runs of one id that lie inside are
// written to their row at once, a run that crosses a border leaves its share in the
// workspace, and embedding_join_kernel adds the shares of such a run in the
// segments' order. So a token that fills half of the batch is as much work for each
// group as any other, and nothing depends on which block is first. Rows without
// a token are zeroed by blocks of their own, which the sort's marks guide.
// Bytes: dy once, the whole gradient once.
#include <algorithm>

#include "rows.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdPieces = 4;  // of a lane
constexpr int kRun = 8;        // rows of dy in flight a lane
constexpr int kZeroBytes = 16384;

struct FwdKernelArgs {
    KeySource k;
    const void* table;
    void* y;
    int64_t table_stride, y_stride;
    RowShape shape;
    float scale;
    int* status;
};

template <typename TT, typename TA, int E>
__global__ void __launch_bounds__(kThreads) embedding_fwd_kernel(const __grid_constant__ FwdKernelArgs a) {
    const unsigned lane = threadIdx.x & (a.shape.lanes - 1);
    const unsigned group = group_index<kThreads>(a.shape.lanes);
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const unsigned item = group / a.shape.chunks;
    if (item >= a.k.n) return;
    const int first = (group - item * a.shape.chunks) * (a.shape.lanes * kFwdPieces) + lane;
    const uint32_t row = key_at(a.k, item);
    const TT* src = static_cast<const TT*>(a.table) + row * a.table_stride;
    TA* dst = static_cast<TA*>(a.y) + item * a.y_stride;
    Piece<TT, E> in[kFwdPieces];
#pragma unroll
    for (int u = 0; u < kFwdPieces; ++u) {
        const int p = first + u * a.shape.lanes;
        in[u].zero();
        if (p < a.shape.pieces && row < a.k.limit) in[u].load(src + static_cast<int64_t>(p) * E);
    }
#pragma unroll
    for (int u = 0; u < kFwdPieces; ++u) {
        const int p = first + u * a.shape.lanes;
        float f[E];
        in[u].unpack(f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] *= a.scale;
        Piece<TA, E> out;
        out.pack(f);
        TA* to = dst + static_cast<int64_t>(p) * E;
        if (p < a.shape.pieces &&
            RMSN_OK(span_in(to, E * sizeof(TA), a.y,
                            rows_bytes(a.k.n, a.y_stride, static_cast<int64_t>(a.shape.pieces) * E, sizeof(TA))),
                    a.status))
            out.store(to);
    }
}

struct BwdKernelArgs {
    const uint32_t* keys;   // sorted
    const int32_t* items;
    const uint8_t* present;  // null: rows without a token stay
    const void* dy;
    void* grad;
    float* partial;  // [segments][2][width]: of the run that comes in, of the one that goes out
    int64_t dy_stride, grad_stride;
    int64_t rows;  // of the table
    int64_t zero_units;
    uint32_t n, limit;
    RowShape shape;  // lanes of a group, one piece each
    unsigned sum_blocks;  // blocks that add; the others zero rows
    int segment;
    unsigned segments;
    int zero_rows, zero_pieces, zero_slices;  // of a warp's share
    int accumulate;
    float scale;
    int* status;
};

// Row v's columns: scale * sum, on top of what is there with accumulate.
template <typename TG, int E>
__device__ __forceinline__ void put_row(const BwdKernelArgs& a, uint32_t v, int piece, const float (&sum)[E]) {
    TG* to = static_cast<TG*>(a.grad) + v * a.grad_stride + static_cast<int64_t>(piece) * E;
    if (!RMSN_OK(span_in(to, E * sizeof(TG), a.grad,
                         rows_bytes(a.rows, a.grad_stride, static_cast<int64_t>(a.shape.pieces) * E, sizeof(TG))),
                 a.status))
        return;
    Piece<TG, E> out;
    float f[E];
    if (a.accumulate) {
        out.load_plain(to);
        out.unpack(f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = fmaf(a.scale, sum[e], f[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = a.scale * sum[e];
    }
    out.pack(f);
    out.store(to);
}

template <int E>
__device__ __forceinline__ float* partial_at(const BwdKernelArgs& a, unsigned segment, int slot, int piece) {
    return a.partial + (static_cast<int64_t>(segment) * 2 + slot) * a.shape.pieces * E + static_cast<int64_t>(piece) * E;
}

template <typename TA, typename TG, int E>
__device__ __forceinline__ void add_segment(const BwdKernelArgs& a, unsigned segment, int piece) {
    const uint32_t first = segment * static_cast<uint32_t>(a.segment);
    const uint32_t end = min(first + a.segment, a.n);
    uint32_t run = a.keys[first];
    // the run that this segment starts with began before
    bool came_in = first > 0 && a.keys[first - 1] == run;
    const uint32_t behind = end < a.n ? a.keys[end] : 0xffffffffu;
    float sum[E] = {};
    auto flush = [&](bool goes_on) {
        if (run >= a.limit) return;
        if (!came_in && !goes_on) {
            put_row<TG, E>(a, run, piece, sum);
            return;
        }
        float* to = partial_at<E>(a, segment, came_in ? 0 : 1, piece);
        if (!RMSN_OK(span_in(to, E * 4, a.partial, static_cast<int64_t>(a.segments) * 8 * a.shape.pieces * E), a.status))
            return;
        Piece<float, E> out;
        out.pack(sum);
        out.store(to);
    };
    const TA* dy = static_cast<const TA*>(a.dy) + static_cast<int64_t>(piece) * E;
    for (uint32_t i = first; i < end; i += kRun) {
        uint32_t key[kRun];
        Piece<TA, E> in[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            key[j] = a.limit;
            in[j].zero();
            if (i + j < end) {
                key[j] = a.keys[i + j];
                if (key[j] < a.limit) in[j].load(dy + a.items[i + j] * a.dy_stride);
            }
        }
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            if (i + j >= end) break;
            if (key[j] != run) {
                flush(false);
                run = key[j];
                came_in = false;
#pragma unroll
                for (int e = 0; e < E; ++e) sum[e] = 0.f;
            }
            float f[E];
            in[j].unpack(f);
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] += f[e];
        }
    }
    flush(behind == run);
}

// Zeroes rows without a token: a warp takes a few rows' columns.
template <typename TG, int E>
__device__ __forceinline__ void zero_unit(const BwdKernelArgs& a, int64_t unit) {
    const int lane = threadIdx.x % 32;
    const int64_t part = unit / a.zero_slices;
    const int slice = static_cast<int>(unit - part * a.zero_slices);
    const int64_t row0 = part * a.zero_rows;
    const int rows = static_cast<int>(min(static_cast<int64_t>(a.zero_rows), a.rows - row0));
    const bool absent = lane < rows && a.present[row0 + lane] == 0;
    unsigned todo = __ballot_sync(0xffffffffu, absent);
    const int from = slice * a.zero_pieces, to = min(from + a.zero_pieces, a.shape.pieces);
    Piece<TG, E> z;
    z.zero();
    while (todo) {
        const int r = __ffs(todo) - 1;
        todo &= todo - 1;
        TG* row = static_cast<TG*>(a.grad) + (row0 + r) * a.grad_stride;
        for (int p = from + lane; p < to; p += 32)
            if (RMSN_OK(span_in(row + static_cast<int64_t>(p) * E, E * sizeof(TG), a.grad,
                                rows_bytes(a.rows, a.grad_stride, static_cast<int64_t>(a.shape.pieces) * E, sizeof(TG))),
                        a.status))
                z.store(row + static_cast<int64_t>(p) * E);
    }
}

template <typename TA, typename TG, int E>
__global__ void __launch_bounds__(kThreads) embedding_sum_kernel(const __grid_constant__ BwdKernelArgs a) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x < a.sum_blocks) {
        const unsigned group = group_index<kThreads>(a.shape.lanes);
        const unsigned segment = group / a.shape.chunks;
        const int piece = (group - segment * a.shape.chunks) * a.shape.lanes + (threadIdx.x & (a.shape.lanes - 1));
        if (segment < a.segments && piece < a.shape.pieces) add_segment<TA, TG, E>(a, segment, piece);
    } else {
        const int64_t unit =
            static_cast<int64_t>(blockIdx.x - a.sum_blocks) * (kThreads / 32) + threadIdx.x / 32;
        if (unit < a.zero_units) zero_unit<TG, E>(a, unit);
    }
}

// Runs that cross segments: the group of the segment where one begins adds the
// shares in order, in runs of 64.
template <typename TG, int E>
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const __grid_constant__ BwdKernelArgs a) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const unsigned group = group_index<kThreads>(a.shape.lanes);
    const unsigned segment = group / a.shape.chunks;
    const int piece = (group - segment * a.shape.chunks) * a.shape.lanes + (threadIdx.x & (a.shape.lanes - 1));
    if (segment >= a.segments || piece >= a.shape.pieces) return;
    const uint32_t first = segment * static_cast<uint32_t>(a.segment);
    const uint32_t end = min(first + a.segment, a.n);
    if (end >= a.n) return;
    const uint32_t run = a.keys[end - 1];
    if (run >= a.limit || a.keys[end] != run) return;
    if (first > 0 && a.keys[first] == run && a.keys[first - 1] == run) return;  // began before
    // the last segment with a share: the last one that starts with this id
    uint32_t last = segment + 1;
    for (uint32_t other = a.segments; other - last > 1;) {
        const uint32_t mid = last + (other - last) / 2;
        if (a.keys[mid * static_cast<uint32_t>(a.segment)] == run) last = mid;
        else other = mid;
    }
    float sum[E];
    Piece<float, E> in;
    in.load_plain(partial_at<E>(a, segment, 1, piece));
    in.unpack(sum);
    for (uint32_t s = segment + 1; s <= last;) {
        const uint32_t stop = min(last + 1, s + 64);
        float part[E] = {};
#pragma unroll 8
        for (; s < stop; ++s) {
            float f[E];
            in.load_plain(partial_at<E>(a, s, 0, piece));
            in.unpack(f);
#pragma unroll
            for (int e = 0; e < E; ++e) part[e] += f[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sum[e] += part[e];
    }
    put_row<TG, E>(a, run, piece, sum);
}

// Widest piece (elements) of rows of `width` of two types.
int piece_of(const void* p, int64_t ps, int size_p, const void* q, int64_t qs, int size_q, int width) {
    for (int e : {8, 4, 2}) {
        if (e * (size_p < size_q ? size_p : size_q) > 16 || width % e) continue;
        if (piece_fits(p, ps, size_p, e) && piece_fits(q, qs, size_q, e)) return e;
    }
    return 1;
}

template <typename TT, typename TA>
cudaError_t fwd_typed(int e, const FwdKernelArgs& a, int64_t blocks, cudaStream_t s) {
    auto go = [&](auto fn) { return launch_pdl(fn, static_cast<int>(blocks), kThreads, 0, 1, s, a); };
    if constexpr (sizeof(TA) == 2) {
        if (e == 8) return go(embedding_fwd_kernel<TT, TA, 8>);
    }
    if (e == 4) return go(embedding_fwd_kernel<TT, TA, 4>);
    if (e == 2) return go(embedding_fwd_kernel<TT, TA, 2>);
    return go(embedding_fwd_kernel<TT, TA, 1>);
}

template <typename TA, typename TG, int E>
cudaError_t bwd_launches(const BwdKernelArgs& a, int64_t sum_blocks, int64_t zero_blocks, cudaStream_t s) {
    cudaError_t err = launch_pdl(embedding_sum_kernel<TA, TG, E>, static_cast<int>(sum_blocks + zero_blocks), kThreads,
                                 0, 1, s, a);
    if (err != cudaSuccess || a.segments < 2) return err;
    return launch_pdl(embedding_join_kernel<TG, E>, static_cast<int>(sum_blocks), kThreads, 0, 1, s, a);
}
template <typename TA, typename TG>
cudaError_t bwd_typed(int e, const BwdKernelArgs& a, int64_t sum_blocks, int64_t zero_blocks, cudaStream_t s) {
    if constexpr (sizeof(TA) == 2) {
        if (e == 8) return bwd_launches<TA, TG, 8>(a, sum_blocks, zero_blocks, s);
    }
    if (e == 4) return bwd_launches<TA, TG, 4>(a, sum_blocks, zero_blocks, s);
    if (e == 2) return bwd_launches<TA, TG, 2>(a, sum_blocks, zero_blocks, s);
    return bwd_launches<TA, TG, 1>(a, sum_blocks, zero_blocks, s);
}

// Tokens of a segment: as many as 32, but groups enough for every SM to have
// some 32 warps.
constexpr int kMaxSegment = 32, kMinSegment = 8;
int segment_of(int64_t n, int64_t width) {
    int seg = kMaxSegment;
    while (seg > kMinSegment && cdiv(n, seg) * cdiv(width, 256) < 152 * 32) seg /= 2;
    return seg;
}

struct BwdLayout {
    size_t keys[2], items[2], present, counts, partial, bytes;
    BwdLayout(int64_t n, int64_t rows, int64_t width) {
        size_t at = 0;
        auto take = [&](size_t b) {
            const size_t here = at;
            at += (b + 255) / 256 * 256;
            return here;
        };
        for (int i = 0; i < 2; ++i) keys[i] = take(n * 4);
        for (int i = 0; i < 2; ++i) items[i] = take(n * 4);
        present = take(rows);
        counts = take(sort_counts_words(n, sort_max_bins(rows)) * 4);
        partial = take(static_cast<size_t>(cdiv(n, segment_of(n, width))) * 2 * width * 4);
        bytes = at;
    }
};

int64_t fwd_blocks(const EmbeddingArgs& a, int e, RowShape* shape) {
    *shape = row_shape(a.width / e, kFwdPieces);
    return cdiv(static_cast<int64_t>(a.k.n) * shape->chunks * shape->lanes, kThreads);
}

}  // namespace

bool embedding_fits(int64_t n, int64_t width) {
    // element by element, which takes the most groups; they are counted in 32 bits
    return n * cdiv(width, 32 * kFwdPieces) <= kMaxGrid && cdiv(n, kMinSegment) * cdiv(width, 32) <= kMaxGrid;
}

cudaError_t embedding_fwd_launch(const DeviceInfo&, int dtype, const EmbeddingArgs& in, cudaStream_t s) {
    const int st = weight_size(dtype), sa = dtype_size(dtype);
    const int e = piece_of(in.src, in.src_stride, st, in.dst, in.dst_stride, sa, in.width);
    FwdKernelArgs a{in.k, in.src, in.dst, in.src_stride, in.dst_stride, {}, in.scale, in.status};
    const int64_t blocks = fwd_blocks(in, e, &a.shape);
    switch (dtype) {
        case RMSNORM_F32: return fwd_typed<float, float>(e, a, blocks, s);
        case RMSNORM_BF16: return fwd_typed<__nv_bfloat16, __nv_bfloat16>(e, a, blocks, s);
        case RMSNORM_F16: return fwd_typed<__half, __half>(e, a, blocks, s);
        case RMSNORM_BF16_W_F32: return fwd_typed<float, __nv_bfloat16>(e, a, blocks, s);
        default: return fwd_typed<float, __half>(e, a, blocks, s);
    }
}

size_t embedding_bwd_workspace(int64_t n, int64_t rows, int64_t width) {
    return n == 0 ? 0 : BwdLayout(n, rows, width).bytes;
}

cudaError_t embedding_bwd_launch(const DeviceInfo& dev, int dtype, const EmbeddingArgs& in, bool accumulate,
                                 void* workspace, cudaStream_t s) {
    const int sg = weight_size(dtype), sa = dtype_size(dtype);
    const int e = piece_of(in.dst, in.dst_stride, sg, in.src, in.src_stride, sa, in.width);
    const int64_t n = in.k.n;
    const BwdLayout l(n, in.rows, in.width);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    SortBuffers b{};
    for (int i = 0; i < 2; ++i) {
        b.keys[i] = reinterpret_cast<uint32_t*>(ws + l.keys[i]);
        b.items[i] = reinterpret_cast<int32_t*>(ws + l.items[i]);
    }
    b.present = accumulate ? nullptr : ws + l.present;
    b.counts = reinterpret_cast<uint32_t*>(ws + l.counts);
    b.status = in.status;
    const cudaError_t err = sort_launch(dev, in.k, b, s);
    if (err != cudaSuccess) return err;
    const int result = sort_result(sort_passes(in.k.limit));
    BwdKernelArgs a{};
    a.keys = b.keys[result];
    a.items = b.items[result];
    a.present = b.present;
    a.dy = in.src;
    a.grad = in.dst;
    a.partial = reinterpret_cast<float*>(ws + l.partial);
    a.dy_stride = in.src_stride;
    a.grad_stride = in.dst_stride;
    a.rows = in.rows;
    a.n = in.k.n;
    a.limit = static_cast<uint32_t>(in.k.limit);
    a.shape = row_shape(in.width / e, 1);
    a.segment = segment_of(n, in.width);
    a.segments = static_cast<unsigned>(cdiv(n, a.segment));
    a.accumulate = accumulate;
    a.scale = in.scale;
    a.status = in.status;
    const int64_t sum_blocks =
        cdiv(static_cast<int64_t>(a.segments) * a.shape.chunks * a.shape.lanes, kThreads);
    a.sum_blocks = static_cast<unsigned>(sum_blocks);
    int64_t zero_blocks = 0;
    if (!accumulate) {
        // some 16 KB a warp: a few rows, or a part of a long one
        const int64_t row_bytes = static_cast<int64_t>(in.width) * sg;
        a.zero_rows = static_cast<int>(row_bytes >= kZeroBytes ? 1 : std::min<int64_t>(32, kZeroBytes / row_bytes));
        a.zero_pieces = a.zero_rows > 1 ? a.shape.pieces : kZeroBytes / (e * sg);
        a.zero_slices = static_cast<int>(cdiv(a.shape.pieces, a.zero_pieces));
        a.zero_units = cdiv(in.rows, a.zero_rows) * a.zero_slices;
        zero_blocks = cdiv(a.zero_units, kThreads / 32);
    }
    if (sum_blocks + zero_blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    switch (dtype) {
        case RMSNORM_F32: return bwd_typed<float, float>(e, a, sum_blocks, zero_blocks, s);
        case RMSNORM_BF16: return bwd_typed<__nv_bfloat16, __nv_bfloat16>(e, a, sum_blocks, zero_blocks, s);
        case RMSNORM_F16: return bwd_typed<__half, __half>(e, a, sum_blocks, zero_blocks, s);
        case RMSNORM_BF16_W_F32: return bwd_typed<__nv_bfloat16, float>(e, a, sum_blocks, zero_blocks, s);
        default: return bwd_typed<__half, float>(e, a, sum_blocks, zero_blocks, s);
    }
}

}  // namespace rmsn
