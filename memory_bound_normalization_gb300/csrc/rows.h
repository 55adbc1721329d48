// What the host side of the operators that move rows by an index (embedding.cu,
// experts.cu, sort.cu) and the C ABI (rows_api.cu) share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace rmsn {

// The SMs that shapes and workspaces are made for, a GB300's: constant, as a workspace's
// size is asked without a device. On another number the work is shared less evenly.
constexpr int kSms = 152;

// ------------------------------------------------------------- sorting keys
// n small whole numbers, read where they lie: `outer` runs of `inner` with a
// stride each. A key is the number itself where it lies in [0, limit) and is
// not `skip`, else `limit` (dropped: behind every other).
struct KeySource {
    const void* ids;  // int32 or int64
    int64_t stride_outer, stride_inner;
    unsigned n, inner;
    int64_t limit;  // 1 .. 2^31 - 1
    int64_t skip;   // negative: none
    int ids_64;
};

// Rows to be zeroed, of any alignment: `rows` rows of `bytes`, `stride` apart, inside the
// `extent` bytes from `base` on.
struct ZeroJob {
    char* at;
    int64_t bytes, stride, rows;
    const void* base;
    int64_t extent;
};

// Stable order of the keys by radix passes: pairs of a key and the item it came
// from. `present`, unless null: limit bytes, 1 where the key occurs.
struct KeyItem {
    uint32_t key;
    int32_t item;
};
struct SortBuffers {
    KeyItem* pairs[2];
    uint8_t* present;
    uint32_t* counts;  // sort_counts_words(n, bins) words, null if that is 0
    ZeroJob zero;      // done beside the launches, on the SMs they leave idle
    int* status;
};
int sort_passes(int64_t limit);
// Launches of a sort.
int sort_launches(int64_t n, int64_t limit);
// Words of counts for n items: 0 where one cluster of blocks takes them all.
int64_t sort_counts_words(int64_t n, int bins);
int sort_max_bins(int64_t limit);
// Which of the two buffers holds the result.
inline int sort_result(int passes) { return (passes - 1) & 1; }
cudaError_t sort_launch(const DeviceInfo& dev, const KeySource& k, const SortBuffers& b, cudaStream_t s);

// One pass over experts: the row of each choice, the choice of each row, and
// where every expert's rows start.
struct ExpertSortArgs {
    KeySource k;  // limit: the experts
    int32_t* position;
    int32_t* source;
    int32_t* offsets;
    int32_t* counts;
    int32_t rows;
    int32_t align;
    uint32_t* block_counts;  // sort_counts_words(n, experts + 1)
    int* status;
};
cudaError_t expert_sort_launch(const DeviceInfo& dev, const ExpertSortArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- embedding
struct EmbeddingArgs {
    KeySource k;  // limit: rows of the table
    const void* src;  // forward: the table; backward: dy
    void* dst;        // forward: y; backward: the table's gradient
    int64_t src_stride, dst_stride;  // elements between rows
    int64_t rows;                    // of the table
    int width;
    float scale;
    int* status;
};
cudaError_t embedding_fwd_launch(const DeviceInfo& dev, int dtype, const EmbeddingArgs& a, cudaStream_t s);
// Whether the calls' groups can be counted.
bool embedding_fits(int64_t n, int64_t width);
size_t embedding_bwd_workspace(int64_t n, int64_t rows, int64_t width);
cudaError_t embedding_bwd_launch(const DeviceInfo& dev, int dtype, const EmbeddingArgs& a, bool accumulate,
                                 void* workspace, cudaStream_t s);

// ------------------------------------------------------------------ experts
struct ExpertArgs {
    const int32_t* position;  // [tokens, choices]
    const int32_t* source;    // [rows]
    const void* weights;      // [tokens, choices], or nullptr: 1
    const void* x;            // by token: dispatch forward's x, combine's residual or dy
    const void* in;           // by row: rows combined, rows of a gradient
    void* out;                // by row: dispatched rows, drows; by token: y, dx
    float* dweights;
    int64_t x_stride, in_stride, out_stride;
    int64_t tokens;
    int rows, choices, width;
    int* status;
};
bool experts_fit(const ExpertArgs& a);
// Whether choice k is one of a token's. Unsigned: a few behind the last of 2^31 - 1 pass
// 31 bits.
__host__ __device__ constexpr bool more_choices(unsigned k, int choices) { return k < static_cast<unsigned>(choices); }
// rows[position[t, k]] = x[t] (times nothing), rows without a choice zero
cudaError_t expert_scatter_launch(const DeviceInfo& dev, int dtype, const ExpertArgs& a, cudaStream_t s);
// y[t] = x[t] + sum_k w[t, k] in[position[t, k]]
cudaError_t expert_gather_launch(const DeviceInfo& dev, int dtype, const ExpertArgs& a, cudaStream_t s);
// out[position[t, k]] = w[t, k] x[t], dweights[t, k] = <x[t], in[position[t, k]]>
cudaError_t expert_gather_bwd_launch(const DeviceInfo& dev, int dtype, const ExpertArgs& a, cudaStream_t s);

// Blocks a grid may have.
constexpr int64_t kMaxGrid = 0x7fffffff;

}  // namespace rmsn
