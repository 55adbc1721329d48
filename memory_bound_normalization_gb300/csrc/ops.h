// Internal interface between the C-ABI layer (api.cu) and the translation
// units of the operators that go with the norm: rotary positions after the
// query/key norm (rope.cu) and group norm (group_norm.cu). Host code only.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace rmsn {

constexpr int kRopeMaxHeadDim = 256;
constexpr int kRopeMaxPairs = kRopeMaxHeadDim / 2;

// One of the two tensors (queries, keys) of a rotary call. Strides in
// elements over (batch, token, head); the last dimension is dense.
struct RopeTensor {
    const void* x;   // forward: the input; backward: the forward's input
    const void* dy;  // backward: the gradient of the forward's output
    void* out;       // forward: the output; backward: the input's gradient
    const void* w;   // [D], or nullptr without the norm
    float* dw;       // backward with the norm: [D]
    int64_t xs[3], dys[3], os[3];
    int heads;
};

struct RopeArgs {
    RopeTensor t[2];
    const void* pos;  // int32 or int64
    int64_t ps[3];    // strides of positions over (axis, batch, token)
    const float* inv_freq;
    int64_t tokens;   // batch * length
    int length;
    int head_dim, rot, axes;
    float eps;
    int pos64, w_f32;
    float sign;       // -1 turns back (the backward)
    int* status;
    // launch geometry (rope_launch fills it in)
    int units, lanes, tile, splits;
    int per_warp, inv_lanes;  // groups of a warp; 2^16 / lanes, rounded up
    float* partial;   // backward: dw partial rows of t[0], then of t[1]
    int blocks0;      // backward: blocks that take t[0]
    unsigned char axis[kRopeMaxPairs];  // axis of each rotated pair
};

// Rows of partial sums a backward with the norm writes for each tensor.
cudaError_t rope_bwd_rows(const DeviceInfo& dev, int dtype, bool adjacent, const RopeArgs& a,
                          int rows[2]);
// The most rows any call of the device writes, both tensors together.
int rope_bwd_max_rows(const DeviceInfo& dev);
cudaError_t rope_fwd_launch(const DeviceInfo& dev, int dtype, bool adjacent, RopeArgs a,
                            cudaStream_t s);
cudaError_t rope_bwd_launch(const DeviceInfo& dev, int dtype, bool adjacent, RopeArgs a,
                            const int rows[2], cudaStream_t s);

struct GroupNormArgs {
    const void* x;
    const void* w;  // [C], or nullptr (then 1 and 0)
    const void* b;
    const void* dy;
    void* out;      // forward: y; backward: dx
    float* mean;    // [B, G]: written by the forward, read by the backward
    float* rstd;
    float* dw;      // backward: [C]
    float* db;
    int64_t B, S;
    int C, G;
    float eps;
    int act;
    int w_f32;
    int* status;
    uint64_t wait_limit_ns;
};

// The failure-injection hook's unit (-1: none), which is thereby used up.
int64_t take_drop_unit();

// Workspace bytes of a call (0: none), and the call itself. `vec`: every
// pointer is 16-byte aligned and a row of channels is a whole number of
// 16-byte vectors.
// Whether the call's blocks fit a grid.
bool group_norm_fits(const DeviceInfo& dev, int dtype, bool vec, bool bwd, const GroupNormArgs& a);
size_t group_norm_workspace(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                            const GroupNormArgs& a);
cudaError_t group_norm_launch(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                              const GroupNormArgs& a, void* workspace, cudaStream_t s);

// The column sum of dw partial rows: two outputs of n columns each, out[i] =
// the sum of rows[i] rows of `stride` floats from part[i], in a fixed order.
struct PairSum {
    const float* part[2];
    float* out[2];
    int rows[2];
    int n;
    int64_t stride;  // twice the channels of a group norm: past 31 bits from 2^30 on
    int* status;
};
// A thread's next item (a row) in a block of 256: unsigned, since it passes
// 2^31 - 1 behind the last of as many.
constexpr int kItemThreads = 256;
__host__ __device__ inline unsigned next_item(unsigned i) { return i + kItemThreads; }
cudaError_t pair_sum_launch(const PairSum& a, cudaStream_t s);

}  // namespace rmsn
