// The kernel families of the group norm: what the host side (group_norm.cu)
// and the kernels (group_norm_kernels.cuh, one translation unit for each
// activation type) share, and the general path (group_norm_scalar.cu).
#pragma once

#include "ops.h"

namespace rmsn {

// Blocks of 32 channels (any count up to 2^31 - 1).
__host__ __device__ inline int channel_tiles(int C) { return (C - 1) / 32 + 1; }
// Whether a grid has a block for every chunk.
bool gn_scalar_fits(const GroupNormArgs& a);
size_t gn_scalar_workspace(bool bwd, const GroupNormArgs& a);
cudaError_t gn_scalar_launch(int dtype, bool bwd, const GroupNormArgs& a, void* ws, cudaStream_t s);

constexpr int kMaxThreads = 512;
constexpr int kMaxSmem = 227 * 1024;

struct SlabArgs {
    GroupNormArgs a;
    int nvec;      // 16-byte vectors of a slab's row
    int lanes;     // positions a block takes at once
    int splits;    // slabs of a sample (runs of channels)
    int cw, gw;    // channels and groups of a slab
    int D;         // channels of a group
    int cluster;   // resident: blocks of a slab, which join their sums
    int part_rows, part_more;  // positions of a block, and how many blocks take one more
    int join;      // threads that share four channels' sums in a block
    int seg_log;   // log2 of the lanes that join a group's channels: as many as D, 4 to 32
    // stream
    int parts;     // blocks of a slab
    int together;  // slabs of a round
    int rounds;
    int drop;      // L2 is told what is used for the last time
    unsigned* arrived;  // [slab]: blocks that have published their results
    float2* stats;      // [slab][group][part]: (mean, M2), or (sum w P, sum w Q)
    int64_t drop_unit;  // failure injection: the slab block 0 does not count itself in
    // backward: partial rows [2 C] (Q, then P): a sample's, or a sample's part's
    float* rows;
};

// Shared memory besides the slots: the threads' sums, the channels' constants,
// and two values a group, twice (the block's and the slab's).
inline int fixed_smem(int lanes, int cw, int gw) { return (2 * lanes * cw + 4 * cw + 4 * gw) * 4; }

// Positions a thread's copies run ahead, and positions of a group of copies.
constexpr int kDepth = 16, kGroup = 2;
constexpr int kStreamThreads = 256;  // two blocks an SM
constexpr int kStreamMaxParts = 320;
constexpr int stream_depth(bool bwd) { return bwd ? 8 : 12; }
// The stream kernel's shared memory: the ring of copies; the sums of its
// threads; its channels' constants and groups' results.
inline int stream_ring(bool bwd) { return stream_depth(bwd) * kStreamThreads * 16 * (bwd ? 2 : 1); }
inline int stream_smem(bool bwd, int lanes, int cw, int gw) {
    return stream_ring(bwd) + (2 * lanes + 4) * cw * 4 + gw * 8;
}

using SlabFn = void (*)(const SlabArgs);
enum class SlabKind { kResident, kStream };
SlabFn gn_kernel_f32(bool bwd, int act, SlabKind k);
SlabFn gn_kernel_bf16(bool bwd, int act, SlabKind k);
SlabFn gn_kernel_f16(bool bwd, int act, SlabKind k);

}  // namespace rmsn
