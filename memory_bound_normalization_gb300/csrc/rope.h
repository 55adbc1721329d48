// What the host side of the rotary calls (rope.cu) and their kernels
// (rope_kernels.cuh, one translation unit for each activation type) share.
#pragma once

#include "ops.h"

namespace rmsn {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTile = 32;  // tokens of a tile
constexpr int kRopeBwdBlocks = 2;  // blocks an SM holds in the backward
constexpr int kRopeBwdAhead = 3;   // rows a thread's copies run ahead in the backward

// Pieces of a backward block's rows on the way: two of x and two of dy a thread.
constexpr int kRopeRingWords = kRopeBwdAhead * 4 * kRopeThreads;
constexpr int kRopeBwdSmem = 100 * 1024;  // of a backward block at most

using RopeFn = void (*)(const RopeArgs);
// The kernel for pieces of e elements and `units` units a head.
RopeFn rope_kernel_f32(int e, int units, bool bwd, bool adjacent, bool norm);
RopeFn rope_kernel_bf16(int e, int units, bool bwd, bool adjacent, bool norm);
RopeFn rope_kernel_f16(int e, int units, bool bwd, bool adjacent, bool norm);

}  // namespace rmsn
