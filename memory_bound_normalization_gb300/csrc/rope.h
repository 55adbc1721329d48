// What the host side of the rotary calls (rope.cu) and their kernels
// (rope_kernels.cuh, one translation unit for each activation type) share.
#pragma once

#include "ops.h"

namespace rmsn {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTile = 32;  // tokens of a tile
constexpr int kRopeBlocks = 2;    // blocks an SM holds
constexpr int kRopeFwdAhead = 3;  // rows a thread's copies run ahead
constexpr int kRopeBwdAhead = 2;
// Pieces of a block's rows on the way: two a tensor and thread.
constexpr int kRopeFwdWords = kRopeFwdAhead * 2 * kRopeThreads;
constexpr int kRopeBwdWords = kRopeBwdAhead * 4 * kRopeThreads;
constexpr int kRopeMaxSmem = 80 * 1024;  // dynamic shared memory of a block at most

using RopeFn = void (*)(const RopeArgs);
// The kernel for pieces of e elements, `units` units a head and `lanes` lanes a
// group.
RopeFn rope_kernel_f32(int e, int units, int lanes, bool bwd, bool adjacent, bool norm);
RopeFn rope_kernel_bf16(int e, int units, int lanes, bool bwd, bool adjacent, bool norm);
RopeFn rope_kernel_f16(int e, int units, int lanes, bool bwd, bool adjacent, bool norm);

}  // namespace rmsn
