// What the host side of the rotary calls (rope.cu) and their kernels
// (rope_kernels.cuh, one translation unit for each activation type) share.
#pragma once

#include "ops.h"

namespace rmsn {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTile = 32;  // tokens of a tile
constexpr int kRopeBwdBlocks = 2;  // blocks an SM holds in the backward

using RopeFn = void (*)(const RopeArgs);
// The kernel for pieces of e elements and `units` units a head.
RopeFn rope_kernel_f32(int e, int units, bool bwd, bool adjacent, bool norm);
RopeFn rope_kernel_bf16(int e, int units, bool bwd, bool adjacent, bool norm);
RopeFn rope_kernel_f16(int e, int units, bool bwd, bool adjacent, bool norm);

}  // namespace rmsn
