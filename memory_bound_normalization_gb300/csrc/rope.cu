// Rotary positions after the QK-norm, host side: the widest pieces the tensors
// allow, the geometry and the launches.
#include <algorithm>
#include <mutex>

#include "rope.h"

namespace rmsn {
namespace {

// Widest piece (elements of one access) that every offset of the call allows.
bool fits(const void* p, const int64_t (&s)[3], int bytes, int size) {
    if (p == nullptr) return true;
    if (reinterpret_cast<uintptr_t>(p) % bytes) return false;
    for (int64_t v : s)
        if (v * size % bytes) return false;
    return true;
}
int piece_of(const RopeArgs& a, int dtype, bool adjacent) {
    const int size = dtype_size(dtype);
    for (int e : {16 / size, 8 / size, 4}) {
        if (e > 16 / size || e < 4) continue;
        bool ok = adjacent ? a.head_dim % (2 * e) == 0
                           : a.rot / 2 % e == 0 && (a.head_dim - a.rot) / 2 % e == 0;
        for (const RopeTensor& t : a.t) {
            if (t.heads == 0) continue;
            ok = ok && fits(t.x, t.xs, e * size, size) && fits(t.dy, t.dys, e * size, size) &&
                 fits(t.out, t.os, e * size, size);
        }
        if (ok) return e;
    }
    return 1;
}

RopeFn kernel_for(int dtype, int e, const RopeArgs& a, bool bwd, bool adjacent, bool norm) {
    switch (dtype) {
        case RMSNORM_F32: return rope_kernel_f32(e, a.units, a.lanes, bwd, adjacent, norm);
        case RMSNORM_BF16:
        case RMSNORM_BF16_W_F32: return rope_kernel_bf16(e, a.units, a.lanes, bwd, adjacent, norm);
        default: return rope_kernel_f16(e, a.units, a.lanes, bwd, adjacent, norm);
    }
}

// Lanes of a group: the power of two at or above the units of a head, or as many
// as the units where a warp then holds more groups.
void shape_of(RopeArgs* a, int e) {
    a->units = a->head_dim / 2 / e;
    a->lanes = 4;
    while (a->lanes < 32 && a->lanes < a->units) a->lanes *= 2;
    if (e > 1 && 32 / a->units > 32 / a->lanes) a->lanes = a->units;
    a->per_warp = 32 / a->lanes;
    a->inv_lanes = 65536 / a->lanes + 1;
}
int groups_of(const RopeArgs& a) { return kRopeThreads / 32 * a.per_warp; }

// Shared memory of the backward: rows on the way, weights, then the larger of
// the two angle tables and the groups' shares of dw.
int bwd_smem(const RopeArgs& a, int e, int dtype) {
    return (e >= 4 ? kRopeBwdWords * e * dtype_size(dtype) : 0) +
           a.head_dim * 4 * (1 + std::max(2 * a.tile, groups_of(a)));
}

// Lets a kernel have the shared memory that its blocks an SM leave it, once a
// device.
cudaError_t allow_smem(const DeviceInfo& dev, RopeFn fn) {
    static std::mutex mu;
    static struct {
        int device;
        RopeFn fn;
    } done[256];
    static int n = 0;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n; ++i)
        if (done[i].device == dev.device && done[i].fn == fn) return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kRopeMaxSmem);
    if (err == cudaSuccess && n < 256) done[n++] = {dev.device, fn};
    return err;
}

// Tokens of a tile at most: two angle tables fit in 40 KB.
int max_tile(const RopeArgs& a) { return std::min(kRopeMaxTile, 40 * 1024 / (8 * a.head_dim)); }

// Some eight passes of the block's groups over a tile's rows, but no fewer tiles
// than SMs: 25 tokens of 48 bf16 heads of 96 take 5.0 us, where tiles of eight
// passes on a few blocks take 8.3.
int bwd_tile(const DeviceInfo& dev, const RopeArgs& a) {
    const int groups = groups_of(a);
    int heads = 1;
    for (const RopeTensor& t : a.t)
        if (t.heads > 0) heads = std::max(heads, t.heads);
    return static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>({max_tile(a), 8 * groups / heads, a.tokens / dev.sm_count})));
}

}  // namespace

cudaError_t rope_fwd_launch(const DeviceInfo& dev, int dtype, bool adjacent, RopeArgs a,
                            cudaStream_t s) {
    const int e = piece_of(a, dtype, adjacent);
    shape_of(&a, e);
    const bool norm = a.t[0].w != nullptr;
    const int heads = a.t[0].heads + a.t[1].heads;
    const int groups = groups_of(a);
    // some eight passes of the block's groups over a tile's rows, but no fewer
    // tiles than SMs; few tokens share their heads out
    a.tile = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>({max_tile(a), cdiv(8 * groups, heads), a.tokens / (2 * dev.sm_count)})));
    a.splits = 1;
    if (a.tile == 1)
        a.splits = static_cast<int>(std::max<int64_t>(
            1, std::min<int64_t>(cdiv(heads, groups), 2 * dev.sm_count / a.tokens)));
    const int blocks = static_cast<int>(
        std::min<int64_t>(cdiv(a.tokens, a.tile), static_cast<int64_t>(kRopeBlocks) * dev.sm_count));
    const int smem = (e >= 4 ? kRopeFwdWords * e * dtype_size(dtype) : 0) +
                     a.head_dim * 4 * (2 * a.tile + (norm ? 2 : 0));
    const RopeFn fn = kernel_for(dtype, e, a, false, adjacent, norm);
    const cudaError_t err = allow_smem(dev, fn);
    if (err != cudaSuccess) return err;
    return launch_pdl(fn, blocks * a.splits, kRopeThreads, smem, 1, s, a);
}

int rope_bwd_max_rows(const DeviceInfo& dev) { return kRopeBlocks * dev.sm_count + 2; }

cudaError_t rope_bwd_rows(const DeviceInfo& dev, int dtype, bool adjacent, const RopeArgs& in,
                          int rows[2]) {
    RopeArgs a = in;
    shape_of(&a, piece_of(a, dtype, adjacent));
    a.tile = bwd_tile(dev, a);
    const int64_t tiles = cdiv(a.tokens, a.tile);
    // what fits, shared out by the heads of the two tensors
    const int64_t total = rope_bwd_max_rows(dev) - 2;
    // in proportion to their work: a token's angles cost about as much as two rows
    const int64_t q = a.t[0].heads + 2, k = a.t[1].heads == 0 ? 0 : a.t[1].heads + 2;
    rows[0] = static_cast<int>(std::max<int64_t>(1, std::min(tiles, total * q / (q + k))));
    rows[1] = k == 0 ? 0 : static_cast<int>(std::max<int64_t>(1, std::min(tiles, total * k / (q + k))));
    return cudaSuccess;
}

cudaError_t rope_bwd_launch(const DeviceInfo& dev, int dtype, bool adjacent, RopeArgs a,
                            const int rows[2], cudaStream_t s) {
    const int e = piece_of(a, dtype, adjacent);
    shape_of(&a, e);
    a.tile = bwd_tile(dev, a);
    a.blocks0 = rows[0];
    const RopeFn fn = kernel_for(dtype, e, a, true, adjacent, true);
    cudaError_t err = allow_smem(dev, fn);
    if (err != cudaSuccess) return err;
    err = launch_pdl(fn, rows[0] + rows[1], kRopeThreads, bwd_smem(a, e, dtype), 1, s, a);
    if (err != cudaSuccess) return err;
    PairSum p{};
    for (int i = 0; i < 2; ++i) {
        p.part[i] = a.partial + static_cast<int64_t>(i ? rows[0] : 0) * a.head_dim;
        p.out[i] = a.t[i].dw;
        p.rows[i] = rows[i];
    }
    p.n = p.stride = a.head_dim;
    p.status = a.status;
    return pair_sum_launch(p, s);
}

}  // namespace rmsn
