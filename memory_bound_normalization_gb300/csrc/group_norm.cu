// Group norm, host side: the choice of a kernel family, its geometry and the
// launches.
#include <algorithm>
#include <mutex>

#include "group_norm.h"

namespace rmsn {
namespace {

// ---------------------------------------------------------------- host side
SlabFn kernel_for(int dtype, bool bwd, int act, SlabKind k) {
    switch (dtype) {
        case RMSNORM_F32: return gn_kernel_f32(bwd, act, k);
        case RMSNORM_BF16:
        case RMSNORM_BF16_W_F32: return gn_kernel_bf16(bwd, act, k);
        default: return gn_kernel_f16(bwd, act, k);
    }
}

// Clusters of a kernel that the device runs at once (0: it refuses the size);
// the answer is kept, so that a shape's grid is the same on every call.
struct OccEntry {
    int device;
    SlabFn fn;
    int threads, smem, cluster, clusters;
};
std::mutex g_occ_mu;
OccEntry g_occ[512];
int g_occ_n = 0;

int resident_clusters(const DeviceInfo& dev, SlabFn fn, int threads, int smem, int cluster) {
    std::lock_guard<std::mutex> lk(g_occ_mu);
    for (int i = 0; i < g_occ_n; ++i) {
        const OccEntry& e = g_occ[i];
        if (e.device == dev.device && e.fn == fn && e.threads == threads && e.smem == smem &&
            e.cluster == cluster)
            return e.clusters;
    }
    const void* f = reinterpret_cast<const void*>(fn);
    int n = 0;
    cudaError_t err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (err == cudaSuccess && cluster > 8)
        err = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (err == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cluster * dev.sm_count));
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        err = cudaOccupancyMaxActiveClusters(&n, f, &cfg);
    }
    if (err != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    if (g_occ_n < 512) g_occ[g_occ_n++] = {dev.device, fn, threads, smem, cluster, n};
    return n;
}

struct Plan {
    bool ok = false, resident = false;
    int splits = 1, cluster = 1, chunks = 1, lanes = 1, threads = 32, smem = 0, nvec = 0;
    int64_t samples = 1;  // stream: samples of a batch
};

void geometry(Plan* p, int nvec, int threads) {
    p->nvec = nvec;
    p->lanes = std::max(1, threads / nvec);
    p->threads = round_up(p->lanes * nvec, 32);
}

// Bytes of x (and dy) that a batch of the stream family may hold: what L2
// keeps besides the output written meanwhile.
constexpr int64_t kBatchBytes = 64ll << 20;

Plan make_plan(const DeviceInfo& dev, int dtype, bool bwd, const GroupNormArgs& a) {
    Plan best;
    const int size = dtype_size(dtype), tensors = bwd ? 2 : 1;
    const int64_t row_bytes = static_cast<int64_t>(a.C) * size;
    double best_cost = 0;
    // resident: microseconds a wave of blocks needs, by the slice a block keeps
    // (44 KB/us is an SM's share of the DRAM rate, in and out), the blocks'
    // meeting, and a fixed start; rows are split no finer than 128 bytes
    for (int splits = 1; splits <= a.G; splits *= 2) {
        if (a.G % splits) break;
        const int64_t wide = row_bytes / splits;
        if (row_bytes % splits || wide % 16 || (splits > 1 && wide < 128)) break;
        if (wide / 16 > kMaxThreads) continue;
        Plan p;
        p.splits = splits;
        geometry(&p, static_cast<int>(wide / 16), kMaxThreads);
        const int fixed = round_up(fixed_smem(p.lanes, a.C / splits, a.G / splits), 16);
        for (int cluster = 1; cluster <= 16; cluster *= 2) {
            const int64_t rows = cdiv(a.S, cluster);
            const int64_t slice = cdiv(rows, p.lanes) * p.lanes * wide * tensors;
            if (fixed + slice > kMaxSmem) continue;
            if (cluster > 1 && rows < p.lanes) break;
            const int64_t blocks = a.B * splits * cluster;
            if (blocks > INT32_MAX) break;
            const double waves = static_cast<double>(cdiv(blocks, dev.sm_count));
            const double cost = waves * (1.5 + (cluster > 8 ? 1.5 : cluster > 1 ? 1.0 : 0.0) +
                                         slice * (bwd ? 1.5 : 2.0) / 44e3);
            if (best.ok && cost >= best_cost) continue;
            const int smem = static_cast<int>(fixed + slice);
            if (resident_clusters(dev, kernel_for(dtype, bwd, a.act, SlabKind::kResident), p.threads, kMaxSmem, cluster) < 1)
                continue;
            p.ok = p.resident = true;
            p.cluster = cluster;
            p.smem = smem;
            best = p;
            best_cost = cost;
        }
    }
    // stream: all SMs on two launches
    Plan p;
    while (p.splits <= a.G && row_bytes / p.splits / 16 > kMaxThreads) p.splits *= 2;
    if (p.splits > a.G || a.G % p.splits || row_bytes % (16ll * p.splits)) return best;
    geometry(&p, static_cast<int>(row_bytes / p.splits / 16), 256);
    p.smem = fixed_smem(p.lanes, a.C / p.splits, a.G / p.splits) + ring_smem(p.lanes, p.nvec, bwd);
    if (p.smem > kMaxSmem) return best;
    const double total = static_cast<double>(a.B) * a.S * row_bytes * tensors;
    const double cost = 6.0 + total * (bwd ? 2.0 : 2.5) / (44e3 * dev.sm_count);
    if (best.ok && best_cost <= cost) return best;
    if (resident_clusters(dev, kernel_for(dtype, bwd, a.act, SlabKind::kApply), p.threads, p.smem, 1) < 1)
        return best;  // also raises the kernel's shared-memory limit
    // the largest cluster that leaves no more than a few SMs without a block
    int clusters = 0;
    const SlabFn sums = kernel_for(dtype, bwd, a.act, SlabKind::kSums);
    const int most = resident_clusters(dev, sums, p.threads, p.smem, 1);
    for (p.cluster = 8; p.cluster > 1; p.cluster /= 2) {
        clusters = resident_clusters(dev, sums, p.threads, p.smem, p.cluster);
        if (clusters * p.cluster >= most * 0.95) break;
    }
    if (p.cluster == 1) clusters = most;
    if (clusters < 1) return best;
    p.samples = std::max<int64_t>(
        1, std::min<int64_t>(a.B, kBatchBytes / (a.S * row_bytes * tensors)));
    const int64_t slabs = p.samples * p.splits;
    p.chunks = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(clusters / slabs, a.S / (p.cluster * p.lanes))));
    if (slabs * p.chunks * p.cluster > INT32_MAX || a.B * p.chunks > INT32_MAX) return best;
    p.ok = true;
    p.resident = false;
    return p;
}

// The last plans by shape: making one asks the occupancy tables some twenty
// times, a few microseconds of a call that may run for as many on the GPU.
struct PlanEntry {
    int device, dtype, bwd, act, C, G;
    int64_t B, S;
    Plan plan;
};
std::mutex g_plan_mu;
PlanEntry g_plans[64];
int g_plan_n = 0, g_plan_next = 0;

Plan plan_of(const DeviceInfo& dev, int dtype, bool vec, bool bwd, const GroupNormArgs& a) {
    if (!vec) return Plan{};
    {
        std::lock_guard<std::mutex> lk(g_plan_mu);
        for (int i = 0; i < g_plan_n; ++i) {
            const PlanEntry& e = g_plans[i];
            if (e.S == a.S && e.B == a.B && e.C == a.C && e.G == a.G && e.dtype == dtype &&
                e.act == a.act && e.bwd == (bwd ? 1 : 0) && e.device == dev.device)
                return e.plan;
        }
    }
    const Plan p = make_plan(dev, dtype, bwd, a);
    std::lock_guard<std::mutex> lk(g_plan_mu);
    g_plans[g_plan_next] = {dev.device, dtype, bwd ? 1 : 0, a.act, a.C, a.G, a.B, a.S, p};
    g_plan_next = (g_plan_next + 1) % 64;
    g_plan_n = std::min(64, g_plan_n + 1);
    return p;
}

SlabArgs args_of(const Plan& p, bool bwd, const GroupNormArgs& a) {
    SlabArgs g{};
    g.a = a;
    g.nvec = p.nvec;
    g.lanes = p.lanes;
    g.splits = p.splits;
    g.cw = a.C / p.splits;
    g.gw = a.G / p.splits;
    g.D = a.C / a.G;
    g.cluster = p.cluster;
    g.chunks = p.chunks;
    const int parts = p.chunks * p.cluster;
    g.part_rows = static_cast<int>(a.S / parts);
    g.part_more = static_cast<int>(a.S % parts);
    // a power of two of warps a group (forward), or of threads a channel
    const int room = bwd ? p.threads / (2 * g.cw) : p.threads / 32 / g.gw;
    g.join = 1;
    while (g.join < 16 && 2 * g.join <= room) g.join *= 2;
    return g;
}

size_t stats_bytes(const Plan& p, const GroupNormArgs& a) {
    return p.resident ? 0
                      : (static_cast<size_t>(p.samples) * p.chunks * a.G * 8 + 255) / 256 * 256;
}
// Rows of dw partial sums, 0 where the kernel writes dw and db itself.
int64_t partial_rows(const Plan& p, bool bwd, const GroupNormArgs& a) {
    const int64_t rows = a.B * p.chunks;
    return bwd && a.dw != nullptr && rows > 1 ? rows : 0;
}

}  // namespace

size_t group_norm_workspace(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                            const GroupNormArgs& a) {
    const Plan p = plan_of(dev, dtype, vec, bwd, a);
    if (!p.ok) return gn_scalar_workspace(bwd, a);
    return stats_bytes(p, a) + static_cast<size_t>(partial_rows(p, bwd, a)) * 2 * a.C * 4;
}

cudaError_t group_norm_launch(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                              const GroupNormArgs& a, void* workspace, cudaStream_t s) {
    const Plan p = plan_of(dev, dtype, vec, bwd, a);
    if (!p.ok) return gn_scalar_launch(dtype, bwd, a, workspace, s);
    SlabArgs g = args_of(p, bwd, a);
    const int64_t rows = partial_rows(p, bwd, a);
    g.stats = static_cast<float2*>(workspace);
    if (rows > 0) g.rows = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats_bytes(p, a));
    cudaError_t err = cudaSuccess;
    if (p.resident) {
        err = launch_pdl(kernel_for(dtype, bwd, a.act, SlabKind::kResident),
                         static_cast<int>(a.B * p.splits * p.cluster), p.threads, p.smem, p.cluster, s, g);
    } else {
        for (int64_t b = 0; b < a.B && err == cudaSuccess; b += p.samples) {
            g.sample0 = b;
            const int64_t n = std::min<int64_t>(p.samples, a.B - b);
            const int grid = static_cast<int>(n * p.splits * p.chunks * p.cluster);
            err = launch_pdl(kernel_for(dtype, bwd, a.act, SlabKind::kSums), grid, p.threads, p.smem, p.cluster, s, g);
            if (err == cudaSuccess)
                err = launch_pdl(kernel_for(dtype, bwd, a.act, SlabKind::kApply), grid, p.threads,
                                 static_cast<size_t>((g.gw + 1) / 2 * 16 + ring_smem(p.lanes, p.nvec, bwd)),
                                 1, s, g);
        }
    }
    if (err != cudaSuccess || rows == 0) return err;
    PairSum sum{};
    sum.part[0] = g.rows;
    sum.part[1] = g.rows + a.C;
    sum.out[0] = a.dw;
    sum.out[1] = a.db;
    sum.rows[0] = sum.rows[1] = static_cast<int>(rows);
    sum.n = a.C;
    sum.stride = 2 * a.C;
    sum.status = a.status;
    return pair_sum_launch(sum, s);
}

}  // namespace rmsn
