// Group norm, host side: the choice of a kernel family, its geometry and the
// launches.
#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "common.cuh"
#include "group_norm.h"

namespace rmsn {
namespace {

// Sets the streamed kernel's arrival counters to zero. A kernel of its own, not
// a memset: it lets the streamed kernel start at once, which reads x meanwhile
// and waits for the zeros only before it counts.
__global__ void zero_kernel(unsigned* p, int n) {
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0;
}

// ---------------------------------------------------------------- host side
SlabFn kernel_for(int dtype, bool bwd, int act, SlabKind k) {
    switch (dtype) {
        case RMSNORM_F32: return gn_kernel_f32(bwd, act, k);
        case RMSNORM_BF16:
        case RMSNORM_BF16_W_F32: return gn_kernel_bf16(bwd, act, k);
        default: return gn_kernel_f16(bwd, act, k);
    }
}

// Places of a table of 1024 entries, by a multiplicative hash of the keys.
unsigned place(std::initializer_list<int64_t> keys) {
    uint64_t h = 0;
    for (int64_t k : keys) h = (h ^ static_cast<uint64_t>(k)) * 0x9E3779B97F4A7C15ull, h ^= h >> 29;
    return static_cast<unsigned>(h % 1024);
}

// Makes a device the current one for as long as it lives: a workspace's size may
// be asked for any device.
class OnDevice {
public:
    explicit OnDevice(int device) {
        ok = cudaGetDevice(&prev) == cudaSuccess && (prev == device || cudaSetDevice(device) == cudaSuccess);
        changed = ok && prev != device;
    }
    ~OnDevice() {
        if (changed) cudaSetDevice(prev);
    }
    OnDevice(const OnDevice&) = delete;
    OnDevice& operator=(const OnDevice&) = delete;
    bool ok = false;

private:
    int prev = -1;
    bool changed = false;
};

// Clusters of a kernel that the device runs at once (0: it refuses the size). The
// kernel is allowed the size there, so that a plan, once kept, launches.
struct OccEntry {
    int device;
    SlabFn fn;  // nullptr: empty
    int threads, smem, cluster, clusters;
};
std::mutex g_occ_mu;
OccEntry g_occ[1024];

int resident_clusters(const DeviceInfo& dev, SlabFn fn, int threads, int smem, int cluster) {
    std::lock_guard<std::mutex> lk(g_occ_mu);
    OccEntry& e = g_occ[place({dev.device, reinterpret_cast<int64_t>(fn), threads, smem, cluster})];
    if (e.device == dev.device && e.fn == fn && e.threads == threads && e.smem == smem && e.cluster == cluster)
        return e.clusters;
    const OnDevice there(dev.device);
    if (!there.ok) {
        cudaGetLastError();
        return 0;
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
    e = {dev.device, fn, threads, smem, cluster, n};
    return n;
}

struct Plan {
    bool ok = false, resident = false;
    int splits = 1, cluster = 1, lanes = 1, threads = 32, smem = 0, nvec = 0;
    int parts = 1, together = 1, rounds = 1;  // stream
    bool drop = false;
};

void geometry(Plan* p, int nvec, int threads) {
    p->nvec = nvec;
    p->lanes = std::max(1, threads / nvec);
    p->threads = round_up(p->lanes * nvec, 32);
}

// Microseconds that a resident plan takes, near enough to choose by: a wave's
// fixed part, the meeting of a cluster (whose blocks read one another's sums),
// the joins (by channels and threads of a block), and the slice each SM keeps
// (44 KB/us is an SM's share of the DRAM rate, in and out), with few warps at
// less than that rate in the forward. The backward's column sum comes once.
// Measured (GPU time, forward unless said): 4 samples of 4096 positions of 320
// f16 channels in clusters of 16 blocks of 256 threads 10.4 us, of 8 of 256 11.6,
// of 8 of 512 with twice the slice 11.6; 2 of 64 of 1280 bf16 in single blocks of
// 256 threads 4.0, of 512 4.8, in clusters of 8 5.6; backward 4 of 1069 of 192 in
// clusters of 8 of 256 8.3, of 16 9.7, of 8 of 512 9.0.
double resident_cost(const DeviceInfo& dev, bool bwd, int64_t clusters, int at_once, int cluster, int threads,
                     int64_t slice, int channels) {
    const double waves = static_cast<double>(cdiv(clusters, at_once));
    const int64_t per_sm = cdiv(std::min<int64_t>(clusters, at_once) * cluster, dev.sm_count);
    const double meet = cluster > 8 ? (bwd ? 2.3 : 1.0) : cluster > 4 ? (bwd ? 1.0 : 0.5) : cluster > 1 ? 0.2 : 0.0;
    const int64_t busy = per_sm * threads;
    const double slow = bwd || busy >= 512 ? 1.0 : busy >= 256 ? 1.25 : 1.7;
    return (bwd ? 1.0 : 0.0) + waves * (2.4 + meet + 0.003 * channels + 1.9 * threads / 512 +
                                        per_sm * slice * (bwd ? 1.5 : 2.0) / 44e3 * slow);
}

Plan make_plan(const DeviceInfo& dev, int dtype, bool bwd, const GroupNormArgs& a) {
    Plan best;
    const int size = dtype_size(dtype), tensors = bwd ? 2 : 1;
    const int64_t row_bytes = static_cast<int64_t>(a.C) * size;
    double best_cost = 0;
    // resident: rows are split no finer than 128 bytes; the backward's two tensors
    // want 256 threads
    for (int splits = 1; splits <= a.G; splits *= 2) {
        if (a.G % splits) break;
        const int64_t wide = row_bytes / splits;
        if (row_bytes % splits || wide % 16 || (splits > 1 && wide < 128)) break;
        for (int threads = kMaxThreads; threads >= (bwd ? 256 : 128); threads /= 2) {
            if (wide / 16 > threads) continue;
            Plan p;
            p.splits = splits;
            geometry(&p, static_cast<int>(wide / 16), threads);
            const int fixed = round_up(fixed_smem(p.lanes, a.C / splits, a.G / splits), 16);
            for (int cluster = 1; cluster <= 16; cluster *= 2) {
                const int64_t rows = cdiv(a.S, cluster);
                const int64_t slice = cdiv(rows, p.lanes) * p.lanes * wide * tensors;
                if (fixed + slice > kMaxSmem) continue;
                if (cluster > 1 && rows < p.lanes) break;
                if (a.B * splits * cluster > INT32_MAX) break;
                // how many run at once: clusters of 8 or 16 large blocks leave some
                // SMs of a GPC unused, so that 16 clusters of 8 are two waves
                const int smem = static_cast<int>(fixed + slice);
                const int at_once = resident_clusters(dev, kernel_for(dtype, bwd, a.act, SlabKind::kResident),
                                                      p.threads, std::min(kMaxSmem, round_up(smem, 16 * 1024)),
                                                      cluster);
                if (at_once < 1) continue;
                const double cost = resident_cost(dev, bwd, a.B * splits, at_once, cluster, threads, slice, a.C / splits);
                if (best.ok && cost >= best_cost) continue;
                p.ok = p.resident = true;
                p.cluster = cluster;
                p.smem = smem;
                best = p;
                best_cost = cost;
            }
        }
    }
    // stream: rounds of slabs that half of L2 holds (the other half holds what
    // is written meanwhile), rows split no finer than 128 bytes, the width of an
    // L2 line: narrower pieces read at half the DRAM rate
    const int64_t budget = std::max<int64_t>(1 << 20, static_cast<int64_t>(dev.l2_bytes) * 9 / 16);
    const int64_t slab_rows = a.S * tensors;
    Plan p;
    auto wide = [&] { return row_bytes / p.splits; };
    auto splittable = [&] {
        return a.G % (2 * p.splits) == 0 && row_bytes % (2 * p.splits) == 0 && wide() / 2 % 16 == 0;
    };
    while ((wide() > 16 * kStreamThreads || (wide() >= 256 && wide() * slab_rows > budget)) && splittable())
        p.splits *= 2;
    if (wide() > 16 * kStreamThreads) return best;
    const int64_t slabs = a.B * p.splits;
    if (slabs > INT32_MAX / 1024) return best;
    p.nvec = static_cast<int>(wide() / 16);
    p.lanes = kStreamThreads / p.nvec;
    p.threads = kStreamThreads;
    p.smem = stream_smem(bwd, p.lanes, a.C / p.splits, a.G / p.splits);
    if (p.smem > kMaxSmem) return best;
    const double total = static_cast<double>(a.B) * slab_rows * row_bytes;
    const SlabFn fn = kernel_for(dtype, bwd, a.act, SlabKind::kStream);
    const int64_t most = resident_clusters(dev, fn, p.threads, p.smem, 1);
    if (most < 1) return best;
    // two at least, as long as what both keep is near L2's size
    const int64_t fit = budget / (wide() * slab_rows);
    p.together = static_cast<int>(std::min<int64_t>(
        {slabs, most, fit >= 2 ? fit : wide() * slab_rows <= budget ? 2 : 1}));
    p.rounds = static_cast<int>(cdiv(slabs, p.together));
    p.together = static_cast<int>(cdiv(slabs, p.rounds));
    // at least two groups of positions a thread, where the slab has them
    p.parts = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>({most / p.together, kStreamMaxParts, a.S / (4 * p.lanes)})));
    if ((a.S / p.parts + 1) * row_bytes > UINT32_MAX || a.B * p.parts > INT32_MAX) return best;
    // Where both families fit, the cheaper by this estimate ran faster: 13 samples
    // of 3439 positions of 264 f16 channels take 23.5 us resident (two waves of
    // clusters) and 17.6 streamed, 3 of 13452 of 128 take 9.7 and 12.5, backwards
    // 7 of 6021 of 96 bf16 take 13.8 and 15.7.
    // The fixed part counts a launch more on the host: a near tie goes to resident.
    const double cost = (bwd ? 8.5 : 7.5) + 3.0 * p.rounds + total * (bwd ? 1.5 : 2.0) / (44e3 * dev.sm_count);
    if (best.ok && best_cost <= cost) return best;
    p.ok = true;
    p.drop = total * (bwd ? 1.5 : 2.0) > dev.l2_bytes / 2;
    return p;
}

// Plans by shape: making one asks the occupancy tables some dozens of times,
// longer than a call may run on the GPU. A plan depends on its key alone, so it
// may be dropped and made again.
struct PlanEntry {
    int device, dtype, bwd, act, C, G;
    int64_t B, S;  // B 0: empty
    Plan plan;
};
std::mutex g_plan_mu;
PlanEntry g_plans[1024];

Plan plan_of(const DeviceInfo& dev, int dtype, bool vec, bool bwd, const GroupNormArgs& a) {
    if (!vec) return Plan{};
    PlanEntry& e = g_plans[place({a.S, a.B, a.C, a.G, dtype, a.act, bwd ? 1 : 0, dev.device})];
    {
        std::lock_guard<std::mutex> lk(g_plan_mu);
        if (e.S == a.S && e.B == a.B && e.C == a.C && e.G == a.G && e.dtype == dtype && e.act == a.act &&
            e.bwd == (bwd ? 1 : 0) && e.device == dev.device)
            return e.plan;
    }
    const Plan p = make_plan(dev, dtype, bwd, a);
    std::lock_guard<std::mutex> lk(g_plan_mu);
    e = {dev.device, dtype, bwd ? 1 : 0, a.act, a.C, a.G, a.B, a.S, p};
    return p;
}

SlabArgs args_of(const Plan& p, const GroupNormArgs& a) {
    SlabArgs g{};
    g.a = a;
    g.nvec = p.nvec;
    g.lanes = p.lanes;
    g.splits = p.splits;
    g.cw = a.C / p.splits;
    g.gw = a.G / p.splits;
    g.D = a.C / a.G;
    g.cluster = p.cluster;
    g.parts = p.parts;
    g.together = p.together;
    g.rounds = p.rounds;
    g.drop = p.drop;
    const int parts = p.resident ? p.cluster : p.parts;
    g.part_rows = static_cast<int>(a.S / parts);
    g.part_more = static_cast<int>(a.S % parts);
    // threads that share four channels' lanes: as many as there are, up to 16
    g.join = std::max(1, std::min({16, g.lanes, p.threads / (g.cw / 2)}));
    g.seg_log = 2;
    while (g.seg_log < 5 && (1 << g.seg_log) < g.D) ++g.seg_log;
    g.drop_unit = -1;
    return g;
}

// Workspace of the stream family: arrivals, then results, then partial rows.
size_t rounded(size_t n) { return (n + 255) / 256 * 256; }
size_t arrived_bytes(const Plan& p, const GroupNormArgs& a) {
    return p.resident ? 0 : rounded(static_cast<size_t>(a.B) * p.splits * 4);
}
size_t stats_bytes(const Plan& p, const GroupNormArgs& a) {
    return p.resident ? 0 : rounded(static_cast<size_t>(a.B) * a.G * p.parts * 8);
}
// Rows of dw partial sums, 0 where the kernel writes dw and db itself.
int64_t partial_rows(const Plan& p, bool bwd, const GroupNormArgs& a) {
    const int64_t rows = a.B * (p.resident ? 1 : p.parts);
    return bwd && a.dw != nullptr && (rows > 1 || !p.resident) ? rows : 0;
}

}  // namespace

bool group_norm_fits(const DeviceInfo& dev, int dtype, bool vec, bool bwd, const GroupNormArgs& a) {
    return gn_scalar_fits(a) || plan_of(dev, dtype, vec, bwd, a).ok;
}

size_t group_norm_workspace(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                            const GroupNormArgs& a) {
    const Plan p = plan_of(dev, dtype, vec, bwd, a);
    if (!p.ok) return gn_scalar_workspace(bwd, a);
    return arrived_bytes(p, a) + stats_bytes(p, a) +
           static_cast<size_t>(partial_rows(p, bwd, a)) * 2 * a.C * 4;
}

cudaError_t group_norm_launch(const DeviceInfo& dev, int dtype, bool vec, bool bwd,
                              const GroupNormArgs& a, void* workspace, cudaStream_t s) {
    const Plan p = plan_of(dev, dtype, vec, bwd, a);
    if (!p.ok) return gn_scalar_launch(dtype, bwd, a, workspace, s);
    SlabArgs g = args_of(p, a);
    const int64_t rows = partial_rows(p, bwd, a);
    char* ws = static_cast<char*>(workspace);
    const size_t arrived = arrived_bytes(p, a);
    g.arrived = reinterpret_cast<unsigned*>(ws);
    g.stats = reinterpret_cast<float2*>(ws + arrived);
    if (rows > 0) g.rows = reinterpret_cast<float*>(ws + arrived + stats_bytes(p, a));
    cudaError_t err;
    if (p.resident) {
        err = launch_pdl(kernel_for(dtype, bwd, a.act, SlabKind::kResident),
                         static_cast<int>(a.B * p.splits * p.cluster), p.threads, p.smem, p.cluster, s, g);
    } else {
        g.drop_unit = take_drop_unit();
        const int words = static_cast<int>(a.B * p.splits);
        err = launch_pdl(&zero_kernel, static_cast<int>(std::min<int64_t>(64, cdiv(words, 256))), 256, 0, 1, s,
                         g.arrived, words);
        if (err != cudaSuccess) return err;
        // the blocks wait for one another: all of them run at once, or none
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(p.together * p.parts));
        cfg.blockDim = dim3(kStreamThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(p.smem);
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = pdl_allowed();
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        err = cudaLaunchKernelEx(&cfg, kernel_for(dtype, bwd, a.act, SlabKind::kStream), g);
    }
    if (err != cudaSuccess || rows == 0) return err;
    PairSum sum{};
    sum.part[0] = g.rows;
    sum.part[1] = g.rows + a.C;
    sum.out[0] = a.dw;
    sum.out[1] = a.db;
    sum.rows[0] = sum.rows[1] = static_cast<int>(rows);
    sum.n = a.C;
    sum.stride = 2 * static_cast<int64_t>(a.C);
    sum.status = a.status;
    return pair_sum_launch(sum, s);
}

}  // namespace rmsn
