// Stable sort of small whole numbers (token ids, experts) with the items they
// came from, by radix passes.
//
// A pass: a warp takes 32 neighbouring items a round. Lanes with the same digit
// find one another (votes), the first of them advances the warp's count of that
// digit in shared memory, and an item's rank in its warp is the count so
// far and the equal lanes before it. The counts then become sums over the warps
// before (a digit a thread), over the blocks before, and over the digits before:
// item i goes to sum + rank. No count depends on which block or warp comes first, so
// the order is the same on every run.
//
// A few thousand to some hundred thousand keys of 4 to 8 bytes: the time is a
// chain of launches and barriers, not bytes. Up to kClusterItems one cluster of
// up to eight blocks does every pass in one launch and joins its counts through
// distributed shared memory. More items take two launches a pass over up to 152
// blocks (counts, placement).
#include <algorithm>
#include <mutex>

#include "rows.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
// One cluster's scattered stores are slow: 1.3 us for every 8192 items. 16384 items take
// it 6.6 us, 32768 9.0; 131073 take many blocks 7.
constexpr int64_t kClusterItems = 2 * kThreads * kCluster;
constexpr int kManyBlocks = kSms;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxExperts = RMSNORM_MAX_EXPERTS;

struct SortArgs {
    KeySource k;
    KeyItem* pairs[2];
    uint8_t* present;
    // many blocks, in clusters of kCluster: [blocks][bins] counts of the cluster's blocks
    // before, then [clusters][bins] counts of the clusters
    uint32_t* counts;
    int64_t counts_bytes;
    int blocks, tiles;  // kThreads * R items a tile
    int passes, pass, bits, bins;
    // experts
    int32_t* position;
    int32_t* source;
    int32_t* offsets;
    int32_t* expert_counts;
    int experts, rows, align;
    ZeroJob zero;
    int* status;
};

__host__ __device__ inline int bins_stride(int bins) { return (bins + 1) & ~1; }
inline int sort_smem(int bins, int warps) { return warps * bins_stride(bins) * 2 + 16 + 5 * 4 * (bins + 1); }

struct Smem {
    uint16_t* cnt;    // [warps][stride]
    uint32_t* hist;   // [bins]: the block's
    uint32_t* base;   // [bins]: where the block's items of a digit start
    uint32_t* start;  // [bins]: where the digit starts
    uint32_t* total;  // [bins]
    uint32_t* seen;   // [bins]: the key of the block's first item of a digit
};
__device__ __forceinline__ Smem smem_of(int bins) {
    Smem s;
    const int warps = blockDim.x / 32, stride = bins_stride(bins);
    s.cnt = reinterpret_cast<uint16_t*>(rmsn_dynamic_smem);
    s.hist = reinterpret_cast<uint32_t*>(rmsn_dynamic_smem + ((warps * stride * 2 + 15) & ~15));
    s.base = s.hist + bins + 1;
    s.start = s.base + bins + 1;
    s.total = s.start + bins + 1;
    s.seen = s.total + bins + 1;
    return s;
}

// Keys of the warp's items (0xffffffff behind the last).
template <int R>
__device__ __forceinline__ void load_keys(const SortArgs& a, int pass, unsigned first, uint32_t (&key)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const unsigned i = first + r * 32 + threadIdx.x % 32;
        key[r] = 0xffffffffu;
        if (i < a.k.n) key[r] = pass == 0 ? key_at(a.k, i) : a.pairs[(pass - 1) & 1][i].key;
    }
}
__device__ __forceinline__ uint32_t digit_of(const SortArgs& a, int pass, uint32_t key) {
    return a.experts > 0 ? key : (key >> (pass * a.bits)) & ((1u << a.bits) - 1);
}

// Ranks of the warp's items among its items of the same digit, and its counts. Lanes
// of one digit find one another by a vote a bit of the digit (up to nine in a radix pass,
// eleven for 1024 experts), where a match instruction on 32 mostly different digits took
// 1.7 us a round of 32 warps.
template <int R>
__device__ __forceinline__ void rank_keys(const SortArgs& a, int pass, unsigned first, const uint32_t (&key)[R],
                                          uint16_t* cnt, uint32_t (&rank)[R]) {
    const unsigned lane = threadIdx.x % 32, before_me = (1u << lane) - 1;
    unsigned peers[R];
#pragma unroll
    for (int r = 0; r < R; ++r) peers[r] = __ballot_sync(0xffffffffu, first + r * 32 + lane < a.k.n);
    for (int b = 0; b < a.bits; ++b) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool one = (digit_of(a, pass, key[r]) >> b) & 1;
            const unsigned ones = __ballot_sync(0xffffffffu, one);
            peers[r] &= one ? ones : ~ones;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool valid = first + r * 32 + lane < a.k.n;
        const uint32_t d = digit_of(a, pass, key[r]);
        const unsigned before = __popc(peers[r] & before_me);
        const unsigned so_far = valid ? cnt[d] : 0;
        __syncwarp();
        if (valid && before == 0) cnt[d] = static_cast<uint16_t>(so_far + __popc(peers[r]));
        rank[r] = so_far + before;
        __syncwarp();
    }
}

// Sum of the values of the threads before, over the block.
__device__ __forceinline__ uint32_t scan_before(uint32_t v, uint32_t* sum) {
    __shared__ uint32_t warp_sum[33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t s = v;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    if (warp == 0) {
        uint32_t w = lane < static_cast<int>(blockDim.x) / 32 ? warp_sum[lane] : 0, t = w;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, t, off);
            if (lane >= off) t += o;
        }
        warp_sum[lane] = t - w;
        if (lane == 31) warp_sum[32] = t;
    }
    __syncthreads();
    *sum = warp_sum[32];
    const uint32_t before = warp_sum[warp] + s - v;
    __syncthreads();
    return before;
}

__device__ __forceinline__ uint32_t rounded(uint32_t v, uint32_t align) { return (v + align - 1) / align * align; }

// From the digit's total and the blocks' before (a digit a thread) to where the
// block's items go; experts: starts and counts, by block 0.
__device__ __forceinline__ void place_digits(const SortArgs& a, const Smem& s, uint32_t total, uint32_t mine,
                                             unsigned block) {
    const int d = threadIdx.x;
    const int digits = a.experts > 0 ? a.experts : a.bins;
    uint32_t all;
    const uint32_t room = a.experts > 0 ? rounded(total, a.align) : total;
    const uint32_t start = scan_before(d < digits ? room : 0, &all);
    if (d < digits) {
        s.base[d] = start + mine;
        s.start[d] = start;
        s.total[d] = total;
        if (a.experts > 0 && block == 0) {
            if (RMSN_OK(span_in(a.offsets + d, 4, a.offsets, 4ll * (a.experts + 1)), a.status)) a.offsets[d] = start;
            if (RMSN_OK(span_in(a.expert_counts + d, 4, a.expert_counts, 4ll * a.experts), a.status))
                a.expert_counts[d] = total;
        }
    }
    if (d == 0) {
        s.start[digits] = all;
        if (a.experts > 0) {
            s.base[digits] = 0;  // the dropped ones go nowhere
            if (block == 0 && RMSN_OK(span_in(a.offsets + digits, 4, a.offsets, 4ll * (a.experts + 1)), a.status))
                a.offsets[digits] = all;
        }
    }
    __syncthreads();
}

template <int R>
__device__ __forceinline__ void scatter(const SortArgs& a, int pass, const Smem& s, const uint16_t* cnt, unsigned first,
                                        const uint32_t (&key)[R], const uint32_t (&rank)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const unsigned i = first + r * 32 + threadIdx.x % 32;
        if (i >= a.k.n) continue;
        const uint32_t d = digit_of(a, pass, key[r]);
        const uint32_t at = s.base[d] + cnt[d] + rank[r];
        if (a.experts > 0) {
            const bool dropped = d >= static_cast<uint32_t>(a.experts);
            if (RMSN_OK(span_in(a.position + i, 4, a.position, 4ll * a.k.n), a.status))
                a.position[i] = dropped ? -1 : static_cast<int32_t>(at);
            if (!dropped && RMSN_OK(span_in(a.source + at, 4, a.source, 4ll * a.rows), a.status))
                a.source[at] = static_cast<int32_t>(i);
        } else {
            const int to = pass & 1;
            const uint32_t item = pass == 0 ? i : static_cast<uint32_t>(a.pairs[to ^ 1][i].item);
            // one store of 8 bytes: scattered ones cost by their number
            if (RMSN_OK(at < a.k.n, a.status)) *reinterpret_cast<uint2*>(a.pairs[to] + at) = make_uint2(key[r], item);
        }
    }
}

// Marks the keys of a tile. A frequent one is marked by its digit's first item alone: a
// store from every warp to the same few bytes took longer than the rest of the pass.
template <int R>
__device__ __forceinline__ void mark_present(const SortArgs& a, const Smem& s, const uint16_t* cnt, unsigned first,
                                             const uint32_t (&key)[R], const uint32_t (&rank)[R]) {
    bool is_first[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t d = digit_of(a, 0, key[r]);
        is_first[r] = first + r * 32 + threadIdx.x % 32 < a.k.n && cnt[d] + rank[r] == 0;
        if (is_first[r]) s.seen[d] = key[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool live = first + r * 32 + threadIdx.x % 32 < a.k.n && key[r] < a.k.limit;
        if (live && (is_first[r] || s.seen[digit_of(a, 0, key[r])] != key[r]) &&
            RMSN_OK(span_in(a.present + key[r], 1, a.present, a.k.limit), a.status))
            a.present[key[r]] = 1;
    }
}

// Rows without a choice: behind each expert's, and behind the last expert.
__device__ __forceinline__ void mark_unused(const SortArgs& a, const Smem& s, unsigned block, unsigned blocks) {
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    // as many experts a warp as there are too many for one each, neighbours on other blocks
    const int each = min(32, (a.experts + static_cast<int>(blocks) * warps - 1) / (static_cast<int>(blocks) * warps));
    for (int e0 = ((threadIdx.x / 32) * blocks + block) * each; e0 < a.experts; e0 += blocks * warps * each) {
        const int e = e0 + lane;
        unsigned todo =
            __ballot_sync(0xffffffffu, lane < each && e < a.experts && s.start[e] + s.total[e] < s.start[e + 1]);
        for (; todo; todo &= todo - 1) {
            const int x = e0 + __ffs(todo) - 1;
            const int64_t to = s.start[x + 1];
            for (int64_t i = static_cast<int64_t>(s.start[x]) + s.total[x] + lane; i < to; i += 32)
                if (RMSN_OK(span_in(a.source + i, 4, a.source, 4ll * a.rows), a.status)) a.source[i] = -1;
        }
    }
    for (int64_t i = static_cast<int64_t>(s.start[a.experts]) + block * blockDim.x + threadIdx.x; i < a.rows;
         i += static_cast<int64_t>(blocks) * blockDim.x)
        if (RMSN_OK(span_in(a.source + i, 4, a.source, 4ll * a.rows), a.status)) a.source[i] = -1;
}

__device__ __forceinline__ void clear_present(const SortArgs& a, unsigned block, unsigned blocks) {
    if (a.present == nullptr) return;
    // limit bytes from a 16-byte boundary, room up to the next one
    uint4* p = reinterpret_cast<uint4*>(a.present);
    for (int64_t i = static_cast<int64_t>(block) * blockDim.x + threadIdx.x; i < (a.k.limit + 15) / 16;
         i += static_cast<int64_t>(blocks) * blockDim.x)
        if (RMSN_OK(span_in(p + i, 16, p, (a.k.limit + 15) / 16 * 16), a.status)) p[i] = make_uint4(0, 0, 0, 0);
}

// Clears the counts of the warps in use; their number.
template <int R>
__device__ __forceinline__ int clear_counts(const SortArgs& a, const Smem& s, unsigned block_first) {
    const unsigned left = block_first < a.k.n ? a.k.n - block_first : 0;
    const int warps = static_cast<int>(min((left + 32 * R - 1) / (32 * R), blockDim.x / 32));
    uint32_t* z = reinterpret_cast<uint32_t*>(s.cnt);
    for (int i = threadIdx.x; i < warps * bins_stride(a.bins) / 2; i += blockDim.x) z[i] = 0;
    return warps;
}
// Counts of the warps become sums over the warps before; the block's counts. The
// counts are read eight together: one trip to shared memory instead of one a warp.
__device__ __forceinline__ void sum_warps(const SortArgs& a, const Smem& s, int warps) {
    const int stride = bins_stride(a.bins);
    for (int d = threadIdx.x; d < a.bins; d += blockDim.x) {
        uint32_t sum = 0;
        for (int w0 = 0; w0 < warps; w0 += 8) {
            uint32_t c[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? s.cnt[(w0 + w) * stride + d] : 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < warps) s.cnt[(w0 + w) * stride + d] = static_cast<uint16_t>(sum);
                sum += c[w];
            }
        }
        s.hist[d] = sum;
    }
}

// Rows that are zeroed beside the sort, by block `block` of `blocks`.
constexpr int64_t kZeroUnit = 65536;  // bytes
__device__ __forceinline__ void zero_beside(const SortArgs& a, unsigned block, unsigned blocks) {
    const ZeroJob& z = a.zero;
    const int64_t slices = ceil_div(z.bytes, kZeroUnit);
    auto slice = [&](char* row, int64_t from) {
        zero_span(row + from, min(kZeroUnit, z.bytes - from), threadIdx.x, blockDim.x, z.base, z.extent, a.status);
    };
    if (z.rows == 1) {
        for (int64_t i = block; i < slices; i += blocks) slice(z.at, i * kZeroUnit);
    } else {
        for (int64_t r = block; r < z.rows; r += blocks)
            for (int64_t i = 0; i < slices; ++i) slice(z.at + r * z.stride, i * kZeroUnit);
    }
}

// Every pass, by one cluster.
template <int R>
__global__ void __launch_bounds__(kThreads) sort_cluster_kernel(const __grid_constant__ SortArgs a) {
    const Smem s = smem_of(a.bins);
    const unsigned rank = cluster_rank(), blocks = cluster_size();
    const unsigned block_first = rank * blockDim.x * R, warp = threadIdx.x / 32;
    const unsigned first = block_first + warp * 32 * R;
    uint16_t* cnt = s.cnt + warp * bins_stride(a.bins);
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x >= blocks) {  // not of the first cluster
        zero_beside(a, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    clear_present(a, rank, blocks);
    for (int pass = 0; pass < a.passes; ++pass) {
        uint32_t key[R], place[R];
        load_keys<R>(a, pass, first, key);
        const int warps = clear_counts<R>(a, s, block_first);
        __syncthreads();
        rank_keys<R>(a, pass, first, key, cnt, place);
        __syncthreads();
        sum_warps(a, s, warps);
        uint32_t total = 0, mine = 0;
        if (blocks > 1) {
            cluster_sync_all();
            if (threadIdx.x < a.bins) {
                uint32_t v[kCluster];  // one trip for all
#pragma unroll
                for (int b = 0; b < kCluster; ++b)
                    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                                 : "=r"(v[b])
                                 : "r"(cluster_map(s.hist + threadIdx.x, b)));
#pragma unroll
                for (int b = 0; b < kCluster; ++b) {
                    total += v[b];
                    if (b < static_cast<int>(rank)) mine += v[b];
                }
            }
        } else {
            __syncthreads();
            if (threadIdx.x < a.bins) total = s.hist[threadIdx.x];
        }
        place_digits(a, s, total, mine, rank);
        scatter<R>(a, pass, s, cnt, first, key, place);
        if (a.experts > 0) mark_unused(a, s, rank, blocks);
        else if (pass == 0 && a.present != nullptr) mark_present<R>(a, s, cnt, first, key, place);
        // every block has read the others' counts, and the next pass reads what they placed
        if (blocks > 1) cluster_sync_all();
        else __syncthreads();
    }
}

// One pass over many blocks: the counts of each block's digits, ...
template <int R>
__global__ void __launch_bounds__(kThreads) sort_count_kernel(const __grid_constant__ SortArgs a) {
    uint32_t* hist = reinterpret_cast<uint32_t*>(rmsn_dynamic_smem);
    for (int d = threadIdx.x; d < a.bins; d += blockDim.x) hist[d] = 0;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x >= a.blocks) {  // whole clusters
        zero_beside(a, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    if (a.pass == 0) clear_present(a, blockIdx.x, a.blocks);
    __syncthreads();
    for (int tile = 0; tile < a.tiles; ++tile) {
        uint32_t key[R];
        const unsigned first = (blockIdx.x * a.tiles + tile) * (kThreads * R) + threadIdx.x / 32 * 32 * R;
        load_keys<R>(a, a.pass, first, key);
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (first + r * 32 + threadIdx.x % 32 < a.k.n) atomicAdd(hist + digit_of(a, a.pass, key[r]), 1u);
    }
    // a cluster adds its blocks' counts up, so that the next kernel reads an eighth of them
    cluster_sync_all();
    const int rank = static_cast<int>(cluster_rank());
    for (int d = threadIdx.x; d < a.bins; d += blockDim.x) {
        uint32_t v[kCluster], total = 0, before = 0;
#pragma unroll
        for (int b = 0; b < kCluster; ++b)
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v[b]) : "r"(cluster_map(hist + d, b)));
#pragma unroll
        for (int b = 0; b < kCluster; ++b) {
            total += v[b];
            if (b < rank) before += v[b];
        }
        uint32_t* own = a.counts + static_cast<int64_t>(blockIdx.x) * a.bins + d;
        uint32_t* all = a.counts + static_cast<int64_t>(a.blocks + blockIdx.x / kCluster) * a.bins + d;
        if (RMSN_OK(span_in(own, 4, a.counts, a.counts_bytes), a.status)) *own = before;
        if (rank == 0 && RMSN_OK(span_in(all, 4, a.counts, a.counts_bytes), a.status)) *all = total;
    }
    cluster_sync_all();  // the others have read this block's
}
// ... and the items go to their places.
template <int R>
__global__ void __launch_bounds__(kThreads) sort_place_kernel(const __grid_constant__ SortArgs a) {
    const Smem s = smem_of(a.bins);
    const unsigned warp = threadIdx.x / 32;
    uint16_t* cnt = s.cnt + warp * bins_stride(a.bins);
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x >= a.blocks) {
        zero_beside(a, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    uint32_t key[R];
    load_keys<R>(a, a.pass, blockIdx.x * a.tiles * (kThreads * R) + warp * 32 * R, key);  // on their way meanwhile
    uint32_t total = 0, mine = 0;
    if (threadIdx.x < a.bins) {
        const uint32_t* clusters = a.counts + static_cast<int64_t>(a.blocks) * a.bins + threadIdx.x;
        const int count = a.blocks / kCluster, own = blockIdx.x / kCluster;
        mine = a.counts[static_cast<int64_t>(blockIdx.x) * a.bins + threadIdx.x];
        uint32_t c[kManyBlocks / kCluster];
#pragma unroll
        for (int b = 0; b < kManyBlocks / kCluster; ++b) c[b] = b < count ? clusters[b * a.bins] : 0;
#pragma unroll
        for (int b = 0; b < kManyBlocks / kCluster; ++b) {
            total += c[b];
            if (b < own) mine += c[b];
        }
    }
    place_digits(a, s, total, mine, blockIdx.x);
    for (int tile = 0; tile < a.tiles; ++tile) {
        const unsigned block_first = (blockIdx.x * a.tiles + tile) * (kThreads * R), first = block_first + warp * 32 * R;
        uint32_t place[R];
        if (tile > 0) load_keys<R>(a, a.pass, first, key);
        const int warps = clear_counts<R>(a, s, block_first);
        __syncthreads();
        rank_keys<R>(a, a.pass, first, key, cnt, place);
        __syncthreads();
        sum_warps(a, s, warps);
        __syncthreads();
        scatter<R>(a, a.pass, s, cnt, first, key, place);
        if (a.pass == 0 && a.present != nullptr) mark_present<R>(a, s, cnt, first, key, place);
        if (tile + 1 == a.tiles) break;
        __syncthreads();  // the next tile's items start behind these
        for (int d = threadIdx.x; d < a.bins; d += blockDim.x) s.base[d] += s.hist[d];
    }
    if (a.experts > 0) mark_unused(a, s, blockIdx.x, a.blocks);
}

int bits_of(int64_t limit) {
    int b = 1;
    while ((limit >> b) != 0) ++b;
    return b;
}

// A pass over many blocks, whole clusters of them: a tile (kThreads items, twice as many
// past kManyBlocks of them) each, or as many as keep them at kManyBlocks. A block's
// scattered stores drain at some two cycles each, so more SMs come before fuller ones.
struct Many {
    int rounds, tiles, blocks;
    explicit Many(int64_t n) {
        rounds = n <= kThreads * kManyBlocks ? 1 : 2;
        const int64_t tile = kThreads * rounds;
        tiles = static_cast<int>(cdiv(n, tile * kManyBlocks));
        blocks = static_cast<int>(cdiv(cdiv(n, tile * tiles), kCluster)) * kCluster;
    }
};

using SortFn = void (*)(const SortArgs);
// Lets a kernel have the shared memory of the most bins, once a device.
cudaError_t allow_smem(const DeviceInfo& dev, SortFn fn) {
    static std::mutex mu;
    static struct {
        int device;
        SortFn fn;
    } done[1024];
    static int n = 0;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n; ++i)
        if (done[i].device == dev.device && done[i].fn == fn) return cudaSuccess;
    const cudaError_t err =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sort_smem(kMaxExperts + 1, kThreads / 32));
    if (err == cudaSuccess && n < 1024) done[n++] = {dev.device, fn};
    return err;
}

// Blocks that zero rows beside `blocks` that sort: whole clusters, up to the SMs left,
// or to as many as sort.
int zero_blocks(const DeviceInfo& dev, const ZeroJob& z, int blocks, int threads, int cluster) {
    const int64_t units = z.rows == 1 ? cdiv(z.bytes, kZeroUnit) : z.rows;
    if (z.bytes == 0 || units == 0) return 0;
    const int64_t room = std::max(dev.sm_count - blocks, dev.sm_count / 2) * (kThreads / threads);
    return static_cast<int>(std::max<int64_t>(std::min(units, room) / cluster, 1) * cluster);
}

cudaError_t run(const DeviceInfo& dev, SortArgs a, cudaStream_t s) {
    const int64_t n = a.k.n;
    if (n <= kClusterItems) {
        // one block while its items and the rows it marks are few; then eight
        const int blocks = n <= kThreads && a.rows <= 4 * kThreads ? 1 : kCluster;
        const int rounds = n <= blocks * kThreads ? 1 : 2;
        // no more threads than items, digits or rows to mark need
        const int digits = a.experts > 0 ? a.experts : a.bins;
        const int need = static_cast<int>(
            std::max<int64_t>(digits, std::min<int64_t>(std::max<int64_t>(cdiv(n, rounds), a.rows / 4), kThreads)));
        const int threads = blocks > 1 ? kThreads : std::min(kThreads, std::max(128, round_up(need, 32)));
        const SortFn fn = rounds == 1 ? sort_cluster_kernel<1> : SortFn(sort_cluster_kernel<2>);
        const cudaError_t err = allow_smem(dev, fn);
        if (err != cudaSuccess) return err;
        const int zero = zero_blocks(dev, a.zero, blocks, threads, blocks);
        return launch_pdl(fn, blocks + zero, threads, sort_smem(a.bins, threads / 32), blocks, s, a);
    }
    const Many m(n);
    a.counts_bytes = sort_counts_words(n, a.bins) * 4;
    a.blocks = m.blocks;
    a.tiles = m.tiles;
    // each launch zeroes its part of the rows
    const ZeroJob all = a.zero;
    auto part = [&](int i) {
        ZeroJob z = all;
        const int64_t parts = 2 * a.passes;
        if (all.rows == 1) {  // by 16 bytes
            const int64_t each = cdiv(cdiv(all.bytes, parts), 16) * 16, from = std::min(all.bytes, each * i);
            z.at += from;
            z.bytes = std::min(each, all.bytes - from);
        } else {
            const int64_t each = cdiv(all.rows, parts), from = std::min(all.rows, each * i);
            z.at += from * all.stride;
            z.rows = std::min(each, all.rows - from);
        }
        return z;
    };
    for (a.pass = 0; a.pass < a.passes; ++a.pass) {
        a.zero = part(2 * a.pass);
        int zero = zero_blocks(dev, a.zero, m.blocks, kThreads, kCluster);
        cudaError_t err = launch_pdl(m.rounds == 1 ? sort_count_kernel<1> : SortFn(sort_count_kernel<2>),
                                     m.blocks + zero, kThreads, a.bins * 4, kCluster, s, a);
        if (err != cudaSuccess) return err;
        const SortFn fn = m.rounds == 1 ? sort_place_kernel<1> : SortFn(sort_place_kernel<2>);
        err = allow_smem(dev, fn);
        if (err != cudaSuccess) return err;
        a.zero = part(2 * a.pass + 1);
        zero = zero_blocks(dev, a.zero, m.blocks, kThreads, 1);
        err = launch_pdl(fn, m.blocks + zero, kThreads, sort_smem(a.bins, kThreads / 32), 1, s, a);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace

int sort_passes(int64_t limit) { return static_cast<int>(cdiv(bits_of(limit), kMaxDigitBits)); }
int sort_launches(int64_t n, int64_t limit) { return n <= kClusterItems ? 1 : 2 * sort_passes(limit); }
int sort_max_bins(int64_t limit) { return 1 << cdiv(bits_of(limit), sort_passes(limit)); }

int64_t sort_counts_words(int64_t n, int bins) {
    if (n <= kClusterItems) return 0;
    // past a tile for each of the most blocks their number falls and grows again; the room does not
    const int64_t blocks = n > kThreads * kManyBlocks ? kManyBlocks : Many(n).blocks;
    return bins * (blocks + blocks / kCluster);
}

cudaError_t sort_launch(const DeviceInfo& dev, const KeySource& k, const SortBuffers& b, cudaStream_t s) {
    SortArgs a{};
    a.k = k;
    for (int i = 0; i < 2; ++i) a.pairs[i] = b.pairs[i];
    a.present = b.present;
    a.zero = b.zero;
    a.counts = b.counts;
    a.passes = sort_passes(k.limit);
    a.bits = static_cast<int>(cdiv(bits_of(k.limit), a.passes));
    a.bins = 1 << a.bits;
    a.status = b.status;
    return run(dev, a, s);
}

cudaError_t expert_sort_launch(const DeviceInfo& dev, const ExpertSortArgs& e, cudaStream_t s) {
    SortArgs a{};
    a.k = e.k;
    a.counts = e.block_counts;
    a.passes = 1;
    a.bits = bits_of(e.k.limit);
    a.experts = static_cast<int>(e.k.limit);
    a.bins = a.experts + 1;
    a.position = e.position;
    a.source = e.source;
    a.offsets = e.offsets;
    a.expert_counts = e.counts;
    a.rows = e.rows;
    a.align = e.align;
    a.status = e.status;
    return run(dev, a, s);
}

}  // namespace rmsn
