// A CUDA runtime of two devices that launches nothing, preloaded in front of the
// real one by tests of the library's host code: it keeps which device is current,
// what each function was allowed on which device, and the launches.
#include <cuda_runtime.h>
#include <string.h>

#include <map>
#include <tuple>
#include <utility>
#include <vector>

#include "group_norm.h"
#include "ops.h"

namespace {

int g_device = 0;
std::map<std::pair<int, const void*>, int> g_smem;  // (device, function): its dynamic shared memory
std::map<std::pair<int, const void*>, int> g_wide;  // clusters of 16 are allowed
std::vector<int> g_asked;                           // the device of each occupancy question
int g_words[2];
struct Launch {
    int device, grid, rows, threads, smem, cluster;
    int allowed;  // the function may have this shared memory and cluster on this device
};
std::vector<Launch> g_launches;
rmsn::PairSum g_sum;  // of the last column sum

}  // namespace

extern "C" {

cudaError_t cudaGetDevice(int* d) {
    *d = g_device;
    return cudaSuccess;
}
cudaError_t cudaSetDevice(int d) {
    if (d < 0 || d > 1) return cudaErrorInvalidDevice;
    g_device = d;
    return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : a == cudaDevAttrL2CacheSize ? 126 << 20 : 227 * 1024;
    return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
    *p = &g_words[g_device];
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_smem[{g_device, f}] = v;
    if (a == cudaFuncAttributeNonPortableClusterSizeAllowed) g_wide[{g_device, f}] = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
    const int cluster = static_cast<int>(c->attrs[0].val.clusterDim.x);
    g_asked.push_back(g_device);
    const int blocks = c->dynamicSmemBytes > 110 * 1024 || c->blockDim.x > 256 ? 1 : 2;
    *n = 144 * blocks / cluster;
    return cudaSuccess;
}
cudaError_t cudaMallocAsync(void** p, size_t, cudaStream_t) {
    *p = reinterpret_cast<void*>(1ull << 40);
    return cudaSuccess;
}
cudaError_t cudaFreeAsync(void*, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
    Launch l{g_device, static_cast<int>(c->gridDim.x), static_cast<int>(c->gridDim.y),
             static_cast<int>(c->blockDim.x), static_cast<int>(c->dynamicSmemBytes), 1, 1};
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension)
            l.cluster = static_cast<int>(c->attrs[i].val.clusterDim.x);
    l.allowed = (l.smem <= 48 * 1024 || g_smem[{g_device, f}] >= l.smem) &&
                (l.cluster <= 8 || g_wide[{g_device, f}] != 0);
    g_launches.push_back(l);
    if (l.rows == 2) memcpy(&g_sum, args[0], sizeof g_sum);  // the column sum alone has two rows of blocks
    return l.allowed ? cudaSuccess : cudaErrorInvalidValue;
}

int fake_launches() { return static_cast<int>(g_launches.size()); }
const int* fake_launch(int i) { return &g_launches[i].device; }
int fake_asked(int device) {
    int n = 0;
    for (int d : g_asked) n += d == device;
    return n;
}
long long fake_sum_stride() { return g_sum.stride; }
int fake_channel_tiles(int C) { return rmsn::channel_tiles(C); }
// Items that a thread takes from p on.
int fake_items_from(int p, int items) {
    int n = 0;
    for (auto i = rmsn::next_item(p - rmsn::kItemThreads); i < static_cast<decltype(i)>(items) && n < 1000;
         i = rmsn::next_item(i))
        ++n;
    return n;
}
long long fake_sum_rows() { return g_sum.rows[0]; }
}
