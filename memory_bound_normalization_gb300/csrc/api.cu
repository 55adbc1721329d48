// C ABI of librmsnorm.so (declared in include/rmsnorm.h): argument checks,
// per-device properties, the device status word, workspace handling and
// dispatch to the kernel translation units.
#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <utility>

#include "kernels.h"
#include "ops.h"

namespace rmsn {

// One status word per device (a module-scope variable lives once in every
// device context that loads the library). Kernels receive its address.
__device__ int g_status_word;

namespace {

constexpr int kMaxDevices = 64;
constexpr uint64_t kDefaultWaitLimitNs = 1000000000ull;  // one second

std::mutex g_dev_mu;
DeviceInfo g_dev[kMaxDevices];
bool g_dev_ready[kMaxDevices] = {};

std::atomic<uint64_t> g_wait_limit_ns{kDefaultWaitLimitNs};
std::atomic<int64_t> g_drop_unit{-1};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Maps a CUDA result to a status. A failure is also cleared from the
// runtime's last-error slot, so it does not surface in the caller's next,
// unrelated CUDA call.
int cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return RMSNORM_OK;
    cudaGetLastError();
    return RMSNORM_ERR_CUDA;
}

int shape_status(int64_t M, int64_t N, int dtype) {
    if (M < 0 || N <= 0 || N > INT32_MAX) return RMSNORM_ERR_INVALID_ARG;
    if (!dtype_known(dtype)) return RMSNORM_ERR_INVALID_ARG;
    return RMSNORM_OK;
}

int current_device(const DeviceInfo** out) {
    int dev = -1;
    if (cuda_status(cudaGetDevice(&dev)) != RMSNORM_OK) return RMSNORM_ERR_CUDA;
    *out = device_info(dev);
    return *out ? RMSNORM_OK : RMSNORM_ERR_CUDA;
}

// Backward checks shared by rmsnorm_bwd and rmsnorm_bwd_ws. On success fills
// the plan (with M > 0) or reports that there is nothing to do besides
// clearing dw (M == 0).
int bwd_prepare(const void* x, const void* w, const void* dy, const float* rstd, void* dx,
                float* dw, int64_t M, int64_t N, int dtype, const DeviceInfo** dev,
                rmsnorm_plan_t* plan, const void* dres = nullptr) {
    int st = shape_status(M, N, dtype);
    if (st != RMSNORM_OK) return st;
    if (M == 0) {
        if (dw != nullptr && !aligned(dw, 4)) return RMSNORM_ERR_MISALIGNED;
        *plan = rmsnorm_plan_t{};
        return RMSNORM_OK;
    }
    if (!x || !w || !dy || !rstd || !dx || !dw) return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype), wsz = weight_size(dtype);
    if (!aligned(x, sz) || !aligned(w, wsz) || !aligned(dy, sz) || !aligned(dx, sz) ||
        !aligned(rstd, 4) || !aligned(dw, 4) || (dres && !aligned(dres, sz)))
        return RMSNORM_ERR_MISALIGNED;
    const bool vec = aligned(x, 16) && aligned(w, 16) && aligned(dy, 16) && aligned(dx, 16) &&
                     (!dres || aligned(dres, 16)) && (N * sz) % 16 == 0 && (N * wsz) % 16 == 0;
    bwd_choose(N, dtype, vec, plan, dres != nullptr);
    st = current_device(dev);
    if (st != RMSNORM_OK) return st;
    return cuda_status(bwd_finish_plan(**dev, dtype, M, N, plan, dres != nullptr));
}

int bwd_run(const void* x, const void* w, const void* dy, const float* rstd, void* dx, float* dw,
            int64_t M, int64_t N, int dtype, const DeviceInfo& dev, const rmsnorm_plan_t& plan,
            void* workspace, cudaStream_t stream, const void* dres = nullptr) {
    BwdArgs a{};
    a.x = x;
    a.w = w;
    a.dy = dy;
    a.rstd = rstd;
    a.dx = dx;
    a.partial = static_cast<float*>(workspace);
    a.dw = dw;
    a.M = M;
    a.N = static_cast<int>(N);
    a.status = dev.status_word;
    a.sm_count = dev.sm_count;
    a.wait_limit_ns = g_wait_limit_ns.load();
    a.drop_unit = plan.variant != RMSNORM_VARIANT_SCALAR ? g_drop_unit.exchange(-1) : -1;
    a.dres = dres;
    return cuda_status(bwd_launch(plan, dtype, a, stream));
}

// Forward checks, plan and launch shared by rmsnorm_fwd and rmsnorm_add_fwd
// (res and h are both NULL for the plain forward).
int fwd_run(const void* x, const void* res, const void* w, void* h, void* y, float* rstd,
            int64_t M, int64_t N, float eps, int dtype, cudaStream_t stream) {
    int st = shape_status(M, N, dtype);
    if (st != RMSNORM_OK) return st;
    if (!(eps >= 0.f)) return RMSNORM_ERR_INVALID_ARG;  // negative or NaN
    if (M == 0) return RMSNORM_OK;
    const bool add = res != nullptr || h != nullptr;
    if (!x || !w || !y || !rstd || (add && (!res || !h))) return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype), wsz = weight_size(dtype);
    if (!aligned(x, sz) || !aligned(w, wsz) || !aligned(y, sz) || !aligned(rstd, 4) ||
        (add && (!aligned(res, sz) || !aligned(h, sz))))
        return RMSNORM_ERR_MISALIGNED;
    const bool vec = aligned(x, 16) && aligned(w, 16) && aligned(y, 16) && (N * sz) % 16 == 0 &&
                     (N * wsz) % 16 == 0 && (!add || (aligned(res, 16) && aligned(h, 16)));
    rmsnorm_plan_t plan;
    fwd_choose(N, dtype, vec, &plan, add);
    const DeviceInfo* dev = nullptr;
    st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    st = cuda_status(fwd_finish_plan(*dev, dtype, M, N, &plan, add));
    if (st != RMSNORM_OK) return st;
    if (static_cast<int64_t>(plan.grid) <= 0 ||
        ((plan.variant == RMSNORM_VARIANT_ROWGROUP || plan.variant == RMSNORM_VARIANT_CTA_ROW ||
          plan.variant == RMSNORM_VARIANT_CLUSTER_ROW) &&
         cdiv(M, plan.variant == RMSNORM_VARIANT_ROWGROUP ? plan.rows_per_unit : 1) * plan.cluster >
             INT32_MAX))
        return RMSNORM_ERR_UNSUPPORTED;
    FwdArgs a{x, w, y, rstd, M, static_cast<int>(N), eps, dev->status_word, g_wait_limit_ns.load(),
              res, h};
    a.drop_unit = plan.variant == RMSNORM_VARIANT_RING ? g_drop_unit.exchange(-1) : -1;
    return cuda_status(fwd_launch(plan, dtype, a, stream));
}

// rmsnorm_bwd and rmsnorm_add_bwd: workspace from the stream-ordered pool.
int bwd_alloc_run(const void* x, const void* w, const void* dy, const float* rstd,
                  const void* dres, void* dx, float* dw, int64_t M, int64_t N, int dtype,
                  cudaStream_t stream) {
    const DeviceInfo* dev = nullptr;
    rmsnorm_plan_t plan;
    int st = bwd_prepare(x, w, dy, rstd, dx, dw, M, N, dtype, &dev, &plan, dres);
    if (st != RMSNORM_OK) return st;
    if (M == 0) {
        if (dw == nullptr) return RMSNORM_OK;
        return cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * 4, stream));
    }
    if (plan.workspace_bytes == 0)  // one partial row: written straight to dw
        return bwd_run(x, w, dy, rstd, dx, dw, M, N, dtype, *dev, plan, nullptr, stream, dres);
    void* ws = nullptr;
    if (cuda_status(cudaMallocAsync(&ws, static_cast<size_t>(plan.workspace_bytes), stream)) !=
        RMSNORM_OK)
        return RMSNORM_ERR_NOMEM;
    st = bwd_run(x, w, dy, rstd, dx, dw, M, N, dtype, *dev, plan, ws, stream, dres);
    const int freed = cuda_status(cudaFreeAsync(ws, stream));
    if (st == RMSNORM_OK) st = freed;
    return st;
}

// Workspace of a call: the caller's, or one from the stream-ordered allocator.
struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
    bool given = false;

    int take(size_t need, cudaStream_t s) {
        if (given) {
            if (need > 0 && (p == nullptr || bytes < need)) return RMSNORM_ERR_INVALID_ARG;
            return aligned(p, 16) ? RMSNORM_OK : RMSNORM_ERR_MISALIGNED;
        }
        if (need == 0) return RMSNORM_OK;
        return cuda_status(cudaMallocAsync(&p, need, s)) == RMSNORM_OK ? RMSNORM_OK : RMSNORM_ERR_NOMEM;
    }
    int give(int status, cudaStream_t s) {
        if (given || p == nullptr) return status;
        const int freed = cuda_status(cudaFreeAsync(p, s));
        return status != RMSNORM_OK ? status : freed;
    }
};

// ------------------------------------------------ rotary positions
// Checks of the descriptor; on success fills everything of `a` that does not
// depend on the tensors.
int rope_descriptor(const rmsnorm_rope_t* r, int dtype, RopeArgs* a) {
    if (r == nullptr || !dtype_known(dtype)) return RMSNORM_ERR_INVALID_ARG;
    if (r->batch < 0 || r->length < 0 || r->q_heads < 0 || r->k_heads < 0)
        return RMSNORM_ERR_INVALID_ARG;
    if (r->length > INT32_MAX || (r->length > 0 && r->batch > INT32_MAX / r->length))
        return RMSNORM_ERR_INVALID_ARG;
    if (static_cast<int64_t>(r->q_heads) + r->k_heads > 65536) return RMSNORM_ERR_INVALID_ARG;
    if (r->head_dim < 2 || r->head_dim > RMSNORM_ROPE_MAX_HEAD_DIM || r->head_dim % 2 ||
        r->rotary_dim < 2 || r->rotary_dim > r->head_dim || r->rotary_dim % 2)
        return RMSNORM_ERR_INVALID_ARG;
    if (r->axes < 1 || r->axes > RMSNORM_ROPE_MAX_AXES) return RMSNORM_ERR_INVALID_ARG;
    int left[RMSNORM_ROPE_MAX_AXES];
    int64_t sum = 0;
    for (int i = 0; i < r->axes; ++i) {
        if (r->sections[i] < 0) return RMSNORM_ERR_INVALID_ARG;
        left[i] = r->sections[i];
        sum += r->sections[i];
    }
    if (sum != r->rotary_dim / 2) return RMSNORM_ERR_INVALID_ARG;
    for (int64_t v : r->position_stride)
        if (v < 0) return RMSNORM_ERR_INVALID_ARG;
    int next = 0;
    for (int p = 0; p < r->rotary_dim / 2; ++p) {
        while (left[next] == 0) next = (next + 1) % r->axes;
        a->axis[p] = static_cast<unsigned char>(next);
        if (--left[next] == 0 || r->interleaved) next = (next + 1) % r->axes;
    }
    a->tokens = r->batch * r->length;
    a->length = static_cast<int>(r->length);
    a->head_dim = r->head_dim;
    a->rot = r->rotary_dim;
    a->axes = r->axes;
    a->pos64 = r->positions_64 != 0;
    a->w_f32 = weight_size(dtype) == 4;
    for (int i = 0; i < 3; ++i) a->ps[i] = r->position_stride[i];
    a->t[0].heads = r->q_heads;
    a->t[1].heads = r->k_heads;
    return RMSNORM_OK;
}

// A tensor of a rotary call: non-null, aligned to its elements, strides not
// negative and the heads' below 2^32 bytes.
int rope_tensor(const void* p, const rmsnorm_strides_t& s, int size, int64_t (&out)[3]) {
    if (p == nullptr || s.batch < 0 || s.token < 0 || s.head < 0 || s.head > UINT32_MAX / size)
        return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(p, size)) return RMSNORM_ERR_MISALIGNED;
    out[0] = s.batch;
    out[1] = s.token;
    out[2] = s.head;
    return RMSNORM_OK;
}

// Whether a dimension of more than one element has stride 0.
bool overlaps_itself(const rmsnorm_rope_t* r, const rmsnorm_strides_t& s, int heads) {
    return (r->batch > 1 && s.batch == 0) || (r->length > 1 && s.token == 0) || (heads > 1 && s.head == 0);
}
// Whether two tensors at one address lie differently.
bool differ(const rmsnorm_rope_t* r, const rmsnorm_strides_t& s, const rmsnorm_strides_t& t, int heads) {
    return (r->batch > 1 && s.batch != t.batch) || (r->length > 1 && s.token != t.token) ||
           (heads > 1 && s.head != t.head);
}

// Both directions of the rotary call, the descriptor checked and tokens > 0.
// Without weights the backward is the forward of the gradient with the angle
// turned back.
int rope_run(const rmsnorm_rope_t* r, RopeArgs& a, const void* q, const void* k, const void* wq,
             const void* wk, const void* positions, const float* inv_freq, const void* dq_out,
             const void* dk_out, void* oq, void* ok, float* dwq, float* dwk, float eps, int dtype,
             bool bwd, const Workspace& given, cudaStream_t stream) {
    const int sz = dtype_size(dtype), wsz = weight_size(dtype);
    const bool has[2] = {a.t[0].heads > 0, a.t[1].heads > 0};
    const void* w[2] = {wq, wk};
    float* dw[2] = {dwq, dwk};
    if (has[0] && has[1] && (wq == nullptr) != (wk == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    const bool norm = (has[0] ? wq : wk) != nullptr;
    if (positions == nullptr || inv_freq == nullptr) return RMSNORM_ERR_INVALID_ARG;
    const void* x[2] = {q, k};
    const void* dy[2] = {dq_out, dk_out};
    void* o[2] = {oq, ok};
    const rmsnorm_strides_t* xs[2] = {&r->q, &r->k};
    const rmsnorm_strides_t* ys[2] = {&r->q_out, &r->k_out};
    const rmsnorm_strides_t* ds[2] = {&r->dq, &r->dk};
    for (int i = 0; i < 2; ++i) {
        if (!has[i]) continue;
        RopeTensor& t = a.t[i];
        int st;
        if (!bwd || norm) {
            st = rope_tensor(x[i], *xs[i], sz, t.xs);
            if (st != RMSNORM_OK) return st;
            t.x = x[i];
        }
        if (bwd) {
            st = rope_tensor(dy[i], *ys[i], sz, norm ? t.dys : t.xs);
            if (st != RMSNORM_OK) return st;
            (norm ? t.dy : t.x) = dy[i];
        }
        const rmsnorm_strides_t& os = bwd ? *ds[i] : *ys[i];
        st = rope_tensor(o[i], os, sz, t.os);
        if (st != RMSNORM_OK) return st;
        if (overlaps_itself(r, os, t.heads) || (o[i] == t.x && differ(r, os, bwd && !norm ? *ys[i] : *xs[i], t.heads)) ||
            (o[i] == t.dy && differ(r, os, *ys[i], t.heads)))
            return RMSNORM_ERR_INVALID_ARG;
        t.out = o[i];
        if (norm) {
            if (bwd && dw[i] == nullptr) return RMSNORM_ERR_INVALID_ARG;
            if (!aligned(w[i], wsz)) return RMSNORM_ERR_MISALIGNED;
            t.w = w[i];
            t.dw = dw[i];
        }
    }
    if (!aligned(positions, a.pos64 ? 8 : 4) || !aligned(inv_freq, 4)) return RMSNORM_ERR_MISALIGNED;
    // a call without queries has its keys first
    if (!has[0]) std::swap(a.t[0], a.t[1]);
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.eps = eps;
    a.sign = bwd ? -1.f : 1.f;
    const DeviceInfo* dev = nullptr;
    int st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    a.status = dev->status_word;
    const bool adjacent = r->adjacent != 0;
    if (!bwd || !norm) return cuda_status(rope_fwd_launch(*dev, dtype, adjacent, a, stream));
    int rows[2];
    st = cuda_status(rope_bwd_rows(*dev, dtype, adjacent, a, rows));
    if (st != RMSNORM_OK) return st;
    Workspace ws = given;
    st = ws.take(static_cast<size_t>(rows[0] + rows[1]) * a.head_dim * 4, stream);
    if (st != RMSNORM_OK) return st;
    a.partial = static_cast<float*>(ws.p);
    st = cuda_status(rope_bwd_launch(*dev, dtype, adjacent, a, rows, stream));
    return ws.give(st, stream);
}

int rope_bwd_any(const rmsnorm_rope_t* rope, const void* q, const void* k, const void* wq,
                 const void* wk, const void* positions, const float* inv_freq, const void* dq_out,
                 const void* dk_out, void* dq, void* dk, float* dwq, float* dwk, float eps,
                 int dtype, const Workspace& ws, cudaStream_t stream) {
    RopeArgs a{};
    int st = rope_descriptor(rope, dtype, &a);
    if (st != RMSNORM_OK) return st;
    if (!(eps >= 0.f)) return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(dwq, 4) || !aligned(dwk, 4)) return RMSNORM_ERR_MISALIGNED;
    if (a.tokens == 0 || a.t[0].heads + a.t[1].heads == 0) {
        float* dws[2] = {a.t[0].heads ? dwq : nullptr, a.t[1].heads ? dwk : nullptr};
        for (float* p : dws)
            if (p != nullptr) {
                st = cuda_status(cudaMemsetAsync(p, 0, static_cast<size_t>(a.head_dim) * 4, stream));
                if (st != RMSNORM_OK) return st;
            }
        return RMSNORM_OK;
    }
    return rope_run(rope, a, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq, dwk,
                    eps, dtype, true, ws, stream);
}

// ------------------------------------------------------- group norm
int group_norm_shape(GroupNormArgs* a, int64_t C, int64_t G, int dtype) {
    if (!dtype_known(dtype) || a->B < 0 || a->S < 0 || C <= 0 || C > INT32_MAX || G <= 0 || C % G)
        return RMSNORM_ERR_INVALID_ARG;
    if (a->S > INT32_MAX / (C / G)) return RMSNORM_ERR_INVALID_ARG;
    if (a->S > 0 && a->B > INT64_MAX / 16 / a->S / C) return RMSNORM_ERR_INVALID_ARG;
    a->C = static_cast<int>(C);
    a->G = static_cast<int>(G);
    return RMSNORM_OK;
}

int group_norm_run(bool bwd, GroupNormArgs& a, int64_t C, int64_t G, int dtype,
                   const Workspace& given, cudaStream_t stream) {
    int st = group_norm_shape(&a, C, G, dtype);
    if (st != RMSNORM_OK) return st;
    if (a.act < RMSNORM_ACT_NONE || a.act > RMSNORM_ACT_GELU) return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype), wsz = weight_size(dtype);
    if (!aligned(a.mean, 4) || !aligned(a.rstd, 4) || !aligned(a.dw, 4) || !aligned(a.db, 4))
        return RMSNORM_ERR_MISALIGNED;
    if (a.B == 0 || a.S == 0) {
        for (float* p : {a.dw, a.db})
            if (p != nullptr) {
                st = cuda_status(cudaMemsetAsync(p, 0, static_cast<size_t>(C) * 4, stream));
                if (st != RMSNORM_OK) return st;
            }
        return RMSNORM_OK;
    }
    if (a.x == nullptr || a.out == nullptr || a.mean == nullptr || a.rstd == nullptr ||
        (bwd && a.dy == nullptr) || (a.w == nullptr) != (a.b == nullptr) ||
        (bwd && a.w != nullptr && (a.dw == nullptr || a.db == nullptr)))
        return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(a.x, sz) || !aligned(a.out, sz) || !aligned(a.dy, sz) || !aligned(a.w, wsz) ||
        !aligned(a.b, wsz))
        return RMSNORM_ERR_MISALIGNED;
    if (bwd && a.w == nullptr) a.dw = a.db = nullptr;
    a.w_f32 = wsz == 4;
    const bool vec = aligned(a.x, 16) && aligned(a.out, 16) && aligned(a.dy, 16) && (C * sz) % 16 == 0;
    const DeviceInfo* dev = nullptr;
    st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    a.status = dev->status_word;
    a.wait_limit_ns = g_wait_limit_ns.load();
    if (!group_norm_fits(*dev, dtype, vec, bwd, a)) return RMSNORM_ERR_INVALID_ARG;
    Workspace ws = given;
    st = ws.take(group_norm_workspace(*dev, dtype, vec, bwd, a), stream);
    if (st != RMSNORM_OK) return st;
    st = cuda_status(group_norm_launch(*dev, dtype, vec, bwd, a, ws.p, stream));
    return ws.give(st, stream);
}

GroupNormArgs group_norm_fwd_args(const void* x, const void* w, const void* b, void* y, float* mean,
                                  float* rstd, int64_t B, int64_t S, float eps, int act) {
    GroupNormArgs a{};
    a.x = x;
    a.w = w;
    a.b = b;
    a.out = y;
    a.mean = mean;
    a.rstd = rstd;
    a.B = B;
    a.S = S;
    a.eps = eps;
    a.act = act;
    return a;
}
GroupNormArgs group_norm_bwd_args(const void* x, const void* w, const void* b, const void* dy,
                                  const float* mean, const float* rstd, void* dx, float* dw,
                                  float* db, int64_t B, int64_t S, int act) {
    // mean and rstd are only read in this direction
    GroupNormArgs a = group_norm_fwd_args(x, w, b, dx, const_cast<float*>(mean),
                                          const_cast<float*>(rstd), B, S, 0.f, act);
    a.dy = dy;
    a.dw = dw;
    a.db = db;
    return a;
}

}  // namespace

int64_t take_drop_unit() { return g_drop_unit.exchange(-1); }

int pdl_mode() {
    static const int mode = [] {
        const char* v = getenv("RMSNORM_PDL");
        return (v == nullptr || *v == 0) ? 1 : (atoi(v) != 0 ? 1 : 0);
    }();
    return mode;
}

const DeviceInfo* device_info(int device) {
    if (device < 0 || device >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (g_dev_ready[device]) return &g_dev[device];
    int prev = -1;
    if (cudaGetDevice(&prev) != cudaSuccess || (prev != device && cudaSetDevice(device) != cudaSuccess)) {
        cudaGetLastError();
        return nullptr;
    }
    DeviceInfo d;
    d.device = device;
    bool ok = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, device) == cudaSuccess &&
              cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device) == cudaSuccess &&
              cudaDeviceGetAttribute(&d.l2_bytes, cudaDevAttrL2CacheSize, device) == cudaSuccess &&
              cudaGetSymbolAddress(reinterpret_cast<void**>(&d.status_word), g_status_word) == cudaSuccess;
    if (prev != device) cudaSetDevice(prev);
    if (!ok || d.sm_count <= 0) {
        cudaGetLastError();
        return nullptr;
    }
    g_dev[device] = d;
    g_dev_ready[device] = true;
    return &g_dev[device];
}

}  // namespace rmsn

using namespace rmsn;

extern "C" {

int rmsnorm_fwd(const void* x, const void* w, void* y, float* rstd, int64_t M, int64_t N,
                float eps, int dtype, cudaStream_t stream) {
    return fwd_run(x, nullptr, w, nullptr, y, rstd, M, N, eps, dtype, stream);
}

int rmsnorm_add_fwd(const void* x, const void* residual, const void* w, void* h, void* y,
                    float* rstd, int64_t M, int64_t N, float eps, int dtype,
                    cudaStream_t stream) {
    if (M > 0 && (residual == nullptr || h == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    return fwd_run(x, residual, w, h, y, rstd, M, N, eps, dtype, stream);
}

size_t rmsnorm_bwd_workspace_size(int64_t M, int64_t N, int dtype, int device) {
    if (shape_status(M, N, dtype) != RMSNORM_OK || M == 0) return 0;
    const DeviceInfo* dev = device_info(device);
    if (!dev) return 0;
    rmsnorm_plan_t plan;
    // the workspace only depends on the partial-row count; take the largest
    // of the vector and scalar plans so either alignment class fits
    size_t need = 0;
    for (int vec = 0; vec < 2; ++vec) {
        if (vec && (N * dtype_size(dtype)) % 16 != 0) continue;
        bwd_choose(N, dtype, vec != 0, &plan);
        if (cuda_status(bwd_finish_plan(*dev, dtype, M, N, &plan)) != RMSNORM_OK) return 0;
        if (static_cast<size_t>(plan.workspace_bytes) > need) need = static_cast<size_t>(plan.workspace_bytes);
    }
    return need;
}

int rmsnorm_bwd_ws(const void* x, const void* w, const void* dy, const float* rstd, void* dx,
                   float* dw, int64_t M, int64_t N, int dtype, void* workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
    const DeviceInfo* dev = nullptr;
    rmsnorm_plan_t plan;
    int st = bwd_prepare(x, w, dy, rstd, dx, dw, M, N, dtype, &dev, &plan);
    if (st != RMSNORM_OK) return st;
    if (M == 0) {
        if (dw == nullptr) return RMSNORM_OK;
        return cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * 4, stream));
    }
    if (plan.workspace_bytes > 0 &&
        (workspace == nullptr || workspace_bytes < static_cast<size_t>(plan.workspace_bytes)))
        return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return RMSNORM_ERR_MISALIGNED;
    return bwd_run(x, w, dy, rstd, dx, dw, M, N, dtype, *dev, plan, workspace, stream);
}

int rmsnorm_bwd(const void* x, const void* w, const void* dy, const float* rstd, void* dx,
                float* dw, int64_t M, int64_t N, int dtype, cudaStream_t stream) {
    return bwd_alloc_run(x, w, dy, rstd, nullptr, dx, dw, M, N, dtype, stream);
}

int rmsnorm_add_bwd(const void* h, const void* w, const void* dy, const float* rstd,
                    const void* dres, void* dx, float* dw, int64_t M, int64_t N, int dtype,
                    cudaStream_t stream) {
    return bwd_alloc_run(h, w, dy, rstd, dres, dx, dw, M, N, dtype, stream);
}

int rmsnorm_bwd_naive(const void* x, const void* w, const void* dy, void* dx, float* dw,
                      int64_t M, int64_t N, float eps, int dtype, cudaStream_t stream) {
    int st = shape_status(M, N, dtype);
    if (st != RMSNORM_OK) return st;
    if (!(eps >= 0.f)) return RMSNORM_ERR_INVALID_ARG;
    if (dw != nullptr && !aligned(dw, 4)) return RMSNORM_ERR_MISALIGNED;
    if (M == 0) {
        if (dw == nullptr) return RMSNORM_OK;
        return cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * 4, stream));
    }
    if (!x || !w || !dy || !dx || !dw) return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype), wsz = weight_size(dtype);
    if (!aligned(x, sz) || !aligned(w, wsz) || !aligned(dy, sz) || !aligned(dx, sz))
        return RMSNORM_ERR_MISALIGNED;
    const bool vec = aligned(x, 16) && aligned(w, 16) && aligned(dy, 16) && aligned(dx, 16) &&
                     (N * sz) % 16 == 0 && (N * wsz) % 16 == 0;
    if (!vec || N / dtype_vec(dtype) > kNaiveMaxVectors || M > INT32_MAX)
        return RMSNORM_ERR_UNSUPPORTED;
    const DeviceInfo* dev = nullptr;
    st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    void* ws = nullptr;
    if (cuda_status(cudaMallocAsync(&ws, naive_workspace_bytes(M, N, dtype), stream)) != RMSNORM_OK)
        return RMSNORM_ERR_NOMEM;
    st = cuda_status(naive_launch(dtype, x, w, dy, dx, dw, M, static_cast<int>(N), eps, ws, stream));
    const int freed = cuda_status(cudaFreeAsync(ws, stream));
    if (st == RMSNORM_OK) st = freed;
    return st;
}

int rmsnorm_qk_rope_fwd(const rmsnorm_rope_t* rope, const void* q, const void* k, const void* wq,
                        const void* wk, const void* positions, const float* inv_freq, void* q_out,
                        void* k_out, float eps, int dtype, cudaStream_t stream) {
    RopeArgs a{};
    int st = rope_descriptor(rope, dtype, &a);
    if (st != RMSNORM_OK) return st;
    if (!(eps >= 0.f)) return RMSNORM_ERR_INVALID_ARG;
    if (a.tokens == 0 || a.t[0].heads + a.t[1].heads == 0) return RMSNORM_OK;
    return rope_run(rope, a, q, k, wq, wk, positions, inv_freq, nullptr, nullptr, q_out, k_out,
                    nullptr, nullptr, eps, dtype, false, Workspace{}, stream);
}

int rmsnorm_qk_rope_bwd(const rmsnorm_rope_t* rope, const void* q, const void* k, const void* wq,
                        const void* wk, const void* positions, const float* inv_freq,
                        const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                        float* dwk, float eps, int dtype, cudaStream_t stream) {
    return rope_bwd_any(rope, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq, dwk,
                        eps, dtype, Workspace{}, stream);
}

int rmsnorm_qk_rope_bwd_ws(const rmsnorm_rope_t* rope, const void* q, const void* k, const void* wq,
                           const void* wk, const void* positions, const float* inv_freq,
                           const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                           float* dwk, float eps, int dtype, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    return rope_bwd_any(rope, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq, dwk,
                        eps, dtype, Workspace{workspace, workspace_bytes, true}, stream);
}

size_t rmsnorm_qk_rope_bwd_workspace_size(int head_dim, int device) {
    if (head_dim < 2 || head_dim > RMSNORM_ROPE_MAX_HEAD_DIM || head_dim % 2) return 0;
    const DeviceInfo* dev = device_info(device);
    return dev == nullptr ? 0 : static_cast<size_t>(rope_bwd_max_rows(*dev)) * head_dim * 4;
}

int rmsnorm_group_norm_fwd(const void* x, const void* w, const void* b, void* y, float* mean,
                           float* rstd, int64_t B, int64_t S, int64_t C, int64_t G, float eps,
                           int act, int dtype, cudaStream_t stream) {
    if (!(eps >= 0.f)) return RMSNORM_ERR_INVALID_ARG;
    GroupNormArgs a = group_norm_fwd_args(x, w, b, y, mean, rstd, B, S, eps, act);
    return group_norm_run(false, a, C, G, dtype, Workspace{}, stream);
}

int rmsnorm_group_norm_fwd_ws(const void* x, const void* w, const void* b, void* y, float* mean,
                              float* rstd, int64_t B, int64_t S, int64_t C, int64_t G, float eps,
                              int act, int dtype, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
    if (!(eps >= 0.f)) return RMSNORM_ERR_INVALID_ARG;
    GroupNormArgs a = group_norm_fwd_args(x, w, b, y, mean, rstd, B, S, eps, act);
    return group_norm_run(false, a, C, G, dtype, Workspace{workspace, workspace_bytes, true}, stream);
}

int rmsnorm_group_norm_bwd(const void* x, const void* w, const void* b, const void* dy,
                           const float* mean, const float* rstd, void* dx, float* dw, float* db,
                           int64_t B, int64_t S, int64_t C, int64_t G, int act, int dtype,
                           cudaStream_t stream) {
    GroupNormArgs a = group_norm_bwd_args(x, w, b, dy, mean, rstd, dx, dw, db, B, S, act);
    return group_norm_run(true, a, C, G, dtype, Workspace{}, stream);
}

int rmsnorm_group_norm_bwd_ws(const void* x, const void* w, const void* b, const void* dy,
                              const float* mean, const float* rstd, void* dx, float* dw, float* db,
                              int64_t B, int64_t S, int64_t C, int64_t G, int act, int dtype,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    GroupNormArgs a = group_norm_bwd_args(x, w, b, dy, mean, rstd, dx, dw, db, B, S, act);
    return group_norm_run(true, a, C, G, dtype, Workspace{workspace, workspace_bytes, true}, stream);
}

size_t rmsnorm_group_norm_workspace_size(int64_t B, int64_t S, int64_t C, int64_t G, int dtype,
                                         int backward, int device) {
    GroupNormArgs a = group_norm_fwd_args(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, B, S,
                                          0.f, RMSNORM_ACT_NONE);
    if (group_norm_shape(&a, C, G, dtype) != RMSNORM_OK || B == 0 || S == 0) return 0;
    const DeviceInfo* dev = device_info(device);
    if (dev == nullptr) return 0;
    float one = 0.f;
    a.dw = a.db = &one;  // the largest need: with weight gradients
    // whatever the tensors' alignment and the activation, whose kernels may
    // differ in how many blocks run at once
    size_t need = group_norm_workspace(*dev, dtype, false, backward != 0, a);
    for (int act = RMSNORM_ACT_NONE; act <= RMSNORM_ACT_GELU; ++act) {
        a.act = act;
        if ((C * dtype_size(dtype)) % 16 == 0)
            need = std::max(need, group_norm_workspace(*dev, dtype, true, backward != 0, a));
    }
    return need;
}

int rmsnorm_get_last_device_error(cudaStream_t stream) {
    if (cuda_status(cudaStreamSynchronize(stream)) != RMSNORM_OK) return RMSNORM_ERR_CUDA;
    const DeviceInfo* dev = nullptr;
    if (current_device(&dev) != RMSNORM_OK) return RMSNORM_ERR_CUDA;
    int v = 0;
    if (cuda_status(cudaMemcpy(&v, dev->status_word, sizeof v, cudaMemcpyDeviceToHost)) != RMSNORM_OK)
        return RMSNORM_ERR_CUDA;
    if (v != 0 && cuda_status(cudaMemset(dev->status_word, 0, sizeof v)) != RMSNORM_OK)
        return RMSNORM_ERR_CUDA;
    return v;
}

const char* rmsnorm_status_string(int status) {
    switch (status) {
        case RMSNORM_OK: return "RMSNORM_OK";
        case RMSNORM_ERR_INVALID_ARG: return "RMSNORM_ERR_INVALID_ARG";
        case RMSNORM_ERR_UNSUPPORTED: return "RMSNORM_ERR_UNSUPPORTED";
        case RMSNORM_ERR_MISALIGNED: return "RMSNORM_ERR_MISALIGNED";
        case RMSNORM_ERR_CUDA: return "RMSNORM_ERR_CUDA";
        case RMSNORM_ERR_NOMEM: return "RMSNORM_ERR_NOMEM";
        case RMSNORM_ERR_DEVICE_TIMEOUT: return "RMSNORM_ERR_DEVICE_TIMEOUT";
        case RMSNORM_ERR_OUT_OF_BOUNDS: return "RMSNORM_ERR_OUT_OF_BOUNDS";
        default: return "RMSNORM_STATUS_UNKNOWN";
    }
}

void rmsnorm_set_wait_limit_ns(uint64_t ns) {
    g_wait_limit_ns.store(ns == 0 ? kDefaultWaitLimitNs : ns);
}

void rmsnorm_test_drop_copy(int64_t unit) { g_drop_unit.store(unit < 0 ? -1 : unit); }

int rmsnorm_probe(int kind, void* dst, const void* a, const void* b, size_t bytes,
                  int blocks_per_sm, cudaStream_t stream) {
    if (kind < RMSNORM_PROBE_COPY || kind > RMSNORM_PROBE_2R1W) return RMSNORM_ERR_INVALID_ARG;
    if (bytes % 16 != 0 || blocks_per_sm < 1) return RMSNORM_ERR_INVALID_ARG;
    if (bytes == 0) return RMSNORM_OK;
    if (dst == nullptr) return RMSNORM_ERR_INVALID_ARG;
    if (kind != RMSNORM_PROBE_WRITE && a == nullptr) return RMSNORM_ERR_INVALID_ARG;
    if (kind == RMSNORM_PROBE_2R1W && b == nullptr) return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(dst, 16) || (a && !aligned(a, 16)) || (b && !aligned(b, 16)))
        return RMSNORM_ERR_MISALIGNED;
    const DeviceInfo* dev = nullptr;
    int st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    const int grid = dev->sm_count * blocks_per_sm;
    return cuda_status(probe_launch(kind, dst, a, b, bytes, grid, stream));
}

int rmsnorm_plan(int64_t M, int64_t N, int dtype, int pass, int device, rmsnorm_plan_t* out) {
    if (out == nullptr) return RMSNORM_ERR_INVALID_ARG;
    int st = shape_status(M, N, dtype);
    if (st != RMSNORM_OK) return st;
    if (pass < RMSNORM_PASS_FWD || pass > RMSNORM_PASS_FWD_ADD) return RMSNORM_ERR_INVALID_ARG;
    const bool fwd = pass == RMSNORM_PASS_FWD || pass == RMSNORM_PASS_FWD_ADD;
    if (M == 0) {
        *out = rmsnorm_plan_t{};
        return RMSNORM_OK;
    }
    const bool vec = (N * dtype_size(dtype)) % 16 == 0;
    if (fwd)
        fwd_choose(N, dtype, vec, out, pass == RMSNORM_PASS_FWD_ADD);
    else
        bwd_choose(N, dtype, vec, out, pass == RMSNORM_PASS_BWD_RES);
    if (device < 0) return RMSNORM_OK;
    const DeviceInfo* dev = device_info(device);
    if (!dev) return RMSNORM_ERR_CUDA;
    cudaError_t e = fwd ? fwd_finish_plan(*dev, dtype, M, N, out, pass == RMSNORM_PASS_FWD_ADD)
                                             : bwd_finish_plan(*dev, dtype, M, N, out,
                                                               pass == RMSNORM_PASS_BWD_RES);
    return cuda_status(e);
}

#ifdef RMSNORM_CHECKS
const char* rmsnorm_version(void) { return "0.2.0+checks"; }
#else
const char* rmsnorm_version(void) { return "0.2.0"; }
#endif

}  // extern "C"
