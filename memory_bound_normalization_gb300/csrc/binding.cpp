// Python binding of the tensor-level calls of group norm and of the rotary
// QK-norm: checks of the arguments, outputs and workspaces from PyTorch's
// caching allocator, and the C entry point on the tensors' device. A call costs
// the launch and the allocations, where the same steps in Python took three
// times as long as the kernels of a decode step.
//
// The module holds no computation: it calls the entry points whose addresses
// image_ops.py hands to setup(), of whichever build of the library is loaded.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstdint>
#include <limits>
#include <optional>
#include <string>

#include "rmsnorm.h"

namespace {

struct Entry {
    decltype(&rmsnorm_group_norm_fwd_ws) gn_fwd_ws;
    decltype(&rmsnorm_group_norm_bwd_ws) gn_bwd_ws;
    decltype(&rmsnorm_group_norm_workspace_size) gn_need;
    decltype(&rmsnorm_qk_rope_fwd) rope_fwd;
    decltype(&rmsnorm_qk_rope_bwd_ws) rope_bwd_ws;
    decltype(&rmsnorm_qk_rope_bwd_workspace_size) rope_need;
} g_entry;
PyObject* g_error = nullptr;  // RMSNormError(status, what)

// Raised as the Python exception it stands for.
struct Refused {
    int status;  // 0: a ValueError
    std::string what;
};
[[noreturn]] void refuse(std::string what) { throw Refused{RMSNORM_ERR_INVALID_ARG, std::move(what)}; }
[[noreturn]] void bad_value(std::string what) { throw Refused{0, std::move(what)}; }

PyObject* raise(const Refused& r) {
    if (r.status == 0) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    }
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.what.c_str());
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

using Optional = std::optional<at::Tensor>;

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad_value(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}
Optional optional(PyObject* o, const char* name) {
    if (o == Py_None) return std::nullopt;
    return tensor(o, name);
}
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

std::string text(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t n : t.sizes()) s += std::to_string(n) + ", ";
    return s + ") " + c10::toString(t.scalar_type());
}

int dtype_code(const at::Tensor& x, const Optional& w) {
    const auto t = x.scalar_type(), u = w ? w->scalar_type() : t;
    const bool wide = u == at::kFloat && t != at::kFloat;
    if (u == t || wide) {
        if (t == at::kFloat) return RMSNORM_F32;
        if (t == at::kBFloat16) return wide ? RMSNORM_BF16_W_F32 : RMSNORM_BF16;
        if (t == at::kHalf) return wide ? RMSNORM_F16_W_F32 : RMSNORM_F16;
    }
    refuse(std::string("unsupported dtypes x=") + c10::toString(t) + " w=" + c10::toString(u));
}

void same_device(const at::Tensor& x, const at::Tensor& t) {
    if (t.device() != x.device()) refuse("tensors on " + t.device().str() + " and " + x.device().str());
}
void same_device(const at::Tensor& x, const Optional& t) {
    if (t) same_device(x, *t);
}
void on_gpu(const at::Tensor& x) {
    if (!x.is_cuda()) bad_value("tensor argument on " + x.device().str() + ": the library takes CUDA tensors");
}
void dense(const at::Tensor& t) {
    if (!t.is_contiguous())
        bad_value("tensor argument is not contiguous: the library takes dense row-major tensors "
                  "(call .contiguous() first)");
}
void dense(const Optional& t) {
    if (t) dense(*t);
}
const void* data(const Optional& t) { return t ? t->const_data_ptr() : nullptr; }

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& like) {
    return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

// The call's device, stream and workspace. A stream that is given is the current
// one meanwhile: the caching allocator then gives memory ordered on it, for the
// outputs as for the workspace.
struct Run {
    c10::cuda::CUDAGuard guard;
    std::optional<c10::cuda::CUDAStreamGuard> on;
    cudaStream_t stream;
    void* ws = nullptr;
    Run(const at::Tensor& x, PyObject* s) : guard(x.device()) {
        const auto device = x.get_device();
        stream = c10::cuda::getCurrentCUDAStream(device).stream();
        if (s == Py_None) return;
        const cudaStream_t there = reinterpret_cast<cudaStream_t>(integer(s));
        if (there == stream) return;
        on.emplace(there == nullptr ? c10::cuda::getDefaultCUDAStream(device)
                                    : c10::cuda::getStreamFromExternal(there, device));
        stream = there;
    }
    ~Run() {
        if (ws != nullptr) c10::cuda::CUDACachingAllocator::raw_delete(ws);
    }
    Run(const Run&) = delete;
    Run& operator=(const Run&) = delete;
    void* workspace(size_t need) {
        if (need > 0) ws = c10::cuda::CUDACachingAllocator::raw_alloc(need);
        return ws;
    }
};

template <typename Call>
void check(const char* what, Call call) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    if (st != RMSNORM_OK) throw Refused{st, what};
}

template <typename F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused& r) {
        return raise(r);
    }
    END_HANDLE_TH_ERRORS
}

PyObject* wrap(const Optional& t) {
    if (!t) Py_RETURN_NONE;
    return THPVariable_Wrap(*t);
}
template <typename... T>
PyObject* tuple(const T&... t) {
    PyObject* items[] = {wrap(Optional(t))...};
    constexpr Py_ssize_t n = sizeof...(T);
    PyObject* out = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (out != nullptr && items[i] != nullptr) PyTuple_SET_ITEM(out, i, items[i]);
        else Py_XDECREF(items[i]);
    }
    return out;
}

// ------------------------------------------------------------- group norm
struct GroupNorm {
    int64_t B, S, C, G;
    int act, code;
};

int activation(PyObject* o) {
    const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    const std::string a = s != nullptr ? s : "?";
    if (a == "none") return RMSNORM_ACT_NONE;
    if (a == "silu") return RMSNORM_ACT_SILU;
    if (a == "gelu") return RMSNORM_ACT_GELU;
    refuse("activation " + a + ": one of none, silu, gelu");
}

GroupNorm group_norm_shape(const at::Tensor& x, int64_t groups, const Optional& w, const Optional& b,
                           PyObject* act) {
    GroupNorm g;
    if (x.dim() < 2) refuse("group norm of " + text(x) + ": expected [B, ..., C]");
    g.act = activation(act);
    g.B = x.size(0);
    g.C = x.size(-1);
    g.G = groups;
    if (groups < 1 || g.C == 0 || g.C % groups != 0)
        refuse(std::to_string(g.C) + " channels in " + std::to_string(groups) + " groups");
    g.S = 1;
    for (int64_t i = 1; i + 1 < x.dim(); ++i) g.S *= x.size(i);
    if (w.has_value() != b.has_value()) refuse("group norm takes a weight and a bias, or neither");
    if (w) {
        if (w->dim() != 1 || w->size(0) != g.C || b->dim() != 1 || b->size(0) != g.C)
            refuse("weight " + text(*w) + " and bias " + text(*b) + " of " + std::to_string(g.C) + " channels");
        if (w->scalar_type() != b->scalar_type()) refuse("weight " + text(*w) + " and bias " + text(*b) + " differ");
    }
    return g;
}

// Workspace needs by shape, the last ones: the library answers for every
// alignment and activation, which takes a few lookups of its own.
size_t group_norm_need(const GroupNorm& g, int backward, int device) {
    struct Kept {
        GroupNorm g;
        int backward, device;
        size_t need;
        bool set;
    };
    static std::array<Kept, 1024> kept{};  // under the interpreter's lock
    const uint64_t h = (g.B * 1000003ull + g.S) * 1000003ull + g.C * 31ull + g.G * 7ull + g.code + backward * 5ull;
    Kept& k = kept[(h ^ (h >> 17)) % kept.size()];
    if (!(k.set && k.g.B == g.B && k.g.S == g.S && k.g.C == g.C && k.g.G == g.G && k.g.code == g.code &&
          k.backward == backward && k.device == device))
        k = {g, backward, device, g_entry.gn_need(g.B, g.S, g.C, g.G, g.code, backward, device), true};
    return k.need;
}

// group_norm_forward(x, num_groups, weight, bias, eps, activation, stream)
PyObject* group_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const Optional w = optional(a[2], "weight"), b = optional(a[3], "bias");
        GroupNorm g = group_norm_shape(x, integer(a[1]), w, b, a[5]);
        const float eps = static_cast<float>(real(a[4]));
        g.code = dtype_code(x, w);
        same_device(x, w);
        same_device(x, b);
        on_gpu(x);
        dense(x);
        dense(w);
        dense(b);
        Run run(x, a[6]);
        const at::Tensor y = make(x.sizes(), x.scalar_type(), x);
        const at::Tensor mean = make({g.B, g.G}, at::kFloat, x), rstd = make({g.B, g.G}, at::kFloat, x);
        if (g.S == 0) {  // means of nothing, which the library leaves unwritten
            mean.fill_(std::numeric_limits<float>::quiet_NaN());
            rstd.fill_(std::numeric_limits<float>::quiet_NaN());
        }
        const size_t need = group_norm_need(g, 0, x.get_device());
        void* ws = run.workspace(need);
        const void *px = x.const_data_ptr(), *pw = data(w), *pb = data(b);
        void* py = y.mutable_data_ptr();
        float *pm = mean.mutable_data_ptr<float>(), *pr = rstd.mutable_data_ptr<float>();
        check("rmsnorm_group_norm_fwd", [&] {
            return g_entry.gn_fwd_ws(px, pw, pb, py, pm, pr, g.B, g.S, g.C, g.G, eps, g.act, g.code, ws, need,
                                     run.stream);
        });
        return tuple(y, mean, rstd);
    });
}

// group_norm_backward(x, num_groups, weight, bias, dy, mean, rstd, activation, stream)
PyObject* group_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor& x = tensor(a[0], "x");
        const Optional w = optional(a[2], "weight"), b = optional(a[3], "bias");
        const at::Tensor &dy = tensor(a[4], "dy"), &mean = tensor(a[5], "mean"), &rstd = tensor(a[6], "rstd");
        GroupNorm g = group_norm_shape(x, integer(a[1]), w, b, a[7]);
        if (dy.sizes() != x.sizes() || dy.scalar_type() != x.scalar_type())
            refuse("dy " + text(dy) + " of x " + text(x));
        for (const at::Tensor* t : {&mean, &rstd})
            if (t->dim() != 2 || t->size(0) != g.B || t->size(1) != g.G || t->scalar_type() != at::kFloat)
                refuse("mean or rstd " + text(*t) + ": expected fp32 [B, num_groups]");
        g.code = dtype_code(x, w);
        same_device(x, w);
        same_device(x, b);
        same_device(x, dy);
        same_device(x, mean);
        same_device(x, rstd);
        on_gpu(x);
        dense(x);
        dense(w);
        dense(b);
        dense(dy);
        dense(mean);
        dense(rstd);
        Run run(x, a[8]);
        const at::Tensor dx = make(x.sizes(), x.scalar_type(), x);
        Optional dw, db;
        if (w) {
            dw = make({g.C}, at::kFloat, x);
            db = make({g.C}, at::kFloat, x);
        }
        const size_t need = group_norm_need(g, 1, x.get_device());
        void* ws = run.workspace(need);
        const void *px = x.const_data_ptr(), *pw = data(w), *pb = data(b), *pdy = dy.const_data_ptr();
        const float *pm = mean.const_data_ptr<float>(), *pr = rstd.const_data_ptr<float>();
        void* pdx = dx.mutable_data_ptr();
        float* pdw = dw ? dw->mutable_data_ptr<float>() : nullptr;
        float* pdb = db ? db->mutable_data_ptr<float>() : nullptr;
        check("rmsnorm_group_norm_bwd", [&] {
            return g_entry.gn_bwd_ws(px, pw, pb, pdy, pm, pr, pdx, pdw, pdb, g.B, g.S, g.C, g.G, g.act, g.code, ws,
                                     need, run.stream);
        });
        return tuple(dx, dw, db);
    });
}

// ------------------------------------------------- rotary positions, QK-norm
// Strides over (batch, token, head) of [T, H, D] or [B, T, H, D].
rmsnorm_strides_t strides(const at::Tensor& t) {
    const auto s = t.strides();
    const int64_t n = t.dim();
    if (s[n - 1] != 1)
        bad_value("the last dimension of a head is not dense (call .contiguous() first)");
    return {n == 4 ? s[0] : 0, s[n - 3], s[n - 2]};
}

void like(const char* name, const at::Tensor& t, const at::Tensor& of) {
    if (t.sizes() != of.sizes() || t.scalar_type() != of.scalar_type() || t.device() != of.device())
        refuse(std::string(name) + " " + text(t) + " on " + t.device().str() + ": expected " + text(of) + " on " +
               of.device().str());
}

struct Rope {
    rmsnorm_rope_t d{};
    int code;
    Rope(const at::Tensor& q, const Optional& k, const Optional& wq, const Optional& wk, const at::Tensor& pos,
         const at::Tensor& freq, PyObject* sections, bool interleaved, bool adjacent) {
        if (q.dim() != 3 && q.dim() != 4)
            refuse("queries " + text(q) + ": expected [T, H, D] or [B, T, H, D]");
        const int64_t n = q.dim(), D = q.size(-1);
        if (k && (k->dim() != n || k->sizes().slice(0, n - 2) != q.sizes().slice(0, n - 2) || k->size(-1) != D ||
                  k->scalar_type() != q.scalar_type()))
            refuse("keys " + text(*k) + " of queries " + text(q));
        if (!k && wk) refuse("a key weight without keys");
        if (k && wq.has_value() != wk.has_value()) refuse("weights for queries and keys, or for neither");
        for (const Optional* w : {&wq, &wk})
            if (*w && ((*w)->dim() != 1 || (*w)->size(0) != D || (*w)->scalar_type() != wq->scalar_type()))
                refuse("weight " + text(**w) + " of heads of " + std::to_string(D));
        const int64_t B = n == 4 ? q.size(0) : 1, T = q.size(n - 3);
        PyObject* seq = PySequence_Fast(sections, "sections: a sequence of numbers of pairs");
        if (seq == nullptr) throw python_error();
        const Py_ssize_t axes = PySequence_Fast_GET_SIZE(seq);
        int64_t pairs = 0;
        try {
            if (axes < 1 || axes > RMSNORM_ROPE_MAX_AXES) refuse(std::to_string(axes) + " position axes");
            for (Py_ssize_t i = 0; i < axes; ++i) {
                const int64_t v = integer(PySequence_Fast_GET_ITEM(seq, i));
                if (v < 0 || v > RMSNORM_ROPE_MAX_HEAD_DIM) refuse("a section of " + std::to_string(v) + " pairs");
                d.sections[i] = static_cast<int32_t>(v);
                pairs += v;
            }
        } catch (...) {
            Py_DECREF(seq);
            throw;
        }
        Py_DECREF(seq);
        if (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong)
            refuse("positions " + text(pos) + ": int32 or int64");
        const bool whole = pos.dim() == n - 1 && (n == 3 || pos.size(1) == B);
        const bool shared = n == 4 && pos.dim() == 2;
        if (!(whole || shared) || pos.size(0) != axes || pos.size(-1) != T)
            refuse("positions " + text(pos) + " of " + std::to_string(axes) + " axes and queries " + text(q));
        if (freq.scalar_type() != at::kFloat || freq.dim() != 1 || freq.size(0) != pairs)
            refuse("inv_freq " + text(freq) + ": expected fp32, a value for each of " + std::to_string(pairs) +
                   " pairs");
        code = dtype_code(q, wq);
        same_device(q, k);
        same_device(q, wq);
        same_device(q, wk);
        same_device(q, pos);
        same_device(q, freq);
        const int64_t Hq = q.size(n - 2), Hk = k ? k->size(n - 2) : 0;
        if (Hq > INT32_MAX || Hk > INT32_MAX || D > INT32_MAX) refuse("queries " + text(q));
        d.batch = B;
        d.length = T;
        d.q_heads = static_cast<int32_t>(Hq);
        d.k_heads = static_cast<int32_t>(Hk);
        d.head_dim = static_cast<int32_t>(D);
        d.rotary_dim = static_cast<int32_t>(2 * pairs);
        d.axes = static_cast<int32_t>(axes);
        d.interleaved = interleaved;
        d.adjacent = adjacent;
        d.positions_64 = pos.scalar_type() == at::kLong;
        d.position_stride[0] = pos.stride(0);
        d.position_stride[1] = pos.dim() == 3 ? pos.stride(1) : 0;
        d.position_stride[2] = pos.stride(-1);
        d.q = strides(q);
        if (k) d.k = strides(*k);
    }
};

// qk_rope_forward(q, k, wq, wk, positions, inv_freq, sections, interleaved, adjacent, eps,
//                 q_out, k_out, stream)
PyObject* qk_rope_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const Optional k = optional(a[1], "k"), wq = optional(a[2], "wq"), wk = optional(a[3], "wk");
        const at::Tensor &pos = tensor(a[4], "positions"), &freq = tensor(a[5], "inv_freq");
        Rope r(q, k, wq, wk, pos, freq, a[6], truth(a[7]), truth(a[8]));
        const float eps = static_cast<float>(real(a[9]));
        Optional qo = optional(a[10], "out of the queries"), ko = optional(a[11], "out of the keys");
        if (qo || ko) {
            if (!qo) refuse("an output for the queries");
            like("out of the queries", *qo, q);
            if (ko.has_value() != k.has_value()) refuse("an output for the keys where there are keys");
            if (k) like("out of the keys", *ko, *k);
        }
        on_gpu(q);
        dense(wq);
        dense(wk);
        dense(freq);
        Run run(q, a[12]);
        if (!qo) {
            qo = make(q.sizes(), q.scalar_type(), q);
            if (k) ko = make(k->sizes(), q.scalar_type(), q);
        } else {
            // autograd is told that what it may have saved has changed
            for (const Optional* o : {&qo, &ko})
                if (*o && !(*o)->is_inference()) (*o)->unsafeGetTensorImpl()->bump_version();
        }
        r.d.q_out = strides(*qo);
        if (k) r.d.k_out = strides(*ko);
        const void *pq = q.const_data_ptr(), *pk = data(k), *pwq = data(wq), *pwk = data(wk),
                   *pp = pos.const_data_ptr();
        const float* pf = freq.const_data_ptr<float>();
        void *po = qo->mutable_data_ptr(), *pko = ko ? ko->mutable_data_ptr() : nullptr;
        check("rmsnorm_qk_rope_fwd", [&] {
            return g_entry.rope_fwd(&r.d, pq, pk, pwq, pwk, pp, pf, po, pko, eps, r.code, run.stream);
        });
        return tuple(qo, ko);
    });
}

// qk_rope_backward(q, k, wq, wk, positions, inv_freq, sections, dq_out, dk_out, interleaved,
//                  adjacent, eps, stream)
PyObject* qk_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor& q = tensor(a[0], "q");
        const Optional k = optional(a[1], "k"), wq = optional(a[2], "wq"), wk = optional(a[3], "wk");
        const at::Tensor &pos = tensor(a[4], "positions"), &freq = tensor(a[5], "inv_freq");
        const at::Tensor& dqo = tensor(a[7], "dq_out");
        const Optional dko = optional(a[8], "dk_out");
        Rope r(q, k, wq, wk, pos, freq, a[6], truth(a[9]), truth(a[10]));
        const float eps = static_cast<float>(real(a[11]));
        like("dq_out", dqo, q);
        if (dko.has_value() != k.has_value()) refuse("a gradient for the keys where there are keys");
        if (k) like("dk_out", *dko, *k);
        r.d.q_out = strides(dqo);
        if (k) r.d.k_out = strides(*dko);
        on_gpu(q);
        dense(wq);
        dense(wk);
        dense(freq);
        Run run(q, a[12]);
        const at::Tensor dq = make(q.sizes(), q.scalar_type(), q);
        r.d.dq = strides(dq);
        Optional dk, dwq, dwk;
        if (k) {
            dk = make(k->sizes(), q.scalar_type(), q);
            r.d.dk = strides(*dk);
        }
        size_t need = 0;
        if (wq) {
            dwq = make(wq->sizes(), at::kFloat, q);
            if (k) dwk = make(wk->sizes(), at::kFloat, q);
            need = g_entry.rope_need(r.d.head_dim, q.get_device());
        }
        void* ws = run.workspace(need);
        const void *pq = q.const_data_ptr(), *pk = data(k), *pwq = data(wq), *pwk = data(wk),
                   *pp = pos.const_data_ptr(), *pdqo = dqo.const_data_ptr(), *pdko = data(dko);
        const float* pf = freq.const_data_ptr<float>();
        void *pdq = dq.mutable_data_ptr(), *pdk = dk ? dk->mutable_data_ptr() : nullptr;
        float* pdwq = dwq ? dwq->mutable_data_ptr<float>() : nullptr;
        float* pdwk = dwk ? dwk->mutable_data_ptr<float>() : nullptr;
        check("rmsnorm_qk_rope_bwd", [&] {
            return g_entry.rope_bwd_ws(&r.d, pq, pk, pwq, pwk, pp, pf, pdqo, pdko, pdq, pdk, pdwq, pdwk, eps, r.code,
                                       ws, need, run.stream);
        });
        return tuple(dq, dk, dwq, dwk);
    });
}

// setup(error type, addresses in the order of Entry)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 7) bad_value("setup: an error type and six addresses");
        void* p[6];
        for (int i = 0; i < 6; ++i) p[i] = reinterpret_cast<void*>(integer(a[i + 1]));
        g_entry = {reinterpret_cast<decltype(g_entry.gn_fwd_ws)>(p[0]),
                   reinterpret_cast<decltype(g_entry.gn_bwd_ws)>(p[1]),
                   reinterpret_cast<decltype(g_entry.gn_need)>(p[2]),
                   reinterpret_cast<decltype(g_entry.rope_fwd)>(p[3]),
                   reinterpret_cast<decltype(g_entry.rope_bwd_ws)>(p[4]),
                   reinterpret_cast<decltype(g_entry.rope_need)>(p[5])};
        Py_INCREF(a[0]);
        Py_XSETREF(g_error, a[0]);
        Py_RETURN_NONE;
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), Py_ssize_t N>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    if (g_error == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "the binding is not set up");
        return nullptr;
    }
    return F(self, a, n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction as_method() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F));
}

PyMethodDef g_methods[] = {
    {"setup", as_method<setup>(), METH_FASTCALL, nullptr},
    {"group_norm_forward", as_method<counted<group_norm_forward, 7>>(), METH_FASTCALL, nullptr},
    {"group_norm_backward", as_method<counted<group_norm_backward, 9>>(), METH_FASTCALL, nullptr},
    {"qk_rope_forward", as_method<counted<qk_rope_forward, 13>>(), METH_FASTCALL, nullptr},
    {"qk_rope_backward", as_method<counted<qk_rope_backward, 13>>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) {
    return PyModule_Create(&g_module);
}
