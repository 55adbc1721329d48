// Tensor-level calls of the operators that move rows by an index: the embedding
// lookup and its gradient, and experts' rows. Host code only, part of binding.cpp.
#pragma once

#include <torch/csrc/Dtype.h>

#include "binding_util.h"

namespace {

struct RowsEntry {
    decltype(&rmsnorm_embedding_fwd) embedding_fwd;
    decltype(&rmsnorm_embedding_bwd_ws) embedding_bwd_ws;
    decltype(&rmsnorm_embedding_bwd_workspace_size) embedding_need;
    decltype(&rmsnorm_expert_rows) expert_rows;
    decltype(&rmsnorm_expert_sort_ws) expert_sort_ws;
    decltype(&rmsnorm_expert_sort_workspace_size) expert_sort_need;
    decltype(&rmsnorm_expert_dispatch_fwd) dispatch_fwd;
    decltype(&rmsnorm_expert_dispatch_bwd) dispatch_bwd;
    decltype(&rmsnorm_expert_combine_fwd) combine_fwd;
    decltype(&rmsnorm_expert_combine_bwd) combine_bwd;
} g_rows;
constexpr int kRowsEntries = 10;

void set_rows_entries(void* const* p) {
    g_rows = {reinterpret_cast<decltype(g_rows.embedding_fwd)>(p[0]),
              reinterpret_cast<decltype(g_rows.embedding_bwd_ws)>(p[1]),
              reinterpret_cast<decltype(g_rows.embedding_need)>(p[2]),
              reinterpret_cast<decltype(g_rows.expert_rows)>(p[3]),
              reinterpret_cast<decltype(g_rows.expert_sort_ws)>(p[4]),
              reinterpret_cast<decltype(g_rows.expert_sort_need)>(p[5]),
              reinterpret_cast<decltype(g_rows.dispatch_fwd)>(p[6]),
              reinterpret_cast<decltype(g_rows.dispatch_bwd)>(p[7]),
              reinterpret_cast<decltype(g_rows.combine_fwd)>(p[8]),
              reinterpret_cast<decltype(g_rows.combine_bwd)>(p[9])};
}

// A tensor as rows of its last dimension: their number and the elements between
// them.
struct Rows {
    int64_t n = 1, stride, width;
    Rows(const at::Tensor& t, const char* name) {
        if (t.dim() < 1) refuse(std::string(name) + " " + text(t) + ": expected rows along the last dimension");
        width = t.size(-1);
        if (t.numel() > 0 && width > 1 && t.stride(-1) != 1)
            bad_value(std::string(name) + ": the last dimension is not dense (call .contiguous() first)");
        stride = width;
        bool any = false;
        for (int64_t i = t.dim() - 2; i >= 0; --i) {
            const int64_t size = t.size(i);
            if (size != 1 && t.numel() > 0) {
                if (!any) stride = t.stride(i);
                else if (t.stride(i) != n * stride)
                    bad_value(std::string(name) + ": its rows have no one stride (call .contiguous() first)");
                any = true;
            }
            n *= size;
        }
    }
};

bool is_index(const at::Tensor& t) { return t.scalar_type() == at::kInt || t.scalar_type() == at::kLong; }

void same_leading(const char* a, const at::Tensor& x, const char* b, const at::Tensor& y) {
    if (x.sizes().slice(0, x.dim() - 1) != y.sizes().slice(0, y.dim() - 1))
        refuse(std::string(a) + " " + text(x) + " of " + b + " " + text(y));
}

at::ScalarType dtype_of(PyObject* o, at::ScalarType otherwise) {
    if (o == Py_None) return otherwise;
    if (!THPDtype_Check(o)) bad_value("expected a torch dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// ---------------------------------------------------------------- embedding
// The ids as outer runs of inner, with a stride each.
void id_strides(const at::Tensor& ids, rmsnorm_embedding_t* d) {
    if (!is_index(ids)) refuse("ids " + text(ids) + ": int32 or int64");
    int64_t size[2] = {1, 1}, stride[2] = {0, 1};  // [1]: the inner
    int level = -1;
    for (int64_t i = ids.dim() - 1; i >= 0 && ids.numel() > 0; --i) {
        if (ids.size(i) == 1) continue;
        if (level >= 0 && ids.stride(i) == size[1 - level] * stride[1 - level]) {
            size[1 - level] *= ids.size(i);
            continue;
        }
        if (++level > 1)
            bad_value("ids: more than two strides (call .contiguous() first)");
        size[1 - level] = ids.size(i);
        stride[1 - level] = ids.stride(i);
    }
    d->outer = ids.numel() > 0 ? size[0] : 0;
    d->inner = size[1];
    d->id_stride[0] = stride[0];
    d->id_stride[1] = stride[1];
    d->ids_64 = ids.scalar_type() == at::kLong;
}

// embedding_forward(ids, table, scale, out_dtype, stream)
PyObject* embedding_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &ids = tensor(a[0], "ids"), &table = tensor(a[1], "table");
        rmsnorm_embedding_t d{};
        if (table.dim() != 2 || table.size(0) < 1 || table.size(1) < 1)
            refuse("table " + text(table) + ": expected [rows, width]");
        d.scale = static_cast<float>(real(a[2]));
        const at::ScalarType type = dtype_of(a[3], table.scalar_type());
        const int code = pair_code(type, table.scalar_type());
        id_strides(ids, &d);
        same_device(table, ids);
        on_gpu(table);
        const Rows rows(table, "table");
        d.num_rows = rows.n;
        d.width = d.row_stride = rows.width;
        d.table_stride = rows.stride;
        Run run(table, a[4]);
        c10::DimVector sizes(ids.sizes());
        sizes.push_back(rows.width);
        const at::Tensor y = make(sizes, type, table);
        const void *pi = ids.const_data_ptr(), *pt = table.const_data_ptr();
        void* py = y.mutable_data_ptr();
        check("rmsnorm_embedding_fwd", [&] { return g_rows.embedding_fwd(&d, pi, pt, py, code, run.stream); });
        return wrap(y);
    });
}

// embedding_backward(ids, dy, num_embeddings, scale, padding_idx, grad_dtype, out, accumulate, stream)
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &ids = tensor(a[0], "ids"), &dy = tensor(a[1], "dy");
        const int64_t V = integer(a[2]);
        rmsnorm_embedding_t d{};
        d.scale = static_cast<float>(real(a[3]));
        if (V < 1) refuse(std::to_string(V) + " embeddings");
        int64_t padding = -1;
        if (a[4] != Py_None) {
            padding = integer(a[4]);
            if (padding < -V || padding >= V)
                refuse("padding_idx " + std::to_string(padding) + " of " + std::to_string(V) + " embeddings");
            if (padding < 0) padding += V;
        }
        Optional out = optional(a[6], "out");
        const bool accumulate = truth(a[7]);
        if (accumulate && !out) refuse("a gradient to accumulate into (out)");
        if (dy.dim() != ids.dim() + 1 || dy.sizes().slice(0, ids.dim()) != ids.sizes() || dy.size(-1) < 1)
            refuse("dy " + text(dy) + " of ids " + text(ids));
        const at::ScalarType type = dtype_of(a[5], out ? out->scalar_type() : dy.scalar_type());
        const int code = pair_code(dy.scalar_type(), type);
        id_strides(ids, &d);
        const Rows rows(dy, "dy");
        d.num_rows = V;
        d.width = rows.width;
        d.row_stride = rows.stride;
        if (out && (out->dim() != 2 || out->size(0) != V || out->size(1) != rows.width || out->scalar_type() != type))
            refuse("out " + text(*out) + ": expected [" + std::to_string(V) + ", " + std::to_string(rows.width) +
                   "] " + c10::toString(type));
        same_device(dy, ids);
        same_device(dy, out);
        on_gpu(dy);
        Run run(dy, a[8]);
        if (!out) out = make({V, rows.width}, type, dy);
        else if (!out->is_inference()) out->unsafeGetTensorImpl()->bump_version();  // autograd is told
        d.table_stride = Rows(*out, "out").stride;
        const size_t need = g_rows.embedding_need(ids.numel(), V, rows.width);
        void* ws = run.workspace(need);
        const void *pi = ids.const_data_ptr(), *pdy = dy.const_data_ptr();
        void* pg = out->mutable_data_ptr();
        check("rmsnorm_embedding_bwd", [&] {
            return g_rows.embedding_bwd_ws(&d, pi, pdy, pg, padding, accumulate, code, ws, need, run.stream);
        });
        return wrap(out);
    });
}

// ------------------------------------------------------------------ experts
// expert_sort(experts, num_experts, align, stream)
PyObject* expert_sort(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor& experts = tensor(a[0], "experts");
        const int64_t E = integer(a[1]), align = integer(a[2]);
        if (!is_index(experts) || experts.dim() < 1 || experts.size(-1) < 1)
            refuse("experts " + text(experts) + ": expected int32 or int64 [..., choices]");
        const int64_t K = experts.size(-1), T = experts.numel() / K;
        const int64_t R = g_rows.expert_rows(T, K, E, align);
        if (R < 0)
            refuse("experts " + text(experts) + " of " + std::to_string(E) + " experts aligned to " +
                   std::to_string(align) + ": 1 to " + std::to_string(RMSNORM_MAX_EXPERTS) +
                   " experts, an alignment of 1 or more, rows up to 2^31-1");
        on_gpu(experts);
        dense(experts);
        Run run(experts, a[3]);
        // one allocation for the four: each cost as much as a fourth of the kernel
        auto room = [](int64_t n) { return (n + 3) / 4 * 4; };
        const at::Tensor all = make({room(T * K) + room(R) + room(E + 1) + E}, at::kInt, experts);
        int64_t used = 0;
        auto part = [&](at::IntArrayRef sizes, int64_t n) {
            at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                                    all.dtype());
            t.unsafeGetTensorImpl()->set_storage_offset(used);
            t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
            used += room(n);
            return t;
        };
        const at::Tensor position = part(experts.sizes(), T * K), source = part({R}, R), offsets = part({E + 1}, E + 1),
                         counts = part({E}, E);
        const size_t need = g_rows.expert_sort_need(T, K, E);
        void* ws = run.workspace(need);
        const void* pe = experts.const_data_ptr();
        const int wide = experts.scalar_type() == at::kLong;
        int32_t *pp = position.mutable_data_ptr<int32_t>(), *ps = source.mutable_data_ptr<int32_t>(),
                *po = offsets.mutable_data_ptr<int32_t>(), *pc = counts.mutable_data_ptr<int32_t>();
        check("rmsnorm_expert_sort", [&] {
            return g_rows.expert_sort_ws(pe, wide, T, K, E, align, R, pp, ps, po, pc, ws, need, run.stream);
        });
        return tuple(position, source, offsets, counts);
    });
}

struct Experts {
    rmsnorm_experts_t d{};
    Experts(const at::Tensor& like, const at::Tensor& position) {
        if (position.scalar_type() != at::kInt || position.dim() < 1 || position.size(-1) < 1 ||
            position.size(-1) > INT32_MAX)
            refuse("position " + text(position) + ": expected int32 [..., choices]");
        same_device(like, position);
        dense(position);
        d.choices = static_cast<int32_t>(position.size(-1));
        d.tokens = position.numel() / d.choices;
    }
    void source(const at::Tensor& like, const at::Tensor& s, int64_t rows) {
        if (s.scalar_type() != at::kInt || s.dim() != 1 || (rows >= 0 && s.size(0) != rows))
            refuse("source " + text(s) + ": expected int32, a value for each row");
        same_device(like, s);
        dense(s);
        d.rows = s.size(0);
    }
};
void sorted_rows(const at::Tensor& t) {
    if (t.dim() != 2 || t.size(1) < 1) refuse("rows " + text(t) + ": expected [rows, width]");
}
at::Tensor by_token(const at::Tensor& position, int64_t width, const at::Tensor& like) {
    c10::DimVector sizes(position.sizes());
    sizes.back() = width;
    return make(sizes, like.scalar_type(), like);
}

// expert_dispatch_forward(x, position, source, stream)
PyObject* expert_dispatch_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &x = tensor(a[0], "x"), &position = tensor(a[1], "position"), &source = tensor(a[2], "source");
        Experts e(x, position);
        e.source(x, source, -1);
        if (x.dim() < 1 || x.size(-1) < 1) refuse("x " + text(x) + ": expected [..., width]");
        same_leading("x", x, "position", position);
        const int code = pair_code(x.scalar_type(), x.scalar_type());
        on_gpu(x);
        const Rows r(x, "x");
        e.d.width = e.d.row_stride = r.width;
        e.d.token_stride = r.stride;
        Run run(x, a[3]);
        const at::Tensor rows = make({e.d.rows, r.width}, x.scalar_type(), x);
        const void* px = x.const_data_ptr();
        const int32_t *pp = position.const_data_ptr<int32_t>(), *ps = source.const_data_ptr<int32_t>();
        void* pr = rows.mutable_data_ptr();
        check("rmsnorm_expert_dispatch_fwd", [&] { return g_rows.dispatch_fwd(&e.d, px, pp, ps, pr, code, run.stream); });
        return wrap(rows);
    });
}

// expert_dispatch_backward(drows, position, stream)
PyObject* expert_dispatch_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &drows = tensor(a[0], "drows"), &position = tensor(a[1], "position");
        sorted_rows(drows);
        Experts e(drows, position);
        const int code = pair_code(drows.scalar_type(), drows.scalar_type());
        on_gpu(drows);
        const Rows r(drows, "drows");
        e.d.rows = r.n;
        e.d.width = e.d.token_stride = r.width;
        e.d.row_stride = r.stride;
        Run run(drows, a[2]);
        const at::Tensor dx = by_token(position, r.width, drows);
        const void* pr = drows.const_data_ptr();
        const int32_t* pp = position.const_data_ptr<int32_t>();
        void* px = dx.mutable_data_ptr();
        check("rmsnorm_expert_dispatch_bwd", [&] { return g_rows.dispatch_bwd(&e.d, pr, pp, px, code, run.stream); });
        return wrap(dx);
    });
}

// weights [..., choices] like position, or none
void check_weights(const Optional& w, const at::Tensor& position, const at::Tensor& like) {
    if (!w) return;
    if (w->sizes() != position.sizes()) refuse("weights " + text(*w) + " of position " + text(position));
    same_device(like, *w);
    dense(*w);
}

// expert_combine_forward(rows, position, weights, residual, stream)
PyObject* expert_combine_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &rows = tensor(a[0], "rows"), &position = tensor(a[1], "position");
        const Optional w = optional(a[2], "weights"), residual = optional(a[3], "residual");
        sorted_rows(rows);
        Experts e(rows, position);
        check_weights(w, position, rows);
        const int code = dtype_code(rows, w);
        const Rows r(rows, "rows");
        e.d.rows = r.n;
        e.d.width = e.d.token_stride = r.width;
        e.d.row_stride = r.stride;
        if (residual) {
            if (residual->dim() != position.dim() || residual->size(-1) != r.width ||
                residual->scalar_type() != rows.scalar_type())
                refuse("residual " + text(*residual) + " of rows " + text(rows));
            same_leading("residual", *residual, "position", position);
            same_device(rows, residual);
            e.d.residual_stride = Rows(*residual, "residual").stride;
        }
        on_gpu(rows);
        Run run(rows, a[4]);
        const at::Tensor y = by_token(position, r.width, rows);
        const void *pr = rows.const_data_ptr(), *pw = data(w), *ph = data(residual);
        const int32_t* pp = position.const_data_ptr<int32_t>();
        void* py = y.mutable_data_ptr();
        check("rmsnorm_expert_combine_fwd",
              [&] { return g_rows.combine_fwd(&e.d, pr, pp, pw, ph, py, code, run.stream); });
        return wrap(y);
    });
}

// expert_combine_backward(dy, rows, position, source, weights, stream)
PyObject* expert_combine_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    return guarded([&]() -> PyObject* {
        const at::Tensor &dy = tensor(a[0], "dy"), &rows = tensor(a[1], "rows"), &position = tensor(a[2], "position"),
                         &source = tensor(a[3], "source");
        const Optional w = optional(a[4], "weights");
        sorted_rows(rows);
        Experts e(rows, position);
        e.source(rows, source, rows.size(0));
        check_weights(w, position, rows);
        const int code = dtype_code(rows, w);
        if (dy.dim() != position.dim() || dy.size(-1) != rows.size(1) || dy.scalar_type() != rows.scalar_type())
            refuse("dy " + text(dy) + " of rows " + text(rows));
        same_leading("dy", dy, "position", position);
        same_device(rows, dy);
        on_gpu(rows);
        const Rows r(rows, "rows"), g(dy, "dy");
        e.d.width = e.d.drow_stride = r.width;
        e.d.row_stride = r.stride;
        e.d.token_stride = g.stride;
        Run run(rows, a[5]);
        const at::Tensor drows = make({r.n, r.width}, rows.scalar_type(), rows);
        Optional dw;
        if (w) dw = make(position.sizes(), at::kFloat, rows);
        const void *pdy = dy.const_data_ptr(), *pr = rows.const_data_ptr(), *pw = data(w);
        const int32_t *pp = position.const_data_ptr<int32_t>(), *ps = source.const_data_ptr<int32_t>();
        void* pd = drows.mutable_data_ptr();
        float* pdw = dw ? dw->mutable_data_ptr<float>() : nullptr;
        check("rmsnorm_expert_combine_bwd",
              [&] { return g_rows.combine_bwd(&e.d, pdy, pr, pp, ps, pw, pd, pdw, code, run.stream); });
        return tuple(drows, dw);
    });
}

}  // namespace
