// C ABI of the operators that move rows by an index (declared in rmsnorm.h):
// argument checks, workspaces and the calls into embedding.cu, sort.cu and
// experts.cu.
#include <algorithm>
#include <cstdint>

#include "api_util.h"
#include "rows.h"

namespace rmsn {
namespace {

constexpr int64_t kMaxCount = INT32_MAX;

// Rows of `width` elements `stride` apart: none overlaps the next where they are
// written, and no offset passes 2^60 bytes.
int row_stride_status(int64_t rows, int64_t width, int64_t stride, bool written) {
    if (stride < 0 || (written && rows > 1 && stride < width)) return RMSNORM_ERR_INVALID_ARG;
    if (rows > 1 && stride > (int64_t{1} << 58) / rows) return RMSNORM_ERR_INVALID_ARG;
    return RMSNORM_OK;
}

// ---------------------------------------------------------------- embedding
int embedding_args(const rmsnorm_embedding_t* d, const void* ids, int dtype, bool bwd, int64_t skip,
                   EmbeddingArgs* a) {
    if (d == nullptr || !dtype_known(dtype)) return RMSNORM_ERR_INVALID_ARG;
    if (d->outer < 0 || d->inner < 0 || (d->inner > 0 && d->outer > kMaxCount / d->inner))
        return RMSNORM_ERR_INVALID_ARG;
    if (d->num_rows < 1 || d->num_rows > kMaxCount || d->width < 1 || d->width > kMaxCount)
        return RMSNORM_ERR_INVALID_ARG;
    const int64_t n = d->outer * d->inner;
    if (d->id_stride[0] < 0 || d->id_stride[1] < 0 || d->id_stride[0] > (int64_t{1} << 40) ||
        d->id_stride[1] > (int64_t{1} << 40))
        return RMSNORM_ERR_INVALID_ARG;
    int st = row_stride_status(d->num_rows, d->width, d->table_stride, bwd);
    if (st == RMSNORM_OK) st = row_stride_status(n, d->width, d->row_stride, !bwd);
    if (st != RMSNORM_OK) return st;
    if (!embedding_fits(n, d->width)) return RMSNORM_ERR_INVALID_ARG;
    if (n > 0 && ids == nullptr) return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(ids, d->ids_64 ? 8 : 4)) return RMSNORM_ERR_MISALIGNED;
    a->k = {ids, d->id_stride[0], d->id_stride[1], static_cast<unsigned>(n), static_cast<unsigned>(d->inner),
            d->num_rows, skip < 0 ? -1 : skip, d->ids_64 != 0};
    a->rows = d->num_rows;
    a->width = static_cast<int>(d->width);
    a->scale = d->scale;
    a->src_stride = bwd ? d->row_stride : d->table_stride;
    a->dst_stride = bwd ? d->table_stride : d->row_stride;
    return RMSNORM_OK;
}

int embedding_bwd(const rmsnorm_embedding_t* d, const void* ids, const void* dy, void* grad, int64_t padding_id,
                  int accumulate, int dtype, const Workspace& given, cudaStream_t stream) {
    EmbeddingArgs a{};
    int st = embedding_args(d, ids, dtype, true, padding_id, &a);
    if (st != RMSNORM_OK) return st;
    const int sz = dtype_size(dtype), gsz = weight_size(dtype);
    if (grad == nullptr || (a.k.n > 0 && dy == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(dy, sz) || !aligned(grad, gsz)) return RMSNORM_ERR_MISALIGNED;
    if (a.k.n == 0) {
        if (accumulate) return RMSNORM_OK;
        const size_t row = static_cast<size_t>(a.width) * gsz;
        return cuda_status(cudaMemset2DAsync(grad, a.rows > 1 ? static_cast<size_t>(a.dst_stride) * gsz : row, 0, row,
                                             static_cast<size_t>(a.rows), stream));
    }
    const DeviceInfo* dev = nullptr;
    st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    a.src = dy;
    a.dst = grad;
    a.status = dev->status_word;
    Workspace ws = given;
    st = ws.take(embedding_bwd_workspace(a.k.n, a.rows, a.width), stream);
    if (st != RMSNORM_OK) return st;
    st = cuda_status(embedding_bwd_launch(*dev, dtype, a, accumulate != 0, ws.p, stream));
    return ws.give(st, stream);
}

// ------------------------------------------------------------------ experts
int64_t expert_rows(int64_t tokens, int64_t choices, int64_t experts, int64_t align) {
    if (tokens < 0 || choices < 1 || choices > kMaxCount || tokens > kMaxCount / choices || experts < 1 ||
        experts > RMSNORM_MAX_EXPERTS || align < 1 || align > kMaxCount)
        return -1;
    const int64_t n = tokens * choices;
    const int64_t rows = (n + std::min(experts, n) * (align - 1)) / align * align;
    return rows > kMaxCount ? -1 : rows;
}

int expert_sort(const void* experts, int experts_64, int64_t tokens, int64_t choices, int64_t num_experts,
                int64_t align, int64_t rows, int32_t* position, int32_t* source, int32_t* offsets, int32_t* counts,
                const Workspace& given, cudaStream_t stream) {
    const int64_t need = expert_rows(tokens, choices, num_experts, align);
    if (need < 0 || rows < need || rows > kMaxCount) return RMSNORM_ERR_INVALID_ARG;
    const int64_t n = tokens * choices;
    if (offsets == nullptr || counts == nullptr || (n > 0 && (experts == nullptr || position == nullptr)) ||
        (rows > 0 && source == nullptr))
        return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(experts, experts_64 ? 8 : 4) || !aligned(position, 4) || !aligned(source, 4) || !aligned(offsets, 4) ||
        !aligned(counts, 4))
        return RMSNORM_ERR_MISALIGNED;
    const DeviceInfo* dev = nullptr;
    int st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    ExpertSortArgs a{};
    a.k = {experts, n, 1, static_cast<unsigned>(n), static_cast<unsigned>(n), num_experts, -1, experts_64 != 0};
    a.position = position;
    a.source = source;
    a.offsets = offsets;
    a.counts = counts;
    a.rows = static_cast<int32_t>(rows);
    a.align = static_cast<int32_t>(align);
    a.status = dev->status_word;
    Workspace ws = given;
    st = ws.take(static_cast<size_t>(sort_counts_words(n, static_cast<int>(num_experts) + 1)) * 4, stream);
    if (st != RMSNORM_OK) return st;
    a.block_counts = static_cast<uint32_t*>(ws.p);
    st = cuda_status(expert_sort_launch(*dev, a, stream));
    return ws.give(st, stream);
}

// What every call by token and row checks; written: which of the two is an output.
int expert_args(const rmsnorm_experts_t* d, const int32_t* position, int dtype, bool tokens_written, bool rows_written,
                ExpertArgs* a) {
    if (d == nullptr || !dtype_known(dtype)) return RMSNORM_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->choices < 1 || d->tokens > kMaxCount / d->choices || d->rows < 0 || d->rows > kMaxCount ||
        d->width < 1 || d->width > kMaxCount)
        return RMSNORM_ERR_INVALID_ARG;
    int st = row_stride_status(d->tokens, d->width, d->token_stride, tokens_written);
    if (st == RMSNORM_OK) st = row_stride_status(d->rows, d->width, d->row_stride, rows_written);
    if (st != RMSNORM_OK) return st;
    a->position = position;
    a->tokens = d->tokens;
    a->rows = static_cast<int>(d->rows);
    a->choices = d->choices;
    a->width = static_cast<int>(d->width);
    if (!experts_fit(*a) || (d->tokens > 0 && position == nullptr)) return RMSNORM_ERR_INVALID_ARG;
    return aligned(position, 4) ? RMSNORM_OK : RMSNORM_ERR_MISALIGNED;
}

template <typename Launch>
int expert_launch(Launch launch, int dtype, ExpertArgs& a, cudaStream_t stream) {
    const DeviceInfo* dev = nullptr;
    const int st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    a.status = dev->status_word;
    return cuda_status(launch(*dev, dtype, a, stream));
}

}  // namespace
}  // namespace rmsn

using namespace rmsn;

extern "C" {

int rmsnorm_embedding_fwd(const rmsnorm_embedding_t* embedding, const void* ids, const void* table, void* y, int dtype,
                          cudaStream_t stream) {
    EmbeddingArgs a{};
    int st = embedding_args(embedding, ids, dtype, false, -1, &a);
    if (st != RMSNORM_OK) return st;
    if (a.k.n == 0) return RMSNORM_OK;
    if (table == nullptr || y == nullptr) return RMSNORM_ERR_INVALID_ARG;
    if (!aligned(table, weight_size(dtype)) || !aligned(y, dtype_size(dtype))) return RMSNORM_ERR_MISALIGNED;
    const DeviceInfo* dev = nullptr;
    st = current_device(&dev);
    if (st != RMSNORM_OK) return st;
    a.src = table;
    a.dst = y;
    a.status = dev->status_word;
    return cuda_status(embedding_fwd_launch(*dev, dtype, a, stream));
}

int rmsnorm_embedding_bwd(const rmsnorm_embedding_t* embedding, const void* ids, const void* dy, void* grad,
                          int64_t padding_id, int accumulate, int dtype, cudaStream_t stream) {
    return embedding_bwd(embedding, ids, dy, grad, padding_id, accumulate, dtype, Workspace{}, stream);
}

int rmsnorm_embedding_bwd_ws(const rmsnorm_embedding_t* embedding, const void* ids, const void* dy, void* grad,
                             int64_t padding_id, int accumulate, int dtype, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
    return embedding_bwd(embedding, ids, dy, grad, padding_id, accumulate, dtype,
                         Workspace{workspace, workspace_bytes, true}, stream);
}

size_t rmsnorm_embedding_bwd_workspace_size(int64_t tokens, int64_t num_rows, int64_t width) {
    if (tokens < 0 || tokens > kMaxCount || num_rows < 1 || num_rows > kMaxCount || width < 1 || width > kMaxCount ||
        !embedding_fits(tokens, width))
        return 0;
    return embedding_bwd_workspace(tokens, num_rows, width);
}

int64_t rmsnorm_expert_rows(int64_t tokens, int64_t choices, int64_t num_experts, int64_t align) {
    return expert_rows(tokens, choices, num_experts, align);
}

int rmsnorm_expert_sort(const void* experts, int experts_64, int64_t tokens, int64_t choices, int64_t num_experts,
                        int64_t align, int64_t rows, int32_t* position, int32_t* source, int32_t* offsets,
                        int32_t* counts, cudaStream_t stream) {
    return expert_sort(experts, experts_64, tokens, choices, num_experts, align, rows, position, source, offsets,
                       counts, Workspace{}, stream);
}

int rmsnorm_expert_sort_ws(const void* experts, int experts_64, int64_t tokens, int64_t choices, int64_t num_experts,
                           int64_t align, int64_t rows, int32_t* position, int32_t* source, int32_t* offsets,
                           int32_t* counts, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return expert_sort(experts, experts_64, tokens, choices, num_experts, align, rows, position, source, offsets,
                       counts, Workspace{workspace, workspace_bytes, true}, stream);
}

size_t rmsnorm_expert_sort_workspace_size(int64_t tokens, int64_t choices, int64_t num_experts) {
    if (expert_rows(tokens, choices, num_experts, 1) < 0) return 0;
    return static_cast<size_t>(sort_counts_words(tokens * choices, static_cast<int>(num_experts) + 1)) * 4;
}

int rmsnorm_expert_dispatch_fwd(const rmsnorm_experts_t* experts, const void* x, const int32_t* position,
                                const int32_t* source, void* rows, int dtype, cudaStream_t stream) {
    ExpertArgs a{};
    int st = expert_args(experts, position, dtype, false, true, &a);
    if (st != RMSNORM_OK) return st;
    if (a.rows == 0) return RMSNORM_OK;
    if ((a.tokens > 0 && x == nullptr) || source == nullptr || rows == nullptr) return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype);
    if (!aligned(x, sz) || !aligned(rows, sz) || !aligned(source, 4)) return RMSNORM_ERR_MISALIGNED;
    a.x = x;
    a.x_stride = experts->token_stride;
    a.source = source;
    a.out = rows;
    a.out_stride = experts->row_stride;
    return expert_launch(expert_scatter_launch, dtype, a, stream);
}

int rmsnorm_expert_dispatch_bwd(const rmsnorm_experts_t* experts, const void* drows, const int32_t* position, void* dx,
                                int dtype, cudaStream_t stream) {
    return rmsnorm_expert_combine_fwd(experts, drows, position, nullptr, nullptr, dx, dtype, stream);
}

int rmsnorm_expert_combine_fwd(const rmsnorm_experts_t* experts, const void* rows, const int32_t* position,
                               const void* weights, const void* residual, void* y, int dtype, cudaStream_t stream) {
    ExpertArgs a{};
    int st = expert_args(experts, position, dtype, true, false, &a);
    if (st != RMSNORM_OK) return st;
    if (residual != nullptr) {
        st = row_stride_status(a.tokens, a.width, experts->residual_stride, false);
        if (st != RMSNORM_OK) return st;
    }
    if (a.tokens == 0) return RMSNORM_OK;
    if ((a.rows > 0 && rows == nullptr) || y == nullptr) return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype);
    if (!aligned(rows, sz) || !aligned(y, sz) || !aligned(residual, sz) || !aligned(weights, weight_size(dtype)))
        return RMSNORM_ERR_MISALIGNED;
    a.x = residual;
    a.x_stride = experts->residual_stride;
    a.in = rows;
    a.in_stride = experts->row_stride;
    a.weights = weights;
    a.out = y;
    a.out_stride = experts->token_stride;
    return expert_launch(expert_gather_launch, dtype, a, stream);
}

int rmsnorm_expert_combine_bwd(const rmsnorm_experts_t* experts, const void* dy, const void* rows,
                               const int32_t* position, const int32_t* source, const void* weights, void* drows,
                               float* dweights, int dtype, cudaStream_t stream) {
    if (weights == nullptr && experts != nullptr) {  // the gradient as it is to every choice's row
        rmsnorm_experts_t d = *experts;
        d.row_stride = d.drow_stride;
        return rmsnorm_expert_dispatch_fwd(&d, dy, position, source, drows, dtype, stream);
    }
    ExpertArgs a{};
    int st = expert_args(experts, position, dtype, false, false, &a);
    if (st != RMSNORM_OK) return st;
    st = row_stride_status(a.rows, a.width, experts->drow_stride, true);
    if (st != RMSNORM_OK) return st;
    if (a.tokens == 0 && a.rows == 0) return RMSNORM_OK;
    if ((a.tokens > 0 && (dy == nullptr || dweights == nullptr)) ||
        (a.rows > 0 && (rows == nullptr || source == nullptr || drows == nullptr)))
        return RMSNORM_ERR_INVALID_ARG;
    const int sz = dtype_size(dtype);
    if (!aligned(dy, sz) || !aligned(rows, sz) || !aligned(drows, sz) || !aligned(weights, weight_size(dtype)) ||
        !aligned(source, 4) || !aligned(dweights, 4))
        return RMSNORM_ERR_MISALIGNED;
    a.x = dy;
    a.x_stride = experts->token_stride;
    a.in = rows;
    a.in_stride = experts->row_stride;
    a.source = source;
    a.weights = weights;
    a.out = drows;
    a.out_stride = experts->drow_stride;
    a.dweights = dweights;
    return expert_launch(expert_gather_bwd_launch, dtype, a, stream);
}

}  // extern "C"
