// Rows of a mixture of experts: tokens' rows sent to the rows of their experts,
// sorted by expert, and weighted sums back, with the gradients.
//
// A row of a token has `choices` rows of its own in the sorted order, anywhere, or
// none. Each kernel goes by token, so that the token's row is moved once and the
// sorted rows once:
//   scatter     out[p_tk] = x_t                           (dispatch)
//   gather      y_t = x_t + sum_k w_tk in[p_tk]           (combine; dispatch backward without x and w)
//   gather_bwd  out[p_tk] = w_tk x_t, dw_tk = <x_t, in[p_tk]>   (combine backward, x the gradient)
// One to three operations a byte: bytes bound all three. The positions are
// what a row's loads wait for, so a thread has the pieces of several choices in
// flight. Sums are fp32 in the choices' order; a result is rounded once.
// Rows of the sorted order without a choice are zeroed by the first blocks, by
// `source` (by the last ones they were the tail of the call).
#include <algorithm>

#include "rows.cuh"

namespace rmsn {
namespace {

constexpr int kThreads = 256;
// Pieces of a lane: small ones need more of them in flight.
__host__ __device__ constexpr int scatter_pieces(int e) { return e >= 4 ? 4 : 8; }
__host__ __device__ constexpr int gather_pieces(int e) { return e >= 4 ? 2 : 8 / e; }
__host__ __device__ constexpr int bwd_pieces(int e) { return e >= 4 ? 2 : 4; }
constexpr int kChoices = 4;     // in flight
constexpr int kBwdChoices = 8;  // dots a thread holds
constexpr int kZeroRows = 64;   // of a block

struct KernelArgs {
    ExpertArgs x;
    RowShape shape;
    unsigned zero_blocks;  // the first ones, which zero rows without a choice
    int team;               // threads of a token (gather_bwd)
};

// Rows without a choice, of kZeroRows: the whole block zeroes one after another.
__device__ __forceinline__ void zero_rows(const KernelArgs& a, int size) {
    const ExpertArgs& x = a.x;
    const int lane = threadIdx.x % 32;
    for (int half = 0; half < kZeroRows; half += 32) {
        const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kZeroRows + half;
        unsigned todo = __ballot_sync(0xffffffffu, row0 + lane < x.rows && x.source[row0 + lane] < 0);
        while (todo) {
            const int r = __ffs(todo) - 1;
            todo &= todo - 1;
            zero_span(static_cast<char*>(x.out) + (row0 + r) * x.out_stride * size, static_cast<int64_t>(x.width) * size,
                      threadIdx.x, kThreads, x.out, rows_bytes(x.rows, x.out_stride, x.width, size), x.status);
        }
    }
}

template <typename T, int E>
__global__ void __launch_bounds__(kThreads) expert_scatter_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kScatterPieces = scatter_pieces(E);
    const ExpertArgs& x = a.x;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x < a.zero_blocks) {
        zero_rows(a, sizeof(T));
        return;
    }
    const unsigned group = group_index<kThreads>(a.shape.lanes, a.zero_blocks);
    const unsigned token = group / a.shape.chunks;
    if (token >= x.tokens) return;
    const int first =
        (group - token * a.shape.chunks) * (a.shape.lanes * kScatterPieces) + (threadIdx.x & (a.shape.lanes - 1));
    const T* src = static_cast<const T*>(x.x) + token * x.x_stride;
    Piece<T, E> v[kScatterPieces];
#pragma unroll
    for (int u = 0; u < kScatterPieces; ++u) {
        const int p = first + u * a.shape.lanes;
        v[u].zero();
        if (p < a.shape.pieces) v[u].load(src + static_cast<int64_t>(p) * E);
    }
    const int32_t* pos = x.position + static_cast<int64_t>(token) * x.choices;
    for (int k = 0; k < x.choices; ++k) {
        const int32_t row = pos[k];
        if (static_cast<uint32_t>(row) >= static_cast<uint32_t>(x.rows)) continue;
        T* to = static_cast<T*>(x.out) + row * x.out_stride;
#pragma unroll
        for (int u = 0; u < kScatterPieces; ++u) {
            const int p = first + u * a.shape.lanes;
            if (p < a.shape.pieces &&
                RMSN_OK(span_in(to + static_cast<int64_t>(p) * E, E * sizeof(T), x.out,
                                rows_bytes(x.rows, x.out_stride, x.width, sizeof(T))),
                        x.status))
                v[u].store(to + static_cast<int64_t>(p) * E);
        }
    }
}

template <typename T, typename TW, int E>
__global__ void __launch_bounds__(kThreads) expert_gather_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kGatherPieces = gather_pieces(E);
    const ExpertArgs& x = a.x;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    const unsigned group = group_index<kThreads>(a.shape.lanes, a.zero_blocks);
    const unsigned token = group / a.shape.chunks;
    if (token >= x.tokens) return;
    const int first =
        (group - token * a.shape.chunks) * (a.shape.lanes * kGatherPieces) + (threadIdx.x & (a.shape.lanes - 1));
    float sum[kGatherPieces][E];
#pragma unroll
    for (int u = 0; u < kGatherPieces; ++u) {
        const int p = first + u * a.shape.lanes;
        Piece<T, E> v;
        v.zero();
        if (x.x != nullptr && p < a.shape.pieces)
            v.load(static_cast<const T*>(x.x) + token * x.x_stride + static_cast<int64_t>(p) * E);
        v.unpack(sum[u]);
    }
    const int32_t* pos = x.position + static_cast<int64_t>(token) * x.choices;
    const TW* wgt = static_cast<const TW*>(x.weights) + static_cast<int64_t>(token) * x.choices;
    for (int k0 = 0; k0 < x.choices; k0 += kChoices) {
        Piece<T, E> v[kChoices][kGatherPieces];
        float w[kChoices];
        bool there[kChoices];
#pragma unroll
        for (int k = 0; k < kChoices; ++k) {
            const int32_t row = k0 + k < x.choices ? pos[k0 + k] : -1;
            there[k] = static_cast<uint32_t>(row) < static_cast<uint32_t>(x.rows);
            w[k] = there[k] && x.weights != nullptr ? to_f32(wgt[k0 + k]) : 1.f;
            const T* src = static_cast<const T*>(x.in) + row * x.in_stride;
#pragma unroll
            for (int u = 0; u < kGatherPieces; ++u) {
                const int p = first + u * a.shape.lanes;
                v[k][u].zero();
                if (there[k] && p < a.shape.pieces) v[k][u].load(src + static_cast<int64_t>(p) * E);
            }
        }
#pragma unroll
        for (int k = 0; k < kChoices; ++k) {
            if (!there[k]) continue;  // also where its weight is infinite or NaN
#pragma unroll
            for (int u = 0; u < kGatherPieces; ++u) {
                float f[E];
                v[k][u].unpack(f);
#pragma unroll
                for (int e = 0; e < E; ++e) sum[u][e] = fmaf(w[k], f[e], sum[u][e]);
            }
        }
    }
    T* to = static_cast<T*>(x.out) + token * x.out_stride;
#pragma unroll
    for (int u = 0; u < kGatherPieces; ++u) {
        const int p = first + u * a.shape.lanes;
        Piece<T, E> out;
        out.pack(sum[u]);
        if (p < a.shape.pieces &&
            RMSN_OK(span_in(to + static_cast<int64_t>(p) * E, E * sizeof(T), x.out,
                            rows_bytes(x.tokens, x.out_stride, x.width, sizeof(T))),
                    x.status))
            out.store(to + static_cast<int64_t>(p) * E);
    }
}

// A team of threads (a power of two, 4 to 256) takes a token and all its columns.
template <typename T, typename TW, int E>
__global__ void __launch_bounds__(kThreads) expert_gather_bwd_kernel(const __grid_constant__ KernelArgs a) {
    constexpr int kBwdPieces = bwd_pieces(E);
    __shared__ float part[kThreads / 32][kBwdChoices];
    const ExpertArgs& x = a.x;
    wait_for_prerequisite_grid();
    allow_dependent_launch();
    if (blockIdx.x < a.zero_blocks) {
        zero_rows(a, sizeof(T));
        return;
    }
    const int team = a.team, lane = threadIdx.x & (team - 1);
    const int64_t token = static_cast<int64_t>(blockIdx.x - a.zero_blocks) * (kThreads / team) + threadIdx.x / team;
    const bool live = token < x.tokens;  // the others keep the barriers company
    const T* dy = static_cast<const T*>(x.x) + token * x.x_stride;
    const int32_t* pos = x.position + token * x.choices;
    const TW* wgt = static_cast<const TW*>(x.weights) + token * x.choices;
    for (int k0 = 0; k0 < x.choices; k0 += kBwdChoices) {
        float dot[kBwdChoices] = {};
        const int here = live ? min(kBwdChoices, x.choices - k0) : 0;
        for (int c = lane; c < (live ? a.shape.pieces : 0); c += team * kBwdPieces) {
            Piece<T, E> g[kBwdPieces];
#pragma unroll
            for (int u = 0; u < kBwdPieces; ++u) {
                const int p = c + u * team;
                g[u].zero();
                if (p < a.shape.pieces) g[u].load(dy + static_cast<int64_t>(p) * E);
            }
#pragma unroll
            for (int k1 = 0; k1 < kBwdChoices; k1 += kChoices) {
                Piece<T, E> v[kChoices][kBwdPieces];
                int32_t row[kChoices];
                if (k1 >= here) break;
#pragma unroll
                for (int k = 0; k < kChoices; ++k) {
                    row[k] = k1 + k < here ? pos[k0 + k1 + k] : -1;
                    if (static_cast<uint32_t>(row[k]) >= static_cast<uint32_t>(x.rows)) row[k] = -1;
                    const T* src = static_cast<const T*>(x.in) + row[k] * x.in_stride;
#pragma unroll
                    for (int u = 0; u < kBwdPieces; ++u) {
                        const int p = c + u * team;
                        v[k][u].zero();
                        if (row[k] >= 0 && p < a.shape.pieces) v[k][u].load(src + static_cast<int64_t>(p) * E);
                    }
                }
#pragma unroll
                for (int k = 0; k < kChoices; ++k) {
                    if (row[k] < 0) continue;
                    const float w = to_f32(wgt[k0 + k1 + k]);
                    T* to = static_cast<T*>(x.out) + row[k] * x.out_stride;
#pragma unroll
                    for (int u = 0; u < kBwdPieces; ++u) {
                        const int p = c + u * team;
                        float f[E], h[E];
                        v[k][u].unpack(f);
                        g[u].unpack(h);
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            dot[k1 + k] = fmaf(f[e], h[e], dot[k1 + k]);
                            f[e] = w * h[e];
                        }
                        Piece<T, E> out;
                        out.pack(f);
                        if (p < a.shape.pieces &&
                            RMSN_OK(span_in(to + static_cast<int64_t>(p) * E, E * sizeof(T), x.out,
                                            rows_bytes(x.rows, x.out_stride, x.width, sizeof(T))),
                                    x.status))
                            out.store(to + static_cast<int64_t>(p) * E);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kBwdChoices; ++k)
            for (int off = min(team, 32) / 2; off >= 1; off /= 2) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], off);
        float* to = x.dweights + token * x.choices + k0;
        if (team <= 32) {
#pragma unroll
            for (int k = 0; k < kBwdChoices; ++k)
                if (lane == 0 && k < here &&
                    RMSN_OK(span_in(to + k, 4, x.dweights, 4 * x.tokens * x.choices), x.status))
                    to[k] = dot[k];
        } else {
            if (threadIdx.x % 32 == 0) {
#pragma unroll
                for (int k = 0; k < kBwdChoices; ++k) part[threadIdx.x / 32][k] = dot[k];
            }
            __syncthreads();
            if (lane < here && RMSN_OK(span_in(to + lane, 4, x.dweights, 4 * x.tokens * x.choices), x.status)) {
                float sum = 0.f;
                for (int w = 0; w < team / 32; ++w) sum += part[threadIdx.x / 32 + w][lane];
                to[lane] = sum;
            }
            __syncthreads();
        }
    }
}

int piece_of(const ExpertArgs& a, int dtype) {
    const int size = dtype_size(dtype);
    for (int e : {8, 4, 2}) {
        if (e * size > 16 || a.width % e) continue;
        if (piece_fits(a.x, a.x_stride, size, e) && piece_fits(a.in, a.in_stride, size, e) &&
            piece_fits(a.out, a.out_stride, size, e))
            return e;
    }
    return 1;
}

unsigned zero_blocks(const ExpertArgs& a) { return static_cast<unsigned>(cdiv(a.rows, kZeroRows)); }

// fn(E) for the piece's width
template <typename T, typename F>
cudaError_t with_piece(int e, F fn) {
    if constexpr (sizeof(T) == 2) {
        if (e == 8) return fn(std::integral_constant<int, 8>());
    }
    if (e == 4) return fn(std::integral_constant<int, 4>());
    if (e == 2) return fn(std::integral_constant<int, 2>());
    return fn(std::integral_constant<int, 1>());
}
// fn(T, TW) for the types
template <typename F>
cudaError_t with_types(int dtype, F fn) {
    switch (dtype) {
        case RMSNORM_F32: return fn(float(), float());
        case RMSNORM_BF16: return fn(__nv_bfloat16(), __nv_bfloat16());
        case RMSNORM_F16: return fn(__half(), __half());
        case RMSNORM_BF16_W_F32: return fn(__nv_bfloat16(), float());
        default: return fn(__half(), float());
    }
}

}  // namespace

bool experts_fit(const ExpertArgs& a) {
    return a.tokens * cdiv(a.width, 32 * gather_pieces(1)) <= kMaxGrid;  // groups, element by element
}

cudaError_t expert_scatter_launch(const DeviceInfo&, int dtype, const ExpertArgs& in, cudaStream_t s) {
    KernelArgs a{in, {}, 0, 0};
    const int e = piece_of(in, dtype);
    a.shape = row_shape(in.width / e, scatter_pieces(e));
    a.zero_blocks = zero_blocks(in);
    const int grid = static_cast<int>(a.zero_blocks + cdiv(in.tokens * a.shape.chunks * a.shape.lanes, kThreads));
    auto go = [&](auto t) {
        using T = decltype(t);
        return with_piece<T>(e, [&](auto n) {
            return launch_pdl(expert_scatter_kernel<T, decltype(n)::value>, grid, kThreads, 0, 1, s, a);
        });
    };
    // a copy: the type's size alone counts
    return dtype_size(dtype) == 4 ? go(float()) : go(__nv_bfloat16());
}

cudaError_t expert_gather_launch(const DeviceInfo&, int dtype, const ExpertArgs& in, cudaStream_t s) {
    KernelArgs a{in, {}, 0, 0};
    const int e = piece_of(in, dtype);
    a.shape = row_shape(in.width / e, gather_pieces(e));
    const int grid = static_cast<int>(cdiv(in.tokens * a.shape.chunks * a.shape.lanes, kThreads));
    return with_types(dtype, [&](auto t, auto w) {
        using T = decltype(t);
        return with_piece<T>(e, [&](auto n) {
            return launch_pdl(expert_gather_kernel<T, decltype(w), decltype(n)::value>, grid, kThreads, 0, 1, s, a);
        });
    });
}

cudaError_t expert_gather_bwd_launch(const DeviceInfo&, int dtype, const ExpertArgs& in, cudaStream_t s) {
    KernelArgs a{in, {}, 0, 0};
    const int e = piece_of(in, dtype);
    a.shape = row_shape(in.width / e, bwd_pieces(e));
    a.team = 4;
    while (a.team < kThreads && a.team * bwd_pieces(e) < a.shape.pieces) a.team *= 2;
    a.zero_blocks = zero_blocks(in);
    const int grid = static_cast<int>(a.zero_blocks + cdiv(in.tokens, kThreads / a.team));
    return with_types(dtype, [&](auto t, auto w) {
        using T = decltype(t);
        return with_piece<T>(e, [&](auto n) {
            return launch_pdl(expert_gather_bwd_kernel<T, decltype(w), decltype(n)::value>, grid, kThreads, 0, 1, s, a);
        });
    });
}

}  // namespace rmsn
