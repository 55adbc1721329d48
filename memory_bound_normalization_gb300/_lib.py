"""ctypes binding of librmsnorm.so (declared in include/rmsnorm.h).

Argument marshalling only: every step of the computation runs in the CUDA
library. Functions keep the C names and argument order. Tensor arguments may
be torch tensors (their ``data_ptr()`` is passed) or raw integer device
addresses; ``stream`` may be a ``torch.cuda.Stream``, an integer handle, or
None (the current torch stream of the current device).

There is no fallback: if the library is missing or fails to load, importing
the first function raises.

With RMSNORM_LIBRARY_VARIANT=checked in the environment the binding loads the
checked debug build of the same sources instead (every kernel access tested
against its extent; see build.py), for tests that look for out-of-range
accesses.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

F32 = 0
BF16 = 1
F16 = 2
BF16_W_F32 = 3  # bf16 activations, fp32 weight
F16_W_F32 = 4  # fp16 activations, fp32 weight

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_MISALIGNED = 3
ERR_CUDA = 4
ERR_NOMEM = 5
ERR_DEVICE_TIMEOUT = 6
ERR_OUT_OF_BOUNDS = 7  # reported by the checked debug build only

PASS_FWD = 0
PASS_BWD = 1
PASS_BWD_RES = 2  # rmsnorm_add_bwd with dres
PASS_FWD_ADD = 3  # rmsnorm_add_fwd

PROBE_COPY = 0
PROBE_WRITE = 1
PROBE_2R1W = 2

ACT_NONE = 0
ACT_SILU = 1
ACT_GELU = 2

ROPE_MAX_AXES = 4
ROPE_MAX_HEAD_DIM = 256

MAX_EXPERTS = 1024

VARIANTS = {0: "none", 1: "rowgroup", 2: "cta_row", 3: "cluster_row", 4: "scalar",
            5: "two_pass", 6: "ring"}

# Exported symbols, in header order (tests check the library against this
# list and the header against the library).
EXPORTS = (
    "rmsnorm_fwd",
    "rmsnorm_bwd",
    "rmsnorm_bwd_workspace_size",
    "rmsnorm_bwd_ws",
    "rmsnorm_add_fwd",
    "rmsnorm_add_bwd",
    "rmsnorm_noalloc_scratch_bytes",
    "rmsnorm_bwd_noalloc",
    "rmsnorm_bwd_naive",
    "rmsnorm_qk_rope_fwd",
    "rmsnorm_qk_rope_bwd",
    "rmsnorm_qk_rope_bwd_ws",
    "rmsnorm_qk_rope_bwd_workspace_size",
    "rmsnorm_group_norm_fwd",
    "rmsnorm_group_norm_bwd",
    "rmsnorm_group_norm_fwd_ws",
    "rmsnorm_group_norm_bwd_ws",
    "rmsnorm_group_norm_workspace_size",
    "rmsnorm_embedding_fwd",
    "rmsnorm_embedding_bwd",
    "rmsnorm_embedding_bwd_ws",
    "rmsnorm_embedding_bwd_workspace_size",
    "rmsnorm_expert_rows",
    "rmsnorm_expert_sort",
    "rmsnorm_expert_sort_ws",
    "rmsnorm_expert_sort_workspace_size",
    "rmsnorm_expert_dispatch_fwd",
    "rmsnorm_expert_dispatch_bwd",
    "rmsnorm_expert_combine_fwd",
    "rmsnorm_expert_combine_bwd",
    "rmsnorm_get_last_device_error",
    "rmsnorm_status_string",
    "rmsnorm_set_wait_limit_ns",
    "rmsnorm_test_drop_copy",
    "rmsnorm_probe",
    "rmsnorm_plan",
    "rmsnorm_version",
)


class RMSNormError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = status_string(status)
        super().__init__(f"{what}: {name}" if what else name)


class Plan(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int),
        ("threads", ctypes.c_int),
        ("vectors_per_thread", ctypes.c_int),
        ("threads_per_row", ctypes.c_int),
        ("rows_per_unit", ctypes.c_int),
        ("cluster", ctypes.c_int),
        ("row_groups", ctypes.c_int),
        ("stages", ctypes.c_int),
        ("smem_bytes", ctypes.c_int),
        ("grid", ctypes.c_int),
        ("partial_rows", ctypes.c_int),
        ("workspace_bytes", ctypes.c_int64),
    ]

    def as_dict(self) -> dict:
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["variant_name"] = VARIANTS.get(self.variant, "?")
        return d


class Strides(ctypes.Structure):
    """rmsnorm_strides_t: strides in elements over (batch, token, head)."""

    _fields_ = [("batch", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class Rope(ctypes.Structure):
    """rmsnorm_rope_t: the shapes, strides and pairs of a rotary call."""

    _fields_ = [
        ("batch", ctypes.c_int64),
        ("length", ctypes.c_int64),
        ("q_heads", ctypes.c_int32),
        ("k_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("axes", ctypes.c_int32),
        ("sections", ctypes.c_int32 * ROPE_MAX_AXES),
        ("interleaved", ctypes.c_int32),
        ("adjacent", ctypes.c_int32),
        ("positions_64", ctypes.c_int32),
        ("position_stride", ctypes.c_int64 * 3),
        ("q", Strides),
        ("k", Strides),
        ("q_out", Strides),
        ("k_out", Strides),
        ("dq", Strides),
        ("dk", Strides),
    ]


class Embedding(ctypes.Structure):
    """rmsnorm_embedding_t: the tokens, sizes and strides of a lookup."""

    _fields_ = [
        ("outer", ctypes.c_int64),
        ("inner", ctypes.c_int64),
        ("id_stride", ctypes.c_int64 * 2),
        ("num_rows", ctypes.c_int64),
        ("width", ctypes.c_int64),
        ("table_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("ids_64", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class Experts(ctypes.Structure):
    """rmsnorm_experts_t: the shapes of a call between tokens and their experts'
    rows."""

    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("width", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("residual_stride", ctypes.c_int64),
        ("drow_stride", ctypes.c_int64),
        ("choices", ctypes.c_int32),
    ]


_lock = threading.Lock()
_lib: ctypes.CDLL | None = None


def checked_variant() -> bool:
    """True when this process is to load the checked debug build."""
    return os.environ.get("RMSNORM_LIBRARY_VARIANT", "") == "checked"


def library_path() -> str:
    return _build.lib_path(checked_variant())


def load_library(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load librmsnorm.so (optionally building it first). Raises OSError if
    it cannot be loaded; there is no other implementation to fall back on."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        checked = checked_variant()
        path = _build.lib_path(checked)
        if build_if_missing and (not os.path.exists(path) or _build.is_stale(checked) or
                                 _build.binding_is_stale()):
            _build.build(checked=checked)
        if not os.path.exists(path):
            raise OSError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp, i64, i, f, sz, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                  ctypes.c_size_t, ctypes.c_uint64)
        lib.rmsnorm_fwd.argtypes = [vp, vp, vp, vp, i64, i64, f, i, vp]
        lib.rmsnorm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i, vp]
        lib.rmsnorm_bwd_workspace_size.argtypes = [i64, i64, i, i]
        lib.rmsnorm_bwd_workspace_size.restype = sz
        lib.rmsnorm_bwd_ws.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i, vp, sz, vp]
        lib.rmsnorm_add_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, f, i, vp]
        lib.rmsnorm_add_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i, vp]
        lib.rmsnorm_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i, vp]
        lib.rmsnorm_noalloc_scratch_bytes.argtypes = []
        lib.rmsnorm_noalloc_scratch_bytes.restype = sz
        lib.rmsnorm_bwd_naive.argtypes = [vp, vp, vp, vp, vp, i64, i64, f, i, vp]
        lib.rmsnorm_qk_rope_fwd.argtypes = [vp] * 9 + [f, i, vp]
        lib.rmsnorm_qk_rope_bwd.argtypes = [vp] * 13 + [f, i, vp]
        lib.rmsnorm_qk_rope_bwd_ws.argtypes = [vp] * 13 + [f, i, vp, sz, vp]
        lib.rmsnorm_qk_rope_bwd_workspace_size.argtypes = [i, i]
        lib.rmsnorm_qk_rope_bwd_workspace_size.restype = sz
        lib.rmsnorm_group_norm_fwd_ws.argtypes = [vp] * 6 + [i64] * 4 + [f, i, i, vp, sz, vp]
        lib.rmsnorm_group_norm_bwd_ws.argtypes = [vp] * 9 + [i64] * 4 + [i, i, vp, sz, vp]
        lib.rmsnorm_group_norm_workspace_size.argtypes = [i64] * 4 + [i, i, i]
        lib.rmsnorm_group_norm_workspace_size.restype = sz
        lib.rmsnorm_group_norm_fwd.argtypes = [vp] * 6 + [i64] * 4 + [f, i, i, vp]
        lib.rmsnorm_group_norm_bwd.argtypes = [vp] * 9 + [i64] * 4 + [i, i, vp]
        lib.rmsnorm_embedding_fwd.argtypes = [vp] * 4 + [i, vp]
        lib.rmsnorm_embedding_bwd.argtypes = [vp] * 4 + [i64, i, i, vp]
        lib.rmsnorm_embedding_bwd_ws.argtypes = [vp] * 4 + [i64, i, i, vp, sz, vp]
        lib.rmsnorm_embedding_bwd_workspace_size.argtypes = [i64, i64, i64]
        lib.rmsnorm_embedding_bwd_workspace_size.restype = sz
        lib.rmsnorm_expert_rows.argtypes = [i64] * 4
        lib.rmsnorm_expert_rows.restype = i64
        lib.rmsnorm_expert_sort.argtypes = [vp, i] + [i64] * 5 + [vp] * 5
        lib.rmsnorm_expert_sort_ws.argtypes = [vp, i] + [i64] * 5 + [vp] * 5 + [sz, vp]
        lib.rmsnorm_expert_sort_workspace_size.argtypes = [i64] * 3
        lib.rmsnorm_expert_sort_workspace_size.restype = sz
        lib.rmsnorm_expert_dispatch_fwd.argtypes = [vp] * 5 + [i, vp]
        lib.rmsnorm_expert_dispatch_bwd.argtypes = [vp] * 4 + [i, vp]
        lib.rmsnorm_expert_combine_fwd.argtypes = [vp] * 6 + [i, vp]
        lib.rmsnorm_expert_combine_bwd.argtypes = [vp] * 8 + [i, vp]
        lib.rmsnorm_get_last_device_error.argtypes = [vp]
        lib.rmsnorm_status_string.argtypes = [i]
        lib.rmsnorm_status_string.restype = ctypes.c_char_p
        lib.rmsnorm_set_wait_limit_ns.argtypes = [u64]
        lib.rmsnorm_set_wait_limit_ns.restype = None
        lib.rmsnorm_test_drop_copy.argtypes = [i64]
        lib.rmsnorm_test_drop_copy.restype = None
        lib.rmsnorm_probe.argtypes = [i, vp, vp, vp, sz, i, vp]
        lib.rmsnorm_plan.argtypes = [i64, i64, i, i, i, ctypes.POINTER(Plan)]
        lib.rmsnorm_version.argtypes = []
        lib.rmsnorm_version.restype = ctypes.c_char_p
        for name in ("rmsnorm_fwd", "rmsnorm_bwd", "rmsnorm_bwd_ws", "rmsnorm_add_fwd",
                     "rmsnorm_add_bwd", "rmsnorm_bwd_noalloc", "rmsnorm_bwd_naive",
                     "rmsnorm_qk_rope_fwd", "rmsnorm_qk_rope_bwd", "rmsnorm_group_norm_fwd",
                     "rmsnorm_group_norm_bwd", "rmsnorm_qk_rope_bwd_ws",
                     "rmsnorm_group_norm_fwd_ws", "rmsnorm_group_norm_bwd_ws",
                     "rmsnorm_embedding_fwd", "rmsnorm_embedding_bwd", "rmsnorm_embedding_bwd_ws",
                     "rmsnorm_expert_sort", "rmsnorm_expert_sort_ws", "rmsnorm_expert_dispatch_fwd",
                     "rmsnorm_expert_dispatch_bwd", "rmsnorm_expert_combine_fwd",
                     "rmsnorm_expert_combine_bwd", "rmsnorm_get_last_device_error",
                     "rmsnorm_probe", "rmsnorm_plan"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _ptr(t) -> int | None:
    """Device address of a tensor argument (None and raw integer addresses
    pass through). Host or non-contiguous tensors are refused here, before
    anything reaches the library: its kernels read every tensor as dense
    row-major device memory."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"tensor argument on {t.device}: the library takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor argument is not contiguous: the library takes dense row-major "
                         "tensors (call .contiguous() first)")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        # the handle alone: building a Stream object for it takes 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def rmsnorm_fwd(x, w, y, rstd, M: int, N: int, eps: float, dtype: int, stream=None) -> int:
    return load_library().rmsnorm_fwd(_ptr(x), _ptr(w), _ptr(y), _ptr(rstd), M, N, eps, dtype,
                                      _stream(stream))


def rmsnorm_bwd(x, w, dy, rstd, dx, dw, M: int, N: int, dtype: int, stream=None) -> int:
    return load_library().rmsnorm_bwd(_ptr(x), _ptr(w), _ptr(dy), _ptr(rstd), _ptr(dx), _ptr(dw),
                                      M, N, dtype, _stream(stream))


def rmsnorm_bwd_workspace_size(M: int, N: int, dtype: int, device: int) -> int:
    return load_library().rmsnorm_bwd_workspace_size(M, N, dtype, device)


def rmsnorm_bwd_ws(x, w, dy, rstd, dx, dw, M: int, N: int, dtype: int, workspace,
                   workspace_bytes: int, stream=None) -> int:
    return load_library().rmsnorm_bwd_ws(_ptr(x), _ptr(w), _ptr(dy), _ptr(rstd), _ptr(dx),
                                         _ptr(dw), M, N, dtype, _ptr(workspace), workspace_bytes,
                                         _stream(stream))


def rmsnorm_add_fwd(x, residual, w, h, y, rstd, M: int, N: int, eps: float, dtype: int,
                    stream=None) -> int:
    return load_library().rmsnorm_add_fwd(_ptr(x), _ptr(residual), _ptr(w), _ptr(h), _ptr(y),
                                          _ptr(rstd), M, N, eps, dtype, _stream(stream))


def rmsnorm_add_bwd(h, w, dy, rstd, dres, dx, dw, M: int, N: int, dtype: int,
                    stream=None) -> int:
    return load_library().rmsnorm_add_bwd(_ptr(h), _ptr(w), _ptr(dy), _ptr(rstd), _ptr(dres),
                                          _ptr(dx), _ptr(dw), M, N, dtype, _stream(stream))


def rmsnorm_bwd_noalloc(x, w, dy, rstd, dx, dw, M: int, N: int, dtype: int, stream=None) -> int:
    """rmsnorm_bwd without any device allocation (fixed in-library scratch),
    for callers that cannot allocate; see include/rmsnorm.h."""
    return load_library().rmsnorm_bwd_noalloc(_ptr(x), _ptr(w), _ptr(dy), _ptr(rstd), _ptr(dx),
                                              _ptr(dw), M, N, dtype, _stream(stream))


def rmsnorm_noalloc_scratch_bytes() -> int:
    """Size of rmsnorm_bwd_noalloc's fixed scratch array, as the library was
    built with it."""
    return int(load_library().rmsnorm_noalloc_scratch_bytes())


def rmsnorm_bwd_naive(x, w, dy, dx, dw, M: int, N: int, eps: float, dtype: int,
                      stream=None) -> int:
    """The naive three-kernel backward (an ablation); see include/rmsnorm.h."""
    return load_library().rmsnorm_bwd_naive(_ptr(x), _ptr(w), _ptr(dy), _ptr(dx), _ptr(dw), M, N,
                                            eps, dtype, _stream(stream))


def _strided_ptr(t) -> int | None:
    """Device address of a tensor whose strides travel in a descriptor."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"tensor argument on {t.device}: the library takes CUDA tensors")
    return t.data_ptr()


def rmsnorm_qk_rope_fwd(rope, q, k, wq, wk, positions, inv_freq, q_out, k_out, eps: float,
                        dtype: int, stream=None) -> int:
    """`rope` is a Rope or None; tensors it gives strides for may be strided."""
    return load_library().rmsnorm_qk_rope_fwd(
        _rope_ptr(rope), _strided_ptr(q), _strided_ptr(k), _ptr(wq), _ptr(wk),
        _strided_ptr(positions), _ptr(inv_freq), _strided_ptr(q_out), _strided_ptr(k_out), eps,
        dtype, _stream(stream))


def rmsnorm_qk_rope_bwd(rope, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq, dwk,
                        eps: float, dtype: int, stream=None) -> int:
    return load_library().rmsnorm_qk_rope_bwd(
        _rope_ptr(rope), _strided_ptr(q), _strided_ptr(k), _ptr(wq), _ptr(wk),
        _strided_ptr(positions), _ptr(inv_freq), _strided_ptr(dq_out), _strided_ptr(dk_out),
        _strided_ptr(dq), _strided_ptr(dk), _ptr(dwq), _ptr(dwk), eps, dtype, _stream(stream))


def rmsnorm_qk_rope_bwd_ws(rope, q, k, wq, wk, positions, inv_freq, dq_out, dk_out, dq, dk, dwq,
                           dwk, eps: float, dtype: int, workspace, workspace_bytes: int,
                           stream=None) -> int:
    return load_library().rmsnorm_qk_rope_bwd_ws(
        _rope_ptr(rope), _strided_ptr(q), _strided_ptr(k), _ptr(wq), _ptr(wk),
        _strided_ptr(positions), _ptr(inv_freq), _strided_ptr(dq_out), _strided_ptr(dk_out),
        _strided_ptr(dq), _strided_ptr(dk), _ptr(dwq), _ptr(dwk), eps, dtype, _ptr(workspace),
        workspace_bytes, _stream(stream))


def rmsnorm_qk_rope_bwd_workspace_size(head_dim: int, device: int) -> int:
    return load_library().rmsnorm_qk_rope_bwd_workspace_size(head_dim, device)


def _rope_ptr(rope: Rope | None):
    return None if rope is None else ctypes.addressof(rope)


def rmsnorm_group_norm_fwd(x, w, b, y, mean, rstd, B: int, S: int, C: int, G: int, eps: float,
                           act: int, dtype: int, stream=None) -> int:
    return load_library().rmsnorm_group_norm_fwd(_ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean),
                                                 _ptr(rstd), B, S, C, G, eps, act, dtype,
                                                 _stream(stream))


def rmsnorm_group_norm_bwd(x, w, b, dy, mean, rstd, dx, dw, db, B: int, S: int, C: int, G: int,
                           act: int, dtype: int, stream=None) -> int:
    return load_library().rmsnorm_group_norm_bwd(_ptr(x), _ptr(w), _ptr(b), _ptr(dy), _ptr(mean),
                                                 _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db), B, S, C,
                                                 G, act, dtype, _stream(stream))


def rmsnorm_group_norm_fwd_ws(x, w, b, y, mean, rstd, B: int, S: int, C: int, G: int, eps: float,
                              act: int, dtype: int, workspace, workspace_bytes: int,
                              stream=None) -> int:
    return load_library().rmsnorm_group_norm_fwd_ws(
        _ptr(x), _ptr(w), _ptr(b), _ptr(y), _ptr(mean), _ptr(rstd), B, S, C, G, eps, act, dtype,
        _ptr(workspace), workspace_bytes, _stream(stream))


def rmsnorm_group_norm_bwd_ws(x, w, b, dy, mean, rstd, dx, dw, db, B: int, S: int, C: int, G: int,
                              act: int, dtype: int, workspace, workspace_bytes: int,
                              stream=None) -> int:
    return load_library().rmsnorm_group_norm_bwd_ws(
        _ptr(x), _ptr(w), _ptr(b), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db),
        B, S, C, G, act, dtype, _ptr(workspace), workspace_bytes, _stream(stream))


def rmsnorm_group_norm_workspace_size(B: int, S: int, C: int, G: int, dtype: int, backward: int,
                                      device: int) -> int:
    return load_library().rmsnorm_group_norm_workspace_size(B, S, C, G, dtype, backward, device)


def _struct_ptr(d):
    return None if d is None else ctypes.addressof(d)


def rmsnorm_embedding_fwd(embedding, ids, table, y, dtype: int, stream=None) -> int:
    """`embedding` is an Embedding or None; tensors it gives strides for may be strided."""
    return load_library().rmsnorm_embedding_fwd(_struct_ptr(embedding), _strided_ptr(ids),
                                                _strided_ptr(table), _strided_ptr(y), dtype,
                                                _stream(stream))


def rmsnorm_embedding_bwd(embedding, ids, dy, grad, padding_id: int, accumulate: int, dtype: int,
                          stream=None) -> int:
    return load_library().rmsnorm_embedding_bwd(_struct_ptr(embedding), _strided_ptr(ids),
                                                _strided_ptr(dy), _strided_ptr(grad), padding_id,
                                                accumulate, dtype, _stream(stream))


def rmsnorm_embedding_bwd_ws(embedding, ids, dy, grad, padding_id: int, accumulate: int,
                             dtype: int, workspace, workspace_bytes: int, stream=None) -> int:
    return load_library().rmsnorm_embedding_bwd_ws(
        _struct_ptr(embedding), _strided_ptr(ids), _strided_ptr(dy), _strided_ptr(grad),
        padding_id, accumulate, dtype, _ptr(workspace), workspace_bytes, _stream(stream))


def rmsnorm_embedding_bwd_workspace_size(tokens: int, num_rows: int, width: int) -> int:
    return load_library().rmsnorm_embedding_bwd_workspace_size(tokens, num_rows, width)


def rmsnorm_expert_rows(tokens: int, choices: int, num_experts: int, align: int) -> int:
    return load_library().rmsnorm_expert_rows(tokens, choices, num_experts, align)


def rmsnorm_expert_sort(experts, experts_64: int, tokens: int, choices: int, num_experts: int,
                        align: int, rows: int, position, source, offsets, counts,
                        stream=None) -> int:
    return load_library().rmsnorm_expert_sort(
        _ptr(experts), experts_64, tokens, choices, num_experts, align, rows, _ptr(position),
        _ptr(source), _ptr(offsets), _ptr(counts), _stream(stream))


def rmsnorm_expert_sort_ws(experts, experts_64: int, tokens: int, choices: int, num_experts: int,
                           align: int, rows: int, position, source, offsets, counts, workspace,
                           workspace_bytes: int, stream=None) -> int:
    return load_library().rmsnorm_expert_sort_ws(
        _ptr(experts), experts_64, tokens, choices, num_experts, align, rows, _ptr(position),
        _ptr(source), _ptr(offsets), _ptr(counts), _ptr(workspace), workspace_bytes,
        _stream(stream))


def rmsnorm_expert_sort_workspace_size(tokens: int, choices: int, num_experts: int) -> int:
    return load_library().rmsnorm_expert_sort_workspace_size(tokens, choices, num_experts)


def rmsnorm_expert_dispatch_fwd(experts, x, position, source, rows, dtype: int,
                                stream=None) -> int:
    """`experts` is an Experts or None; tensors it gives strides for may be strided."""
    return load_library().rmsnorm_expert_dispatch_fwd(
        _struct_ptr(experts), _strided_ptr(x), _ptr(position), _ptr(source), _strided_ptr(rows),
        dtype, _stream(stream))


def rmsnorm_expert_dispatch_bwd(experts, drows, position, dx, dtype: int, stream=None) -> int:
    return load_library().rmsnorm_expert_dispatch_bwd(
        _struct_ptr(experts), _strided_ptr(drows), _ptr(position), _strided_ptr(dx), dtype,
        _stream(stream))


def rmsnorm_expert_combine_fwd(experts, rows, position, weights, residual, y, dtype: int,
                               stream=None) -> int:
    return load_library().rmsnorm_expert_combine_fwd(
        _struct_ptr(experts), _strided_ptr(rows), _ptr(position), _ptr(weights),
        _strided_ptr(residual), _strided_ptr(y), dtype, _stream(stream))


def rmsnorm_expert_combine_bwd(experts, dy, rows, position, source, weights, drows, dweights,
                               dtype: int, stream=None) -> int:
    return load_library().rmsnorm_expert_combine_bwd(
        _struct_ptr(experts), _strided_ptr(dy), _strided_ptr(rows), _ptr(position), _ptr(source),
        _ptr(weights), _strided_ptr(drows), _ptr(dweights), dtype, _stream(stream))


def rmsnorm_get_last_device_error(stream=None) -> int:
    return load_library().rmsnorm_get_last_device_error(_stream(stream))


def rmsnorm_status_string(status: int) -> str:
    return load_library().rmsnorm_status_string(status).decode()


status_string = rmsnorm_status_string


def rmsnorm_set_wait_limit_ns(ns: int) -> None:
    load_library().rmsnorm_set_wait_limit_ns(ns)


def rmsnorm_test_drop_copy(unit: int) -> None:
    load_library().rmsnorm_test_drop_copy(unit)


def rmsnorm_probe(kind: int, dst, a, b, nbytes: int, blocks_per_sm: int, stream=None) -> int:
    return load_library().rmsnorm_probe(kind, _ptr(dst), _ptr(a), _ptr(b), nbytes, blocks_per_sm,
                                        _stream(stream))


def rmsnorm_plan(M: int, N: int, dtype: int, pass_: int, device: int = -1) -> Plan:
    p = Plan()
    st = load_library().rmsnorm_plan(M, N, dtype, pass_, device, ctypes.byref(p))
    if st != OK:
        raise RMSNormError(st, "rmsnorm_plan")
    return p


def rmsnorm_version() -> str:
    return load_library().rmsnorm_version().decode()


def check(status: int, what: str = "") -> None:
    if status != OK:
        raise RMSNormError(status, what)
