"""Group norm with an activation, and the query/key norm with rotary positions
of several axes: tensor-level calls of the C ABI (rmsnorm_group_norm_*,
rmsnorm_qk_rope_* in include/rmsnorm.h).

The functions check their arguments, allocate outputs with PyTorch and raise
``RMSNormError`` on a non-OK status, like ``forward`` and ``backward``. They
run on the tensors' own device and on its current stream, or on ``stream`` as if
that were the current one (outputs belong to it); workspaces come from PyTorch's
allocator too. ``autograd`` holds the differentiable forms.

Their checks, allocations and calls are compiled (csrc/binding.cpp): in Python
they took longer than the kernels of a decode step.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

from . import _lib
from . import build as _build

# the entry points binding.cpp calls, in the order of its tables
_ENTRIES = ("rmsnorm_group_norm_fwd_ws", "rmsnorm_group_norm_bwd_ws",
            "rmsnorm_group_norm_workspace_size", "rmsnorm_qk_rope_fwd", "rmsnorm_qk_rope_bwd_ws",
            "rmsnorm_qk_rope_bwd_workspace_size",
            "rmsnorm_embedding_fwd", "rmsnorm_embedding_bwd_ws",
            "rmsnorm_embedding_bwd_workspace_size", "rmsnorm_expert_rows",
            "rmsnorm_expert_sort_ws", "rmsnorm_expert_sort_workspace_size",
            "rmsnorm_expert_dispatch_fwd", "rmsnorm_expert_dispatch_bwd",
            "rmsnorm_expert_combine_fwd", "rmsnorm_expert_combine_bwd")
_bound = None


def _binding():
    """The compiled binding, set up with the loaded library's entry points.
    OSError if either is missing; there is nothing to fall back on."""
    global _bound
    if _bound is None:
        import torch  # noqa: F401  (the binding's libraries)

        lib = _lib.load_library()
        if not os.path.exists(_build.BINDING_PATH):
            raise OSError(f"{_build.BINDING_PATH} is missing: build the CUDA library first, beside a "
                          "PyTorch with CUDA (python -c 'import __graft_entry__ as g; g.build()')")
        spec = importlib.util.spec_from_file_location("_binding", _build.BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.setup(_lib.RMSNormError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                                          for name in _ENTRIES))
        _bound = module
    return _bound


def _handle(stream):
    return None if stream is None else (_lib._stream(stream) or 0)


def group_norm_forward(x, num_groups: int, weight=None, bias=None, eps: float = 1e-5,
                       activation: str = "none", stream=None):
    """y, mean, rstd of act(group_norm(x) * weight + bias), x [B, ..., C]
    contiguous with the channels last; mean and rstd fp32 [B, num_groups] (NaN
    where there are no positions).
    activation: "none", "silu" or "gelu" (z Phi(z), not a form by tanh). An NCHW tensor in
    channels_last memory format passes as x.permute(0, 2, 3, 1)."""
    return (_bound or _binding()).group_norm_forward(x, num_groups, weight, bias, eps, activation,
                                                     _handle(stream))


def group_norm_backward(x, num_groups: int, weight, bias, dy, mean, rstd,
                        activation: str = "none", stream=None):
    """dx, dweight, dbias (fp32; None without a weight) from the forward's mean
    and rstd."""
    return (_bound or _binding()).group_norm_backward(x, num_groups, weight, bias, dy, mean, rstd,
                                                      activation, _handle(stream))


def qk_rope_forward(q, k, wq, wk, positions, inv_freq, sections, interleaved: bool = False,
                    adjacent: bool = False, eps: float = 1e-6, out=None, stream=None):
    """q_out, k_out: RMSNorm of each head (weights wq, wk [D]; None: no norm),
    then 2 * len(inv_freq) elements of it turned by positions * inv_freq.

    q [T, Hq, D] or [B, T, Hq, D], k likewise with Hk heads (or None), strided
    views allowed as long as a head is dense; positions int32 or int64
    [axes, T] or [axes, B, T]; sections: pairs of each axis, in blocks, or
    dealt in turn with `interleaved`; `adjacent` pairs elements (2p, 2p+1)
    instead of (p, p + rotary/2). `out` gives the output tensors, (q, k) itself
    for an update in place."""
    q_out, k_out = (None, None) if out is None else out
    return (_bound or _binding()).qk_rope_forward(q, k, wq, wk, positions, inv_freq, sections,
                                                  interleaved, adjacent, eps, q_out, k_out,
                                                  _handle(stream))


def qk_rope_backward(q, k, wq, wk, positions, inv_freq, sections, dq_out, dk_out,
                     interleaved: bool = False, adjacent: bool = False, eps: float = 1e-6,
                     stream=None):
    """dq, dk, dwq, dwk (fp32; None without weights) from the forward's inputs
    and the gradients of its outputs."""
    return (_bound or _binding()).qk_rope_backward(q, k, wq, wk, positions, inv_freq, sections,
                                                   dq_out, dk_out, interleaved, adjacent, eps,
                                                   _handle(stream))
