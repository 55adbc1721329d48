"""PyTorch autograd wrappers around the C ABI, for use inside models.

``rms_norm(x, weight, eps)`` and ``fused_add_rms_norm(x, residual, weight,
eps)`` run the library's forward on the call and its backward (with the fp32
rstd saved by the forward) when autograd asks; every step of both runs in the
CUDA library. ``RMSNorm`` is the module form. The weight gradient comes back
in fp32, as the library computes it; autograd casts it to the weight's dtype
(an fp32 master weight needs no cast). Inputs must be contiguous CUDA
tensors; rows are the last dimension.

``group_norm`` / ``GroupNorm`` (channels last, with an activation) and
``qk_norm_rope`` / ``QKNormRope`` (QK-norm and rotary positions of several
axes) do the same over their operators.

Backward passes can be captured into CUDA graphs as PyTorch's own can: not while
an eager graph of the same leaves is alive, whose streams the capture cannot wait
for (PyTorch raises then).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from . import dtype_code
from . import image_ops


def _rows(t: torch.Tensor):
    n = t.shape[-1]
    return (t.numel() // n if n else 0), n


class _RMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps):
        M, N = _rows(x)
        code = dtype_code(x.dtype, weight.dtype)
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        _lib.check(_lib.rmsnorm_fwd(x, weight, y, rstd, M, N, eps, code), "rmsnorm_fwd")
        ctx.save_for_backward(x, weight, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, rstd = ctx.saved_tensors
        M, N = _rows(x)
        dy = dy.contiguous()
        dx = torch.empty_like(x)
        dw = torch.empty(N, dtype=torch.float32, device=x.device)
        _lib.check(_lib.rmsnorm_bwd(x, weight, dy, rstd, dx, dw, M, N,
                                    dtype_code(x.dtype, weight.dtype)), "rmsnorm_bwd")
        return dx, dw, None


class _AddRMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        M, N = _rows(x)
        code = dtype_code(x.dtype, weight.dtype)
        h = torch.empty_like(x)
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        _lib.check(_lib.rmsnorm_add_fwd(x, residual, weight, h, y, rstd, M, N, eps, code),
                   "rmsnorm_add_fwd")
        ctx.save_for_backward(h, weight, rstd)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        M, N = _rows(h)
        dy = dy.contiguous() if dy is not None else torch.zeros_like(h)
        dres = dh.contiguous() if dh is not None else None
        dx = torch.empty_like(h)
        dw = torch.empty(N, dtype=torch.float32, device=h.device)
        _lib.check(_lib.rmsnorm_add_bwd(h, weight, dy, rstd, dres, dx, dw, M, N,
                                        dtype_code(h.dtype, weight.dtype)), "rmsnorm_add_bwd")
        # h = x + residual: both receive the same gradient
        return dx, dx, dw, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6) -> torch.Tensor:
    """y = x * rstd * weight over the last dimension, differentiable."""
    return _RMSNormFn.apply(x.contiguous(), weight.contiguous(), float(eps))


def fused_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
                       eps: float = 1e-6):
    """(y, h): h = x + residual rounded into x's dtype, y = rms_norm(h),
    differentiable in x, residual and weight (h's own gradient, from its
    later uses, flows back through the same call)."""
    return _AddRMSNormFn.apply(x.contiguous(), residual.contiguous(), weight.contiguous(),
                               float(eps))


class RMSNorm(torch.nn.Module):
    """``torch.nn.RMSNorm``-like module over the last dimension, backed by
    the CUDA library. ``weight_dtype`` lets an fp32 master weight serve 16-bit
    activations."""

    def __init__(self, dim: int, eps: float = 1e-6, device=None,
                 weight_dtype: torch.dtype = torch.float32):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(dim, device=device, dtype=weight_dtype))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        w = self.weight
        if w.dtype != x.dtype and not (w.dtype == torch.float32 and x.dtype in
                                       (torch.bfloat16, torch.float16)):
            raise TypeError(f"weight {w.dtype} cannot serve activations {x.dtype}")
        return rms_norm(x, w, self.eps)


class _GroupNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, num_groups, eps, activation):
        y, mean, rstd = image_ops.group_norm_forward(x, num_groups, weight, bias, eps, activation)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.num_groups, ctx.activation = num_groups, activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        dx, dw, db = image_ops.group_norm_backward(x, ctx.num_groups, weight, bias,
                                                   dy.contiguous(), mean, rstd, ctx.activation)
        return dx, dw, db, None, None, None


def group_norm(x: torch.Tensor, num_groups: int, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5,
               activation: str = "none") -> torch.Tensor:
    """act(group norm of x over its positions and each group's channels), x
    [B, ..., C] with the channels last, differentiable in x, weight and bias."""
    return _GroupNormFn.apply(x.contiguous(), None if weight is None else weight.contiguous(),
                              None if bias is None else bias.contiguous(), int(num_groups),
                              float(eps), activation)


class GroupNorm(torch.nn.Module):
    """Group norm with an activation over [B, ..., C]; fp32 weight and bias by
    default, which serve 16-bit activations as they are."""

    def __init__(self, num_groups: int, num_channels: int, eps: float = 1e-5,
                 activation: str = "none", affine: bool = True, device=None,
                 weight_dtype: torch.dtype = torch.float32):
        super().__init__()
        if num_channels % num_groups:
            raise ValueError(f"{num_channels} channels do not divide into {num_groups} groups")
        self.num_groups, self.eps, self.activation = num_groups, eps, activation
        if affine:
            self.weight = torch.nn.Parameter(torch.ones(num_channels, device=device,
                                                        dtype=weight_dtype))
            self.bias = torch.nn.Parameter(torch.zeros(num_channels, device=device,
                                                       dtype=weight_dtype))
        else:
            self.register_parameter("weight", None)
            self.register_parameter("bias", None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return group_norm(x, self.num_groups, self.weight, self.bias, self.eps, self.activation)


def _dense_heads(t):
    return t if t is None or t.stride(-1) == 1 else t.contiguous()


class _QKRopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, positions, inv_freq, sections, interleaved, adjacent, eps):
        qo, ko = image_ops.qk_rope_forward(q, k, wq, wk, positions, inv_freq, sections,
                                           interleaved, adjacent, eps)
        ctx.save_for_backward(q, k, wq, wk, positions, inv_freq)
        ctx.style = (interleaved, adjacent, eps)
        ctx.sections = sections
        return qo, ko

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, wq, wk, positions, inv_freq = ctx.saved_tensors
        dq, dk, dwq, dwk = image_ops.qk_rope_backward(
            q, k, wq, wk, positions, inv_freq, ctx.sections, _dense_heads(dq_out),
            None if k is None else _dense_heads(dk_out), *ctx.style)
        return dq, dk, dwq, dwk, None, None, None, None, None, None


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, wq: torch.Tensor | None,
                 wk: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
                 sections, interleaved: bool = False, adjacent: bool = False, eps: float = 1e-6):
    """(q, k) after the RMSNorm of their heads (without weights: no norm) and
    the rotation by positions of several axes, differentiable in q, k, wq and
    wk; see image_ops.qk_rope_forward for the layouts."""
    return _QKRopeFn.apply(_dense_heads(q), _dense_heads(k),
                           None if wq is None else wq.contiguous(),
                           None if wk is None else wk.contiguous(), positions,
                           inv_freq.contiguous(), tuple(int(n) for n in sections),
                           bool(interleaved), bool(adjacent), float(eps))


class QKNormRope(torch.nn.Module):
    """QK-norm and rotary positions of several axes for heads of `head_dim`.
    `sections`: pairs of each axis; frequencies theta^(-p / pairs) over all
    pairs. norm=False leaves the rotation alone."""

    def __init__(self, head_dim: int, sections, theta: float = 10000.0, eps: float = 1e-6,
                 interleaved: bool = False, adjacent: bool = False, norm: bool = True,
                 device=None, weight_dtype: torch.dtype = torch.float32):
        super().__init__()
        self.sections = tuple(int(n) for n in sections)
        self.interleaved, self.adjacent, self.eps = interleaved, adjacent, eps
        pairs = sum(self.sections)
        if not 0 < 2 * pairs <= head_dim:
            raise ValueError(f"{pairs} pairs do not fit in heads of {head_dim}")
        self.theta = float(theta)
        self.inv_freq = self._frequencies(device)
        for name in ("q_weight", "k_weight"):
            w = torch.ones(head_dim, device=device, dtype=weight_dtype) if norm else None
            self.register_parameter(name, None if w is None else torch.nn.Parameter(w))

    def _frequencies(self, device):
        pairs = sum(self.sections)
        freq = torch.arange(pairs, device=device, dtype=torch.float64).div_(-pairs)
        return torch.pow(self.theta, freq).float()

    def _apply(self, fn, *args, **kwargs):
        # the frequencies follow the module's device but stay fp32; from the meta
        # device they have no values to take along
        super()._apply(fn, *args, **kwargs)
        device = fn(self.inv_freq).device
        self.inv_freq = (self._frequencies(device) if self.inv_freq.is_meta
                         else self.inv_freq.to(device))
        return self

    def forward(self, q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor):
        # queries alone: the key weight has nothing to scale
        return qk_norm_rope(q, k, self.q_weight, None if k is None else self.k_weight, positions,
                            self.inv_freq, self.sections, self.interleaved, self.adjacent,
                            self.eps)
