"""Group norm with an activation, and the query/key norm with rotary positions
of several axes: tensor-level calls of the C ABI (rmsnorm_group_norm_*,
rmsnorm_qk_rope_* in include/rmsnorm.h).

The functions check their arguments, allocate outputs with PyTorch and raise
``RMSNormError`` on a non-OK status, like ``forward`` and ``backward``. They
run on the tensors' own device and, unless ``stream`` is given, on its current
stream. ``autograd`` holds the differentiable forms.

A call's checks, its type code, workspace size and packed descriptor depend on
the layouts of its arguments alone, so they are kept per layout (shapes,
strides, types, device and options; never an address or a value): a decode
step's call spends its time in the launch and the two allocations.
"""
from __future__ import annotations

import struct

from . import _lib
from ._lib import ERR_INVALID_ARG, RMSNormError, check

ACTIVATIONS = {"none": _lib.ACT_NONE, "silu": _lib.ACT_SILU, "gelu": _lib.ACT_GELU}

# rmsnorm_rope_t: 2 int64, 12 int32, 3 + 18 int64 (no padding)
_ROPE = struct.Struct("=2q12i21q")


def _refuse(what: str):
    raise RMSNormError(ERR_INVALID_ARG, what)


def _codes(dtype, w_dtype):
    from . import dtype_code

    return dtype_code(dtype, w_dtype)


def _here(device: int) -> bool:
    """Whether `device` (a tensor's get_device()) is the current one; a call on
    another runs again with it made current."""
    import torch

    if device < 0:
        raise ValueError("tensor argument on the host: the library takes CUDA tensors")
    return device == torch.cuda.current_device()


_KEPT: dict = {}


def _keep(key, made):
    if len(_KEPT) >= 1024:
        _KEPT.clear()
    _KEPT[key] = made
    return made


_NOTHING = (None,)


def _layout(t):
    return _NOTHING if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _foreign(stream, here: int):
    """(the handle to run on, whether it is another stream than the current one,
    whose handle is `here`). The caching allocator's memory is ordered on the
    current stream, so a call on another leaves its workspace to the library,
    which takes it in that stream's order."""
    there = _lib._stream(stream)
    return there, there != here


def _one_device(device: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != device:
            _refuse(f"tensors on devices {t.get_device()} and {device}")


# ------------------------------------------------------------- group norm
def _group_norm_shape(x, num_groups, weight, bias, activation):
    if x.dim() < 2:
        _refuse(f"group norm of a tensor of {x.dim()} dimensions: expected [B, ..., C]")
    if activation not in ACTIVATIONS:
        _refuse(f"activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    B, C = x.shape[0], x.shape[-1]
    if num_groups < 1 or C % num_groups or C == 0:
        _refuse(f"{C} channels in {num_groups} groups")
    S = 1
    for n in x.shape[1:-1]:
        S *= n
    if (weight is None) != (bias is None):
        _refuse("group norm takes a weight and a bias, or neither")
    if weight is not None:
        if weight.shape != (C,) or bias.shape != (C,):
            _refuse(f"weight {tuple(weight.shape)} and bias {tuple(bias.shape)} of {C} channels")
        if weight.dtype != bias.dtype:
            _refuse(f"weight {weight.dtype} and bias {bias.dtype} differ")
    return B, S, C


def _group_norm_forward_layout(x, num_groups, weight, bias, activation):
    B, S, C = _group_norm_shape(x, num_groups, weight, bias, activation)
    code = _codes(x.dtype, None if weight is None else weight.dtype)
    dev = x.get_device()
    _one_device(dev, weight, bias)
    _here(dev)
    for t in (x, weight, bias):
        _lib._ptr(t)  # dense device memory
    need = _lib.rmsnorm_group_norm_workspace_size(B, S, C, num_groups, code, 0, dev)
    return (B, S, C, num_groups), code, ACTIVATIONS[activation], need, dev, (B, num_groups)


def group_norm_forward(x, num_groups: int, weight=None, bias=None, eps: float = 1e-5,
                       activation: str = "none", stream=None):
    """y, mean, rstd of act(group_norm(x) * weight + bias), x [B, ..., C]
    contiguous with the channels last; mean and rstd fp32 [B, num_groups].
    activation: "none", "silu" or "gelu" (exact). An NCHW tensor in
    channels_last memory format passes as x.permute(0, 2, 3, 1)."""
    import torch

    key = ("gn", num_groups, activation, *_layout(x), *_layout(weight), *_layout(bias))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _group_norm_forward_layout(x, num_groups, weight, bias, activation))
    size, code, act, need, dev, per_group = kept
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return group_norm_forward(x, num_groups, weight, bias, eps, activation, stream)
    handle, foreign = torch._C._cuda_getCurrentRawStream(dev), False
    if stream is not None:
        handle, foreign = _foreign(stream, handle)
    lib, where = _lib.load_library(), x.device
    y = torch.empty_like(x)
    mean = torch.empty(per_group, dtype=torch.float32, device=where)
    rstd = torch.empty_like(mean)
    w, b = (None, None) if weight is None else (weight.data_ptr(), bias.data_ptr())
    if foreign:
        st = lib.rmsnorm_group_norm_fwd(x.data_ptr(), w, b, y.data_ptr(), mean.data_ptr(),
                                        rstd.data_ptr(), *size, eps, act, code, handle)
    else:
        ws = torch.empty(need, dtype=torch.uint8, device=where) if need else None
        st = lib.rmsnorm_group_norm_fwd_ws(
            x.data_ptr(), w, b, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), *size, eps, act,
            code, ws.data_ptr() if need else None, need, handle)
    if st:
        check(st, "rmsnorm_group_norm_fwd")
    return y, mean, rstd


def _group_norm_backward_layout(x, num_groups, weight, bias, dy, mean, rstd, activation):
    import torch

    B, S, C = _group_norm_shape(x, num_groups, weight, bias, activation)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        _refuse(f"dy {tuple(dy.shape)} {dy.dtype} of x {tuple(x.shape)} {x.dtype}")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.shape != (B, num_groups) or t.dtype != torch.float32:
            _refuse(f"{name} {tuple(t.shape)} {t.dtype}: expected fp32 {(B, num_groups)}")
    code = _codes(x.dtype, None if weight is None else weight.dtype)
    dev = x.get_device()
    _one_device(dev, weight, bias, dy, mean, rstd)
    _here(dev)
    for t in (x, weight, bias, dy, mean, rstd):
        _lib._ptr(t)  # dense device memory
    need = _lib.rmsnorm_group_norm_workspace_size(B, S, C, num_groups, code, 1, dev)
    return (B, S, C, num_groups), code, ACTIVATIONS[activation], need, dev, (C,)


def group_norm_backward(x, num_groups: int, weight, bias, dy, mean, rstd,
                        activation: str = "none", stream=None):
    """dx, dweight, dbias (fp32; None without a weight) from the forward's mean
    and rstd."""
    import torch

    key = ("gnb", num_groups, activation, *_layout(x), *_layout(weight), *_layout(bias),
           *_layout(dy), *_layout(mean), *_layout(rstd))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _group_norm_backward_layout(x, num_groups, weight, bias, dy, mean, rstd,
                                                      activation))
    size, code, act, need, dev, per_channel = kept
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return group_norm_backward(x, num_groups, weight, bias, dy, mean, rstd, activation,
                                       stream)
    handle, foreign = torch._C._cuda_getCurrentRawStream(dev), False
    if stream is not None:
        handle, foreign = _foreign(stream, handle)
    lib, where = _lib.load_library(), x.device
    dx = torch.empty_like(x)
    dw = db = w = b = pw = pb = None
    if weight is not None:
        dw = torch.empty(per_channel, dtype=torch.float32, device=where)
        db = torch.empty_like(dw)
        w, b, pw, pb = weight.data_ptr(), bias.data_ptr(), dw.data_ptr(), db.data_ptr()
    if foreign:
        st = lib.rmsnorm_group_norm_bwd(x.data_ptr(), w, b, dy.data_ptr(), mean.data_ptr(),
                                        rstd.data_ptr(), dx.data_ptr(), pw, pb, *size, act, code,
                                        handle)
    else:
        ws = torch.empty(need, dtype=torch.uint8, device=where) if need else None
        st = lib.rmsnorm_group_norm_bwd_ws(
            x.data_ptr(), w, b, dy.data_ptr(), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), pw,
            pb, *size, act, code, ws.data_ptr() if need else None, need, handle)
    if st:
        check(st, "rmsnorm_group_norm_bwd")
    return dx, dw, db


# ------------------------------------------------- rotary positions, QK-norm
def _strides(t):
    """(batch, token, head) strides of [T, H, D] or [B, T, H, D]."""
    s = t.stride()
    if s[-1] != 1:
        raise ValueError("the last dimension of a head is not dense (call .contiguous() first)")
    return (s[-4] if len(s) == 4 else 0, s[-3], s[-2])


_NONE = (0, 0, 0)


def _rope_shape(q, k, wq, wk, positions, inv_freq, sections):
    import torch

    if q.dim() not in (3, 4):
        _refuse(f"queries of {q.dim()} dimensions: expected [T, H, D] or [B, T, H, D]")
    D = q.shape[-1]
    if k is not None and (k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] or
                          k.shape[-1] != D or k.dtype != q.dtype):
        _refuse(f"keys {tuple(k.shape)} {k.dtype} of queries {tuple(q.shape)} {q.dtype}")
    if k is None:
        if wk is not None:
            _refuse("a key weight without keys")
    elif (wq is None) != (wk is None):
        _refuse("weights for queries and keys, or for neither")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None and (w.shape != (D,) or w.dtype != wq.dtype):
            _refuse(f"{name} {tuple(w.shape)} {w.dtype} of heads of {D}")
    lead = tuple(q.shape[:-2])
    B, T = lead if len(lead) == 2 else (1, lead[0])
    axes = len(sections)
    if not 1 <= axes <= _lib.ROPE_MAX_AXES:
        _refuse(f"{axes} position axes: 1 to {_lib.ROPE_MAX_AXES}")
    if positions.dtype not in (torch.int32, torch.int64):
        _refuse(f"positions of {positions.dtype}: int32 or int64")
    shape = tuple(positions.shape)
    if shape not in ((axes,) + lead, (axes, T)):
        _refuse(f"positions {shape} of {axes} axes and tokens {lead}")
    ps = positions.stride()
    ps = (ps[0], ps[1], ps[2]) if len(shape) == 3 else (ps[0], 0, ps[1])
    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or inv_freq.numel() != sum(sections):
        _refuse(f"inv_freq {tuple(inv_freq.shape)} {inv_freq.dtype}: expected fp32, a value for "
                f"each of {sum(sections)} pairs")
    code = _codes(q.dtype, None if wq is None else wq.dtype)
    head = (B, T, q.shape[-2], 0 if k is None else k.shape[-2], D, 2 * inv_freq.numel(), axes,
            *sections, *((0,) * (_lib.ROPE_MAX_AXES - axes)))
    dev = q.get_device()
    _one_device(dev, k, wq, wk, positions, inv_freq)
    return head, positions.dtype == torch.int64, ps, code, dev


def _pack(head, interleaved, adjacent, pos64, ps, *strides):
    try:
        return _ROPE.pack(*head, bool(interleaved), bool(adjacent), pos64, *ps,
                          *(v for s in strides for v in s))
    except struct.error as e:
        _refuse(f"rotary descriptor: {e}")


def _like(name, t, of):
    if t.shape != of.shape or t.dtype != of.dtype or t.device != of.device:
        _refuse(f"{name} {tuple(t.shape)} {t.dtype} on {t.device}: expected {tuple(of.shape)} "
                f"{of.dtype} on {of.device}")


def _dense(t):
    """Strides that torch.empty(t.shape) has."""
    *lead, H, D = t.shape
    return (lead[0] and lead[1] * H * D if len(lead) == 2 else 0, H * D, D)


def _rope_forward_layout(q, k, wq, wk, positions, inv_freq, sections, interleaved, adjacent, qo, ko):
    head, pos64, ps, code, dev = _rope_shape(q, k, wq, wk, positions, inv_freq, sections)
    keys = k is not None
    if qo is not None or ko is not None:
        if qo is None:
            _refuse("an output for the queries")
        _like("out of the queries", qo, q)
        if (ko is not None) != keys:
            _refuse("an output for the keys where there are keys")
        if keys:
            _like("out of the keys", ko, k)
    desc = _pack(head, interleaved, adjacent, pos64, ps, _strides(q),
                 _strides(k) if keys else _NONE, _dense(q) if qo is None else _strides(qo),
                 (_dense(k) if ko is None else _strides(ko)) if keys else _NONE, _NONE, _NONE)
    _here(dev)
    for t in (wq, wk, inv_freq):
        _lib._ptr(t)  # dense device memory
    return desc, code, dev


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
    import torch

    qo, ko = (None, None) if out is None else out
    sections = tuple(sections)
    key = ("qk", sections, interleaved, adjacent, *_layout(q), *_layout(k), *_layout(wq),
           *_layout(wk), *_layout(positions), *_layout(inv_freq), *_layout(qo), *_layout(ko))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _rope_forward_layout(q, k, wq, wk, positions, inv_freq, sections,
                                               interleaved, adjacent, qo, ko))
    desc, code, dev = kept
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return qk_rope_forward(q, k, wq, wk, positions, inv_freq, sections, interleaved,
                                   adjacent, eps, out, stream)
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _lib._stream(stream)
    pk = pko = None
    if qo is None:
        where = q.device
        qo = torch.empty(q.shape, dtype=q.dtype, device=where)
        if k is not None:
            ko = torch.empty(k.shape, dtype=q.dtype, device=where)
    if k is not None:
        pk, pko = k.data_ptr(), ko.data_ptr()
    st = _lib.load_library().rmsnorm_qk_rope_fwd(
        desc, q.data_ptr(), pk, None if wq is None else wq.data_ptr(),
        None if wk is None else wk.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(),
        qo.data_ptr(), pko, eps, code, handle)
    if st:
        check(st, "rmsnorm_qk_rope_fwd")
    return qo, ko


def _rope_backward_layout(q, k, wq, wk, positions, inv_freq, sections, interleaved, adjacent,
                          dq_out, dk_out):
    head, pos64, ps, code, dev = _rope_shape(q, k, wq, wk, positions, inv_freq, sections)
    keys = k is not None
    _like("dq_out", dq_out, q)
    if (dk_out is not None) != keys:
        _refuse("a gradient for the keys where there are keys")
    if keys:
        _like("dk_out", dk_out, k)
    desc = _pack(head, interleaved, adjacent, pos64, ps, _strides(q),
                 _strides(k) if keys else _NONE, _strides(dq_out),
                 _strides(dk_out) if keys else _NONE, _dense(q), _dense(k) if keys else _NONE)
    _here(dev)
    for t in (wq, wk, inv_freq):
        _lib._ptr(t)  # dense device memory
    need = 0 if wq is None else _lib.rmsnorm_qk_rope_bwd_workspace_size(q.shape[-1], dev)
    return desc, code, dev, need


def qk_rope_backward(q, k, wq, wk, positions, inv_freq, sections, dq_out, dk_out,
                     interleaved: bool = False, adjacent: bool = False, eps: float = 1e-6,
                     stream=None):
    """dq, dk, dwq, dwk (fp32; None without weights) from the forward's inputs
    and the gradients of its outputs."""
    import torch

    sections = tuple(sections)
    key = ("qkb", sections, interleaved, adjacent, *_layout(q), *_layout(k), *_layout(wq),
           *_layout(wk), *_layout(positions), *_layout(inv_freq), *_layout(dq_out),
           *_layout(dk_out))
    kept = _KEPT.get(key)
    if kept is None:
        kept = _keep(key, _rope_backward_layout(q, k, wq, wk, positions, inv_freq, sections,
                                                interleaved, adjacent, dq_out, dk_out))
    desc, code, dev, need = kept
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return qk_rope_backward(q, k, wq, wk, positions, inv_freq, sections, dq_out, dk_out,
                                    interleaved, adjacent, eps, stream)
    handle, foreign = torch._C._cuda_getCurrentRawStream(dev), False
    if stream is not None:
        handle, foreign = _foreign(stream, handle)
    lib, where, dtype = _lib.load_library(), q.device, q.dtype
    dq = torch.empty(q.shape, dtype=dtype, device=where)
    dk = dwq = dwk = pk = pdko = pdk = pwq = pwk = pdwq = pdwk = None
    if k is not None:
        dk = torch.empty(k.shape, dtype=dtype, device=where)
        pk, pdko, pdk = k.data_ptr(), dk_out.data_ptr(), dk.data_ptr()
    if need:
        dwq = torch.empty(wq.shape, dtype=torch.float32, device=where)
        pwq, pdwq = wq.data_ptr(), dwq.data_ptr()
        if k is not None:
            dwk = torch.empty_like(dwq)
            pwk, pdwk = wk.data_ptr(), dwk.data_ptr()
    if foreign or not need:
        st = lib.rmsnorm_qk_rope_bwd(
            desc, q.data_ptr(), pk, pwq, pwk, positions.data_ptr(), inv_freq.data_ptr(),
            dq_out.data_ptr(), pdko, dq.data_ptr(), pdk, pdwq, pdwk, eps, code, handle)
    else:
        ws = torch.empty(need, dtype=torch.uint8, device=where)
        st = lib.rmsnorm_qk_rope_bwd_ws(
            desc, q.data_ptr(), pk, pwq, pwk, positions.data_ptr(), inv_freq.data_ptr(),
            dq_out.data_ptr(), pdko, dq.data_ptr(), pdk, pdwq, pdwk, eps, code, ws.data_ptr(),
            need, handle)
    if st:
        check(st, "rmsnorm_qk_rope_bwd")
    return dq, dk, dwq, dwk
