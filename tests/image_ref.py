"""64-bit references of the image and video operators on the CPU, with the
bounds that the kernels' results are held to.

Bounds. U is the unit roundoff of the output's type (finfo.eps / 2), F that of
fp32 (2^-24). An output is one rounding (U |ref|, plus half the smallest
subnormal) of an fp32 result whose own error is a number of fp32 roundings of
the terms it is made of:
  rotary forward   n = x rstd w: the row sum is a chain of at most 64 roundings
                   halved by the square root, then rsqrt and two products;
                   cos and sin carry the angle's rounding (pi F) and 2 ulp; the
                   rotation two more: 64 F (|n_a| + |n_b|) holds all of it.
  rotary backward  the same 64 F on every term of dx, each weighted by rstd.
  sums over rows   a chain of n roundings costs n F of the sum of magnitudes;
                   a lane takes at most rows / 8 of them, then 64 in the trees.
  group norm       K = 64 + n/1024 roundings in a slab sum of n values. The mean
                   is K F mean|x| off, so xhat is K F (|xhat| + rstd mean|x|)
                   off, and z by that times |w| plus 4 F (|b| + |z|); an
                   activation's slope is below 1.2 and its value 8 F |z| off; the
                   slope's own slope is below 1 (silu 0.5, gelu 0.8).
"""
from __future__ import annotations

import math

import numpy as np
import torch

F = 2.0 ** -24


def rounding(dtype, ref):
    """One rounding of ref into dtype: half a step, or half a subnormal step."""
    fi = torch.finfo(dtype)
    return fi.eps / 2 * ref.abs() + fi.smallest_normal * fi.eps / 2


def check(got, ref, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN at other places"
    fin = ref.isfinite()
    assert torch.equal(got[~fin].nan_to_num(7.0), ref[~fin].nan_to_num(7.0)), f"{what}: infinities"
    err = (got - ref).abs()[fin]
    over = err > bound.expand(ref.shape)[fin]
    if over.any():
        i = int((err - bound.expand(ref.shape)[fin]).argmax())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} out of bounds, worst "
                             f"{float(err[i]):.3g} over {float(bound.expand(ref.shape)[fin][i]):.3g} at {float(ref[fin][i]):.3g}")


# --------------------------------------------------------------- group norm
def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def slope(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _slabs(t, G):
    """[B, ..., C] -> [B, S, G, C/G] in 64 bits."""
    return t.detach().double().cpu().reshape(t.shape[0], -1, G, t.shape[-1] // G)


def group_norm(x, G, w, b, eps, name):
    """Everything of the forward, as [B, S, G, D] and [B, 1, G, 1] tensors."""
    X = _slabs(x, G)
    D = X.shape[-1]
    one = lambda v, d: (torch.full((G, D), d, dtype=torch.float64) if v is None  # noqa: E731
                        else v.detach().double().cpu().reshape(G, D))
    W, Bv = one(w, 1.0), one(b, 0.0)
    mean = X.mean((1, 3), keepdim=True)
    var = ((X - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xhat = (X - mean) * rstd
    z = xhat * W + Bv
    n = X.shape[1] * D
    K = 64 + n / 1024
    e_hat = K * F * (xhat.abs() + rstd * X.abs().mean((1, 3), keepdim=True))
    # squares about an fp32 mean that is itself off: second order in mean / std
    e_var = (K * F * rstd * X.abs().mean((1, 3), keepdim=True)) ** 2
    e_hat = e_hat + xhat.abs() * e_var
    e_z = e_hat * W.abs() + 4 * F * (Bv.abs() + z.abs())
    return dict(X=X, W=W, B=Bv, mean=mean, rstd=rstd, xhat=xhat, z=z, K=K, e_hat=e_hat, e_z=e_z,
                e_var=e_var, n=n)


def check_group_norm(x, G, w, b, eps, name, y, mean, rstd):
    r = group_norm(x, G, w, b, eps, name)
    ref = act(r["z"], name)
    bound = rounding(x.dtype, ref) * 1.01 + 1.2 * r["e_z"] + 8 * F * r["z"].abs()
    check(y.reshape(r["X"].shape), ref, bound, "y")
    m = r["mean"].reshape(mean.shape)
    check(mean, m, r["K"] * F * r["X"].abs().mean((1, 3)).reshape(mean.shape) + 1e-45, "mean")
    s = r["rstd"].reshape(rstd.shape)
    check(rstd, s, s * (r["K"] * F + r["e_var"].reshape(s.shape)), "rstd")


def check_group_norm_grads(x, G, w, b, dy, eps, name, dx, dw, db):
    r = group_norm(x, G, w, b, eps, name)
    dY, W, xhat, rstd, K = _slabs(dy, G), r["W"], r["xhat"], r["rstd"], r["K"]
    sl = slope(r["z"], name)
    dz = dY * sl
    e_dz = dY.abs() * ((r["e_z"] if name != "none" else 0) + 8 * F * (1 + sl.abs()))
    g, e_g = dz * W, e_dz * W.abs()
    mean = lambda t: t.mean((1, 3), keepdim=True)  # noqa: E731
    A, Bq = mean(g), mean(g * xhat)
    ref = rstd * (g - A - xhat * Bq)
    e_A = mean(e_g) + K * F * mean(g.abs())
    e_B = mean(e_g * xhat.abs() + g.abs() * r["e_hat"]) + K * F * mean((g * xhat).abs())
    e = rstd * (e_g + e_A + xhat.abs() * e_B + r["e_hat"] * Bq.abs() +
                8 * F * (g.abs() + A.abs() + (xhat * Bq).abs()))
    e = e + (K * F + r["e_var"]) * ref.abs()
    check(dx.reshape(ref.shape), ref, rounding(x.dtype, ref) * 1.01 + e, "dx")
    if dw is not None:
        rows = dz.shape[0] * dz.shape[1]
        chain = (64 + rows / 8) * F
        flat = lambda t: t.sum((0, 1)).reshape(-1)  # noqa: E731
        check(db, flat(dz), flat(e_dz) + chain * flat(dz.abs()) + 1e-45, "db")
        check(dw, flat(dz * xhat), flat(e_dz * xhat.abs() + dz.abs() * r["e_hat"]) +
              chain * flat((dz * xhat).abs()) + 1e-45, "dw")


# ------------------------------------------------------------------- rotary
def axis_of_pairs(sections, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def angles(positions, inv_freq, sections, interleaved, lead):
    """cos, sin [*lead, 1, pairs]: the product of an integer and an fp32 value
    is formed in extended precision and reduced there."""
    pos = positions.detach().cpu().numpy()
    f = inv_freq.detach().cpu().numpy().astype(np.longdouble)
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    cols = []
    for p, a in enumerate(axis_of_pairs(sections, interleaved)):
        t = np.broadcast_to(pos[a], lead).astype(np.longdouble) * f[p]
        cols.append((t - two_pi * np.round(t / two_pi)).astype(np.float64))
    theta = torch.from_numpy(np.stack(cols, -1)).unsqueeze(-2)
    return torch.cos(theta), torch.sin(theta)


def members(D, rot, adjacent):
    p = torch.arange(rot // 2)
    return (2 * p, 2 * p + 1) if adjacent else (p, p + rot // 2)


def rotate(n, cos, sin, rot, adjacent):
    i, j = members(n.shape[-1], rot, adjacent)
    out = n.clone()
    out[..., i] = n[..., i] * cos - n[..., j] * sin
    out[..., j] = n[..., j] * cos + n[..., i] * sin
    return out


def spread(n, rot, adjacent):
    """|n_a| + |n_b| at both members of each pair, |n| elsewhere."""
    i, j = members(n.shape[-1], rot, adjacent)
    out = n.abs()
    s = out[..., i] + out[..., j]
    out = out.clone()
    out[..., i] = s
    out[..., j] = s
    return out


def rope_one(x, w, cos, sin, rot, adjacent, eps):
    X = x.detach().double().cpu()
    if w is None:
        return rotate(X, cos, sin, rot, adjacent), X
    n = X / torch.sqrt((X * X).mean(-1, keepdim=True) + eps) * w.detach().double().cpu()
    return rotate(n, cos, sin, rot, adjacent), n


def check_rope(x, w, cos, sin, rot, adjacent, eps, y, what):
    ref, n = rope_one(x, w, cos, sin, rot, adjacent, eps)
    check(y, ref, rounding(x.dtype, ref) * 1.01 + 64 * F * spread(n, rot, adjacent), what)


def check_rope_grads(x, w, cos, sin, rot, adjacent, eps, dy, dx, dw, what):
    X, G = x.detach().double().cpu(), dy.detach().double().cpu()
    g = rotate(G, cos, -sin, rot, adjacent)
    e_g = 64 * F * spread(G, rot, adjacent)
    if w is None:
        check(dx, g, rounding(x.dtype, g) * 1.01 + e_g, "d" + what)
        return
    W = w.detach().double().cpu()
    rstd = 1 / torch.sqrt((X * X).mean(-1, keepdim=True) + eps)
    xhat = X * rstd
    h = g * W
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    c = mean(h * xhat)
    ref = rstd * (h - xhat * c)
    e = rstd * (e_g * W.abs() + xhat.abs() * mean(e_g * (W * xhat).abs()) +
                64 * F * (h.abs() + xhat.abs() * (c.abs() + mean((h * xhat).abs()))))
    check(dx, ref, rounding(x.dtype, ref) * 1.01 + e, "d" + what)
    rows = g.numel() // g.shape[-1]
    flat = lambda t: t.reshape(rows, -1).sum(0)  # noqa: E731
    check(dw, flat(g * xhat), flat(e_g * xhat.abs()) + (96 + rows / 8) * F * flat((g * xhat).abs()) +
          1e-45, "dw of " + what)
