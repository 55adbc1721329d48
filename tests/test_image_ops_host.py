"""Group norm and the rotary QK-norm without a GPU: arguments are refused
before anything reaches CUDA, in the C ABI and in the tensor-level calls, and
the references the GPU tests use agree with differences of their forwards."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import image_ref as ref
import memory_bound_normalization_gb300 as pkg
from memory_bound_normalization_gb300 import build as libbuild

A = 1 << 20  # aligned non-null addresses; never dereferenced by these calls


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    pkg.load_library()


def gn(x=A, w=A, b=A, y=A, mean=A, rstd=A, B=2, S=4, C=64, G=8, eps=1e-5, act=1, dtype=pkg.BF16):
    return pkg.rmsnorm_group_norm_fwd(x, w, b, y, mean, rstd, B, S, C, G, eps, act, dtype, 0)


def gn_bwd(x=A, w=A, b=A, dy=A, mean=A, rstd=A, dx=A, dw=A, db=A, B=2, S=4, C=64, G=8, act=1,
           dtype=pkg.BF16):
    return pkg.rmsnorm_group_norm_bwd(x, w, b, dy, mean, rstd, dx, dw, db, B, S, C, G, act, dtype,
                                      0)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(S=-1), dict(C=0), dict(C=-8), dict(G=0),
                                 dict(G=7), dict(act=3), dict(act=-1), dict(dtype=5),
                                 dict(dtype=-1), dict(x=None), dict(w=None), dict(b=None),
                                 dict(mean=None), dict(rstd=None), dict(C=1 << 31, G=1 << 31),
                                 dict(S=1 << 30), dict(B=1 << 60)])
def test_group_norm_invalid(bad):
    assert gn(**bad) == pkg.ERR_INVALID_ARG
    assert gn_bwd(**bad) == pkg.ERR_INVALID_ARG


def test_group_norm_invalid_of_one_direction():
    for eps in (-1e-6, math.nan):
        assert gn(eps=eps) == pkg.ERR_INVALID_ARG
    assert gn(y=None) == pkg.ERR_INVALID_ARG
    for name in ("dy", "dx", "dw", "db"):
        assert gn_bwd(**{name: None}) == pkg.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(x=A + 1), dict(mean=A + 2), dict(rstd=A + 1), dict(w=A + 1),
                                 dict(b=A + 1)])
def test_group_norm_misaligned(bad):
    assert gn(**bad) == pkg.ERR_MISALIGNED
    assert gn_bwd(**bad) == pkg.ERR_MISALIGNED
    if set(bad) <= {"w", "b"}:  # an fp32 weight beside 16-bit activations
        assert gn(**{k: A + 2 for k in bad}, dtype=pkg.BF16_W_F32) == pkg.ERR_MISALIGNED


def test_group_norm_nothing_to_do():
    assert gn(B=0) == pkg.OK and gn(S=0) == pkg.OK
    assert gn_bwd(B=0, dw=None, db=None) == pkg.OK and gn_bwd(S=0, dw=None, db=None) == pkg.OK


def desc(**over):
    r = pkg.Rope()
    base = dict(batch=2, length=3, q_heads=4, k_heads=2, head_dim=64, rotary_dim=64, axes=3,
                interleaved=0, adjacent=0, positions_64=0)
    sections = over.pop("sections", (8, 12, 12))
    for k, v in {**base, **{k: v for k, v in over.items() if hasattr(r, k) and k not in
                            ("q", "k", "q_out", "k_out", "dq", "dk", "position_stride")}}.items():
        setattr(r, k, v)
    for i, v in enumerate(sections):
        r.sections[i] = v
    for i, v in enumerate(over.get("position_stride", (6, 3, 1))):
        r.position_stride[i] = v
    for name in ("q", "k", "q_out", "k_out", "dq", "dk"):
        b, t, h = over.get(name, (768, 256, 64))
        setattr(r, name, pkg.Strides(b, t, h))
    return r


def rope(r=None, q=A, k=A, wq=A, wk=A, pos=A, freq=A, qo=A, ko=A, eps=1e-6, dtype=pkg.BF16):
    return pkg.rmsnorm_qk_rope_fwd(desc() if r is None else r, q, k, wq, wk, pos, freq, qo, ko,
                                   eps, dtype, 0)


def rope_bwd(r=None, q=A, k=A, wq=A, wk=A, pos=A, freq=A, dqo=A, dko=A, dq=A, dk=A, dwq=A, dwk=A,
             eps=1e-6, dtype=pkg.BF16):
    return pkg.rmsnorm_qk_rope_bwd(desc() if r is None else r, q, k, wq, wk, pos, freq, dqo, dko,
                                   dq, dk, dwq, dwk, eps, dtype, 0)


BAD_DESC = [dict(batch=-1), dict(length=-1), dict(q_heads=-1), dict(k_heads=-1), dict(head_dim=63),
            dict(head_dim=0), dict(head_dim=258), dict(rotary_dim=66), dict(rotary_dim=0),
            dict(rotary_dim=63), dict(axes=0), dict(axes=5), dict(axes=2),
            dict(sections=(8, 12, 11)), dict(sections=(-4, 18, 18)),
            dict(sections=(2 ** 31 - 1, 2 ** 31 - 1, 34)), dict(position_stride=(-1, 3, 1)),
            dict(batch=1 << 20, length=1 << 20), dict(length=1 << 40),
            dict(q_heads=1 << 30, k_heads=1 << 30)]


@pytest.mark.parametrize("bad", BAD_DESC)
def test_rope_descriptor(bad):
    assert rope(desc(**dict(bad))) == pkg.ERR_INVALID_ARG
    assert rope_bwd(desc(**dict(bad))) == pkg.ERR_INVALID_ARG


def test_rope_arguments():
    for name in ("q", "k", "wq", "wk", "pos", "freq"):
        assert rope(**{name: None}) == pkg.ERR_INVALID_ARG, name
        assert rope_bwd(**{name: None}) == pkg.ERR_INVALID_ARG, name
    for name in ("qo", "ko"):
        assert rope(**{name: None}) == pkg.ERR_INVALID_ARG, name
    for name in ("dqo", "dko", "dq", "dk", "dwq", "dwk"):
        assert rope_bwd(**{name: None}) == pkg.ERR_INVALID_ARG, name
    for eps in (-1.0, math.nan):
        assert rope(eps=eps) == pkg.ERR_INVALID_ARG and rope_bwd(eps=eps) == pkg.ERR_INVALID_ARG
    assert rope(dtype=5) == pkg.ERR_INVALID_ARG and rope_bwd(dtype=-1) == pkg.ERR_INVALID_ARG
    assert pkg.load_library().rmsnorm_qk_rope_fwd(None, *[A] * 8, 1e-6, 1, 0) == pkg.ERR_INVALID_ARG
    for name in ("q", "k", "q_out", "k_out"):
        assert rope(desc(**{name: (768, -256, 64)})) == pkg.ERR_INVALID_ARG
    for name in ("dq", "dk"):
        assert rope_bwd(desc(**{name: (768, 256, -64)})) == pkg.ERR_INVALID_ARG
    for name in ("q", "k", "wq", "wk", "pos", "freq"):
        assert rope(**{name: A + 1}) == pkg.ERR_MISALIGNED, name
        assert rope_bwd(**{name: A + 1}) == pkg.ERR_MISALIGNED, name
    assert rope(desc(positions_64=1), pos=A + 4) == pkg.ERR_MISALIGNED
    assert rope_bwd(dwq=A + 2) == pkg.ERR_MISALIGNED


def test_rope_nothing_to_do():
    for empty in (dict(batch=0), dict(length=0), dict(q_heads=0, k_heads=0)):
        assert rope(desc(**empty)) == pkg.OK
        assert rope_bwd(desc(**empty), dwq=None, dwk=None) == pkg.OK


def test_descriptor_matches_the_header(tmp_path):
    """The ctypes structure has the layout the header's compiler gives it."""
    src = tmp_path / "layout.c"
    names = [n for n, _ in pkg.Rope._fields_]
    lines = "".join(f'printf("{n} %zu\\n", offsetof(rmsnorm_rope_t, {n}));' for n in names)
    src.write_text('#include <stdio.h>\n#include "rmsnorm.h"\nint main(void) {' + lines +
                   'printf("size %zu\\n", sizeof(rmsnorm_rope_t)); return 0; }')
    cuda = os.path.join(os.path.dirname(os.path.dirname(libbuild._nvcc())), "include")
    subprocess.run(["gcc", "-I", libbuild.INCLUDE, "-I", cuda, str(src), "-o",
                    str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True)
    got = dict(line.split() for line in out.stdout.splitlines())
    assert int(got.pop("size")) == ctypes.sizeof(pkg.Rope)
    assert {n: int(v) for n, v in got.items()} == {n: getattr(pkg.Rope, n).offset for n in names}


def test_missing_binding_raises():
    """Without the compiled binding the tensor-level calls raise; nothing else
    computes in its place."""
    code = ("import torch, memory_bound_normalization_gb300 as p\n"
            "from memory_bound_normalization_gb300 import build\n"
            "build.BINDING_PATH = '/nonexistent/_binding.so'\n"
            "x = torch.zeros(2, 4, 8)\n"
            "try:\n    p.group_norm_forward(x, 2)\nexcept OSError:\n    print('raised')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root,
                         timeout=120)
    assert "raised" in res.stdout, res.stderr[-2000:]


def test_calls_take_tensors():
    with pytest.raises(ValueError, match="expected a tensor"):
        pkg.group_norm_forward([1.0], 1)
    with pytest.raises(ValueError, match="expected a tensor"):
        pkg.qk_rope_forward(None, None, None, None, None, None, (1,))
    with pytest.raises(TypeError):
        pkg.group_norm_forward(torch.zeros(2, 8), "two")


def test_group_norm_calls_refuse():
    x, w = torch.zeros(2, 5, 8), torch.ones(8)
    m = torch.zeros(2, 4)
    refuse = [lambda: pkg.group_norm_forward(torch.zeros(8), 4, w, w),
              lambda: pkg.group_norm_forward(x, 3, w, w),
              lambda: pkg.group_norm_forward(x, 0, w, w),
              lambda: pkg.group_norm_forward(x, 4, w, None),
              lambda: pkg.group_norm_forward(x, 4, w[:4], w),
              lambda: pkg.group_norm_forward(x, 4, w, w.double()),
              lambda: pkg.group_norm_forward(x, 4, w, w, activation="relu"),
              lambda: pkg.group_norm_forward(x.double(), 4, w.double(), w.double()),
              lambda: pkg.group_norm_forward(x, 4, w.half(), w.half()),
              lambda: pkg.group_norm_backward(x, 4, w, w, x[:1], m, m),
              lambda: pkg.group_norm_backward(x, 4, w, w, x.half(), m, m),
              lambda: pkg.group_norm_backward(x, 4, w, w, x, m.double(), m),
              lambda: pkg.group_norm_backward(x, 4, w, w, x, m, m[:1])]
    for call in refuse:
        with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
            call()
    with pytest.raises(ValueError, match="CUDA tensors"):
        pkg.group_norm_forward(x, 4, w, w)


def test_rope_calls_refuse():
    q, k, w = torch.zeros(2, 3, 4, 16), torch.zeros(2, 3, 2, 16), torch.ones(16)
    pos, f, s = torch.zeros(2, 2, 3, dtype=torch.int64), torch.ones(8), (4, 4)
    ok = dict(q=q, k=k, wq=w, wk=w, positions=pos, inv_freq=f, sections=s)
    bad = [dict(q=torch.zeros(3, 16)), dict(k=k[:1]), dict(k=k[..., :8]), dict(k=k.half()),
           dict(wk=None), dict(k=None), dict(wq=w[:8]), dict(wk=w.double()), dict(sections=()),
           dict(sections=(1,) * 5), dict(positions=pos.float()), dict(positions=pos[:1]),
           dict(positions=pos[:, :, :2]), dict(inv_freq=f.double()), dict(inv_freq=f[:7]),
           dict(sections=(4, 3)), dict(wq=w.half(), wk=w.half())]
    for change in bad:
        with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
            pkg.qk_rope_forward(**{**ok, **change})
        with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
            pkg.qk_rope_backward(**{**ok, **change}, dq_out=q, dk_out=k)
    with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
        pkg.qk_rope_forward(**ok, out=(q[:1], k))
    with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
        pkg.qk_rope_backward(**ok, dq_out=q, dk_out=None)
    with pytest.raises(ValueError, match="not dense"):
        pkg.qk_rope_forward(**{**ok, "q": torch.zeros(2, 3, 16, 4).transpose(2, 3)})
    with pytest.raises(ValueError, match="CUDA tensors"):
        pkg.qk_rope_forward(**ok)


# ------------------------------------------- the references, by differences
def _directional(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_group_norm_reference_gradient(name):
    g = torch.Generator().manual_seed(3)
    x, dy, v = (torch.randn(2, 7, 12, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(12, generator=g, dtype=torch.float64) for _ in range(2))

    def loss(t, wt=w, bt=b):
        r = ref.group_norm(t, 3, wt, bt, 1e-5, name)
        return float((ref.act(r["z"], name).reshape(t.shape) * dy).sum())

    xr, wr, br = (t.clone().requires_grad_(True) for t in (x, w, b))
    X = xr.reshape(2, 7, 3, 4)
    m = X.mean((1, 3), keepdim=True)
    z = ((X - m) / torch.sqrt(((X - m) ** 2).mean((1, 3), keepdim=True) + 1e-5)).reshape(2, 7, 12)
    (ref.act(z * wr + br, name) * dy).sum().backward()
    # the formula of check_group_norm_grads, held to autograd and to differences
    ref.check_group_norm_grads(x, 3, w, b, dy, 1e-5, name, xr.grad, wr.grad, br.grad)
    assert abs(_directional(loss, x, v) - float((xr.grad * v).sum())) < 1e-7
    vw = v[0, 0]
    assert abs(_directional(lambda t: loss(x, wt=t), w, vw) - float((wr.grad * vw).sum())) < 1e-7
    assert abs(_directional(lambda t: loss(x, bt=t), b, vw) - float((br.grad * vw).sum())) < 1e-7


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_reference_gradient(adjacent):
    g = torch.Generator().manual_seed(4)
    x, dy, v = (torch.randn(2, 5, 3, 16, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(16, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 1000, (3, 2, 5), generator=g)
    freq = torch.rand(6, generator=g)
    cos, sin = ref.angles(pos, freq, (1, 3, 2), True, (2, 5))
    args = (cos, sin, 12, adjacent, 1e-6)
    loss = lambda t, wt=w: float((ref.rope_one(t, wt, *args)[0] * dy).sum())  # noqa: E731
    xr, wr = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    n = xr / torch.sqrt((xr * xr).mean(-1, keepdim=True) + 1e-6) * wr
    (ref.rotate(n, cos, sin, 12, adjacent) * dy).sum().backward()
    ref.check_rope_grads(x, w, *args, dy, xr.grad, wr.grad, "q")
    assert abs(_directional(loss, x, v) - float((xr.grad * v).sum())) < 1e-7
    assert abs(_directional(lambda t: loss(x, t), w, v[0, 0, 0]) -
               float((wr.grad * v[0, 0, 0]).sum())) < 1e-7


def test_axis_order():
    assert ref.axis_of_pairs((2, 1, 3), False) == [0, 0, 1, 2, 2, 2]
    assert ref.axis_of_pairs((2, 1, 3), True) == [0, 1, 2, 0, 2, 2]
