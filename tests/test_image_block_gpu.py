"""The operators together, as an image model runs them: group norm + SiLU over
a picture, a projection, QK-norm with (height, width) positions, attention, and
the library's RMSNorm behind it; outputs and gradients against the same block
in 64 bits."""
from __future__ import annotations

import pytest
import torch

import image_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    pkg.load_library(build_if_missing=True)
    yield


def plain(x, p, pos, freq, G, H):
    """The block in the dtype of its inputs, by elementary operations."""
    B, S, C = x.shape
    X = x.reshape(B, S, G, C // G)
    m = X.mean((1, 3), keepdim=True)
    z = ((X - m) / torch.sqrt(((X - m) ** 2).mean((1, 3), keepdim=True) + 1e-5)).reshape(B, S, C)
    z = z * p["gw"] + p["gb"]
    h = z * torch.sigmoid(z)
    q, k, v = (t.reshape(B, S, H, C // H) for t in (h @ p["wqkv"]).split(C, -1))
    D = C // H
    half = freq.numel()
    cos, sin = (f.to(x.dtype).to(x.device) for f in ref.angles(pos, freq, (half // 2, half // 2), False, (B, S)))

    def turn(t, w):
        n = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        a, b = n[..., :half], n[..., half:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    q, k = turn(q, p["q"]), turn(k, p["k"])
    s = torch.softmax(torch.einsum("bshd,bthd->bhst", q, k) / D ** 0.5, -1)
    o = torch.einsum("bhst,bthd->bshd", s, v).reshape(B, S, C) + x
    return o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * p["ow"]


def test_block_with_gradients():
    from memory_bound_normalization_gb300.autograd import group_norm, qk_norm_rope, rms_norm

    B, hh, ww, C, G, H = 2, 6, 5, 64, 8, 4
    S, D = hh * ww, C // H
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = rnd(B, S, C)
    p = {"gw": 1 + 0.1 * rnd(C), "gb": 0.1 * rnd(C), "wqkv": rnd(C, 3 * C) / 8, "q": 1 + 0.1 * rnd(D),
         "k": 1 + 0.1 * rnd(D), "ow": 1 + 0.1 * rnd(C)}
    dy = rnd(B, S, C)
    i = torch.arange(S)
    pos = torch.stack([i // ww, i % ww]).unsqueeze(1).expand(2, B, S)
    freq = (100.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float()

    xd = x.double().requires_grad_(True)
    pd = {k: v.double().requires_grad_(True) for k, v in p.items()}
    want = plain(xd, pd, pos, freq, G, H)
    (want * dy.double()).sum().backward()

    xg = x.to(DEV).requires_grad_(True)
    pg = {k: v.to(DEV).requires_grad_(True) for k, v in p.items()}
    posd, freqd = pos.to(DEV), freq.to(DEV)
    h = group_norm(xg.view(B, hh, ww, C), G, pg["gw"], pg["gb"], 1e-5, "silu").view(B, S, C)
    qkv = h @ pg["wqkv"]
    q, k, v = (t.view(B, S, H, D) for t in qkv.split(C, -1))
    q, k = qk_norm_rope(q, k, pg["q"], pg["k"], posd, freqd, (D // 4, D // 4))
    s = torch.softmax(torch.einsum("bshd,bthd->bhst", q, k) / D ** 0.5, -1)
    o = torch.einsum("bhst,bthd->bshd", s, v).reshape(B, S, C) + xg
    got = rms_norm(o, pg["ow"], 1e-6)
    got.backward(dy.to(DEV))
    torch.cuda.synchronize()
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK

    # fp32 throughout: products of 64 terms and slabs of 240 values, a few
    # hundred roundings deep; relative to each tensor's norm
    def close(a, b, what):
        rel = float((a.detach().double().cpu() - b).norm() / b.norm())
        assert rel < 512 * ref.F, f"{what}: {rel:.3g}"

    close(got, want.detach(), "output")
    close(xg.grad, xd.grad, "dx")
    for name in p:
        close(pg[name].grad, pd[name].grad, name)
