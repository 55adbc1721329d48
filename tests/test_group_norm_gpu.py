"""Group norm with an activation, channels last, against 64-bit references on
the CPU, through the tensor-level calls, the C ABI and autograd."""
from __future__ import annotations

import threading

import pytest
import torch

import image_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    pkg.load_library(build_if_missing=True)
    yield


@pytest.fixture(autouse=True)
def _status():
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK


def make(B, S, C, dtype, w_dtype, seed=0, mean=0.5, affine=True):
    g = torch.Generator().manual_seed(seed + 1)
    x = (torch.randn(B, S, C, generator=g) * (1 + 0.3 * torch.randn(C, generator=g)) +
         mean * torch.randn(C, generator=g)).to(dtype)
    w = (1 + 0.1 * torch.randn(C, generator=g)).to(w_dtype) if affine else None
    b = (0.1 * torch.randn(C, generator=g)).to(w_dtype) if affine else None
    dy = torch.randn(B, S, C, generator=g).to(dtype)
    dev = [t if t is None else t.to(DEV) for t in (x, w, b, dy)]
    return dev


def both(x, w, b, dy, G, act, eps=1e-5):
    y, mean, rstd = pkg.group_norm_forward(x, G, w, b, eps, act)
    dx, dw, db = pkg.group_norm_backward(x, G, w, b, dy, mean, rstd, act)
    torch.cuda.synchronize()
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
    ref.check_group_norm(x, G, w, b, eps, act, y, mean, rstd)
    ref.check_group_norm_grads(x, G, w, b, dy, eps, act, dx, dw, db)
    return y, mean, rstd, dx, dw, db


# (B, S, C, G): one position, one channel a group, one group, odd positions,
# groups that end inside a 16-byte vector, channel counts that no vector fits,
# more samples than blocks share, wide channels
SHAPES = [(1, 1, 8, 1), (1, 1, 8, 8), (2, 1, 64, 4), (3, 5, 32, 32), (2, 64, 1280, 32),
          (1, 997, 320, 32), (2, 37 * 5, 120, 8), (1, 300, 36, 6), (2, 129, 13, 1), (1, 70, 7, 7),
          (5, 33, 100, 5), (1, 4096, 64, 32), (200, 9, 64, 8), (1, 50, 4096, 32),
          (2, 11, 8200, 8), (1, 3, 16416, 2), (1, 6000, 128, 32), (2, 2000, 512, 16)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype,w_dtype", [(BF16, BF16), (F16, F32), (F32, F32)],
                         ids=["bf16", "f16_wf32", "f32"])
def test_silu(shape, dtype, w_dtype):
    B, S, C, G = shape
    x, w, b, dy = make(B, S, C, dtype, w_dtype)
    both(x, w, b, dy, G, "silu")


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype,w_dtype", [(BF16, F32), (F16, F16), (F32, F32)],
                         ids=["bf16_wf32", "f16", "f32"])
@pytest.mark.parametrize("shape", [(2, 100, 320, 32), (1, 1500, 64, 8), (2, 31, 13, 13)],
                         ids=lambda s: "x".join(map(str, s)))
def test_other_activations(act, dtype, w_dtype, shape):
    B, S, C, G = shape
    x, w, b, dy = make(B, S, C, dtype, w_dtype, seed=7)
    both(x, w, b, dy, G, act)


@pytest.mark.parametrize("C", [64, 36])
def test_no_affine(C):
    x, w, b, dy = make(2, 77, C, BF16, BF16, affine=False)
    both(x, None, None, dy, 4, "silu")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S,C", [(5000, 64), (90, 36)])
def test_mean_far_from_zero(dtype, S, C):
    """A mean thousands of deviations from zero keeps the variance's digits."""
    g = torch.Generator().manual_seed(5)
    x = (1000 + (0.25 if dtype == F32 else 8) * torch.randn(2, S, C, generator=g)).to(dtype).to(DEV)
    x[:, 0] = 0  # a border of zeros is where the first values come from
    _, w, b, dy = make(2, S, C, dtype, dtype)
    both(x, w, b, dy, 4, "none")


def test_constant_slab():
    """No variance: rstd is 1/sqrt(eps), y the activation of the bias."""
    x = torch.full((2, 50, 64), 3.0, device=DEV)
    _, w, b, dy = make(2, 50, 64, F32, F32)
    y, mean, rstd, *_ = both(x, w, b, dy, 8, "silu")
    assert torch.equal(mean, torch.full_like(mean, 3.0))


@pytest.mark.parametrize("C", [64, 36])
def test_nan_and_inf_stay_in_their_slab(C):
    G = 4
    x, w, b, dy = make(3, 200, C, F32, F32)
    clean = pkg.group_norm_forward(x, G, w, b, 1e-5, "silu")
    bad = x.clone()
    bad[1, 17, 0] = float("nan")
    bad[2, 3, C - 1] = float("inf")
    y, mean, rstd = pkg.group_norm_forward(bad, G, w, b, 1e-5, "silu")
    D = C // G
    sick = torch.zeros(3, 200, C, dtype=torch.bool, device=DEV)
    sick[1, :, :D] = True
    sick[2, :, C - D:] = True
    assert torch.equal(y[~sick], clean[0][~sick])
    assert y[sick].isnan().all()
    dx, _, _ = pkg.group_norm_backward(bad, G, w, b, dy, mean, rstd, "silu")
    dx0, _, _ = pkg.group_norm_backward(x, G, w, b, dy, clean[1], clean[2], "silu")
    assert torch.equal(dx[~sick], dx0[~sick])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_extreme_arguments_of_the_activation(act):
    """Large weights drive z past every exponent: no NaN, the limits."""
    x, w, b, dy = make(1, 300, 32, F32, F32)
    both(x, w * 60, b, dy, 4, act)


def test_empty():
    for B, S in ((0, 5), (3, 0)):
        x, w, b, dy = make(B, S, 16, F32, F32)
        y, mean, rstd = pkg.group_norm_forward(x, 4, w, b)
        dx, dw, db = pkg.group_norm_backward(x, 4, w, b, dy, mean, rstd)
        assert y.shape == x.shape and dx.shape == x.shape
        assert not dw.any() and not db.any()


def test_leading_shape_and_refusals():
    x, w, b, _ = make(2, 12, 16, F32, F32)
    y = pkg.group_norm_forward(x.view(2, 3, 4, 16), 4, w, b)[0]
    assert torch.equal(y.view(2, 12, 16), pkg.group_norm_forward(x, 4, w, b)[0])
    with pytest.raises(ValueError, match="contiguous"):
        pkg.group_norm_forward(x.transpose(1, 2), 4, w[:12], b[:12])
    with pytest.raises(pkg.RMSNormError):
        pkg.group_norm_forward(x, 4, w.cpu(), b)
    with pytest.raises(pkg.RMSNormError):
        pkg.group_norm_forward(x, 4, w, b, eps=-1.0)
    two = pkg.group_norm_forward(x.reshape(24, 16), 4, w, b)[0]  # [B, C]: one position
    ref.check_group_norm(x.reshape(24, 16), 4, w, b, 1e-5, "none", two,
                         *pkg.group_norm_forward(x.reshape(24, 16), 4, w, b)[1:])


@pytest.mark.parametrize("offset", [1, 4])
def test_guard_bands_and_alignment(offset):
    """Buffers that start off 16 bytes, surrounded by values that must stay."""
    B, S, C, G = 2, 45, 64, 8
    x, w, b, dy = make(B, S, C, BF16, BF16)
    n = x.numel()

    def inside(t=None):
        buf = torch.full((n + 64,), 7.0, dtype=BF16, device=DEV)
        v = buf[32 + offset:32 + offset + n].view(B, S, C)
        if t is not None:
            v.copy_(t)
        return buf, v

    _, xv = inside(x)
    _, dv = inside(dy)
    yb, y = inside()
    db_, dx = inside()
    mean, rstd = (torch.full((B * G + 8,), 9.0, device=DEV) for _ in range(2))
    dw, db = (torch.full((C + 8,), 9.0, device=DEV) for _ in range(2))
    code = pkg.BF16
    assert pkg.rmsnorm_group_norm_fwd(xv, w, b, y, mean[4:], rstd[4:], B, S, C, G, 1e-5, 1, code) == pkg.OK
    assert pkg.rmsnorm_group_norm_bwd(xv, w, b, dv, mean[4:], rstd[4:], dx, dw[4:], db[4:], B, S, C,
                                      G, 1, code) == pkg.OK
    m, r = mean[4:4 + B * G].view(B, G), rstd[4:4 + B * G].view(B, G)
    ref.check_group_norm(x, G, w, b, 1e-5, "silu", y, m, r)
    ref.check_group_norm_grads(x, G, w, b, dy, 1e-5, "silu", dx, dw[4:-4], db[4:-4])
    for buf in (yb, db_):
        assert (buf[:32 + offset] == 7).all() and (buf[32 + offset + n:] == 7).all()
    for t in (mean, rstd, dw, db):
        assert (t[:4] == 9).all() and (t[-4:] == 9).all()


def test_dx_over_dy():
    x, w, b, dy = make(2, 600, 64, BF16, BF16)
    y, mean, rstd = pkg.group_norm_forward(x, 8, w, b, 1e-5, "silu")
    want = pkg.group_norm_backward(x, 8, w, b, dy, mean, rstd, "silu")
    dw, db = (torch.empty(64, device=DEV) for _ in range(2))
    assert pkg.rmsnorm_group_norm_bwd(x, w, b, dy, mean, rstd, dy, dw, db, 2, 600, 64, 8, 1,
                                      pkg.BF16) == pkg.OK
    assert torch.equal(dy, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])


@pytest.mark.parametrize("shape", [(2, 3000, 320, 32), (1, 40000, 64, 8), (16, 300, 640, 32),
                                   (2, 100, 36, 6)], ids=lambda s: "x".join(map(str, s)))
def test_bitwise_repeatable(shape):
    B, S, C, G = shape
    x, w, b, dy = make(B, S, C, BF16, F32)
    runs = []
    for _ in range(10):
        y, mean, rstd = pkg.group_norm_forward(x, G, w, b, 1e-5, "silu")
        runs.append((y, mean, rstd, *pkg.group_norm_backward(x, G, w, b, dy, mean, rstd, "silu")))
    for r in runs[1:]:
        for a, c in zip(runs[0], r):
            assert torch.equal(a, c)


FULL = [(1, 300 * 300, 128, 32), (3, 128 * 128, 512, 32), (2, 20000, 96, 8), (1, 700 * 701, 64, 16)]


@pytest.mark.parametrize("shape", FULL, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_full_size(shape, dtype):
    """Slabs split over many blocks, kept on chip or past what the chip keeps."""
    B, S, C, G = shape
    x, w, b, dy = make(B, S, C, dtype, F32)
    both(x, w, b, dy, G, "silu")


def test_full_size_offsets_past_32_bits():
    """Two samples of 2^31 + bytes each: the second one's offsets pass 32 bits."""
    S, C, G = 1 << 17, 8192, 8
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.zeros(2, S, C, dtype=BF16, device=DEV)
    x[1, :, ::2] = 1.0
    x[1, :, 1::2] = -1.0
    y, mean, rstd = pkg.group_norm_forward(x, G, None, None, 0.0 + 1e-5)
    assert not y[0].any()
    assert (mean.abs() < 1e-5).all()
    assert (rstd[1] - 1).abs().max() < 1e-4
    assert torch.equal(y[1, -3:], x[1, -3:]) and torch.equal(y[1, :3], x[1, :3])
    dx, _, _ = pkg.group_norm_backward(x, G, None, None, x, mean, rstd)
    # dy is xhat there: its gradient is rstd (xhat - 0 - xhat) ~ 0
    assert dx[1].abs().max() < 1e-2 and not dx[0].any()


def test_streams_and_threads():
    """Calls at once on their own streams give what they give alone."""
    cases = [(2, 64, 1280, 32), (1, 20000, 64, 8), (4, 4096, 320, 32), (2, 129, 13, 1)]
    made = [make(*c[:3], BF16, F32, seed=i) for i, c in enumerate(cases)]

    def step(i):
        x, w, b, dy = made[i]
        G = cases[i][3]
        y, mean, rstd = pkg.group_norm_forward(x, G, w, b, 1e-5, "silu")
        return (y, mean, rstd, *pkg.group_norm_backward(x, G, w, b, dy, mean, rstd, "silu"))

    alone = [step(i) for i in range(len(cases))]
    torch.cuda.synchronize()
    got, failed = {}, []

    def worker(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [step(i) for _ in range(8)]
            s.synchronize()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed, failed
    for i, want in enumerate(alone):
        for r in got[i]:
            for a, c in zip(want, r):
                assert torch.equal(a, c), cases[i]


@pytest.mark.parametrize("shape", [(2, 64, 1280, 32), (1, 9000, 128, 32), (2, 129, 13, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_captured_and_replayed(shape):
    """Two graphs over the same inputs, replayed in turn and at once."""
    B, S, C, G = shape
    x, w, b, dy = make(B, S, C, BF16, BF16)
    want = both(x, w, b, dy, G, "silu")

    def step():
        y, mean, rstd = pkg.group_norm_forward(x, G, w, b, 1e-5, "silu")
        return (y, mean, rstd, *pkg.group_norm_backward(x, G, w, b, dy, mean, rstd, "silu"))

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(s):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        for a, c in zip(want, out):
            assert torch.equal(a, c)
    # new values in the captured buffers
    x.mul_(0.5).add_(0.25)
    want = both(x, w, b, dy, G, "silu")
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for a, c in zip(want, graphs[0][1]):
        assert torch.equal(a, c)


def test_explicit_stream():
    x, w, b, _ = make(1, 5000, 64, BF16, BF16)
    want = pkg.group_norm_forward(x, 8, w, b, 1e-5, "silu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pkg.group_norm_forward(x, 8, w, b, 1e-5, "silu", stream=s)
    s.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)


@pytest.mark.parametrize("w_dtype", [F32, BF16], ids=["wf32", "wbf16"])
def test_autograd(w_dtype):
    from memory_bound_normalization_gb300.autograd import GroupNorm, group_norm

    x, w, b, dy = make(2, 60, 320, BF16, w_dtype)
    xr, wr, br = (t.clone().requires_grad_(True) for t in (x.view(2, 6, 10, 320), w, b))
    y = group_norm(xr, 32, wr, br, 1e-5, "silu")
    y.backward(dy.view(2, 6, 10, 320))
    y2, mean, rstd = pkg.group_norm_forward(x, 32, w, b, 1e-5, "silu")
    dx, dw, db = pkg.group_norm_backward(x, 32, w, b, dy, mean, rstd, "silu")
    assert torch.equal(y.view_as(y2), y2) and torch.equal(xr.grad.view_as(dx), dx)
    assert torch.equal(wr.grad, dw.to(w_dtype)) and torch.equal(br.grad, db.to(w_dtype))
    layer = GroupNorm(32, 320, activation="silu", device=DEV, weight_dtype=w_dtype)
    with torch.no_grad():
        layer.weight.copy_(w)
        layer.bias.copy_(b)
    assert torch.equal(layer(x), y2)
    # an NCHW tensor in channels_last memory format, and a broadcast gradient
    img = x.view(2, 6, 10, 320).permute(0, 3, 1, 2)
    assert img.is_contiguous(memory_format=torch.channels_last)
    z = layer(img.permute(0, 2, 3, 1))
    z.sum().backward()
    ones = torch.ones_like(x)
    _, dw1, db1 = pkg.group_norm_backward(x, 32, w, b, ones, mean, rstd, "silu")
    assert torch.equal(layer.weight.grad, dw1.to(w_dtype))
    assert torch.equal(layer.bias.grad, db1.to(w_dtype))
    bare = GroupNorm(4, 320, affine=False)
    assert bare(x).shape == x.shape and not list(bare.parameters())
