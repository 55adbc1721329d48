"""Values of the group norm that random inputs do not reach: the activations over
their whole range, many positions that differ little, none.

Bounds. F is 2^-24 (an fp32 rounding). With weights of zero z is the bias, exactly,
so that y = act(b) and, for one position and dy = 1, db = act'(b) in fp32."""
from __future__ import annotations

import pytest
import torch

import image_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
F = 2.0 ** -24


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


# ------------------------------------------------------------- activations
# 4096 arguments by 16-byte vectors, and 4097 element by element; every exponent
# from 2^-20 to the largest argument, both signs
def arguments(n, largest):
    g = torch.Generator().manual_seed(n)
    a = torch.cat([torch.linspace(-largest, largest, n // 2),
                   torch.exp2(torch.empty(n - n // 2).uniform_(-20, torch.tensor(largest).log2().item(), generator=g))])
    a[n // 2::2] *= -1
    return a.to(DEV)


def value_and_slope(z, dtype, name, positions):
    """y and act' of every argument, through the public calls."""
    C = z.numel()
    groups = 64 if C % 64 == 0 else 1
    x = torch.randn(1, positions, C, device=DEV).to(dtype)
    w = torch.zeros(C, device=DEV)
    y, mean, rstd = pkg.group_norm_forward(x, groups, w, z, 1e-5, name)
    dy = torch.zeros_like(x)
    dy[:, -1] = 1  # one position's slope, so that db holds nothing else
    _, dw, db = pkg.group_norm_backward(x, groups, w, z, dy, mean, rstd, name)
    assert (y == y[:, :1]).all()
    return y[0, 0], db


def exact(z, name):
    Z = z.double().cpu()
    if name == "silu":
        s, o = torch.sigmoid(Z), torch.sigmoid(-Z)
        return Z, Z * s, s * (1 + Z * o), s, o
    tail = torch.special.erfcx(Z.abs() / 2 ** 0.5) * torch.exp(-Z * Z / 2) / 2
    phi = torch.where(Z < 0, tail, 1 - tail)
    density = torch.exp(-Z * Z / 2) / (2 * torch.pi) ** 0.5
    return Z, Z * phi, phi + Z * density, phi, density


TINY = 2.0 ** -118  # results below may be flushed, or lose bits of a subnormal fp32 factor


# fp32: with the exponential and the reciprocal good to 2^-22 of their values (4 F)
# and some ten roundings of products and sums behind them, 16 F of a value. A slope
# is a sum of two terms that cancel near its zero: 16 F of either. Silu's takes
# 1 - s for the other side, in either path: s = 1 / (1 + e^-z) is F (the sum) and 2 F
# (the reciprocal) of s off, the difference F more, and z s times that is 4 F |z| s.
# GELU has its polynomial (6 F) and sum of ten steps: 32 F. Its e^(-z^2/2) is a power
# of a product that is rounded twice, F each, of a constant that is 0.2 F off: the
# exponent, z^2/2, is 2.2 F of itself off and the power 1.1 z^2 F of itself.
@pytest.mark.parametrize("C,positions", [(4096, 1), (4097, 2), (512, 30000)], ids=["vectors", "elements", "streamed"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activation_in_32_bits(name, C, positions):
    z = arguments(C, 80.0 if name == "silu" else 12.5)
    y, db = value_and_slope(z, F32, name, positions)
    Z, value, slope, s, o = exact(z, name)
    k = 16 if name == "silu" else 32 + 1.25 * Z * Z
    err = (y.double().cpu() - value).abs()
    bound = k * F * value.abs() + TINY
    assert (err <= bound).all(), f"value {float((err / bound).max()):.2f} of the bound at {float(Z[(err / bound).argmax()])}"
    terms = s + (Z * s * o).abs() if name == "silu" else s + (Z * o).abs()
    err = (db.double().cpu() - slope).abs()
    bound = k * F * terms + (4 * F * Z.abs() * s if name == "silu" else 0) + TINY
    assert (err <= bound).all(), f"slope {float((err / bound).max()):.2f} of the bound at {float(Z[(err / bound).argmax()])}"


# 16 bits: an approximation is a sixteenth of half an f16 step (2^-16) where f16 has
# normal values and 2^-13, a sixteenth of half a bf16 step, behind; then one rounding.
# A slope is summed in 32 bits (db): 16 F of 1 from the approximation, or the same
# parts of the value where that is less, and 16 F of its terms from the arithmetic.
@pytest.mark.parametrize("C,positions", [(4096, 1), (4097, 2), (512, 30000)], ids=["vectors", "elements", "streamed"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activation_in_16_bits(name, dtype, C, positions):
    z = arguments(C, 80.0 if name == "silu" else 12.5)
    y, db = value_and_slope(z, dtype, name, positions)
    Z, value, slope, s, o = exact(z, name)
    near = torch.where(Z.abs() <= 4.5, 2.0 ** -16, 2.0 ** -13)
    err = (y.double().cpu() - value).abs()
    bound = near * value.abs() + ref.rounding(dtype, value) * 1.001 + TINY
    assert (err <= bound).all(), f"value {float((err / bound).max()):.2f} of the bound at {float(Z[(err / bound).argmax()])}"
    terms = s + (Z * s * o).abs() if name == "silu" else s + (Z * o).abs()
    err = (db.double().cpu() - slope).abs()
    bound = torch.minimum(near * terms, torch.tensor(16 * F)) + 16 * F * terms + TINY
    assert (err <= bound).all(), f"slope {float((err / bound).max()):.2f} of the bound at {float(Z[(err / bound).argmax()])}"


# ------------------------------------------------------------- statistics
# Element by element (3 channels), millions of positions that differ little: the mean
# is a few roundings off (4 F of it), and what its error leaves in the deviations is
# rstd times that; their own sums are K F of the mean deviation: n values over 64 blocks
# of 256 threads, in runs of 64, which are added up, then 13 in a block, 64 over the
# blocks and a few: K = 149 + n / 16384 / 64.
@pytest.mark.parametrize("level", [1000.0 / 3, 1.0 / 3])
@pytest.mark.parametrize("S", [1 << 22, 1000003])
def test_mean_of_many_positions_element_by_element(S, level):
    g = torch.Generator().manual_seed(1)
    x = (level * (1 + 2.0 ** -20 * torch.randn(1, S, 3, generator=g))).to(DEV)
    y, mean, rstd = pkg.group_norm_forward(x, 1, None, None, 1e-12)
    X = x.double()
    m = X.mean()
    d = X - m
    var = (d * d).mean()
    r = (var + 1e-12).rsqrt()
    K = 149 + X.numel() / 16384 / 64
    spread = d.abs().mean()
    e_mean = 4 * F * m.abs() + K * F * spread
    assert (mean.double() - m).abs() <= e_mean, float((mean.double() - m).abs() / (F * m.abs()))
    # squares about a mean that is off by e: e^2 more, beside their own roundings
    e_r = K * F + (e_mean * r) ** 2
    assert (rstd.double() / r - 1).abs() <= e_r
    err = (y.double() - d * r).abs()
    assert (err <= r * e_mean + (e_r + 4 * F) * (d * r).abs()).all(), float((err / (r * e_mean)).max())


def test_one_sided_gradients_element_by_element():
    """Weight gradients over millions of positions whose terms have one sign: sums
    in runs of 64, some 128 runs a thread, then 8, 64 blocks and the column sum's
    trees: 256 roundings hold them."""
    S = 1 << 22
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, S, 3, generator=g).abs().to(DEV)
    dy = (1.0 / 3 + 2.0 ** -22 * torch.randn(1, S, 3, generator=g)).to(DEV)
    w, b = torch.ones(3, device=DEV), torch.zeros(3, device=DEV)
    mean, rstd = torch.zeros(1, 1, device=DEV), torch.ones(1, 1, device=DEV)
    dx, dw, db = pkg.group_norm_backward(x, 1, w, b, dy, mean, rstd)
    X, D = x.double(), dy.double()
    for got, terms in ((db, D), (dw, D * X)):
        want = terms.sum((0, 1))
        assert ((got.double() - want).abs() <= 256 * F * terms.abs().sum((0, 1))).all(), \
            float(((got.double() - want).abs() / want / F).max())
    A, Bq = D.mean(), (D * X).mean()
    e = 300 * F * (A.abs() + X * Bq.abs()) + 8 * F * (D.abs() + A + X * Bq)
    assert ((dx.double() - (D - A - X * Bq)).abs() <= e).all()


@pytest.mark.parametrize("C", [8, 3], ids=["vectors", "elements"])
def test_one_sided_gradients_of_many_samples(C):
    """A partial row a sample, a million of them: 4096 rows a thread of the column
    sum in runs of 64, 13 in its trees: 256 roundings hold them."""
    B = 1 << 20
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, 1, C, generator=g).abs().to(DEV)
    dy = (0.4 + 2.0 ** -22 * torch.randn(B, 1, C, generator=g)).to(DEV)
    w, b = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    mean, rstd = torch.zeros(B, 1, device=DEV), torch.ones(B, 1, device=DEV)
    _, dw, db = pkg.group_norm_backward(x, 1, w, b, dy, mean, rstd)
    for got, terms in ((db, dy.double()), (dw, dy.double() * x.double())):
        want = terms.sum((0, 1))
        assert ((got.double() - want).abs() <= 256 * F * want).all(), float(((got.double() - want).abs() / want / F).max())


def test_statistics_of_no_positions():
    """They are means of nothing: NaN, not what the memory held."""
    for shape in ((3, 0, 16), (3, 4, 0, 16)):
        x = torch.empty(shape, device=DEV)
        junk = torch.full((64, 12), 5.0, device=DEV)
        del junk
        y, mean, rstd = pkg.group_norm_forward(x, 4)
        assert y.shape == x.shape and mean.shape == rstd.shape == (3, 4)
        assert mean.isnan().all() and rstd.isnan().all()
