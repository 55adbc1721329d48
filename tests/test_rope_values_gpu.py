"""Values of the rotary calls that random inputs do not reach: infinities and NaN
in the elements that pass, far positions."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest
import torch

import image_ref as ref
import test_rope_gpu as rp

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


# pieces of 16, 8 bytes and one element; constant and run-time lanes
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,rot", [(128, 64), (128, 52), (64, 32), (80, 16), (96, 32), (256, 64), (112, 56), (100, 50),
                                   (112, 8)])
@pytest.mark.parametrize("norm", [False, True], ids=["rot", "norm"])
@pytest.mark.parametrize("where", ["inputs", "gradients"])
def test_infinities_in_elements_that_pass(where, D, rot, dtype, adjacent, norm):
    """An element that passes is its own value, whatever lies beside it: an
    infinity or NaN reaches no other element without the norm, and with it only
    as far as the row's sum takes it."""
    half = rot // 2
    a, dq, dk = rp.make((2, 9), 3, 2, D, (half - half // 2, half // 2), dtype, dtype if norm else None, seed=D)
    inf, nan = float("inf"), float("nan")
    for t in (a["q"], a["k"]) if where == "inputs" else (dq, dk):
        t[0, 2, 0, rot] = inf
        t[0, 4, 1, D - 1] = -inf
        t[1, 1, 0, rot + (D - rot) // 2] = nan
        t[1, 7, 1, rot + 1] = inf
    rp.verify(a, dq, dk, adjacent=adjacent)


# 80 digits of pi
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089, 10 ** 79)


def exact_angles(positions, freq, axis):
    """cos and sin of the exact product, reduced in rational arithmetic, and how far
    the angle may be off: the position times 2^-63 turns."""
    theta, off = np.empty((positions.shape[1], len(axis))), np.empty((positions.shape[1], len(axis)))
    for p, a in enumerate(axis):
        turns = Fraction(float(freq[p])) / (2 * PI)
        for t in range(positions.shape[1]):
            at = int(positions[a, t]) * turns
            at -= round(at)
            theta[t, p] = float(at * 2 * PI)
            off[t, p] = abs(int(positions[a, t])) * 2.0 ** -63 * 2 * np.pi
    theta, off = (torch.from_numpy(v).unsqueeze(-2) for v in (theta, off))
    return torch.cos(theta), torch.sin(theta), off


@pytest.mark.parametrize("dtype", [F32, F16], ids=["f32", "f16"])
@pytest.mark.parametrize("D", [64, 100])
@pytest.mark.parametrize("theta", [10000.0, 0.0001])
def test_far_positions(dtype, D, theta):
    """An angle is off by its rounding and the position times 2^-63 turns: a chord of
    the pair's length by that angle."""
    n, half = 16, D // 2
    g = torch.Generator().manual_seed(4)
    a, dq, dk = rp.make((n,), 2, 1, D, (half - 5, 5), dtype, None)
    pos = torch.tensor([0, 1, -1, (1 << 31) - 1, -(1 << 31), (1 << 32) + 1, 1 << 36, -(1 << 36) - 1, (1 << 40) + 3,
                        -(1 << 40) + 1, (1 << 44) - 1, (1 << 48) + 12345, -(1 << 53) - 1, (1 << 53) + 1, (1 << 56) - 1,
                        0x123456789abcde])
    a["positions"] = torch.stack([pos, pos[torch.randperm(n, generator=g)]]).to(DEV)
    a["inv_freq"] = (theta ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEV)
    qo, ko = pkg.qk_rope_forward(**a)
    gq, gk, _, _ = pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk)
    cos, sin, off = exact_angles(a["positions"].cpu(), a["inv_freq"].cpu(), ref.axis_of_pairs(a["sections"], False))
    off = torch.cat((off, off), -1)
    for x, y, turn, what in ((a["q"], qo, sin, "q"), (a["k"], ko, sin, "k"), (dq, gq, -sin, "dq"), (dk, gk, -sin, "dk")):
        X = x.double().cpu()
        want, length = ref.rotate(X, cos, turn, D, False), ref.spread(X, D, False)
        ref.check(y, want, ref.rounding(dtype, want) * 1.01 + (64 * ref.F + off) * length, what)
