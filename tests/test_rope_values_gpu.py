"""Values of the rotary calls that random inputs do not reach: infinities and NaN
in the elements that pass."""
from __future__ import annotations

import pytest
import torch

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
