"""The modules of the image operators on the device."""
from __future__ import annotations

import pytest
import torch

import test_rope_gpu as rp

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")
from memory_bound_normalization_gb300.autograd import QKNormRope  # noqa: E402

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    pkg.load_library(build_if_missing=True)


def test_queries_alone_with_the_norm():
    """What the tensor-level calls give without keys; the key weight has no part in it."""
    a, dq, _ = rp.make((2, 20), 4, 2, 64, (8, 12, 12), BF16, F32)
    layer = QKNormRope(64, (8, 12, 12), device=DEV)
    with torch.no_grad():
        layer.q_weight.copy_(a["wq"])
    q = a["q"].clone().requires_grad_(True)
    y, k = layer(q, None, a["positions"])
    assert k is None
    y.backward(dq)
    alone = {**a, "k": None, "wk": None}
    want = pkg.qk_rope_forward(**alone)
    dx, _, dw, _ = pkg.qk_rope_backward(**alone, dq_out=dq, dk_out=None)
    assert torch.equal(y, want[0])
    assert torch.equal(q.grad, dx) and torch.equal(layer.q_weight.grad, dw)
    assert layer.k_weight.grad is None
