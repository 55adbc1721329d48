"""The modules of the image operators without a GPU."""
from __future__ import annotations

import pytest
import torch

import memory_bound_normalization_gb300 as pkg
from memory_bound_normalization_gb300 import build as libbuild
from memory_bound_normalization_gb300.autograd import QKNormRope


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    pkg.load_library()


@pytest.mark.parametrize("norm", [True, False])
def test_queries_alone_reach_the_device_check(norm):
    """Keys are optional, with the norm as without."""
    layer = QKNormRope(16, (4, 4), norm=norm)
    pos = torch.zeros(2, 3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA tensors"):
        layer(torch.zeros(3, 4, 16), None, pos)


@pytest.mark.parametrize("norm", [True, False])
def test_materialised_from_the_meta_device(norm):
    """A module built without memory gets its frequencies with its memory: they
    are no parameter that a checkpoint would bring."""
    want = QKNormRope(16, (5, 2), theta=500.0, norm=norm)
    layer = QKNormRope(16, (5, 2), theta=500.0, norm=norm, device="meta")
    assert layer.inv_freq.is_meta
    outer = torch.nn.Sequential(layer).to_empty(device="cpu")
    assert outer[0].inv_freq.dtype == torch.float32
    assert torch.equal(outer[0].inv_freq, want.inv_freq)
    assert torch.equal(want.to_empty(device="cpu").inv_freq, layer.inv_freq)
    assert layer.to("meta").inv_freq.is_meta


def test_frequencies_follow_the_module():
    layer = QKNormRope(16, (5, 2))
    before = layer.inv_freq.clone()
    layer = layer.to(torch.bfloat16).double().cpu()
    assert layer.inv_freq.dtype == torch.float32 and torch.equal(layer.inv_freq, before)
    assert layer.q_weight.dtype == torch.float64
