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
