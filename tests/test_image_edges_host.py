"""Refusals of the image operators' workspace forms and of outputs that overlap
(no GPU: every check precedes the first CUDA call)."""
from __future__ import annotations

import ctypes

import pytest

pkg = pytest.importorskip("memory_bound_normalization_gb300")
from memory_bound_normalization_gb300 import _lib  # noqa: E402

A = 1 << 20  # addresses that no call gets to read


@pytest.fixture(scope="module", autouse=True)
def _built():
    pkg.load_library(build_if_missing=True)


def rope(batch=2, length=3, hq=2, hk=2, D=16):
    d = _lib.Rope(batch=batch, length=length, q_heads=hq, k_heads=hk, head_dim=D, rotary_dim=D, axes=1,
                  positions_64=1)
    d.sections[0] = D // 2
    d.position_stride[2] = 1
    for name, h in (("q", hq), ("q_out", hq), ("dq", hq), ("k", hk), ("k_out", hk), ("dk", hk)):
        setattr(d, name, _lib.Strides(length * h * D, h * D, D))
    return d


def forward(d, q_out=5 * A, k_out=6 * A):
    return pkg.load_library().rmsnorm_qk_rope_fwd(ctypes.byref(d), A, 2 * A, 3 * A, 3 * A, 4 * A, 4 * A, q_out,
                                                  k_out, 1e-6, _lib.BF16, None)


def backward(d, dq=7 * A, dk=8 * A):
    return pkg.load_library().rmsnorm_qk_rope_bwd(ctypes.byref(d), A, 2 * A, 3 * A, 3 * A, 4 * A, 4 * A, 5 * A,
                                                  6 * A, dq, dk, 9 * A, 9 * A + 64, 1e-6, _lib.BF16, None)


@pytest.mark.parametrize("dim", ["batch", "token", "head"])
@pytest.mark.parametrize("which", ["q", "k"])
def test_outputs_that_overlap_themselves(which, dim):
    d = rope()
    setattr(getattr(d, which + "_out"), dim, 0)
    assert forward(d) == _lib.ERR_INVALID_ARG
    d = rope()
    setattr(getattr(d, "d" + which), dim, 0)
    assert backward(d) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("dim", ["batch", "token", "head"])
def test_in_place_with_other_strides(dim):
    d = rope()
    setattr(d.q_out, dim, getattr(d.q, dim) * 2)
    assert forward(d, q_out=A) == _lib.ERR_INVALID_ARG
    d = rope()
    setattr(d.dk, dim, getattr(d.k_out, dim) * 2)
    assert backward(d, dk=6 * A) == _lib.ERR_INVALID_ARG


def test_group_norm_more_pairs_than_blocks():
    """2^31 pairs of channels that no vector fits (with a device the check is
    made; without one the call ends at the device)."""
    lib = pkg.load_library()
    C = 7
    st = lib.rmsnorm_group_norm_fwd(A, None, None, 2 * A, 3 * A, 4 * A, (1 << 31) // C + 1, 1, C, C, 1e-5, 0,
                                    _lib.F32, None)
    assert st in (_lib.ERR_INVALID_ARG, _lib.ERR_CUDA)


def test_workspace_sizes_of_invalid_arguments():
    lib = pkg.load_library()
    assert lib.rmsnorm_group_norm_workspace_size(1, 1, 8, 3, _lib.F32, 0, 0) == 0
    assert lib.rmsnorm_group_norm_workspace_size(1, 1, 8, 4, 99, 0, 0) == 0
    assert lib.rmsnorm_group_norm_workspace_size(1, 1, 8, 4, _lib.F32, 0, -1) == 0
    assert lib.rmsnorm_qk_rope_bwd_workspace_size(15, 0) == 0
    assert lib.rmsnorm_qk_rope_bwd_workspace_size(258, 0) == 0
    assert lib.rmsnorm_qk_rope_bwd_workspace_size(16, -1) == 0
