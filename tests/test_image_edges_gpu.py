"""Edges of the image operators on the device: workspace forms, streams that are
not the current one, the bounded wait of a split group norm, few heads and many
tokens, in-place calls and autograd, and the suites under the checked build."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import image_ref as ref
import test_group_norm_gpu as gn
import test_rope_gpu as rp

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")
from memory_bound_normalization_gb300 import _lib  # noqa: E402

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    pkg.load_library(build_if_missing=True)
    yield
    pkg.rmsnorm_test_drop_copy(-1)
    pkg.rmsnorm_set_wait_limit_ns(0)


@pytest.fixture(autouse=True)
def _status():
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK


def p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------- workspaces
# resident clusters, streamed, element by element
@pytest.mark.parametrize("shape", [(3, 64, 320, 32), (1, 60000, 64, 8), (2, 300, 13, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_group_norm_workspace(shape):
    lib = pkg.load_library()
    B, S, C, G = shape
    x, w, b, dy = gn.make(B, S, C, BF16, F32)
    y, mean, rstd, dx, dw, db = gn.both(x, w, b, dy, G, "silu")
    code = _lib.BF16_W_F32
    stream = torch.cuda.current_stream().cuda_stream
    for bwd in (0, 1):
        need = lib.rmsnorm_group_norm_workspace_size(B, S, C, G, code, bwd, 0)
        room = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)  # not zeroed
        base = room.data_ptr()
        assert base % 16 == 0
        outs = [torch.empty_like(t) for t in ((dx, dw, db) if bwd else (y, mean, rstd))]

        def call(at, n):
            if bwd:
                return lib.rmsnorm_group_norm_bwd_ws(p(x), p(w), p(b), p(dy), p(mean), p(rstd), *map(p, outs),
                                                     B, S, C, G, _lib.ACT_SILU, code, at, n, stream)
            return lib.rmsnorm_group_norm_fwd_ws(p(x), p(w), p(b), *map(p, outs), B, S, C, G, 1e-5,
                                                 _lib.ACT_SILU, code, at, n, stream)

        if shape == (3, 64, 320, 32) and not bwd:
            # a slab that a cluster keeps: none is needed where 16-byte vectors fit
            assert call(None, 0) == _lib.OK
        else:
            assert need > 0 and call(None, need) == _lib.ERR_INVALID_ARG
            assert call(base, 16) == _lib.ERR_INVALID_ARG
        if S > 1000:
            assert call(base, need - 1) == _lib.ERR_INVALID_ARG
        assert call(base + 8, need + 16) == _lib.ERR_MISALIGNED
        assert call(base, need) == _lib.OK
        torch.cuda.synchronize()
        assert (room[need:] == 255).all()
        for got, want in zip(outs, (dx, dw, db) if bwd else (y, mean, rstd)):
            assert torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 100, 128])
def test_rope_workspace(D):
    lib = pkg.load_library()
    a, dq, dk = rp.make((2, 70), 4, 2, D, (D // 2,), BF16, F32)
    want = rp.verify(a, dq, dk)[2:]
    d = _lib.Rope(batch=2, length=70, q_heads=4, k_heads=2, head_dim=D, rotary_dim=D, axes=1, positions_64=1)
    d.sections[0] = D // 2
    d.position_stride[1], d.position_stride[2] = 70, 1
    for name, h in (("q", 4), ("q_out", 4), ("dq", 4), ("k", 2), ("k_out", 2), ("dk", 2)):
        setattr(d, name, _lib.Strides(70 * h * D, h * D, D))
    need = lib.rmsnorm_qk_rope_bwd_workspace_size(D, 0)
    assert need > 0
    room = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    base = room.data_ptr()
    outs = [torch.empty_like(t) for t in want]

    def call(at, n):
        return lib.rmsnorm_qk_rope_bwd_ws(ctypes.byref(d), p(a["q"]), p(a["k"]), p(a["wq"]), p(a["wk"]),
                                          p(a["positions"]), p(a["inv_freq"]), p(dq), p(dk), *map(p, outs),
                                          1e-6, _lib.BF16_W_F32, at, n,
                                          torch.cuda.current_stream().cuda_stream)

    assert call(None, need) == _lib.ERR_INVALID_ARG
    assert call(base, 0) == _lib.ERR_INVALID_ARG
    assert call(base + 8, need) == _lib.ERR_MISALIGNED
    assert call(base, need) == _lib.OK
    torch.cuda.synchronize()
    assert (room[need:] == 255).all()
    for got, w in zip(outs, want):
        assert torch.equal(got, w)


def test_group_norm_more_pairs_than_blocks():
    lib = pkg.load_library()
    C = 7
    at = torch.zeros(64, device=DEV).data_ptr()
    n = (1 << 31) // C + 1
    assert lib.rmsnorm_group_norm_fwd(at, None, None, at + 16, at + 32, at + 48, n, 1, C, C, 1e-5, 0, _lib.F32,
                                      None) == _lib.ERR_INVALID_ARG
    assert lib.rmsnorm_group_norm_bwd(at, None, None, at, at + 32, at + 48, at + 16, None, None, n, 1, C, C, 0,
                                      _lib.F32, None) == _lib.ERR_INVALID_ARG


# ------------------------------------------------------------- the bounded wait
@pytest.mark.parametrize("bwd", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("shape,unit", [((1, 60000, 64, 8), 0), ((6, 60000, 64, 8), 3)], ids=["one", "rounds"])
def test_lost_share_times_out_and_recovers(shape, unit, bwd):
    """A block that never reports its share: the others give up in time, the
    status says so, and the next call is right. (The share is lost in a slab
    that the first block of the grid has a part of.)"""
    B, S, C, G = shape
    x, w, b, dy = gn.make(B, S, C, BF16, F32)
    y, mean, rstd, dx, dw, db = gn.both(x, w, b, dy, G, "silu")
    call = ((lambda: pkg.group_norm_backward(x, G, w, b, dy, mean, rstd, "silu")) if bwd else
            (lambda: pkg.group_norm_forward(x, G, w, b, 1e-5, "silu")))
    torch.cuda.synchronize()
    pkg.rmsnorm_set_wait_limit_ns(50_000_000)
    try:
        for u in range(unit + 1):  # the slabs of the first block come in turn
            pkg.rmsnorm_test_drop_copy(u)
            call()
            st = pkg.rmsnorm_get_last_device_error()
            if u == 0:
                assert st == pkg.ERR_DEVICE_TIMEOUT
            assert st in (pkg.OK, pkg.ERR_DEVICE_TIMEOUT)
    finally:
        pkg.rmsnorm_test_drop_copy(-1)
        pkg.rmsnorm_set_wait_limit_ns(0)
    got = call()
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
    for g, want in zip(got, (dx, dw, db) if bwd else (y, mean, rstd)):
        assert torch.equal(g, want)


# ------------------------------------------------------------- streams
@pytest.mark.parametrize("shape", [(2, 64, 320, 32), (1, 60000, 64, 8), (2, 300, 13, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_backward_on_another_stream(shape):
    B, S, C, G = shape
    x, w, b, dy = gn.make(B, S, C, BF16, F32)
    y, mean, rstd, dx, dw, db = gn.both(x, w, b, dy, G, "silu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [pkg.group_norm_backward(x, G, w, b, dy, mean, rstd, "silu", stream=s) for _ in range(4)]
    s.synchronize()
    for g in got:
        for u, v in zip(g, (dx, dw, db)):
            assert torch.equal(u, v)


def test_rope_backward_on_another_stream():
    a, dq, dk = rp.make((3, 50), 6, 2, 128, (16, 24, 24), BF16, F32)
    want = rp.verify(a, dq, dk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk, stream=s) for _ in range(4)]
    s.synchronize()
    for g in got:
        for u, v in zip(g, want[2:]):
            assert torch.equal(u, v)


@pytest.mark.parametrize("call", ["group_norm", "rope"])
def test_memory_of_another_stream(call):
    """A call on a given stream takes no memory that the current stream still has
    work queued on."""
    n = 1 << 20
    x = torch.randn(1, n // 64, 64, device=DEV)
    q = x.view(n // 128, 2, 64)
    pos = torch.zeros(1, n // 128, dtype=torch.int32, device=DEV)
    freq = torch.ones(32, device=DEV)
    s = torch.cuda.Stream()
    for _ in range(3):
        t = torch.full((n,), 7.0, device=DEV)
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)
        seen = t.clone()
        del t
        if call == "group_norm":
            got = pkg.group_norm_forward(x, 8, stream=s)
        else:
            got = pkg.qk_rope_forward(q, None, None, None, pos, freq, (32,), stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        assert (seen == 7).all()
        del got


# ------------------------------------------------------------- shapes
# (lead, Hq, Hk, D, sections): tiles of one pass and of a part of one, rows that
# end inside a pass, many heads a token, more tokens than blocks
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype,w_dtype", [(BF16, F32), (F16, None), (F32, F32)], ids=["bf16", "f16_rot", "f32"])
@pytest.mark.parametrize("case", [((20011,), 1, 1, 64, (32,)), ((3, 3333), 2, 1, 128, (10, 22)),
                                  ((5000,), 1, 0, 256, (128,)), ((701,), 64, 16, 64, (16, 16)),
                                  ((40,), 128, 128, 96, (48,)), ((1,), 200, 8, 128, (40, 24)),
                                  ((9001,), 3, 1, 112, (20, 8)), ((4001,), 2, 1, 56, (28,)),
                                  ((3001,), 1, 1, 24, (12,)), ((2500,), 3, 2, 100, (25, 25))],
                         ids=lambda c: f"{'x'.join(map(str, c[0]))}_{c[1]}_{c[2]}_{c[3]}")
def test_rope_rows_and_tiles(case, dtype, w_dtype, adjacent):
    a, dq, dk = rp.make(*case, dtype, w_dtype, seed=3)
    rp.verify(a, dq, dk, adjacent=adjacent)


# every number of units a head can have with 16- and 8-byte pieces, and some of
# single elements: groups of as many lanes, of the next power of two, idle lanes
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dtype,w_dtype", [(F16, F16), (F32, F32)], ids=["f16", "f32"])
@pytest.mark.parametrize("D", [4, 8, 12, 16, 24, 30, 32, 40, 48, 56, 72, 80, 88, 104, 112, 120, 132, 144, 160, 176,
                               192, 208, 224, 240, 248])
def test_rope_every_width(D, dtype, w_dtype, adjacent):
    a, dq, dk = rp.make((37,), 3, 2, D, (D // 2 - D // 4, D // 4), dtype, w_dtype, seed=D)
    rp.verify(a, dq, dk, adjacent=adjacent)


# group widths around the lanes that join them, channels that split over blocks
# or not, fewer positions than lanes
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("S", [1, 7, 260])
@pytest.mark.parametrize("C,G", [(8, 8), (16, 4), (24, 8), (72, 8), (136, 8), (200, 4), (264, 8), (320, 64), (512, 4),
                                 (1056, 32), (2048, 2)])
def test_group_norm_widths(C, G, S, dtype):
    x, w, b, dy = gn.make(3, S, C, dtype, F32, seed=C)
    gn.both(x, w, b, dy, G, "silu")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 20000, 96, 8), (1, 900, 640, 32)], ids=lambda s: "x".join(map(str, s)))
def test_mean_far_from_zero_behind_borders(shape, dtype):
    """A border of zeros and a few zeroed positions inside: what a channel's
    values are taken about is not one of them."""
    B, S, C, G = shape
    g = torch.Generator().manual_seed(9)
    x = (1000 + (0.25 if dtype == F32 else 8) * torch.randn(B, S, C, generator=g)).to(dtype)
    x[:, :40] = 0
    x[:, -40:] = 0
    x[:, S // 2 - 3:S // 2 + 3] = 0
    x = x.to(DEV)
    _, w, b, dy = gn.make(B, S, C, dtype, dtype)
    gn.both(x, w, b, dy, G, "none")


@pytest.mark.parametrize("shape", [(3000, 1, 64, 8), (700, 2, 320, 32), (1, 2, 8, 2), (1, 3, 2048, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_few_positions_many_samples(shape):
    B, S, C, G = shape
    x, w, b, dy = gn.make(B, S, C, F16, F32, seed=5)
    gn.both(x, w, b, dy, G, "gelu")


# ------------------------------------------------------------- autograd
def test_in_place_is_seen_by_autograd():
    """A tensor saved for a backward pass and then turned in place is refused
    there, as for PyTorch's own in-place functions."""
    a, _, _ = rp.make((9,), 2, 1, 64, (32,), F32, F32)
    leaf = torch.ones_like(a["q"], requires_grad=True)
    out = leaf * a["q"]  # saves q
    pkg.qk_rope_forward(**a, out=(a["q"], a["k"]))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    with torch.inference_mode():
        b, _, _ = rp.make((9,), 2, 1, 64, (32,), F32, F32)
        pkg.qk_rope_forward(**b, out=(b["q"], b["k"]))
    assert torch.equal(a["q"], b["q"])


def test_outputs_that_overlap_are_refused():
    a, _, _ = rp.make((9,), 2, 1, 64, (32,), F32, F32)
    wide = torch.empty(1, 2, 64, device=DEV).expand(9, 2, 64)
    with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
        pkg.qk_rope_forward(**a, out=(wide, torch.empty_like(a["k"])))


# ------------------------------------------------------------- checked build
def test_image_suites_under_checks():
    """The image operators' tests with every global store, asynchronous copy and
    shared-memory slot tested against its extent; a failed check is reported as
    RMSNORM_ERR_OUT_OF_BOUNDS, which every test reads back."""
    from memory_bound_normalization_gb300 import build as libbuild

    if _lib.checked_variant():
        pytest.skip("runs the checked build already")
    libbuild.build(checked=True)
    env = dict(os.environ)
    env["RMSNORM_LIBRARY_VARIANT"] = "checked"
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k",
           "not full_size and not bitwise_repeatable", "tests/test_group_norm_gpu.py", "tests/test_rope_gpu.py",
           "tests/test_image_block_gpu.py", "tests/test_image_edges_gpu.py"]
    out = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (out.stdout + out.stderr)[-4000:]
    assert out.returncode == 0, tail
    assert " passed" in tail and " failed" not in tail, tail
