"""The host side of the image operators over a CUDA runtime that launches
nothing (fake_cudart.cpp, preloaded in a process of its own): what is launched,
on which device, with which strides."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import textwrap

import pytest

from memory_bound_normalization_gb300 import build as libbuild

TESTS = os.path.dirname(os.path.abspath(__file__))

PROLOGUE = """
import ctypes, os, sys
import memory_bound_normalization_gb300 as pkg
from memory_bound_normalization_gb300 import _lib
fake = ctypes.CDLL(os.environ["LD_PRELOAD"])
fake.fake_launch.restype = ctypes.POINTER(ctypes.c_int * 7)
fake.fake_sum_stride.restype = fake.fake_sum_rows.restype = ctypes.c_longlong
lib = pkg.load_library()
A = 1 << 44  # addresses that no launch reads


def launches():
    names = ("device", "grid", "rows", "threads", "smem", "cluster", "allowed")
    return [dict(zip(names, fake.fake_launch(i).contents)) for i in range(fake.fake_launches())]
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    libbuild.build()
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")),
                        "include")
    so = str(tmp_path_factory.mktemp("fake") / "fake_cudart.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", cuda, "-I", libbuild.CSRC, "-I",
                    libbuild.INCLUDE, os.path.join(TESTS, "fake_cudart.cpp"), "-o", so], check=True)

    def call(body):
        env = dict(os.environ, LD_PRELOAD=so, PYTHONPATH=os.path.dirname(TESTS))
        out = subprocess.run([sys.executable, "-c", PROLOGUE + textwrap.dedent(body)], env=env,
                             capture_output=True, text=True, timeout=120)
        assert out.returncode == 0, out.stdout + out.stderr
        return out.stdout

    return call


@pytest.mark.parametrize("C,G", [(1 << 20, 8), (1 << 30, 8), ((1 << 30) + 8, 4), ((1 << 31) - 1, 1)])
def test_partial_rows_of_many_channels(run, C, G):
    """A partial row is 2 C floats, which pass 31 bits with C at 2^30. (x lies off
    16 bytes: element by element.)"""
    run(f"""
    C, G = {C}, {G}
    st = lib.rmsnorm_group_norm_bwd_ws(A + 2, A, A, A, A, A, A, A, A, 2, 1, C, G, _lib.ACT_NONE, _lib.BF16, A,
                                       1 << 40, None)
    assert st == _lib.OK, st
    assert [l["rows"] for l in launches()] == [1, 1, 2], launches()
    assert launches()[0]["grid"] == 2 * ((C + 31) // 32)
    assert fake.fake_sum_rows() == 2
    assert fake.fake_sum_stride() == 2 * C, fake.fake_sum_stride()
    """)


@pytest.mark.parametrize("C", [1, 31, 32, 33, (1 << 31) - 33, (1 << 31) - 32, (1 << 31) - 1])
def test_channel_tiles(run, C):
    """Tiles of 32 channels, as the kernels count them."""
    run(f"assert fake.fake_channel_tiles({C}) == {-(-C // 32)}, fake.fake_channel_tiles({C})")


@pytest.mark.parametrize("items", [1000, (1 << 31) - 300, (1 << 31) - 1])
@pytest.mark.parametrize("back", [1, 255, 256, 257, 600])
def test_items_end(run, items, back):
    """A thread ends behind the last item, also of 2^31 - 1 (partial rows, channels)."""
    run(f"assert fake.fake_items_from({items - back}, {items}) == {-(-back // 256)}")


# shapes of clusters of 16, of one streamed slab, of several rounds
SHAPES = "[(4, 4096, 320, 32), (1, 60000, 64, 8), (6, 60000, 640, 8)]"


@pytest.mark.parametrize("bwd", [0, 1])
def test_workspace_of_another_device(run, bwd):
    """Asked for a device that is not current, the size is found out there, the
    current device stays, and a later call there is launched as it may be."""
    run(f"""
    for B, S, C, G in {SHAPES}:
        need = lib.rmsnorm_group_norm_workspace_size(B, S, C, G, _lib.BF16, {bwd}, 1)
        assert fake.fake_asked(0) == 0 and fake.fake_asked(1) > 0
        d = ctypes.c_int(-1)
        assert fake.cudaGetDevice(ctypes.byref(d)) == 0 and d.value == 0
    fake.cudaSetDevice(1)
    for B, S, C, G in {SHAPES}:
        if {bwd}:
            st = lib.rmsnorm_group_norm_bwd_ws(A, A, A, A, A, A, A, A, A, B, S, C, G, 0, _lib.BF16, A, 1 << 40, None)
        else:
            st = lib.rmsnorm_group_norm_fwd_ws(A, A, A, A, A, A, B, S, C, G, 1e-5, 0, _lib.BF16, A, 1 << 40, None)
        assert st == _lib.OK, (B, S, C, G, launches())
    assert all(l["device"] == 1 and l["allowed"] for l in launches()), launches()
    assert max(l["smem"] for l in launches()) > 48 * 1024
    assert {bwd} or max(l["cluster"] for l in launches()) == 16  # the backward plans fewer here
    """)


def test_calls_on_two_devices(run):
    """A shape used on one device and then on the other."""
    run(f"""
    for device in (0, 1, 0, 1):
        fake.cudaSetDevice(device)
        for B, S, C, G in {SHAPES}:
            assert lib.rmsnorm_group_norm_bwd(A, A, A, A, A, A, A, A, A, B, S, C, G, 1, _lib.BF16, None) == _lib.OK
            assert lib.rmsnorm_group_norm_fwd(A, A, A, A, A, A, B, S, C, G, 1e-5, 1, _lib.BF16, None) == _lib.OK
        assert all(l["allowed"] for l in launches()), launches()
        assert launches()[-1]["device"] == device
    """)
