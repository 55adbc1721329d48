"""The host side of the rows by index, and what its kernels count by, at the ends of
their ranges: over a CUDA runtime that launches nothing, or compiled for the host."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

import memory_bound_normalization_gb300 as pkg
from memory_bound_normalization_gb300 import build as libbuild
from test_image_launches_host import run  # noqa: F401  (a fixture)

BIG = (1 << 31) - 1

STEPS_PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "rows.h"
int main(int, char** v) {
    const int choices = atoi(v[1]), step = atoi(v[2]);
    // the loop of a kernel from its last few steps on
    long long taken = 0, steps = 0;
    for (unsigned k0 = static_cast<unsigned>((choices > 1000 ? choices - 1000 : 0) / step) * step;
         rmsn::more_choices(k0, choices); k0 += step) {
        if (++steps > 2000) break;
        for (int k = 0; k < step; ++k) taken += rmsn::more_choices(k0 + k, choices);
    }
    std::printf("%lld\n", taken);
    return 0;
}
"""


@pytest.fixture(scope="module")
def steps(tmp_path_factory):
    d = tmp_path_factory.mktemp("steps")
    (d / "steps.cpp").write_text(STEPS_PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(libbuild._nvcc())), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", cuda, "-I", libbuild.CSRC, "-I", libbuild.INCLUDE,
                    str(d / "steps.cpp"), "-o", str(d / "steps")], check=True)

    def call(*a):
        return int(subprocess.run([str(d / "steps"), *map(str, a)], capture_output=True, text=True, check=True).stdout)

    return call


@pytest.mark.parametrize("step", [1, 2, 4])
@pytest.mark.parametrize("choices", [1, 3, 4, 5, 999, 1000, BIG - 4, BIG - 3, BIG - 2, BIG - 1, BIG])
def test_choices_end(steps, choices, step):
    """Steps of several choices end behind the last one, also of 2^31 - 1 (a signed count
    went on from -2^31, before the token's positions)."""
    first = max(0, choices - 1000) // step * step
    assert steps(choices, step) == choices - first


def test_ring_of_choices(run):  # noqa: F811
    """The combine backward's ring (the one launch with shared memory) takes 5 to 1024
    choices: its blocks count their steps in 32 bits."""
    run(f"""
    for choices, ring in ((4, False), (5, True), (1024, True), (1025, False), (1 << 28, False), ({BIG}, False)):
        d = _lib.Experts(tokens=1, rows=4096, width=4096, token_stride=4096, row_stride=4096, residual_stride=4096,
                         drow_stride=4096, choices=choices)
        assert lib.rmsnorm_expert_combine_bwd(ctypes.byref(d), A, A, A, A, A, A, A, _lib.BF16, None) == _lib.OK
        assert (launches()[-1]["smem"] > 0) == ring, (choices, launches()[-1])
    """)


@pytest.mark.parametrize("dtype,size", [("F32", 4), ("BF16", 2), ("F16_W_F32", 2)])
def test_ring_of_the_widest_rows(run, dtype, size):  # noqa: F811
    """Rows of 2^31 bytes and more go by the ring as shorter ones do."""
    run(f"""
    for width in (512 // {size} - 4, 512 // {size}, 1 << 28, (1 << 31) // {size} - 4, (1 << 31) // {size},
                  (1 << 31) // {size} + 4, (1 << 31) - 4):
        d = _lib.Experts(tokens=1, rows=1 << 17, width=width, token_stride=width, row_stride=width,
                         residual_stride=width, drow_stride=width, choices=6)
        assert lib.rmsnorm_expert_combine_bwd(ctypes.byref(d), A, A, A, A, A, A, A, _lib.{dtype}, None) == _lib.OK
        ring = launches()[-1]["smem"] > 0
        assert ring == (width * {size} >= 512), width
    """)


# ------------------------------------------------------------- workspaces
# around every limit: one launch, one cluster, tiles, segments of 8, 16 and 32 tokens
TOKENS = sorted({257, 300, 1000, 2432, 4863, 4864, 4865, 9727, 9728, 16383, 16384, 16385, 20000, 38911, 38912, 77823, 77824,
                 77825, 100_000, 131_072, 155_647, 155_648, 155_649, 200_000, 311_295, 311_296, 311_297, 400_000, 700_000,
                 1 << 20, 1 << 24})


@pytest.mark.parametrize("width", [1, 8, 129, 256, 1000, 4096, 8192, 100_000])
@pytest.mark.parametrize("rows", [1, 511, 512, 131072])
def test_workspaces_do_not_shrink(rows, width):
    """One for the largest batch serves smaller ones."""
    size = [pkg.rmsnorm_embedding_bwd_workspace_size(n, rows, width) for n in TOKENS if n * width <= 1 << 38]
    assert size == sorted(size), [(n, a, b) for n, a, b in zip(TOKENS, size, size[1:]) if b < a]
    size = [pkg.rmsnorm_expert_sort_workspace_size(n, 1, min(rows, 1024)) for n in TOKENS]
    assert size == sorted(size)


def test_workspaces_hold_what_is_launched(run):  # noqa: F811
    """Room for the spans that the launches have (a block's tokens by its shared memory),
    and no more than a few times that for large calls."""
    run(f"""
    for width in (1, 2, 8, 64, 129, 256, 1000, 4096, 8192, 100000):
        for n in {TOKENS}:
            if n * width > 1 << 38:
                continue
            for rows in (1, 511, 131072):
                e = _lib.Embedding(outer=1, inner=n, num_rows=rows, width=width, table_stride=width, row_stride=width,
                                   ids_64=1, scale=1.0)
                e.id_stride[1] = 1
                need = lib.rmsnorm_embedding_bwd_workspace_size(n, rows, width)
                for at in (A, A + 2):  # by pieces of 16 bytes, element by element
                    before = len(launches())
                    st = lib.rmsnorm_embedding_bwd_ws(ctypes.byref(e), A, at, A, -1, 1, _lib.BF16, A, need, None)
                    assert st == _lib.OK, (n, rows, width)
                    sums = [l for l in launches()[before:] if l["threads"] == 256][0]
                    span = (sums["smem"] // 4 - 2) // 2
                    spans = -(-n // span)
                    used = 16 * n + 8 * spans * width
                    assert used <= need, (n, rows, width, span)
                    if n >= 131072 and at == A:
                        assert need <= 1.5 * used + rows + (1 << 20), (n, rows, width, need, used)
    """)


@pytest.mark.parametrize("n", [1, 200, 3000, 20000])
def test_short_rows_are_shared_out(run, n):  # noqa: F811
    """Rows without a token: a warp looks at 32 after 32, so a share of short ones is
    bounded by their number, not by their bytes alone."""
    run(f"""
    for rows, width, wide in ((5288, 2, 0), (1000000, 1, 0), (40000, 8, 0), (200984, 10, 1), (40000000, 3, 1)):
        e = _lib.Embedding(outer=1, inner={n}, num_rows=rows, width=width, table_stride=width, row_stride=width,
                           ids_64=1, scale=1.0)
        e.id_stride[1] = 1
        dtype = _lib.BF16_W_F32 if wide else _lib.BF16
        def blocks(accumulate):
            before = len(launches())
            assert lib.rmsnorm_embedding_bwd_ws(ctypes.byref(e), A, A, A, -1, accumulate, dtype, A, 1 << 40,
                                                None) == _lib.OK
            return [l for l in launches()[before:] if l["threads"] == 256][0]["grid"]
        size = (4 if wide else 2) * width
        if {n} <= 256:
            left = rows
        else:  # what is zeroed beside the sort
            passes = -(-rows.bit_length() // 9)
            left = rows - min(rows, -(-(48 << 20 if {n} <= 16384 else passes * 24 << 20) // size))
        zero = blocks(0) - blocks(1)  # with nothing to zero there are the sums' blocks alone
        # an even share of 96 warps an SM, in whole 32s; no share is larger than 16 KB
        share = max(32, min(16384 // size // 32 * 32, -(-left // (152 * 96 * 32)) * 32))
        assert zero == -(-(-(-left // share)) // 8), (rows, width, zero, share)
    """)


# ------------------------------------------------------------- the checked build's checks
def unchecked(name, access):
    """Lines with such an access that no check of the checked build stands before."""
    with open(os.path.join(libbuild.CSRC, name)) as fh:
        lines = fh.read().split("\n")
    found = [i for i, line in enumerate(lines) if re.search(access, line)]
    assert found, f"no {access} in {name}"
    return [lines[i].strip() for i in found if not any("RMSN_OK" in near for near in lines[max(0, i - 5):i + 1])]


@pytest.mark.parametrize("access", [r"\ba\.(?!pairs)\w+\[[^=]*\] = (?!b\.)", r"\*(own|all) = ", r"\bp\[i\] = ", r"\*reinterpret_cast<uint2"])
def test_stores_of_sorts_are_checked(access):
    assert unchecked("sort.cu", access) == []


@pytest.mark.parametrize("name,access", [("embedding.cu", r"load_shared_row\("), ("embedding.cu", r"in\[j\]\[u\]\.load\("),
                                         ("embedding.cu", r"load_now\("), ("experts.cu", r"v\[k\]\[u\]\.load\("),
                                         ("experts.cu", r"copy_own<kPiece>\(")])
def test_loads_through_an_index_are_checked(name, access):
    assert unchecked(name, access) == []
