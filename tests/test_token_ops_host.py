"""The operators that move rows by an index, without a GPU: refusals before anything
reaches CUDA, in the C ABI and in the tensor-level calls; what is launched for the
largest sizes; and the references of the GPU tests against autograd in 64 bits."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import memory_bound_normalization_gb300 as pkg
import token_ref as ref
from memory_bound_normalization_gb300 import _lib, autograd
from memory_bound_normalization_gb300 import build as libbuild
from test_image_launches_host import run  # noqa: F401  (a fixture)

A = 1 << 20  # aligned non-null addresses; never dereferenced by these calls
BIG = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _library():
    libbuild.build()
    pkg.load_library()


def emb(**change):
    d = dict(outer=2, inner=3, num_rows=10, width=64, table_stride=64, row_stride=64, ids_64=1, scale=1.0)
    stride = change.pop("id_stride", (3, 1))
    d.update(change)
    e = _lib.Embedding(**d)
    e.id_stride[0], e.id_stride[1] = stride
    return e


def emb_fwd(e, ids=A, table=A, y=A, dtype=pkg.BF16):
    return pkg.rmsnorm_embedding_fwd(e, ids, table, y, dtype, 0)


def emb_bwd(e, ids=A, dy=A, grad=A, padding=-1, acc=0, dtype=pkg.BF16, ws=A, n=1 << 40):
    return pkg.rmsnorm_embedding_bwd_ws(e, ids, dy, grad, padding, acc, dtype, ws, n, 0)


@pytest.mark.parametrize("bad", [dict(outer=-1), dict(inner=-1), dict(outer=1 << 16, inner=1 << 15),
                                 dict(outer=1 << 40), dict(num_rows=0), dict(num_rows=1 << 31), dict(width=0),
                                 dict(width=1 << 31), dict(table_stride=-1), dict(row_stride=-1),
                                 dict(id_stride=(-1, 1)), dict(id_stride=(3, -1)), dict(table_stride=1 << 58),
                                 dict(row_stride=1 << 58), dict(id_stride=(1 << 41, 1)),
                                 dict(outer=1, inner=BIG, width=BIG)])
def test_embedding_descriptor(bad):
    assert emb_fwd(emb(**bad)) == pkg.ERR_INVALID_ARG
    assert emb_bwd(emb(**bad)) == pkg.ERR_INVALID_ARG


def test_embedding_arguments():
    e = emb()
    for call in (emb_fwd, emb_bwd):
        assert call(None) == pkg.ERR_INVALID_ARG
        assert call(e, dtype=5) == pkg.ERR_INVALID_ARG
        assert call(e, ids=None) == pkg.ERR_INVALID_ARG
        assert call(e, ids=A + 4) == pkg.ERR_MISALIGNED
        assert call(emb(ids_64=0), ids=A + 2) == pkg.ERR_MISALIGNED
    assert emb_fwd(e, table=None) == emb_fwd(e, y=None) == pkg.ERR_INVALID_ARG
    assert emb_bwd(e, dy=None) == emb_bwd(e, grad=None) == pkg.ERR_INVALID_ARG
    assert emb_fwd(e, y=A + 1) == emb_fwd(e, table=A + 1) == pkg.ERR_MISALIGNED
    assert emb_fwd(e, table=A + 2, dtype=pkg.BF16_W_F32) == pkg.ERR_MISALIGNED
    assert emb_bwd(e, dy=A + 1) == emb_bwd(e, grad=A + 2, dtype=pkg.F16_W_F32) == pkg.ERR_MISALIGNED
    # outputs whose rows would overlap; inputs may
    assert emb_fwd(emb(row_stride=63)) == pkg.ERR_INVALID_ARG
    assert emb_bwd(emb(table_stride=63)) == pkg.ERR_INVALID_ARG
    # nothing to do
    assert emb_fwd(emb(outer=0), ids=None, table=None, y=None) == pkg.OK
    assert emb_bwd(emb(inner=0), ids=None, dy=None, acc=1) == pkg.OK


def sort(tokens=4, choices=2, experts=8, align=1, rows=8, at=A, position=A, source=A, offsets=A, counts=A, wide=1):
    return pkg.rmsnorm_expert_sort(at, wide, tokens, choices, experts, align, rows, position, source, offsets, counts,
                                   0)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(choices=0), dict(experts=0), dict(experts=pkg.MAX_EXPERTS + 1),
                                 dict(align=0), dict(rows=7), dict(align=4, rows=31), dict(tokens=1 << 30, rows=BIG),
                                 dict(rows=1 << 31), dict(at=None), dict(position=None), dict(source=None),
                                 dict(offsets=None), dict(counts=None), dict(align=1 << 30, rows=BIG)])
def test_expert_sort_refuses(bad):
    assert sort(**bad) == pkg.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(at=A + 4), dict(position=A + 2), dict(source=A + 1), dict(offsets=A + 2),
                                 dict(counts=A + 3), dict(at=A + 2, wide=0)])
def test_expert_sort_misaligned(bad):
    assert sort(**bad) == pkg.ERR_MISALIGNED


@pytest.mark.parametrize("T,K,E,align", [(0, 1, 1, 1), (0, 3, 8, 128), (1, 1, 1, 1), (1, 8, 128, 128), (5, 3, 7, 16),
                                         (16384, 8, 128, 128), (BIG, 1, 1, 1)])
def test_expert_rows(T, K, E, align):
    R = pkg.rmsnorm_expert_rows(T, K, E, align)
    assert R == ref.rows_of(T, K, E, align) and R % align == 0
    # room for the worst case: every expert's rows rounded up
    used = min(E, T * K)
    assert R + align > T * K + used * (align - 1) >= R


@pytest.mark.parametrize("bad", [(-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                                 (1 << 31, 1, 1, 1), (1 << 20, 1 << 12, 8, 1), (1 << 30, 1, 1024, BIG)])
def test_expert_rows_of_invalid_arguments(bad):
    assert pkg.rmsnorm_expert_rows(*bad) == -1


def test_workspace_sizes():
    size = pkg.rmsnorm_embedding_bwd_workspace_size
    assert size(0, 10, 8) == 0 and size(-1, 10, 8) == 0 and size(5, 0, 8) == 0 and size(5, 10, 0) == 0
    assert size(1 << 31, 10, 8) == 0 and size(BIG, 10, BIG) == 0
    assert size(256, 1 << 20, 4096) == 0  # sorted on chip
    assert 0 < size(257, 1, 1) <= size(1000, 10, 8) <= size(100000, 10, 8) <= size(100000, 1 << 20, 8)
    assert pkg.rmsnorm_expert_sort_workspace_size(16, 8, 128) == 0
    assert pkg.rmsnorm_expert_sort_workspace_size(1 << 20, 8, 128) > 0
    assert pkg.rmsnorm_expert_sort_workspace_size(1 << 20, 8, 2000) == 0


def experts(**change):
    d = dict(tokens=4, rows=8, width=64, token_stride=64, row_stride=64, residual_stride=64, drow_stride=64, choices=2)
    d.update(change)
    return _lib.Experts(**d)


def dispatch(d, x=A, position=A, source=A, rows=A, dtype=pkg.BF16):
    return pkg.rmsnorm_expert_dispatch_fwd(d, x, position, source, rows, dtype, 0)


def combine(d, rows=A, position=A, weights=A, residual=A, y=A, dtype=pkg.BF16):
    return pkg.rmsnorm_expert_combine_fwd(d, rows, position, weights, residual, y, dtype, 0)


def combine_bwd(d, dy=A, rows=A, position=A, source=A, weights=A, drows=A, dweights=A, dtype=pkg.BF16):
    return pkg.rmsnorm_expert_combine_bwd(d, dy, rows, position, source, weights, drows, dweights, dtype, 0)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(rows=-1), dict(width=0), dict(choices=0), dict(choices=-3),
                                 dict(tokens=1 << 31), dict(rows=1 << 31), dict(width=1 << 31),
                                 dict(token_stride=-1), dict(row_stride=-1), dict(token_stride=1 << 58),
                                 dict(tokens=1 << 30, choices=4), dict(tokens=BIG, choices=1, width=BIG)])
def test_expert_descriptor(bad):
    d = experts(**bad)
    assert dispatch(d) == combine(d) == combine_bwd(d) == pkg.ERR_INVALID_ARG
    assert pkg.rmsnorm_expert_dispatch_bwd(d, A, A, A, pkg.BF16, 0) == pkg.ERR_INVALID_ARG


def test_expert_arguments():
    d = experts()
    assert dispatch(None) == combine(None) == combine_bwd(None) == combine_bwd(None, weights=None) == \
        pkg.ERR_INVALID_ARG
    for call, names in ((dispatch, ("x", "position", "source", "rows")), (combine, ("rows", "position", "y")),
                        (combine_bwd, ("dy", "rows", "position", "source", "drows", "dweights"))):
        assert call(d, dtype=9) == pkg.ERR_INVALID_ARG
        for name in names:
            assert call(d, **{name: None}) == pkg.ERR_INVALID_ARG, (call, name)
            assert call(d, **{name: A + 1}) == pkg.ERR_MISALIGNED, (call, name)
    assert combine(d, weights=A + 1) == combine(d, residual=A + 1) == combine_bwd(d, weights=A + 1) == \
        pkg.ERR_MISALIGNED
    # outputs whose rows would overlap
    assert dispatch(experts(row_stride=63)) == combine(experts(token_stride=63)) == pkg.ERR_INVALID_ARG
    assert combine_bwd(experts(drow_stride=63)) == combine_bwd(experts(drow_stride=63), weights=None) == \
        pkg.ERR_INVALID_ARG
    assert combine(experts(residual_stride=-1)) == pkg.ERR_INVALID_ARG
    # nothing to do
    assert dispatch(experts(rows=0, tokens=0), x=None, source=None, rows=None, position=None) == pkg.OK
    assert combine(experts(tokens=0), rows=None, y=None, position=None) == pkg.OK


def test_descriptors_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    lines = []
    for name, cls in (("rmsnorm_embedding_t", pkg.Embedding), ("rmsnorm_experts_t", pkg.Experts)):
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "rmsnorm.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn RMSNORM_MAX_EXPERTS != %d;\n}\n" % pkg.MAX_EXPERTS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(libbuild._nvcc())), "include")
    subprocess.run(["gcc", "-I", libbuild.INCLUDE, "-I", cuda, str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, field, value = line.split()
        cls = {"rmsnorm_embedding_t": pkg.Embedding, "rmsnorm_experts_t": pkg.Experts}[name]
        want = ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset
        assert int(value) == want, line


# ------------------------------------------------------------- tensor-level calls
def test_embedding_calls_refuse():
    ids, table = torch.zeros(2, 3, dtype=torch.int64), torch.zeros(5, 8)
    dy = torch.zeros(2, 3, 8)
    bad = [lambda: pkg.embedding_forward(ids.float(), table), lambda: pkg.embedding_forward(ids, table[0]),
           lambda: pkg.embedding_forward(ids, table[:0]), lambda: pkg.embedding_forward(ids, table[:, :0]),
           lambda: pkg.embedding_forward(ids, table.double()),
           lambda: pkg.embedding_forward(ids, table.half(), out_dtype=torch.bfloat16),
           lambda: pkg.embedding_forward(ids, table.half(), out_dtype=torch.float32),
           lambda: pkg.embedding_backward(ids.bool(), dy, 5), lambda: pkg.embedding_backward(ids, dy, 0),
           lambda: pkg.embedding_backward(ids, dy[:1], 5), lambda: pkg.embedding_backward(ids[0], dy, 5),
           lambda: pkg.embedding_backward(ids, dy, 5, padding_idx=5),
           lambda: pkg.embedding_backward(ids, dy, 5, padding_idx=-6),
           lambda: pkg.embedding_backward(ids, dy, 5, grad_dtype=torch.bfloat16),
           lambda: pkg.embedding_backward(ids, dy.double(), 5),
           lambda: pkg.embedding_backward(ids, dy, 5, accumulate=True),
           lambda: pkg.embedding_backward(ids, dy, 5, out=table[:4]),
           lambda: pkg.embedding_backward(ids, dy, 5, out=table[:, :4]),
           lambda: pkg.embedding_backward(ids, dy, 5, out=table, grad_dtype=torch.float16)]
    for call in bad:
        with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
            call()
    with pytest.raises(ValueError, match="expected a tensor"):
        pkg.embedding_forward([1, 2], table)
    with pytest.raises(ValueError, match="torch dtype"):
        pkg.embedding_forward(ids, table, out_dtype="bf16")
    with pytest.raises(ValueError, match="more than two strides"):
        pkg.embedding_forward(torch.zeros(4, 4, 4, dtype=torch.int64)[:2, :2, :2], table)
    with pytest.raises(ValueError, match="not dense"):
        pkg.embedding_backward(ids, torch.zeros(2, 8, 3).transpose(1, 2), 5)
    with pytest.raises(ValueError, match="no one stride"):
        pkg.embedding_backward(ids, torch.zeros(2, 4, 8)[:, :3], 5)
    for call in (lambda: pkg.embedding_forward(ids, table), lambda: pkg.embedding_backward(ids, dy, 5)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


def test_expert_calls_refuse():
    e = torch.zeros(4, 2, dtype=torch.int64)
    x, rows, w = torch.zeros(4, 8), torch.zeros(8, 8), torch.zeros(4, 2)
    p, s = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    bad = [lambda: pkg.expert_sort(e.float(), 8), lambda: pkg.expert_sort(e[0, 0], 8),
           lambda: pkg.expert_sort(e[:, :0], 8), lambda: pkg.expert_sort(e, 0),
           lambda: pkg.expert_sort(e, pkg.MAX_EXPERTS + 1), lambda: pkg.expert_sort(e, 8, align=0),
           lambda: pkg.expert_dispatch_forward(x, p.long(), s), lambda: pkg.expert_dispatch_forward(x[:3], p, s),
           lambda: pkg.expert_dispatch_forward(x, p, s.long()), lambda: pkg.expert_dispatch_forward(x, p, p),
           lambda: pkg.expert_dispatch_forward(x.double(), p, s), lambda: pkg.expert_dispatch_forward(x[:, :0], p, s),
           lambda: pkg.expert_dispatch_backward(x[0], p), lambda: pkg.expert_dispatch_backward(rows.int(), p),
           lambda: pkg.expert_combine_forward(rows, p, w[:3]), lambda: pkg.expert_combine_forward(rows, p, w.half()),
           lambda: pkg.expert_combine_forward(rows, p, w, x[:, :4]),
           lambda: pkg.expert_combine_forward(rows, p, w, x.half()),
           lambda: pkg.expert_combine_forward(rows, p, w, x[:3]),
           lambda: pkg.expert_combine_backward(x[:3], rows, p, s, w),
           lambda: pkg.expert_combine_backward(x, rows, p, s[:7], w),
           lambda: pkg.expert_combine_backward(x.half(), rows, p, s, w),
           lambda: pkg.expert_combine_backward(x, rows, p, s, w.double())]
    for call in bad:
        with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
            call()
    for call in (lambda: pkg.expert_sort(e, 8), lambda: pkg.expert_dispatch_forward(x, p, s),
                 lambda: pkg.expert_dispatch_backward(rows, p), lambda: pkg.expert_combine_forward(rows, p, w, x),
                 lambda: pkg.expert_combine_backward(x, rows, p, s, w)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


def test_one_stride():
    """Which gradients the autograd forms pass on as they are."""
    t = torch.zeros(4, 5, 6)
    for same in (t, t[0], t[0, 0], t[..., :3], t[:, :1], torch.zeros(6).expand(4, 5, 6), t[:0]):
        assert autograd._one_stride(same) is same
    for copied in (t[:, :3], t.transpose(0, 1), t.transpose(1, 2), torch.zeros(()).expand(4, 6),
                   torch.zeros(5, 6).expand(4, 5, 6)):
        assert autograd._one_stride(copied).is_contiguous()


# ------------------------------------------------------------- what is launched
def test_launches_of_the_largest_sizes(run):  # noqa: F811
    """Grids of 2^31 - 1 tokens, choices and rows; clusters and shared memory that the
    kernels are allowed, on two devices."""
    run("""
    BIG = (1 << 31) - 1
    def emb(**k):
        d = dict(outer=1, inner=BIG, num_rows=BIG, width=1, table_stride=1, row_stride=1, ids_64=1, scale=1.0)
        d.update(k)
        e = _lib.Embedding(**d)
        e.id_stride[1] = 1
        return ctypes.byref(e)
    def fine(st):
        assert st == _lib.OK, st
        assert all(l["allowed"] and 0 < l["grid"] < 1 << 31 for l in launches()), launches()
    for device in (0, 1):
        fake.cudaSetDevice(device)
        for dtype in range(5):
            for k in (dict(), dict(width=4096, inner=1 << 20, table_stride=4096, row_stride=4096),
                      dict(inner=5, width=BIG, table_stride=BIG, row_stride=BIG, num_rows=3),
                      dict(inner=40000, num_rows=50000), dict(inner=3000), dict(inner=16385, num_rows=511)):
                fine(lib.rmsnorm_embedding_fwd(emb(**k), A, A, A, dtype, None))
                for acc in (0, 1):
                    fine(lib.rmsnorm_embedding_bwd_ws(emb(**k), A, A, A, 0, acc, dtype, A, 1 << 50, None))
        for T, K, E in ((BIG, 1, 1), (1 << 28, 7, 1024), (1, 8, 1024), (2049, 8, 1024), (1, 1, 1)):
            fine(lib.rmsnorm_expert_sort(A, 0, T, K, E, 1, BIG, A, A, A, A, None))
        for T, K, R, H in ((BIG, 1, BIG, 1), (1 << 20, 8, BIG, 4096), (5, 100, 500, BIG), (1000, 8, 8000, 2048),
                           (0, 1, BIG, 64), (1 << 20, 6, 6 << 20, 2880)):
            d = ctypes.byref(_lib.Experts(tokens=T, rows=R, width=H, token_stride=H, row_stride=H,
                                          residual_stride=H, drow_stride=H, choices=K))
            for dtype in range(5):
                fine(lib.rmsnorm_expert_dispatch_fwd(d, A, A, A, A, dtype, None))
                fine(lib.rmsnorm_expert_dispatch_bwd(d, A, A, A, dtype, None))
                fine(lib.rmsnorm_expert_combine_fwd(d, A, A, A, A, A, dtype, None))
                fine(lib.rmsnorm_expert_combine_bwd(d, A, A, A, A, A, A, A, dtype, None))
        assert launches()[-1]["device"] == device
    """)


# ------------------------------------------------------------- the references
def test_references_against_autograd():
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(-1, 7, (4, 5), generator=g)
    table = torch.randn(6, 3, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(4, 5, 3, generator=g, dtype=torch.float64)
    (ref.embedding(ids, table, 1.5) * dy).sum().backward()
    grad, count, magnitude = ref.embedding_grad(ids, dy, 6, 1.5)
    assert torch.allclose(grad, table.grad, rtol=1e-14, atol=1e-14)
    assert torch.equal(count[:, 0], torch.stack([(ids == v).sum() for v in range(6)]).double())
    assert bool((magnitude >= grad.abs() * (1 - 1e-15)).all())
    grad = ref.embedding_grad(ids, dy, 6, 1.5, padding=2)[0]
    assert not grad[2].any() and torch.equal(grad[3], ref.embedding_grad(ids, dy, 6, 1.5)[0][3])

    experts = torch.randint(-1, 4, (6, 3), generator=g)
    R = ref.rows_of(6, 3, 4, 2)
    position, source, offsets, counts = ref.sort(experts, 4, 2, R)
    assert int(offsets[-1]) <= R and not (offsets % 2).any() and int(counts.sum()) == int((experts >= 0).sum())
    for e in range(4):
        mine = source[int(offsets[e]):int(offsets[e]) + int(counts[e])].long()
        assert mine.tolist() == [i for i, v in enumerate(experts.flatten().tolist()) if v == e]
        assert position.flatten()[mine].tolist() == list(range(int(offsets[e]), int(offsets[e]) + int(counts[e])))
    rows = torch.randn(R, 5, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.rand(6, 3, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(6, 5, generator=g, dtype=torch.float64)
    y = torch.zeros(6, 5, dtype=torch.float64)
    for t in range(6):  # by hand
        for k in range(3):
            if position[t, k] >= 0:
                y[t] = y[t] + w[t, k] * rows[int(position[t, k])]
    assert torch.allclose(y, ref.combine(rows, position, w)[0], rtol=1e-14, atol=1e-14)
    (y * dy).sum().backward()
    drows, dw, _ = ref.combine_grads(dy, rows.detach(), position, w.detach())
    assert torch.allclose(drows, rows.grad, rtol=1e-14) and torch.allclose(dw, w.grad, rtol=1e-13, atol=1e-14)


def test_a_wrong_value_is_seen():
    """The bounds refuse a value that is one step off, and a lost term."""
    r = torch.tensor([1.0, 100.0], dtype=torch.float64)
    for t in (torch.float32, torch.bfloat16, torch.float16):
        ref.close(r.to(t), r)
        off = r.to(t)
        off[1] += 100 * torch.finfo(t).eps
        with pytest.raises(AssertionError):
            ref.close(off, r)
        with pytest.raises(AssertionError):
            ref.close(r.to(t), r + torch.tensor([0.0, 1.0]), 10, r.abs())
