"""Tokens sorted by expert, dispatched and combined, with the gradients, against a
walk over the choices and 64 bits."""
from __future__ import annotations

import pytest
import torch

import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda"
# tokens, choices, experts, alignment
SORTS = [(1, 1, 1, 1), (1, 8, 128, 1), (16, 8, 128, 1), (5, 3, 7, 16), (100, 2, 8, 128),
         (1000, 6, 60, 1), (1025, 4, 1024, 3), (4099, 1, 16, 8), (4099, 9, 33, 128), (65536, 2, 300, 1),
         (43691, 3, 1000, 7), (200000, 1, 2, 128), (30000, 8, 1024, 4)]
# tokens, choices, experts, width, alignment: pieces of 16, 8, 4 and 2 bytes, groups
# of lanes, warps and several warps
ROWS = [(1, 1, 1, 1, 1), (1, 8, 128, 4096, 1), (17, 4, 9, 8, 4), (33, 3, 5, 33, 1), (100, 8, 60, 72, 16),
        (64, 2, 8, 1000, 1), (9, 13, 20, 1412, 8), (40, 6, 8, 2048, 1), (5, 5, 5, 9000, 128),
        (3, 9, 12, 20001, 1), (3000, 2, 16, 130, 1)]


def case_id(s):
    return "x".join(map(str, s))


def choices(T, K, E, seed=0, drop=0.1):
    gen = torch.Generator().manual_seed(seed)
    score = torch.rand(T, max(K, E), generator=gen) + torch.rand(max(K, E), generator=gen)
    e = score.topk(K).indices
    e = torch.where(e < E, e, -1)
    if drop and T > 2:
        e[torch.rand(T, generator=gen) < drop] = -1
        e[torch.randint(0, T, (1,), generator=gen), 0] = E
        e[torch.randint(0, T, (1,), generator=gen), -1] = -(1 << 31)
    return e.to(DEV)


def normal(*shape, dtype, seed=1):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def same_plan(plan, want):
    for got, w, name in zip(plan, want, ("position", "source", "offsets", "counts")):
        assert got.dtype == torch.int32 and torch.equal(got, w), name


@pytest.mark.parametrize("itype", [torch.int32, torch.int64], ids=["i32", "i64"])
@pytest.mark.parametrize("case", SORTS, ids=case_id)
def test_sort(case, itype):
    T, K, E, align = case
    e = choices(T, K, E).to(itype)
    plan = pkg.expert_sort(e, E, align=align)
    same_plan(plan, ref.sort(e, E, align, ref.rows_of(T, K, E, align)))


@pytest.mark.parametrize("which", ["same", "last", "none", "turn", "far"])
@pytest.mark.parametrize("n", [1, 32, 1024, 1025, 4096, 4097, 8192, 9000, 131072, 131073])
def test_sort_of_few_experts_used(which, n):
    E = 256
    i = torch.arange(n, device=DEV)
    e = {"same": i * 0 + 3, "last": i * 0 + E - 1, "none": i * 0 - 1, "turn": i % E,
         "far": i + (1 << 40)}[which][:, None]
    same_plan(pkg.expert_sort(e, E, align=32), ref.sort(e, E, 32, ref.rows_of(n, 1, E, 32)))


def test_sort_shapes():
    e = choices(12, 4, 6).view(3, 4, 4)
    plan = pkg.expert_sort(e, 6)
    assert plan.position.shape == (3, 4, 4)
    same_plan(plan, ref.sort(e, 6, 1, 48))
    empty = pkg.expert_sort(e[:0], 6, align=16)
    assert empty.source.numel() == 0 and empty.position.shape == (0, 4, 4)
    assert not empty.offsets.any() and not empty.counts.any()
    # the same expert twice
    e = torch.tensor([[2, 2, 0], [2, 0, 2]], device=DEV)
    same_plan(pkg.expert_sort(e, 3), ref.sort(e, 3, 1, 6))


def setup(case, dtype, seed=0):
    T, K, E, H, align = case
    plan = pkg.expert_sort(choices(T, K, E, seed), E, align=align)
    return plan, plan.source.numel()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("case", ROWS, ids=case_id)
def test_dispatch(case, dtype):
    T, K, E, H, align = case
    plan, R = setup(case, dtype)
    x = normal(T, H, dtype=dtype)
    rows = pkg.expert_dispatch_forward(x, plan.position, plan.source)
    src = plan.source.long()
    want = torch.where(src[:, None] >= 0, x[src.clamp(min=0) // K], 0)
    assert torch.equal(rows, want)
    drows = normal(R, H, dtype=dtype, seed=2)
    dx = pkg.expert_dispatch_backward(drows, plan.position)
    y, magnitude = ref.combine(drows, plan.position)
    ref.close(dx, y, K, magnitude)


@pytest.mark.parametrize("pair", ref.PAIRS, ids=ref.pair_id)
@pytest.mark.parametrize("case", ROWS, ids=case_id)
def test_combine(case, pair):
    T, K, E, H, align = case
    plan, R = setup(case, pair[0])
    rows, residual = normal(R, H, dtype=pair[0]), normal(T, H, dtype=pair[0], seed=2)
    w = torch.softmax(normal(T, K, dtype=torch.float32, seed=3), -1).to(pair[1])
    for weights in (w, None):
        for res in (residual, None):
            y = pkg.expert_combine_forward(rows, plan.position, weights, res)
            want, magnitude = ref.combine(rows, plan.position, weights, res)
            ref.close(y, want, K + 1, magnitude)
            dropped = (plan.position < 0).all(-1)
            if res is None:
                assert not y[dropped].any()
            else:
                assert torch.equal(y[dropped], res[dropped])


@pytest.mark.parametrize("pair", ref.PAIRS, ids=ref.pair_id)
@pytest.mark.parametrize("case", ROWS, ids=case_id)
def test_combine_backward(case, pair):
    T, K, E, H, align = case
    plan, R = setup(case, pair[0])
    rows, dy = normal(R, H, dtype=pair[0]), normal(T, H, dtype=pair[0], seed=2)
    w = torch.softmax(normal(T, K, dtype=torch.float32, seed=3), -1).to(pair[1])
    drows, dw = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    want, dots, magnitude = ref.combine_grads(dy, rows, plan.position, w)
    ref.close(drows, want)
    assert dw.dtype == torch.float32
    ref.close(dw, dots, H, magnitude)
    again = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    assert torch.equal(again[0], drows) and torch.equal(again[1], dw)
    alone, none = pkg.expert_combine_backward(dy, rows, plan.position, plan.source)
    assert none is None
    assert torch.equal(alone.double(), ref.combine_grads(dy, rows, plan.position, None)[0])


def test_values_that_are_not_read():
    """Rows without a choice, and weights of dropped choices, may be NaN."""
    T, K, E, H = 50, 4, 8, 96
    plan, R = setup((T, K, E, H, 16), torch.bfloat16)
    rows, dy = normal(R, H, dtype=torch.bfloat16), normal(T, H, dtype=torch.bfloat16, seed=2)
    w = torch.rand(T, K, device=DEV)
    clean = pkg.expert_combine_forward(rows, plan.position, w)
    drows, dw = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    rows[plan.source < 0] = float("nan")
    w[plan.position < 0] = float("nan")
    dy2 = dy.clone()
    dy2[(plan.position < 0).all(-1)] = float("nan")
    assert torch.equal(pkg.expert_combine_forward(rows, plan.position, w), clean)
    drows2, dw2 = pkg.expert_combine_backward(dy2, rows, plan.position, plan.source, w)
    assert torch.equal(drows2, drows) and torch.equal(dw2, dw)


def test_strides():
    """Tokens and rows as slices of columns."""
    T, K, E, H = 60, 3, 8, 40
    plan, R = setup((T, K, E, H, 8), torch.bfloat16)
    p4 = plan.position.view(5, 12, K)
    wide = normal(5, 12, 3 * H, dtype=torch.bfloat16)
    x = wide[..., H:2 * H]
    rows = pkg.expert_dispatch_forward(x, p4, plan.source)
    assert torch.equal(rows, pkg.expert_dispatch_forward(x.contiguous(), p4, plan.source))
    big = normal(R, H + 8, dtype=torch.bfloat16)
    r = big[:, 8:]
    w = torch.rand(5, 12, K, device=DEV)
    y = pkg.expert_combine_forward(r, p4, w, x)
    assert y.shape == (5, 12, H)
    assert torch.equal(y, pkg.expert_combine_forward(r.contiguous(), p4, w, x.contiguous()))
    assert torch.equal(pkg.expert_dispatch_backward(r, p4),
                       pkg.expert_dispatch_backward(r.contiguous(), p4))
    a = pkg.expert_combine_backward(x, r, p4, plan.source, w)
    b = pkg.expert_combine_backward(x.contiguous(), r.contiguous(), p4, plan.source, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # rows off 16 bytes: by smaller pieces
    odd = normal(R, H + 1, dtype=torch.bfloat16)[:, 1:]
    ref.close(pkg.expert_combine_forward(odd, p4, w), *ref_with(odd, p4, w, K))


def ref_with(rows, position, w, K):
    y, magnitude = ref.combine(rows, position, w)
    return y, K, magnitude


def test_nothing():
    e = torch.full((7, 2), -1, device=DEV)
    plan = pkg.expert_sort(e, 4)
    R = plan.source.numel()
    x = normal(7, 16, dtype=torch.float32)
    assert R == 14 and not pkg.expert_dispatch_forward(x, plan.position, plan.source).any()
    rows = normal(R, 16, dtype=torch.float32)
    w = torch.ones(7, 2, device=DEV)
    assert torch.equal(pkg.expert_combine_forward(rows, plan.position, w, x), x)
    drows, dw = pkg.expert_combine_backward(x, rows, plan.position, plan.source, w)
    assert not drows.any() and not dw.any()
    empty = pkg.expert_sort(e[:0], 4)
    none = pkg.expert_dispatch_forward(x[:0], empty.position, empty.source)
    assert none.shape == (0, 16)
    assert pkg.expert_combine_forward(none, empty.position, w[:0], x[:0]).shape == (0, 16)
    drows, dw = pkg.expert_combine_backward(x[:0], none, empty.position, empty.source, w[:0])
    assert drows.shape == (0, 16) and dw.shape == (0, 2)
    assert pkg.expert_dispatch_backward(none, empty.position).shape == (0, 16)


def test_offsets_past_32_bits():
    """Rows of more than 2^32 bytes: the last."""
    T, K, H = 66000, 2, 16400
    e = torch.zeros(T, K, dtype=torch.int32, device=DEV)
    e[:, 1] = 1
    plan = pkg.expert_sort(e, 2)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[-1] = normal(H, dtype=torch.bfloat16)
    rows = pkg.expert_dispatch_forward(x, plan.position, plan.source)
    assert torch.equal(rows[-1], x[-1]) and torch.equal(rows[T - 1], x[-1])
    w = torch.tensor([0.25, 0.5], device=DEV).expand(T, K).contiguous()
    y = pkg.expert_combine_forward(rows, plan.position, w)
    ref.close(y[-1], x[-1].double() * 0.75, 2, x[-1].double().abs())
    drows, dw = pkg.expert_combine_backward(x, rows, plan.position, plan.source, w)
    assert torch.equal(drows[-1], (x[-1] * 0.5)) and torch.equal(drows[T - 1], x[-1] * 0.25)
    dots = (x[-1].double() ** 2).sum()
    ref.close(dw[-1], dots.expand(2), H, dots)
    assert not dw[:-1].any()


@pytest.fixture(scope="module", autouse=True)
def _status():
    """No kernel of this module recorded a failure (of the checked build, a store
    outside its tensor)."""
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
