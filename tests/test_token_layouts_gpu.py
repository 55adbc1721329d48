"""The autograd forms of the rows by index on layouts that the tensor-level calls refuse:
the results and gradients of the same values held densely."""
from __future__ import annotations

import pytest
import torch

import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda"


def normal(*shape, seed, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def held(t, how):
    """The same values in another layout."""
    if how == "dense":
        return t.contiguous()
    if how == "transposed":  # the last dimension is not dense
        return t.transpose(-1, -2).contiguous().transpose(-1, -2)
    if how == "swapped":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    whole = torch.zeros(*(n + 2 for n in t.shape), dtype=t.dtype, device=t.device)
    part = whole[tuple(slice(1, n + 1) for n in t.shape)]
    part.copy_(t)
    return part


@pytest.mark.parametrize("how", ["transposed", "swapped", "inside"])
def test_layouts(how):
    from memory_bound_normalization_gb300.autograd import embedding, expert_combine, expert_dispatch

    g = torch.Generator().manual_seed(3)
    ids = torch.randint(-1, 40, (3, 5, 7), generator=g).to(DEV)
    plan = pkg.expert_sort(torch.randint(-1, 6, (3, 5, 7, 2), generator=g).to(DEV), 6, align=4)
    table, dy = normal(39, 24, seed=1), normal(3, 5, 7, 24, seed=2)
    w, up = torch.rand(3, 5, 7, 2, generator=g).to(DEV), normal(plan.source.numel(), 24, seed=4)

    def step(how):
        leaf = {n: held(t, how).detach().requires_grad_(True) for n, t in (("table", table), ("x", dy), ("w", w), ("up", up))}
        h = embedding(held(ids, how), leaf["table"], 2.0)
        rows = expert_dispatch(leaf["x"], plan)
        y = expert_combine(leaf["up"], plan, leaf["w"], leaf["x"])
        outs = [h, rows, y]
        torch.autograd.backward(outs, [held(dy, how), held(up, how) if how != "inside" else up, held(dy, how)])
        return outs + [t.grad for t in leaf.values()]

    names = ("h", "rows", "y", "dtable", "dx", "dw", "dup")
    for name, got, want in zip(names, step(how), step("dense")):
        assert got.shape == want.shape
        if name != "dw":
            assert torch.equal(got, want), name
            continue
        # a dot's order goes by the rows' alignment: each side is off from the exact sum of 24
        # products by 25 roundings of the sum of magnitudes at most
        _, dots, magnitude = ref.combine_grads(dy, up, plan.position, w)
        ref.close(got, dots, 24, magnitude)
        ref.close(want, dots, 24, magnitude)


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
