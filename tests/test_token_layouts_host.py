"""The autograd forms of the rows by index without a GPU: which layouts they copy, and
what they refuse before anything is computed."""
from __future__ import annotations

import pytest
import torch

import memory_bound_normalization_gb300 as pkg
from memory_bound_normalization_gb300 import autograd, token_ops
from memory_bound_normalization_gb300 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def _library():
    libbuild.build()
    pkg.load_library()


def layouts(dtype):
    t = torch.zeros(4, 5, 6, 8, dtype=dtype)
    return [t, t[0], t[0, 0], t[0, 0, 0], t[..., :3], t[:, :3], t[:, :, :4], t[:, :3, :4], t[:, :3, :4, :5], t[::2],
            t[:, ::2], t[:, ::2, ::3], t[..., ::2], t[:, :1, :1], t[:, :1, ::2, ::2], t.transpose(0, 1), t.transpose(0, 2),
            t.transpose(1, 3), t.permute(3, 2, 1, 0), t[:0], t[:, :0], t[:, :, :0, :3],
            torch.zeros(8, dtype=dtype).expand(4, 5, 6, 8), torch.zeros(5, 1, 8, dtype=dtype).expand(4, 5, 6, 8),
            torch.zeros(6, 1, dtype=dtype).expand(4, 5, 6, 8), torch.zeros(1, 1, 1, 1, dtype=dtype),
            torch.zeros((), dtype=dtype).expand(4, 6)]


def refusal(call):
    """Whether a call refuses a layout; one on CPU tensors that it would take ends at that."""
    with pytest.raises(ValueError) as e:
        call()
    text = str(e.value)
    assert ("stride" in text or "dense" in text) != ("CUDA tensors" in text), text
    return "CUDA tensors" not in text


def test_ids_are_copied_where_a_lookup_refuses_them():
    table = torch.zeros(9, 4)
    copied = 0
    for ids in [*layouts(torch.int64), torch.zeros((), dtype=torch.int64)]:
        passed = autograd._two_strides(ids)
        assert (passed is not ids) == refusal(lambda: pkg.embedding_forward(ids, table)), (ids.shape, ids.stride())
        assert not refusal(lambda: pkg.embedding_forward(passed, table))
        copied += passed is not ids
    assert copied > 3


def test_rows_are_copied_where_a_call_refuses_them():
    copied = 0
    for x in layouts(torch.float32):
        if x.shape[-1] == 0:
            continue
        ids = torch.zeros(x.shape[:-1], dtype=torch.int32)
        passed = autograd._one_stride(x)
        call = lambda t: pkg.embedding_backward(ids, t, 7)  # noqa: E731
        assert (passed is not x) == refusal(lambda: call(x)), (x.shape, x.stride())
        assert not refusal(lambda: call(passed))
        copied += passed is not x
    assert copied > 5


class Taken(Exception):
    pass


def taken(monkeypatch, name):
    """A tensor-level call that keeps what it is given and goes no further."""
    seen = []

    def call(*a, **k):
        seen.append(a)
        raise Taken

    monkeypatch.setattr(token_ops, name, call)
    return seen


def test_forms_copy_what_the_calls_refuse(monkeypatch):
    seen = taken(monkeypatch, "embedding_forward")
    ids, table = torch.zeros(4, 4, 4, dtype=torch.int64)[:2, :2, :2], torch.zeros(6, 9).t()
    with pytest.raises(Taken):
        autograd.embedding(ids, table)
    assert seen[0][0].is_contiguous() and seen[0][1].is_contiguous()
    plan = token_ops.ExpertRows(torch.zeros(2, 3, 2, dtype=torch.int32), torch.zeros(12, dtype=torch.int32), None, None)
    x = torch.zeros(3, 2, 8).transpose(0, 1)
    seen = taken(monkeypatch, "expert_dispatch_forward")
    with pytest.raises(Taken):
        autograd.expert_dispatch(x, plan)
    assert seen[0][0].is_contiguous()
    seen = taken(monkeypatch, "expert_combine_forward")
    with pytest.raises(Taken):
        autograd.expert_combine(torch.zeros(8, 12).t(), plan, torch.zeros(2, 2, 3).transpose(1, 2), x)
    rows, position, weights, residual = seen[0]
    assert rows.is_contiguous() and weights.is_contiguous() and residual.is_contiguous()
    # and nothing that they take
    wide = torch.zeros(2, 3, 16)[..., 8:]
    with pytest.raises(Taken):
        autograd.expert_combine(torch.zeros(12, 16)[:, :8], plan, None, wide)
    assert seen[1][0].stride() == (16, 1) and seen[1][3].data_ptr() == wide.data_ptr()


def test_padding_outside_the_table_is_refused_by_the_forward(monkeypatch):
    """Before anything is looked up, as the gradient would refuse it."""
    seen = taken(monkeypatch, "embedding_forward")
    ids, table = torch.zeros(3, dtype=torch.int64), torch.zeros(6, 9)
    for padding in (6, -7, 1 << 40):
        with pytest.raises(pkg.RMSNormError, match="padding_idx .*INVALID_ARG") as e:
            autograd.embedding(ids, table, padding_idx=padding)
        assert e.value.status == pkg.ERR_INVALID_ARG
    assert not seen
    for padding in (5, 0, -1, -6, None):
        with pytest.raises(Taken):
            autograd.embedding(ids, table, padding_idx=padding)
    # the module finds it when it is made
    with pytest.raises(IndexError):
        autograd.Embedding(6, 9, padding_idx=6)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("asked", ["rows", "weights", "residual", "rows and residual"])
def test_combine_gradients_that_nobody_asks_for(monkeypatch, asked, weighted):
    """The residual's gradient is the result's own: nothing is computed for it, and the
    rows are not kept."""
    if asked == "weights" and not weighted:
        pytest.skip("no weights")
    called = []
    monkeypatch.setattr(token_ops, "expert_combine_forward", lambda rows, position, w, residual: residual.clone())
    monkeypatch.setattr(token_ops, "expert_combine_backward",
                        lambda dy, rows, position, source, w: called.append("combine") or (rows * 0 + 1, w * 0 + 1))
    monkeypatch.setattr(token_ops, "expert_dispatch_forward",
                        lambda dy, position, source: called.append("dispatch") or torch.ones(8, 16))
    plan = token_ops.ExpertRows(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), None, None)
    t = {"rows": torch.zeros(8, 16), "weights": torch.zeros(4, 2) if weighted else None, "residual": torch.zeros(4, 16)}
    for name, value in t.items():
        if value is not None:
            value.requires_grad_(name in asked)
    y = autograd.expert_combine(t["rows"], plan, t["weights"], t["residual"])
    kept = [s for s in y.grad_fn.saved_tensors if s is not None and s.shape == (8, 16)]
    needed = asked != "residual"
    assert bool(kept) == (needed and weighted)
    dy = torch.randn(4, 16, generator=torch.Generator().manual_seed(1))
    y.backward(dy)
    assert called == ([] if not needed else ["combine" if weighted else "dispatch"])
    assert (t["rows"].grad is not None) == ("rows" in asked)
    if "residual" in asked:
        assert torch.equal(t["residual"].grad, dy)
