"""The operators together, as a language model runs them: tokens looked up with a
scale, normed, sent to their experts, the experts' rows combined onto the residual,
and the library's fused residual norm behind; outputs and gradients against the same
model in 64 bits. The modules, and a captured training step."""
from __future__ import annotations

import pytest
import torch

import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda"
B, T, V, H, F, E, K = 3, 14, 50, 64, 32, 6, 2
SCALE = 8.0


def parameters(dtype):
    g = torch.Generator().manual_seed(11)
    p = {"table": torch.randn(V, H, generator=g) / 8, "n1": 1 + 0.1 * torch.randn(H, generator=g),
         "router": torch.randn(H, E, generator=g) / 8, "up": torch.randn(E, H, F, generator=g) / 8,
         "down": torch.randn(E, F, H, generator=g) / 6, "n2": 1 + 0.1 * torch.randn(H, generator=g),
         "head": torch.randn(H, V, generator=g) / 8}
    return {n: t.to(DEV, dtype).requires_grad_(True) for n, t in p.items()}


def tokens():
    ids = torch.randint(0, V, (B, T + 1), generator=torch.Generator().manual_seed(12))
    ids[1, 9:] = 0  # padding
    return ids.to(DEV)


def route(x, router):
    """Experts, the weights of the choices; padding goes nowhere."""
    score, experts = (x @ router).topk(K, -1)
    return experts, torch.softmax(score, -1)


def experts_of(rows, offsets, p):
    """Each expert's rows through its two matrices."""
    parts = []
    edge = offsets.tolist()
    for e in range(E):
        h = torch.relu(rows[edge[e]:edge[e + 1]] @ p["up"][e]) @ p["down"][e]
        parts.append(h)
    return torch.cat(parts + [rows[edge[E]:] * 0])


def model(ids, p):
    from memory_bound_normalization_gb300.autograd import (embedding, expert_combine, expert_dispatch,
                                                           fused_add_rms_norm, rms_norm)

    h = embedding(ids, p["table"], SCALE, padding_idx=0)
    x = rms_norm(h, p["n1"])
    experts, w = route(x, p["router"])
    plan = pkg.expert_sort(torch.where(ids[..., None] == 0, -1, experts), E, align=4)
    rows = experts_of(expert_dispatch(x, plan), plan.offsets, p)
    mixed = expert_combine(rows, plan, w, h)
    y, _ = fused_add_rms_norm(mixed, x, p["n2"])
    return y @ p["head"], experts


def plain(ids, p, experts):
    """The same in the parameters' type, by elementary operations, choices given."""
    def norm(t, w):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w

    h = p["table"][ids] * SCALE
    h = torch.where(ids[..., None] == 0, h.detach(), h)  # no gradient of the padding row
    x = norm(h, p["n1"])
    w = torch.softmax((x @ p["router"]).gather(-1, experts), -1)
    mixed = h
    for k in range(K):
        e = experts[..., k]
        out = torch.einsum("btf,btfh->bth", torch.relu(torch.einsum("bth,bthf->btf", x, p["up"][e])), p["down"][e])
        mixed = mixed + torch.where(ids[..., None] == 0, 0.0, w[..., k:k + 1] * out)
    return norm(mixed + x, p["n2"]) @ p["head"]


def loss_of(logits, target):
    return torch.nn.functional.cross_entropy(logits.flatten(0, 1), target.flatten())


def test_model_with_gradients():
    """fp32: 2^-24 a rounding, and some 2^10 of them one on another (sums of 64 columns,
    two norms, two products of experts, the head): 2^-12 of the largest value."""
    batch = tokens()
    ids, target = batch[:, :-1], batch[:, 1:]
    p = parameters(torch.float32)
    logits, experts = model(ids, p)
    loss = loss_of(logits, target)
    loss.backward()
    q = {n: t.detach().double().requires_grad_(True) for n, t in p.items()}
    want = plain(ids, q, experts)
    wloss = loss_of(want, target)
    wloss.backward()
    logits, want = logits.detach().double(), want.detach()
    assert float((logits - want).abs().max()) <= 2.0 ** -12 * float(want.abs().max())
    loss, wloss = float(loss.detach()), float(wloss.detach())
    assert abs(loss - wloss) <= 2.0 ** -12 * abs(wloss)
    for n in p:
        a, b = p[n].grad.double(), q[n].grad
        assert float((a - b).abs().max()) <= 2.0 ** -12 * float(b.abs().max()), n
    assert not p["table"].grad[0].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_model_runs_in_16_bits(dtype):
    batch = tokens()
    p = parameters(dtype)
    logits, _ = model(batch[:, :-1], p)
    loss_of(logits.float(), batch[:, 1:]).backward()
    for n, t in p.items():
        assert t.grad.dtype == dtype and bool(t.grad.isfinite().all()) and bool(t.grad.any()), n


def test_gradients_by_differences():
    """Along a random direction of each parameter: the fp32 loss of 39 tokens is good to
    some 2^-20, a step of 2^-6 makes that 2^-15 of a slope."""
    batch = tokens()
    ids, target = batch[:, :-1], batch[:, 1:]
    p = parameters(torch.float32)
    loss_of(model(ids, p)[0], target).backward()
    g = torch.Generator().manual_seed(3)
    q = {n: t.detach().double() for n, t in p.items()}
    experts = model(ids, p)[1]
    for n, t in p.items():
        v = torch.randn(t.shape, generator=g).to(DEV)
        if n == "table":
            v[0] = 0  # the padding row has no gradient by design
        v = v.double() / v.norm()
        slope = float((t.grad.double() * v).sum())
        h = 2.0 ** -10
        up = float(loss_of(plain(ids, {**q, n: q[n] + h * v}, experts), target))
        down = float(loss_of(plain(ids, {**q, n: q[n] - h * v}, experts), target))
        # the loss's third derivative along v, some units, times h^2 / 6
        assert abs(slope - (up - down) / (2 * h)) <= 1e-4 * float(t.grad.norm()) + 1e-6, n


def test_frozen_inputs():
    """Gradients of what asks for one alone; a residual that is the rows' input."""
    from memory_bound_normalization_gb300.autograd import expert_combine, expert_dispatch

    g = torch.Generator().manual_seed(1)
    plan = pkg.expert_sort(torch.randint(-1, 5, (20, 3), generator=g).to(DEV), 5)
    x = torch.randn(20, 16, generator=g).to(DEV)
    w = torch.rand(20, 3, generator=g).to(DEV)
    rows = expert_dispatch(x, plan)
    for grads in ((True, False, False), (False, True, False), (False, False, True), (True, True, True)):
        r, v, h = (t.detach().clone().requires_grad_(on) for t, on in zip((rows, w, x), grads))
        y = expert_combine(r, plan, v, h)
        y.sum().backward()  # a broadcast gradient
        ones = torch.ones_like(y)
        drows, dw, magnitude = ref.combine_grads(ones, r.detach(), plan.position, v.detach())
        for t, on, want in ((r, grads[0], drows), (v, grads[1], dw), (h, grads[2], ones.double())):
            assert (t.grad is not None) == on
            if on:
                assert torch.allclose(t.grad.double(), want, rtol=0, atol=2.0 ** -18)
    # no weights
    r = rows.detach().clone().requires_grad_(True)
    expert_combine(r, plan).sum().backward()
    assert torch.equal(r.grad, (plan.source >= 0).float()[:, None].expand_as(r))
    # shared: dispatched and added to
    s = x.clone().requires_grad_(True)
    expert_combine(expert_dispatch(s, plan), plan, w, s).sum().backward()
    kept = torch.where(plan.position >= 0, w, 0).sum(-1, keepdim=True)
    assert torch.allclose(s.grad, 1 + kept.expand_as(s), rtol=0, atol=2.0 ** -20)


def test_embedding_module():
    from memory_bound_normalization_gb300.autograd import Embedding

    ids = tokens()
    m = Embedding(V, H, scale=3.0, padding_idx=-1, device=DEV, out_dtype=torch.bfloat16)
    assert not m.weight[V - 1].any()
    y = m(ids)
    assert y.dtype == torch.bfloat16 and y.shape == (*ids.shape, H)
    ref.close(y, ref.embedding(ids, m.weight.detach(), 3.0))
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(2)).to(DEV, torch.bfloat16)
    y.backward(dy)
    assert m.weight.grad.dtype == torch.float32
    ref.close(m.weight.grad, *ref.embedding_grad(ids, dy, V, 3.0, V - 1))
    other = Embedding(V, H, device="meta")
    other = other.to_empty(device=DEV)
    other.load_state_dict(m.state_dict())
    assert torch.equal(other(ids), torch.nn.functional.embedding(ids, m.weight))
    # a frozen table has no gradient to compute
    m.weight.requires_grad_(False)
    assert not m(ids).requires_grad
    # every expand of a scalar's gradient, and a transposed one
    m.weight.requires_grad_(True)
    m.weight.grad = None
    m(ids).float().sum().backward()
    ones = torch.ones(*ids.shape, H, device=DEV)
    ref.close(m.weight.grad, *ref.embedding_grad(ids, ones, V, 3.0, V - 1))
    m.weight.grad = None
    mixed = torch.randn(H, *ids.shape, generator=torch.Generator().manual_seed(4)).to(DEV, torch.bfloat16)
    m(ids).backward(mixed.permute(1, 2, 0))
    ref.close(m.weight.grad, *ref.embedding_grad(ids, mixed.permute(1, 2, 0), V, 3.0, V - 1))


def test_captured_training_step():
    """Lookup, dispatch, combine and their backward passes captured once and replayed
    on other tokens; no eager graph of the same leaves is alive."""
    from memory_bound_normalization_gb300.autograd import embedding, expert_combine, expert_dispatch

    g = torch.Generator().manual_seed(6)
    table = (torch.randn(V, H, generator=g) / 8).to(DEV).requires_grad_(True)
    ids = torch.randint(0, V, (40,), generator=g).to(DEV)
    experts = torch.randint(0, E, (40, K), generator=g).to(DEV)
    w = torch.rand(40, K, generator=g).to(DEV)

    def step():
        table.grad = None
        h = embedding(ids, table, 2.0)
        plan = pkg.expert_sort(experts, E)
        y = expert_combine(expert_dispatch(h, plan) * 3, plan, w, h)
        (y * y).sum().backward()
        return y.detach()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in (1, 2):
        ids.copy_(torch.randint(0, V, (40,), generator=torch.Generator().manual_seed(seed)))
        experts.copy_(torch.randint(-1, E, (40, K), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        # y = h (1 + 3 sum of the weights kept), the loss's gradient 2 y (that)
        gain = 1 + 3 * torch.where(experts >= 0, w, 0).double().sum(-1, keepdim=True)
        want = table.detach().double()[ids] * 2 * gain
        assert torch.allclose(y.double(), want, rtol=2.0 ** -20, atol=2.0 ** -22)
        grad = torch.zeros(V, H, dtype=torch.float64, device=DEV).index_add_(0, ids, 2 * want * gain * 2)
        assert torch.allclose(table.grad.double(), grad, rtol=2.0 ** -18, atol=2.0 ** -18)


@pytest.fixture(scope="module", autouse=True)
def _status():
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
