"""The operators that move rows by an index: workspaces, streams, captured graphs,
guard bands around every output, several calls at once, and the suites under the
checked build."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import test_embedding_gpu as emb
import test_experts_gpu as exp
import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")
from memory_bound_normalization_gb300 import _lib  # noqa: E402

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def descriptor(n, V, H, scale=1.0, table_stride=None, row_stride=None):
    e = _lib.Embedding(outer=1, inner=n, num_rows=V, width=H, table_stride=table_stride or H,
                       row_stride=row_stride or H, ids_64=1, scale=scale)
    e.id_stride[1] = 1
    return e


def expert_descriptor(T, K, R, H, stride=None):
    s = stride or H
    return _lib.Experts(tokens=T, rows=R, width=H, token_stride=s, row_stride=s, residual_stride=s, drow_stride=s,
                        choices=K)


# ------------------------------------------------------------- workspaces
@pytest.mark.parametrize("shape", [(257, 90, 64), (5000, 7001, 40), (20000, 300, 33), (17000, 100000, 8)],
                         ids=emb.shape_id)
def test_embedding_workspace(shape):
    n, V, H = shape
    ids, dy = emb.tokens(n, V), emb.normal(n, H, dtype=BF16)
    want = pkg.embedding_backward(ids, dy, V)
    need = pkg.rmsnorm_embedding_bwd_workspace_size(n, V, H)
    room = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)  # not zeroed
    base = room.data_ptr()
    grad = torch.full_like(want, 3.0)

    def call(at, size):
        return pkg.rmsnorm_embedding_bwd_ws(descriptor(n, V, H), ids, dy, grad, -1, 0, _lib.BF16, at, size)

    assert call(None, need) == call(base, need - 1) == _lib.ERR_INVALID_ARG
    assert call(base + 8, need) == _lib.ERR_MISALIGNED
    assert call(base, need) == _lib.OK
    torch.cuda.synchronize()
    assert (room[need:] == 255).all()
    assert torch.equal(grad, want)
    grad.fill_(3.0)  # one from the stream-ordered allocator
    assert pkg.rmsnorm_embedding_bwd(descriptor(n, V, H), ids, dy, grad, -1, 0, _lib.BF16) == _lib.OK
    assert torch.equal(grad, want)


def test_expert_sort_workspace():
    T, K, E = 20001, 3, 70
    e = exp.choices(T, K, E)
    want = pkg.expert_sort(e, E, align=8)
    R = want.source.numel()
    need = pkg.rmsnorm_expert_sort_workspace_size(T, K, E)
    room = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
    base = room.data_ptr()
    # more rows than are needed: those behind have no choice
    outs = [torch.full((n,), 77, dtype=torch.int32, device=DEV) for n in (T * K, R + 50, E + 1, E)]

    def call(at, size):
        return pkg.rmsnorm_expert_sort_ws(e, 1, T, K, E, 8, R + 50, *outs, at, size)

    assert call(None, need) == call(base, need - 1) == _lib.ERR_INVALID_ARG
    assert call(base + 4, need) == _lib.ERR_MISALIGNED
    assert call(base, need) == _lib.OK
    assert (room[need:] == 255).all()
    assert torch.equal(outs[0].view(T, K), want.position) and torch.equal(outs[1][:R], want.source)
    assert (outs[1][R:] == -1).all()
    assert torch.equal(outs[2], want.offsets) and torch.equal(outs[3], want.counts)
    for t in outs:
        t.fill_(77)
    assert pkg.rmsnorm_expert_sort(e, 1, T, K, E, 8, R + 50, *outs) == _lib.OK
    assert torch.equal(outs[0].view(T, K), want.position) and (outs[1][R:] == -1).all()


# ------------------------------------------------------------- guard bands
def banded(rows, width, stride, dtype, offset):
    """A tensor of rows inside a larger one, `offset` elements off 256 bytes, with
    bands before, between and behind."""
    whole = torch.full((1024 + rows * stride + 1024,), 123.0, dtype=dtype, device=DEV)
    start = 512 + offset
    return whole, torch.as_strided(whole, (rows, width), (stride, 1), start)


def bands_hold(whole, part):
    outside = torch.ones_like(whole, dtype=torch.bool)
    torch.as_strided(outside, part.shape, part.stride(), part.storage_offset()).fill_(False)
    assert bool((whole[outside] == 123).all())


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("H,room", [(64, 0), (64, 8), (40, 3), (33, 0), (33, 7), (1412, 4), (2050, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_bands(dtype, H, room, offset):
    """Nothing but the rows is written, at every alignment."""
    code = _lib.BF16 if dtype == BF16 else _lib.F32
    s = H + room
    n, V = 70, 41
    ids, table, dy = emb.tokens(n, V), emb.normal(V, H, dtype=dtype), emb.normal(n, H, dtype=dtype, seed=4)
    whole, y = banded(n, H, s, dtype, offset)
    assert pkg.rmsnorm_embedding_fwd(descriptor(n, V, H, 2.0, H, s), ids, table, y, code) == _lib.OK
    assert torch.equal(y, pkg.embedding_forward(ids, table, scale=2.0))
    bands_hold(whole, y)
    whole, grad = banded(V, H, s, dtype, offset)
    need = pkg.rmsnorm_embedding_bwd_workspace_size(n, V, H)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert pkg.rmsnorm_embedding_bwd_ws(descriptor(n, V, H, 2.0, s, H), ids, dy, grad, -1, 0, code, ws,
                                        need) == _lib.OK
    ref.close(grad, *ref.embedding_grad(ids, dy, V, 2.0))
    bands_hold(whole, grad)

    T, K, E = 23, 6, 9
    plan = pkg.expert_sort(exp.choices(T, K, E), E, align=4)
    R = plan.source.numel()
    x, rows = emb.normal(T, H, dtype=dtype), emb.normal(R, H, dtype=dtype, seed=2)
    w = torch.rand(T, K, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(dtype)
    d = expert_descriptor(T, K, R, H)
    d.row_stride = s
    whole, out = banded(R, H, s, dtype, offset)
    assert pkg.rmsnorm_expert_dispatch_fwd(d, x, plan.position, plan.source, out, code) == _lib.OK
    assert torch.equal(out, pkg.expert_dispatch_forward(x, plan.position, plan.source))
    bands_hold(whole, out)
    d = expert_descriptor(T, K, R, H)
    d.token_stride = s
    whole, out = banded(T, H, s, dtype, offset)
    assert pkg.rmsnorm_expert_combine_fwd(d, rows, plan.position, w, x, out, code) == _lib.OK
    y, magnitude = ref.combine(rows, plan.position, w, x)
    ref.close(out, y, K + 1, magnitude)
    bands_hold(whole, out)
    d = expert_descriptor(T, K, R, H)
    d.drow_stride = s
    whole, out = banded(R, H, s, dtype, offset)
    dwhole, dw = banded(T, K, K, F32, offset)
    assert pkg.rmsnorm_expert_combine_bwd(d, x, rows, plan.position, plan.source, w, out, dw.view(-1), code) == _lib.OK
    want, dots, magnitude = ref.combine_grads(x, rows, plan.position, w)
    ref.close(out, want)
    ref.close(dw, dots, H, magnitude)
    bands_hold(whole, out)
    bands_hold(dwhole, dw)


@pytest.mark.parametrize("H", [1024, 1028, 1030])
def test_bands_of_the_ring(H):
    """Many choices of many tokens: rows copied ahead in pieces of 16, 8 and 4 bytes."""
    T, K, E = 1500, 7, 30
    plan = pkg.expert_sort(exp.choices(T, K, E), E, align=16)
    R = plan.source.numel()
    dy, rows = emb.normal(T, H, dtype=BF16), emb.normal(R, H, dtype=BF16, seed=2)
    w = torch.softmax(emb.normal(T, K, dtype=F32, seed=3), -1)
    s = H + 6
    d = expert_descriptor(T, K, R, H)
    d.drow_stride = s
    whole, out = banded(R, H, s, BF16, 2)
    dwhole, dw = banded(T, K, K, F32, 1)
    assert pkg.rmsnorm_expert_combine_bwd(d, dy, rows, plan.position, plan.source, w, out, dw.view(-1),
                                          _lib.BF16_W_F32) == _lib.OK
    want, dots, magnitude = ref.combine_grads(dy, rows, plan.position, w)
    ref.close(out, want)
    ref.close(dw, dots, H, magnitude)
    bands_hold(whole, out)
    bands_hold(dwhole, dw)
    again, dagain = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    ref.close(again, want)
    ref.close(dagain, dots, H, magnitude)


@pytest.mark.parametrize("T", [1, 5, 300, 5000])
@pytest.mark.parametrize("K", [5, 8, 9, 20])
@pytest.mark.parametrize("dtype,H", [(BF16, 2048), (F16, 520), (F32, 4100), (BF16, 9006)])
def test_ring_of_many_choices(dtype, H, K, T):
    """Blocks of every team, few tokens and more than the resident blocks take; groups
    of eight choices."""
    if T * K * H > 60_000_000:
        T = 60_000_000 // (K * H)
    E = 40
    plan = pkg.expert_sort(exp.choices(T, K, E), E)
    R = plan.source.numel()
    dy, rows = emb.normal(T, H, dtype=dtype), emb.normal(R, H, dtype=dtype, seed=2)
    w = torch.softmax(emb.normal(T, K, dtype=F32, seed=3), -1)
    drows, dw = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    want, dots, magnitude = ref.combine_grads(dy, rows, plan.position, w)
    ref.close(drows, want)
    ref.close(dw, dots, H, magnitude)


def test_rows_of_the_largest_width():
    """Rows of 2^31 - 1 elements, one by one (no piece of 4 bytes fits): where a thread's
    next element passes 31 bits. Ones and powers of two, whose sums fp32 holds."""
    H = (1 << 31) - 1
    x = torch.ones(1, H, dtype=BF16, device=DEV)
    x[0, -1] = 4
    zero = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    rows = pkg.expert_dispatch_forward(x, zero, zero[0])
    assert torch.equal(rows, x)
    w = torch.full((1, 1), 0.5, device=DEV)
    y = pkg.expert_combine_forward(rows, zero, w, x)
    assert float(y[0, -1]) == 6 and float(y[0, -2]) == 1.5 and float(y.amin()) == 1.5
    del y
    drows, dw = pkg.expert_combine_backward(x, rows, zero, zero[0], w)
    assert float(drows[0, -1]) == 2 and float(drows[0, -2]) == 0.5 and float(drows.amin()) == 0.5
    # a thread's 2^23 ones are exact, as are sums of powers of two; the 4^2 is below a step
    assert abs(float(dw) - 2.0 ** 31) <= 2.0 ** 8
    del drows, rows
    ids = torch.zeros(1, dtype=torch.int64, device=DEV)
    assert torch.equal(pkg.embedding_forward(ids, x), x)
    assert torch.equal(pkg.embedding_backward(ids, x, 1), x)


def test_result_larger_than_the_cache():
    """Stored without being kept: more than half of L2."""
    ids, table = emb.tokens(20001, 900), emb.normal(900, 2056, dtype=BF16)
    y = pkg.embedding_forward(ids, table)
    assert y.numel() * 2 > torch.cuda.get_device_properties(0).L2_cache_size // 2
    there = (ids >= 0) & (ids < 900)
    assert torch.equal(y, torch.where(there[:, None], table[ids.clamp(0, 899)], 0))
    odd = emb.normal(900, 2055, dtype=F16)
    y = pkg.embedding_forward(ids, odd)
    assert torch.equal(y, torch.where(there[:, None], odd[ids.clamp(0, 899)], 0))


# ------------------------------------------------------------- streams and graphs
def calls():
    """Every operator on inputs of its own: name -> (call(stream), what it gave first)."""
    ids, table, dy = emb.tokens(3000, 500), emb.normal(500, 96, dtype=BF16), emb.normal(3000, 96, dtype=BF16)
    many, wide = emb.tokens(30000, 9000), emb.normal(30000, 24, dtype=F16)
    e = exp.choices(700, 6, 20)
    plan = pkg.expert_sort(e, 20, align=8)
    big = exp.choices(9000, 3, 33)
    R = plan.source.numel()
    x, rows = emb.normal(700, 512, dtype=BF16), emb.normal(R, 512, dtype=BF16, seed=2)
    w = torch.rand(700, 6, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    out = {
        "lookup": lambda s=None: (pkg.embedding_forward(ids, table, 3.0, stream=s),),
        "gradient": lambda s=None: (pkg.embedding_backward(ids, dy, 500, stream=s),),
        "gradient_many": lambda s=None: (pkg.embedding_backward(many, wide, 9000, grad_dtype=F32, stream=s),),
        "sort": lambda s=None: tuple(pkg.expert_sort(e, 20, 8, stream=s)),
        "sort_many": lambda s=None: tuple(pkg.expert_sort(big, 33, stream=s)),
        "dispatch": lambda s=None: (pkg.expert_dispatch_forward(x, plan.position, plan.source, stream=s),),
        "dispatch_backward": lambda s=None: (pkg.expert_dispatch_backward(rows, plan.position, stream=s),),
        "combine": lambda s=None: (pkg.expert_combine_forward(rows, plan.position, w, x, stream=s),),
        "combine_backward": lambda s=None: pkg.expert_combine_backward(x, rows, plan.position, plan.source, w,
                                                                       stream=s),
    }
    return {name: (call, call()) for name, call in out.items()}


def same(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_on_another_stream():
    todo = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = {name: [call(s) for _ in range(3)] for name, (call, _) in todo.items()}
    s.synchronize()
    for name, (_, want) in todo.items():
        for g in got[name]:
            same(g, want)


def test_memory_of_another_stream():
    """A call on a given stream takes no memory that the current stream still has
    work queued on."""
    todo = calls()
    s = torch.cuda.Stream()
    for name, (call, want) in todo.items():
        n = max(t.numel() * t.element_size() for t in want)
        t = torch.full((n,), 7, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)
        seen = t.clone()
        del t
        got = call(s)
        s.synchronize()
        torch.cuda.synchronize()
        assert (seen == 7).all(), name
        same(got, want)
        del got


def test_several_at_once():
    """Threads on streams of their own."""
    todo = calls()
    torch.cuda.synchronize()
    failed = []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    for call, want in todo.values():
                        got = call()
                        s.synchronize()
                        same(got, want)
        except Exception as error:  # noqa: BLE001
            failed.append(error)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_captured_together_and_replayed():
    """Two graphs of every operator, replayed in turn and at once."""
    todo = calls()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = {name: call() for name, (call, _) in todo.items()}
        graphs.append((g, got))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, got), s in zip(graphs, streams):
            for ts in got.values():
                for t in ts:
                    t.zero_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            for name, (_, want) in todo.items():
                same(got[name], want)


def test_captured_with_other_tokens():
    """A captured lookup, sort and gradient follow what the ids hold at replay."""
    V, H, n, E = 300, 40, 2000, 12
    ids, table, dy = emb.tokens(n, V), emb.normal(V, H, dtype=BF16), emb.normal(n, H, dtype=BF16)
    e = exp.choices(n, 2, E)
    pkg.embedding_backward(ids, dy, V)
    pkg.expert_sort(e, E)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = pkg.embedding_forward(ids, table)
        grad = pkg.embedding_backward(ids, dy, V)
        plan = pkg.expert_sort(e, E)
        rows = pkg.expert_dispatch_forward(dy, plan.position, plan.source)
    for seed in (3, 4):
        ids.copy_(emb.tokens(n, V, seed))
        e.copy_(exp.choices(n, 2, E, seed, drop=0.3))
        g.replay()
        torch.cuda.synchronize()
        ref.close(y, ref.embedding(ids, table, 1.0))
        ref.close(grad, *ref.embedding_grad(ids, dy, V, 1.0))
        want = ref.sort(e, E, 1, 2 * n)
        exp.same_plan(plan, want)
        src = want[1].long()
        assert torch.equal(rows, torch.where(src[:, None] >= 0, dy[src.clamp(min=0) // 2], 0))


# ------------------------------------------------------------- autograd's versions
def test_accumulating_is_seen_by_autograd():
    ids, dy = emb.tokens(50, 9), emb.normal(50, 8, dtype=F32)
    grad = torch.zeros(9, 8, device=DEV)
    leaf = torch.ones_like(grad, requires_grad=True)
    out = leaf * grad  # saves grad
    pkg.embedding_backward(ids, dy, 9, out=grad, accumulate=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    with torch.inference_mode():
        other = torch.zeros(9, 8, device=DEV)
        pkg.embedding_backward(ids, dy, 9, out=other, accumulate=True)
    assert torch.equal(other, grad)


def test_overlapping_outputs_are_refused():
    ids, dy = emb.tokens(50, 9), emb.normal(50, 8, dtype=F32)
    with pytest.raises(pkg.RMSNormError, match="INVALID_ARG"):
        pkg.embedding_backward(ids, dy, 9, out=torch.zeros(8, device=DEV).expand(9, 8))


# ------------------------------------------------------------- checked build
def test_token_suites_under_checks():
    """These tests with every global store, asynchronous copy and slot tested against
    its extent; a failed check is recorded on the device and read back here."""
    from memory_bound_normalization_gb300 import build as libbuild

    if _lib.checked_variant():
        pytest.skip("runs the checked build already")
    libbuild.build(checked=True)
    env = dict(os.environ, RMSNORM_LIBRARY_VARIANT="checked")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_embedding_gpu.py", "tests/test_experts_gpu.py", "tests/test_token_edges_gpu.py",
           "tests/test_token_block_gpu.py"]
    out = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (out.stdout + out.stderr)[-4000:]
    assert out.returncode == 0, tail
    assert " passed" in tail and " failed" not in tail, tail


@pytest.fixture(scope="module", autouse=True)
def _status():
    """No kernel of this module recorded a failure (of the checked build, a store
    outside its tensor)."""
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
