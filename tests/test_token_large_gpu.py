"""The paths of the rows by index that large calls alone take: gradients larger than
what is zeroed beside the sort (rows zeroed by marks), strided gradients of more than
256 tokens, sorts of several tiles a block, and the combine backward's ring with its
tokens shared out. Against 64 bits and a walk over the choices."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import test_embedding_gpu as emb
import test_experts_gpu as exp
import test_token_edges_gpu as edges
import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")
from memory_bound_normalization_gb300 import _lib  # noqa: E402

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def normal(*shape, dtype, seed=1):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV).to(dtype)


def ids_of(which, n, V, seed=0):
    """Ids of a kind; some lie outside the table."""
    gen = torch.Generator().manual_seed(seed)
    i = torch.arange(n)
    ids = {
        "text": lambda: emb.tokens(n, V, seed).cpu(),
        # one for half of the tokens among others that share its lowest nine bits
        "alike": lambda: torch.where(i % 2 == 0, 512 * (V // 1024),
                                     512 * torch.randint(0, max(1, V // 512), (n,), generator=gen)),
        # the first rows and the last ones, a few times each
        "ends": lambda: torch.where(i % 3 == 0, i // 3 % 40, V - 1 - i % 97),
        "apart": lambda: i * 7919 % V,
        "same": lambda: i * 0 + V // 3,
        "none": lambda: torch.where(i % 2 == 0, -1 - i, V + i),
    }[which]()
    return ids.clamp(max=V + n).to(DEV)


# tokens, rows, width, types of dy and gradient: more than 48 MB for one cluster's sort
# (up to 16384 tokens), more than 12 MB for each launch of a larger one (passes of nine
# bits); rows of several slices; rows of one sector
LARGE = [(257, 70001, 512, BF16, F32), (3000, 70000, 512, BF16, F32), (16384, 70000, 512, F16, F16),
         (16385, 262145, 96, BF16, F32), (20000, 510, 16384, BF16, F32), (20000, 70000, 513, BF16, BF16),
         (5000, 3_000_017, 9, F32, F32), (320_000, 400_000, 64, BF16, F32)]


def budget(n, V):
    """Bytes that are zeroed beside the sort."""
    if n <= 16384:
        return 48 << 20
    return 2 * -(-V.bit_length() // 9) * (12 << 20)


@pytest.mark.parametrize("which", ["text", "alike", "ends", "apart", "same", "none"])
@pytest.mark.parametrize("case", LARGE, ids=lambda c: "x".join(str(v).split(".")[-1] for v in c))
def test_rows_zeroed_by_marks(case, which):
    n, V, H, act, weight = case
    assert V * H * weight.itemsize > budget(n, V)
    ids, dy = ids_of(which, n, V), normal(n, H, dtype=act)
    out = torch.full((V, H), NAN, dtype=weight, device=DEV)
    # the frequent id is padding for one of the kinds
    pad = V // 3 if which == "same" else 0 if which == "text" else None
    grad = pkg.embedding_backward(ids, dy, V, scale=0.5, padding_idx=pad, out=out)
    assert grad is out
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, 0.5, pad)
    ref.close(grad, want, terms, magnitude)
    assert not grad[(terms == 0)[:, 0]].any()
    del want, magnitude
    # other tokens in the same memory: no mark is left of the call before
    ids = ids_of(which, n, V, seed=1).roll(1) if which != "none" else ids_of("ends", n, V)
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, 1.0)
    ref.close(pkg.embedding_backward(ids, dy, V, out=out), want, terms, magnitude)


@pytest.mark.parametrize("n,V,H,room", [(3000, 30000, 512, 8), (20000, 70000, 200, 3), (20000, 510, 16384, 24),
                                        (3000, 400_000, 40, 1), (1000, 60, 300_000, 5)])
def test_strided_rows_zeroed_by_marks(n, V, H, room):
    assert V * H * 4 > budget(n, V)
    ids, dy = ids_of("text", n, V), normal(n, H, dtype=BF16)
    whole, grad = edges.banded(V, H, H + room, F32, 4)
    grad.fill_(NAN)
    pkg.embedding_backward(ids, dy, V, out=grad)
    ref.close(grad, *ref.embedding_grad(ids, dy, V, 1.0))
    edges.bands_hold(whole, grad)


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("H,room", [(64, 0), (64, 8), (40, 3), (33, 7), (1412, 4), (2050, 1)])
@pytest.mark.parametrize("n,V", [(300, 41), (5000, 600), (20000, 41), (17000, 600)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_bands_of_sorted_gradients(dtype, n, V, H, room, offset):
    """Gradients of more than 256 tokens with room between their rows, dy as a slice of
    columns, runs over many blocks; written and added to."""
    ids = ids_of("text", n, V)
    ids[::3] = 7  # over several blocks
    both = normal(n, 2 * H + offset, dtype=dtype, seed=4)
    dy = both[:, offset:offset + H]
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, 2.0)
    whole, grad = edges.banded(V, H, H + room, dtype, offset)
    grad.fill_(NAN)
    pkg.embedding_backward(ids, dy, V, scale=2.0, out=grad)
    ref.close(grad, want, terms, magnitude)
    edges.bands_hold(whole, grad)
    before = normal(V, H, dtype=dtype, seed=5)
    grad.copy_(before)
    pkg.embedding_backward(ids, dy, V, scale=2.0, out=grad, accumulate=True)
    ref.close(grad, want + before.double(), terms + 1, magnitude + before.double().abs())
    untouched = terms[:, 0] == 0
    assert torch.equal(grad[untouched], before[untouched])
    edges.bands_hold(whole, grad)


@pytest.mark.parametrize("n", [300, 20000])
def test_sorted_gradients_past_32_bits(n):
    """A gradient of more than 2^32 bytes, its first, middle and last rows; the others
    zeroed beside the sort and by marks."""
    V, H = 131075, 16400
    at = [0, 1, V // 2, V - 2, V - 1]
    ids = torch.tensor(at, device=DEV)[torch.arange(n, device=DEV) % 5]
    dy = normal(n, H, dtype=BF16)
    out = torch.full((V, H), NAN, dtype=BF16, device=DEV)
    grad = pkg.embedding_backward(ids, dy, V, out=out)
    for i, v in enumerate(at):
        mine = dy[i::5].double()
        ref.close(grad[v], mine.sum(0), mine.shape[0], mine.abs().sum(0))
    hit = grad.count_nonzero(1).nonzero()[:, 0]
    assert hit.tolist() == at
    assert not any(bool(part.isnan().any()) for part in grad.split(8192))


@pytest.mark.parametrize("shape", [(4863, 300, 4096), (9727, 70001, 2048), (2432, 600, 8200), (131_072, 511, 1032),
                                   (311_297, 70001, 66), (40_000, 9, 4096)], ids=emb.shape_id)
def test_a_workspace_is_not_left(shape):
    """A workspace of the bytes that are asked for, and of what a larger batch asks for."""
    n, V, H = shape
    ids, dy = ids_of("text", n, V), normal(n, H, dtype=BF16)
    want = pkg.embedding_backward(ids, dy, V)
    for size in (pkg.rmsnorm_embedding_bwd_workspace_size(n, V, H),
                 pkg.rmsnorm_embedding_bwd_workspace_size(n + n // 3, V, H)):
        room = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
        grad = torch.full_like(want, NAN)
        assert pkg.rmsnorm_embedding_bwd_ws(edges.descriptor(n, V, H), ids, dy, grad, -1, 0, _lib.BF16,
                                            room.data_ptr(), size) == _lib.OK
        assert bool((room[size:] == 255).all()) and torch.equal(grad, want)


# ------------------------------------------------------------- sorts of several tiles
# one cluster takes up to 16384 items, a block one tile of 1024 up to 155648, of 2048 up to
# 311296, then two and more
SIZES = [16383, 16384, 16385, 155648, 155649, 311296, 311297, 700_001]


@pytest.mark.parametrize("which", ["text", "same", "turn", "none"])
@pytest.mark.parametrize("n", SIZES)
def test_expert_sorts(n, which):
    E, align = (1024, 1) if which == "turn" else (300, 32)
    i = torch.arange(n, device=DEV)
    e = {"text": lambda: emb.tokens(n, E, 3), "same": lambda: i * 0 + E - 1, "turn": lambda: i * 7 % E,
         "none": lambda: i * 0 + E}[which]()[:, None]
    exp.same_plan(pkg.expert_sort(e, E, align=align), ref.sort(e, E, align, ref.rows_of(n, 1, E, align)))


@pytest.mark.parametrize("which", ["text", "alike", "same", "apart", "none"])
@pytest.mark.parametrize("V", [511, 70001])
@pytest.mark.parametrize("n", SIZES)
def test_gradients_of_sorts(n, V, which):
    H = 6
    ids, dy = ids_of(which, n, V), normal(n, H, dtype=BF16)
    ref.close(pkg.embedding_backward(ids, dy, V, grad_dtype=F32), *ref.embedding_grad(ids, dy, V, 1.0))


# ------------------------------------------------------------- the ring, shared out
# tokens enough for blocks of each team to share them out, and some over; groups of
# eight choices; several chunks of columns; pieces of 16, 8 and 4 bytes
@pytest.mark.parametrize("T,K,H,dtype", [(38912 + 777, 9, 256, BF16), (38912, 6, 260, F16), (19456 + 31, 12, 512, BF16),
                                         (19456, 17, 130, F32), (9728 + 5, 9, 1024, F16), (9728, 8, 900, BF16),
                                         (5003, 9, 4100, BF16), (4864, 5, 4098, BF16), (4900, 16, 2052, F32)])
def test_ring_shared_out(T, K, H, dtype):
    E = 40
    plan = pkg.expert_sort(exp.choices(T, K, E), E, align=8)
    R = plan.source.numel()
    dy, rows = normal(T, H, dtype=dtype), normal(R, H, dtype=dtype, seed=2)
    w = torch.softmax(normal(T, K, dtype=F32, seed=3), -1).to(dtype)
    drows, dw = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    again = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    assert torch.equal(again[0], drows) and torch.equal(again[1], dw)
    del again
    for part in torch.arange(T, device=DEV).split(4096):  # token by token, as the rows are
        p = plan.position[part]
        keep = p >= 0
        g = dy[part].double()[:, None]
        ref.close(drows[p[keep].long()], (g * w[part].double()[..., None])[keep])
        prod = g * ref.gathered(rows, p)
        ref.close(dw[part], prod.sum(-1), H, prod.abs().sum(-1))
    assert not drows[plan.source < 0].any()


@pytest.mark.parametrize("K", [1024, 1025, 1500])
def test_choices_up_to_the_rings_most_and_past_it(K):
    T, E, H = 5, 1024, 1024
    e = torch.randint(-1, E, (T, K), generator=torch.Generator().manual_seed(K)).to(DEV)
    plan = pkg.expert_sort(e, E)
    R = plan.source.numel()
    dy, rows = normal(T, H, dtype=BF16), normal(R, H, dtype=BF16, seed=2)
    w = torch.softmax(normal(T, K, dtype=F32, seed=3), -1)
    drows, dw = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    want, dots, magnitude = ref.combine_grads(dy, rows, plan.position, w)
    ref.close(drows, want)
    ref.close(dw, dots, H, magnitude)
    y, magnitude = ref.combine(rows, plan.position, w)
    ref.close(pkg.expert_combine_forward(rows, plan.position, w), y, K, magnitude)


@pytest.mark.parametrize("H", [(1 << 29) + 4, (1 << 29) + 1])
def test_ring_of_rows_past_31_bits_of_bytes(H):
    """One token of five choices, by pieces of 16 and of 4 bytes. Ones and powers of two,
    whose sums fp32 holds."""
    K = 5
    plan = pkg.expert_sort(torch.tensor([[3, 0, -1, 1, 2]], device=DEV), 4)
    dy = torch.ones(1, H, device=DEV)
    dy[0, -1] = 4
    rows = torch.ones(K, H, device=DEV)
    rows[2, -1] = 2
    w = torch.tensor([[0.5, 1.0, NAN, 2.0, 4.0]], device=DEV)
    drows, dw = pkg.expert_combine_backward(dy, rows, plan.position, plan.source, w)
    # rows in the experts' order: choices 1, 3, 4 and 0, then none
    for row, weight in enumerate((1.0, 2.0, 4.0, 0.5, 0.0)):
        assert float(drows[row, -1]) == 4 * weight
        assert bool((drows[row, :-1] == weight).all())
    base = float(1 << 29) + (H - (1 << 29) - 1)
    want = [base + 4, base + 4, 0.0, base + 4, base + 8]
    # a thread's sums are exact; joined, half steps of sums of 2^25 to 2^30: 1 + 2 + ... + 32
    assert all(abs(a - b) <= 2.0 ** 6 for a, b in zip(dw[0].tolist(), want))


# ------------------------------------------------------------- checked build
def test_large_calls_under_checks():
    """These tests in the checked build; a failed check is recorded on the device."""
    from memory_bound_normalization_gb300 import build as libbuild

    if _lib.checked_variant():
        pytest.skip("runs the checked build already")
    libbuild.build(checked=True)
    env = dict(os.environ, RMSNORM_LIBRARY_VARIANT="checked")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "-k", "not 700001 and not 311296", "tests/test_token_large_gpu.py"]
    out = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = (out.stdout + out.stderr)[-4000:]
    assert out.returncode == 0, tail
    assert " passed" in tail and " failed" not in tail, tail


@pytest.fixture(scope="module", autouse=True)
def _status():
    """No kernel of this module recorded a failure."""
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
