"""Embedding lookup with a scale and its gradient by sorted tokens, against 64 bits."""
from __future__ import annotations

import pytest
import torch

import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda"
# tokens, rows of the table, width: one of each; less and more than a warp; widths of
# 16-, 8-, 4- and 2-byte pieces; more tokens than one cluster sorts (131072)
SHAPES = [(1, 1, 1), (1, 7, 4096), (3, 5, 8), (33, 10, 40), (256, 70000, 24), (200, 3, 4104),
          (255, 40, 77), (257, 1000, 1412), (1021, 50, 129),
          (4097, 3, 64), (5000, 70000, 24), (31, 300, 20000), (131072, 511, 16), (131073, 512, 6),
          (140001, 5, 3), (300000, 400000, 2)]


def shape_id(s):
    return "x".join(map(str, s))


def tokens(n, V, seed=0, spread=True):
    """Frequent ids are small, and a few lie outside."""
    gen = torch.Generator().manual_seed(seed)
    ids = (torch.rand(n, generator=gen).double() * torch.log(torch.tensor(V + 1.0))).exp().long() - 1
    ids.clamp_(0, V - 1)
    if spread and n > 2:
        ids[torch.randint(0, n, (max(1, n // 16),), generator=gen)] = -1
        ids[torch.randint(0, n, (max(1, n // 16),), generator=gen)] = V
    return ids.to(DEV)


def normal(*shape, dtype, seed=1):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


@pytest.mark.parametrize("pair", ref.PAIRS, ids=ref.pair_id)
@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
def test_forward(shape, pair):
    n, V, H = shape
    ids, table = tokens(n, V), normal(V, H, dtype=pair[1])
    y = pkg.embedding_forward(ids, table, scale=1.7, out_dtype=pair[0])
    assert y.dtype == pair[0]
    ref.close(y, ref.embedding(ids, table, torch.tensor(1.7).float().double()))


@pytest.mark.parametrize("pair", ref.PAIRS, ids=ref.pair_id)
@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
def test_backward(shape, pair):
    n, V, H = shape
    ids, dy = tokens(n, V).int(), normal(n, H, dtype=pair[0])
    pad = V // 2
    grad = pkg.embedding_backward(ids, dy, V, scale=0.3, padding_idx=pad, grad_dtype=pair[1])
    assert grad.dtype == pair[1]
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, torch.tensor(0.3).float().double(), pad)
    ref.close(grad, want, terms, magnitude)
    again = pkg.embedding_backward(ids, dy, V, scale=0.3, padding_idx=pad, grad_dtype=pair[1])
    assert torch.equal(grad, again)


@pytest.mark.parametrize("which", ["same", "two", "none", "each", "outside"])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 255, 256, 257, 2048, 9000, 131073])
def test_runs(which, n):
    """One id for all, two in turn, none, an id for each: runs over many segments
    and none."""
    V, H = 70001, 24
    i = torch.arange(n, device=DEV)
    ids = {"same": i * 0 + 77, "two": i % 2 * 70000, "none": i * 0 - 5, "each": (i * 31) % V,
           "outside": i + V}[which]
    dy = normal(n, H, dtype=torch.bfloat16)
    grad = pkg.embedding_backward(ids, dy, V, grad_dtype=torch.float32)
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, 1.0)
    ref.close(grad, want, terms, magnitude)


@pytest.mark.parametrize("n", [100, 700])
@pytest.mark.parametrize("pair", ref.PAIRS, ids=ref.pair_id)
def test_accumulate(pair, n):
    V, H = 90, 72
    ids, dy = tokens(n, V // 2), normal(n, H, dtype=pair[0])
    grad = normal(V, H, dtype=pair[1], seed=5)
    before = grad.clone()
    version = grad._version
    out = pkg.embedding_backward(ids, dy, V, scale=2.0, out=grad, accumulate=True)
    assert out is grad and grad._version > version
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, 2.0)
    ref.close(grad, want + before.double(), terms + 1, magnitude + before.double().abs())
    untouched = terms[:, 0] == 0
    # the ids are up to V / 2, the one behind those of tokens()
    assert int(untouched.sum()) >= V - V // 2 - 1 and torch.equal(grad[untouched], before[untouched])


def test_padding_from_the_end_and_values_not_read():
    """Rows of padding and of ids outside may hold infinities and NaN."""
    n, V, H = 100, 9, 40
    ids = torch.arange(n, device=DEV) % (V + 1)
    dy = normal(n, H, dtype=torch.bfloat16)
    dy[ids == V] = float("nan")
    dy[ids == V - 1] = float("inf")
    grad = pkg.embedding_backward(ids, dy, V, padding_idx=-1)
    want, terms, magnitude = ref.embedding_grad(ids, torch.where(dy.isfinite(), dy, 0), V, 1.0, V - 1)
    ref.close(grad, want, terms, magnitude)
    assert not grad[V - 1].any()


def test_infinities_and_nan_of_one_row_stay_there():
    n, V, H = 200, 11, 16
    ids = torch.arange(n, device=DEV) % V
    dy = normal(n, H, dtype=torch.float16)
    dy[ids == 3, 2] = float("inf")
    dy[5, 7] = float("nan")
    grad = pkg.embedding_backward(ids, dy, V)
    bad = ~grad.isfinite()
    assert bad.nonzero().tolist() == [[3, 2], [5, 7]]
    table = normal(V, H, dtype=torch.bfloat16)
    table[4] = float("nan")
    y = pkg.embedding_forward(ids, table)
    assert torch.equal(y.isnan().any(1), ids == 4)


@pytest.mark.parametrize("H", [64, 33])
def test_strides(H):
    """Ids without their last column, a table and gradients with room between rows,
    dy as a slice of columns."""
    B, T, V = 5, 37, 60
    batch = tokens(B * (T + 1), V).view(B, T + 1)
    ids = batch[:, :-1]
    wide = normal(V, H + 24, dtype=torch.bfloat16)
    table = wide[:, 8:8 + H]
    y = pkg.embedding_forward(ids, table, scale=3.0)
    assert y.shape == (B, T, H)
    ref.close(y, ref.embedding(ids, table, 3.0))
    both = normal(B, T, 2 * H, dtype=torch.bfloat16)
    dy = both[..., H:]
    out = torch.full((V, H + 3), 7.0, device=DEV)
    grad = pkg.embedding_backward(ids, dy, V, out=out[:, :H])
    want, terms, magnitude = ref.embedding_grad(ids, dy, V, 1.0)
    ref.close(grad, want, terms, magnitude)
    assert bool((out[:, H:] == 7).all())
    # ids down a column, and one id for all
    ref.close(pkg.embedding_forward(batch.t()[:-1], table), ref.embedding(batch.t()[:-1], table, 1.0))
    one = torch.full((), 3, device=DEV).expand(4, 6)
    ref.close(pkg.embedding_forward(one, table), ref.embedding(one, table, 1.0))
    one_dy = normal(H, dtype=torch.float32).expand(4, 6, H)
    want, terms, magnitude = ref.embedding_grad(one, one_dy, V, 1.0)
    ref.close(pkg.embedding_backward(one, one_dy, V), want, terms, magnitude)


def test_nothing():
    table = normal(6, 8, dtype=torch.bfloat16)
    ids = torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    assert pkg.embedding_forward(ids, table).shape == (0, 3, 8)
    dy = torch.zeros(0, 3, 8, device=DEV)
    grad = pkg.embedding_backward(ids, dy, 6)
    assert grad.shape == (6, 8) and not grad.any()
    out = torch.full((6, 11), 2.0, device=DEV)
    pkg.embedding_backward(ids, dy, 6, out=out[:, :8])
    assert not out[:, :8].any() and bool((out[:, 8:] == 2).all())
    out.fill_(2.0)
    pkg.embedding_backward(ids, dy, 6, out=out[:, :8], accumulate=True)
    assert bool((out == 2).all())
    one = torch.tensor(4, device=DEV)
    assert torch.equal(pkg.embedding_forward(one, table), table[4])


def test_gradient_by_differences():
    """fp32, a step of 2^-6 on exactly held values: the forward is linear."""
    n, V, H = 40, 7, 12
    ids = tokens(n, V, spread=False)
    table = (torch.randint(-64, 64, (V, H)) / 64).to(DEV)
    dy = (torch.randint(-64, 64, (n, H)) / 64).to(DEV)
    grad = pkg.embedding_backward(ids, dy, V, scale=2.0)

    def loss(t):
        return (pkg.embedding_forward(ids, t, scale=2.0).double() * dy.double()).sum()

    for v, h in [(0, 0), (3, 5), (6, 11)]:
        up, down = table.clone(), table.clone()
        up[v, h] += 2.0 ** -6
        down[v, h] -= 2.0 ** -6
        slope = (loss(up) - loss(down)) * 2.0 ** 5
        # sums of at most 40 multiples of 2^-5: exact in fp32
        assert float(slope) == float(grad[v, h])


def test_offsets_past_32_bits():
    """A table and a gradient of more than 2^32 bytes: the last rows."""
    V, H = 131075, 16400
    ids = torch.tensor([V - 1, 0, V - 2, V - 1], device=DEV)
    table = torch.zeros(V, H, dtype=torch.bfloat16, device=DEV)
    table[-2:] = normal(2, H, dtype=torch.bfloat16)
    y = pkg.embedding_forward(ids, table)
    assert torch.equal(y, table[ids])
    dy = normal(4, H, dtype=torch.bfloat16)
    grad = pkg.embedding_backward(ids, dy, V, out=table)
    assert torch.equal(grad[V - 2], dy[2]) and torch.equal(grad[0], dy[1])
    ref.close(grad[V - 1], dy[0].double() + dy[3].double())
    assert not grad[1:V - 2].any()


@pytest.fixture(scope="module", autouse=True)
def _status():
    """No kernel of this module recorded a failure (of the checked build, a store
    outside its tensor)."""
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
