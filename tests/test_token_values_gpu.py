"""Values of the rows by index where a formula's zero meets an infinity or NaN."""
from __future__ import annotations

import pytest
import torch

import test_embedding_gpu as emb
import token_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda"
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("scale", [INF, -INF, NAN, 1e39, -1.0, -3e38, 0.0])
@pytest.mark.parametrize("H", [64, 36, 70, 33, 2056])
@pytest.mark.parametrize("pair", ref.PAIRS, ids=ref.pair_id)
def test_rows_outside_the_table_are_zeros_under_any_scale(pair, H, scale):
    """An id outside the table gives a row of zeros, not 0 * scale; rows inside are the
    product, whatever it is."""
    n, V = 300, 11
    ids, table = emb.tokens(n, V), emb.normal(V, H, dtype=pair[1])
    table[3, ::5] = 0
    y = pkg.embedding_forward(ids, table, scale=scale, out_dtype=pair[0])
    there = (ids >= 0) & (ids < V)
    outside = y[~there].float()
    assert outside.shape[0] > 10 and not outside.any() and not outside.signbit().any()
    # one product in fp32, rounded once: the same bits
    want = (table.float()[ids[there]] * torch.tensor(scale, device=DEV).float()).to(pair[0])
    assert torch.equal(y[there].nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.equal(y[there].isnan(), want.isnan())
    # a shard of the table holds nothing of the others' rows: the results add up
    parts = [pkg.embedding_forward(ids - at, table[at:at + 4], scale=scale, out_dtype=pair[0]) for at in (0, 4, 8)]
    total = parts[0] + parts[1] + parts[2]
    assert torch.equal(total.nan_to_num(7.0), y.nan_to_num(7.0)) and torch.equal(total.isnan(), y.isnan())


@pytest.fixture(scope="module", autouse=True)
def _status():
    """No kernel of this module recorded a failure."""
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
