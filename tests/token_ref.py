"""64-bit references of the operators that move rows by an index, and how far
a result may be off: half a step of its type for the one rounding, 2^-24 of it for
the scale's product in fp32, and terms * 2^-24 of the sum of magnitudes for fp32
sums in any order."""
from __future__ import annotations

import torch

TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
# rows' type, type of the table or the weights
PAIRS = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
         (torch.float16, torch.float32)]


def pair_id(p):
    return "-".join(str(t).split(".")[1] for t in p)


def bound(ref, dtype, terms=0, magnitude=0.0):
    """How far a result of this type may be from ref; terms and magnitude of its
    sum (tensors or numbers)."""
    sums = (terms + 2) * 2.0 ** -24 * magnitude
    half = torch.finfo(dtype).eps / 2
    return sums + half * (ref.abs() + sums) + 2.0 ** -24 * ref.abs() + TINY[dtype]


def close(got, ref, terms=0, magnitude=0.0):
    assert got.shape == ref.shape, (got.shape, ref.shape)
    err = (got.double() - ref).abs()
    bad = err > bound(ref, got.dtype, terms, magnitude)
    if bool(bad.any()):
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{float(got[at])} for {float(ref[at])}")


def embedding(ids, table, scale):
    V, H = table.shape
    flat = ids.reshape(-1).long()
    there = (flat >= 0) & (flat < V)
    y = table.double()[flat.clamp(0, V - 1)] * scale * there[:, None]
    return y.view(*ids.shape, H)


def embedding_grad(ids, dy, V, scale, padding=None):
    """gradient, additions of each row [V, 1], sums of magnitudes."""
    H = dy.shape[-1]
    flat = ids.reshape(-1).long()
    there = (flat >= 0) & (flat < V)
    if padding is not None:
        there &= flat != padding
    at = torch.where(there, flat, V)
    g = dy.reshape(-1, H).double()
    rows = torch.zeros(3, V + 1, H, dtype=torch.float64, device=dy.device)
    rows[0].index_add_(0, at, g * scale)
    rows[1].index_add_(0, at, (g * scale).abs())
    count = torch.zeros(V + 1, dtype=torch.float64, device=dy.device)
    count.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    return rows[0, :V], count[:V, None], rows[1, :V]


def rows_of(T, K, E, align):
    n = T * K
    return (n + min(E, n) * (align - 1)) // align * align


def sort(experts, E, align, R):
    """position, source, offsets, counts by a walk over the choices."""
    flat = [int(v) for v in experts.reshape(-1).tolist()]
    mine = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            mine[e].append(i)
    position, source, offsets = [-1] * len(flat), [-1] * R, [0]
    for choices in mine:
        at = offsets[-1]
        for j, i in enumerate(choices):
            position[i] = at + j
            source[at + j] = i
        offsets.append(at + -(-len(choices) // align) * align)
    i32 = {"dtype": torch.int32, "device": experts.device}
    return (torch.tensor(position, **i32).view(experts.shape), torch.tensor(source, **i32),
            torch.tensor(offsets, **i32), torch.tensor([len(c) for c in mine], **i32))


def gathered(rows, position):
    """[..., K, H] in 64 bits, zeros for dropped choices."""
    p = position.long()
    if rows.shape[0] == 0:
        return torch.zeros(*p.shape, rows.shape[1], dtype=torch.float64, device=rows.device)
    return torch.where(p[..., None] >= 0, rows.double()[p.clamp(min=0)], 0.0)


def combine(rows, position, weights=None, residual=None):
    """y and the sum of magnitudes."""
    g = gathered(rows, position)
    if weights is not None:
        g = torch.where(position[..., None] >= 0, g * weights.double()[..., None], 0.0)
    y, magnitude = g.sum(-2), g.abs().sum(-2)
    if residual is not None:
        y, magnitude = y + residual.double(), magnitude + residual.double().abs()
    return y, magnitude


def combine_grads(dy, rows, position, weights):
    """drows, dweights, the dots' sums of magnitudes."""
    p = position.reshape(-1).long()
    K = position.shape[-1]
    H = rows.shape[1]
    g = dy.reshape(-1, 1, H).double().expand(-1, K, H)
    share = g if weights is None else g * weights.reshape(-1, K, 1).double()
    drows = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
    keep = p >= 0
    drows[p[keep]] = share.reshape(-1, H)[keep]
    prod = g * gathered(rows, position).view(-1, K, H)
    return (drows, prod.sum(-1).view(position.shape), prod.abs().sum(-1).view(position.shape))
