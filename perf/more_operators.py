"""The measured calls of the operators that move a language model's rows by an
index: the embedding lookup with a scale and its gradient by sorted tokens, and
a mixture of experts' tokens sorted by expert, dispatched and combined, with
their gradients.

Each case is one call of a direction of one operator. `run` computes it in its
plain form (elementary torch operations in 32 bits, rounded once at the end)
or, with `own` set, through the library's entry points; `exact` computes the
definition in 64 bits, gradients by differentiating the forward.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


def _emb(name, dir, B, T, V, H, table, act, scaled, pad, id64):
    """B x T tokens of a vocabulary of V; `table` is the type of the table (of
    its gradient), `act` of the rows; `pad`: the share of padding tokens."""
    return {"name": name, "op": "embedding", "dir": dir, "B": B, "T": T, "V": V, "H": H,
            "table": table, "act": act, "scaled": scaled, "pad": pad, "id64": id64}


def _moe(name, op, dir, T, K, E, H, act, weight, align, pad, residual, id64):
    """T tokens with K of E experts each; `pad`: the share of tokens without
    any; `weight` "none": the choices count alike."""
    return {"name": name, "op": op, "dir": dir, "T": T, "K": K, "E": E, "H": H, "act": act,
            "weight": weight, "align": align, "pad": pad, "residual": residual, "id64": id64}


def listed():
    return [
        # one new token of eight requests: latency counts
        _emb("emb_fwd_decode", "fwd", 8, 1, 131072, 4096, "bf16", "bf16", True, 0.0, True),
        # the inputs of the 16384 x 4096 training step
        _emb("emb_fwd_train", "fwd", 4, 4096, 131072, 4096, "bf16", "bf16", True, 0.0, True),
        # its gradient: the whole table is written
        _emb("emb_bwd_train", "bwd", 4, 4096, 131072, 4096, "bf16", "bf16", True, 0.0, True),
        # a small model's fp32 gradient of 16-bit rows, odd sizes, padded batches
        _emb("emb_bwd_odd", "bwd", 7, 1021, 32001, 1000, "f32", "bf16", False, 0.2, False),
        # the choices of a decode step of 16 requests: latency counts
        _moe("sort_decode", "sort", "fwd", 16, 8, 128, 0, "bf16", "f32", 1, 0.0, False, True),
        # the choices of a training step, starts fit for tiles of 128 rows
        _moe("sort_train", "sort", "fwd", 32768, 8, 128, 0, "bf16", "f32", 128, 0.02, False, True),
        # tokens of the 16384 x 4096 step to two experts each of eight
        _moe("dispatch_fwd_train", "dispatch", "fwd", 16384, 2, 8, 4096, "bf16", "f32", 128, 0.0,
             False, True),
        # the gradient of many narrow experts' inputs, fp16, a row that is no whole 16 bytes
        _moe("dispatch_bwd_odd", "dispatch", "bwd", 5003, 6, 60, 1412, "f16", "f32", 1, 0.05,
             False, False),
        # a decode step's experts back to their tokens, onto the residual: latency counts
        _moe("combine_fwd_decode", "combine", "fwd", 16, 8, 128, 4096, "bf16", "f32", 1, 0.0, True,
             True),
        # a long prompt's
        _moe("combine_fwd_prompt", "combine", "fwd", 16384, 8, 128, 4096, "bf16", "f32", 128, 0.0,
             True, True),
        # the training step of experts of 2048, weights in the rows' type
        _moe("combine_bwd_train", "combine", "bwd", 16384, 8, 64, 2048, "bf16", "bf16", 128, 0.01,
             False, True),
        # a short step in fp32
        _moe("combine_bwd_f32", "combine", "bwd", 777, 4, 16, 2880, "f32", "f32", 16, 0.0, True,
             False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """Mostly whole 16-byte vectors of any type, one in four whatever comes."""
    if rng.random() < 0.25:
        return _log(rng, 1, 5000)
    return 8 * _log(rng, 8, 1024)


def draw(rng):
    id64 = rng.random() < 0.5
    H = _width(rng)
    if rng.random() < 0.4:
        dir = rng.choice(["fwd", "bwd"])
        act = rng.choice(["bf16", "bf16", "f16", "f32"])
        V = _log(rng, 16, max(16, min(262144, (1 << 28) // H)))
        B = _log(rng, 1, 16)
        T = _log(rng, 1, max(1, min(8192, (1 << 26) // (B * H))))
        c = _emb("", dir, B, T, V, H, rng.choice([act, "f32"]), act, rng.random() < 0.5,
                 rng.choice([0.0, 0.0, 0.1, 0.5]), id64)
    else:
        op = rng.choice(["sort", "dispatch", "combine", "combine"])
        dir = "fwd" if op == "sort" else rng.choice(["fwd", "bwd"])
        act = rng.choice(["bf16", "bf16", "f16", "f32"])
        E = _log(rng, 2, 384)
        K = min(E, rng.choice([1, 2, 4, 6, 8, 8]))
        if op == "sort":
            T, H = _log(rng, 1, 65536), 0
        else:
            T = _log(rng, 1, max(1, min(65536, (1 << 27) // (K * H))))
        c = _moe("", op, dir, T, K, E, H, act, rng.choice(["f32", act, "none"]),
                 rng.choice([1, 1, 8, 128]), rng.choice([0.0, 0.0, 0.05, 0.3]),
                 op == "combine" and rng.random() < 0.5, id64)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _scale(case):
    return math.sqrt(case["H"]) if case["scaled"] else 1.0


def _rows(case):
    """Rows of the sorted choices: room for every expert's start to be rounded
    up."""
    n, align = case["T"] * case["K"], case["align"]
    return (n + min(case["E"], n) * (align - 1)) // align * align


def _inputs(case, seed):
    """Everything a program holds before the call, made from the seed."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    act = DTYPES[case["act"]]
    itype = torch.int64 if case["id64"] else torch.int32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    if case["op"] == "embedding":
        B, T, V, H = case["B"], case["T"], case["V"], case["H"]
        # the r-th token in about 1/r of the text; ids grow with rarity, as vocabularies are built
        ids = torch.exp(uniform(B, T + 1).double() * math.log(V + 1)).long().sub_(1).clamp_(0, V - 1)
        if case["pad"]:  # sequences end early
            left = (1 - case["pad"] * 2 * uniform(B, 1)) * (T + 1)
            ids = torch.where(torch.arange(T + 1, device=DEV) < left, ids, 0)
        s = {"ids": ids.to(itype)[:, :-1]}  # the tokens without the last, which is a target only
        if case["dir"] == "fwd":
            s["table"] = normal(V, H).mul_(1 / math.sqrt(H)).to(DTYPES[case["table"]])
        else:
            s["dy"] = normal(B, T, H).to(act)
        return s
    T, K, E, H = case["T"], case["K"], case["E"], case["H"]
    # a router's choices: some experts are liked more
    score = 0.5 * normal(E) - torch.log(-torch.log(uniform(T, E).clamp_(1e-7, 1 - 1e-7)))
    score, experts = torch.topk(score, K, dim=1)
    if case["pad"]:  # tokens of padding go to no expert
        experts = torch.where(uniform(T, 1) < case["pad"], -1, experts)
    s = {"experts": experts.to(itype)}
    if case["op"] == "sort":
        return s
    R = _rows(case)
    s["position"], s["source"] = _sort_plain(s["experts"], E, case["align"], R)[:2]
    fwd = case["dir"] == "fwd"
    if case["op"] == "dispatch":
        s.update(x=normal(T, H).to(act)) if fwd else s.update(dy=normal(R, H).to(act))
        return s
    s["rows"] = normal(R, H).to(act)
    if case["weight"] != "none":
        s["weights"] = torch.softmax(score, 1).to(DTYPES[case["weight"]])
    if fwd:
        if case["residual"]:
            s["residual"] = normal(T, H).to(act)
    else:
        s["dy"] = normal(T, H).to(act)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------- plain forms
def _emb_fwd_plain(s):
    c = s["case"]
    return (s["table"][s["ids"].long()].float() * _scale(c)).to(DTYPES[c["act"]])


def _padding(case):
    """The row that gets no gradient."""
    return 0 if case["pad"] else None


def _emb_bwd_plain(s):
    c = s["case"]
    grad = torch.zeros(c["V"], c["H"], device=DEV)
    grad.index_add_(0, s["ids"].reshape(-1).long(), s["dy"].reshape(-1, c["H"]).float())
    grad *= _scale(c)
    if _padding(c) is not None:
        grad[_padding(c)] = 0
    return grad.to(DTYPES[c["table"]])


def _sort_plain(experts, E, align, R):
    flat = experts.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    ordered, order = torch.sort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    counts.index_add_(0, key, torch.ones_like(key))
    counts = counts[:E]
    room = (counts + (align - 1)) // align * align
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(room, 0)
    packed = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    packed[1:] = torch.cumsum(counts, 0)
    row = torch.arange(n, device=DEV) - packed[ordered] + offsets[ordered]
    row = torch.where(ordered < E, row, R)
    source = torch.full((R + 1,), -1, dtype=torch.int32, device=DEV)
    source[row] = order.int()
    position = torch.empty(n, dtype=torch.int32, device=DEV)
    position[order] = torch.where(row < R, row, -1).int()
    return position.view(experts.shape), source[:R], offsets.int(), counts.int()


def _dispatch_fwd_plain(s):
    source = s["source"].long()
    rows = s["x"][source.clamp(min=0) // s["case"]["K"]].float()
    return torch.where(source[:, None] >= 0, rows, 0).to(s["x"].dtype)


def _gathered(rows, position):
    """rows [R, H] by position [T, K] in 32 bits, zeros for choices dropped."""
    p = position.long()
    if rows.shape[0] == 0:
        return torch.zeros(*p.shape, rows.shape[1], device=DEV)
    return torch.where(p[..., None] >= 0, rows[p.clamp(min=0)].float(), 0)


def _dispatch_bwd_plain(s):
    return _gathered(s["dy"], s["position"]).sum(1).to(s["dy"].dtype)


def _combine_fwd_plain(s):
    y = _gathered(s["rows"], s["position"])
    if "weights" in s:
        y = y * s["weights"].float()[..., None]
    y = y.sum(1)
    if "residual" in s:
        y = y + s["residual"].float()
    return y.to(s["rows"].dtype)


def _combine_bwd_plain(s):
    K = s["case"]["K"]
    source = s["source"].long()
    at = source.clamp(min=0)
    dy = s["dy"].float()
    drows = dy[at // K]
    if "weights" in s:
        drows = drows * s["weights"].float().reshape(-1)[at][:, None]
    drows = torch.where(source[:, None] >= 0, drows, 0).to(s["rows"].dtype)
    if "weights" not in s:
        return drows
    return drows, (dy[:, None, :] * _gathered(s["rows"], s["position"])).sum(-1)


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "sort":
            return _sort_plain(s["experts"], c["E"], c["align"], _rows(c))
        return {("embedding", "fwd"): _emb_fwd_plain, ("embedding", "bwd"): _emb_bwd_plain,
                ("dispatch", "fwd"): _dispatch_fwd_plain, ("dispatch", "bwd"): _dispatch_bwd_plain,
                ("combine", "fwd"): _combine_fwd_plain, ("combine", "bwd"): _combine_bwd_plain
                }[c["op"], c["dir"]](s)
    import memory_bound_normalization_gb300 as rn

    fwd = c["dir"] == "fwd"
    if c["op"] == "embedding":
        if fwd:
            return rn.embedding_forward(s["ids"], s["table"], scale=_scale(c),
                                        out_dtype=DTYPES[c["act"]])
        return rn.embedding_backward(s["ids"], s["dy"], c["V"], scale=_scale(c),
                                     padding_idx=_padding(c), grad_dtype=DTYPES[c["table"]])
    if c["op"] == "sort":
        return tuple(rn.expert_sort(s["experts"], c["E"], align=c["align"]))
    if c["op"] == "dispatch":
        if fwd:
            return rn.expert_dispatch_forward(s["x"], s["position"], s["source"])
        return rn.expert_dispatch_backward(s["dy"], s["position"])
    if fwd:
        return rn.expert_combine_forward(s["rows"], s["position"], s.get("weights"),
                                         s.get("residual"))
    out = rn.expert_combine_backward(s["dy"], s["rows"], s["position"], s["source"],
                                     s.get("weights"))
    return out if "weights" in s else out[0]


# --------------------------------------------------------------- 64 bits
def _exact_sort(experts, E, align, R):
    """Expert by expert, on the host."""
    flat = experts.reshape(-1).cpu().numpy()
    position = np.full(flat.size, -1, np.int32)
    source = np.full(R, -1, np.int32)
    offsets, counts, at = [0], [], 0
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        source[at:at + mine.size] = mine
        position[mine] = np.arange(at, at + mine.size)
        counts.append(mine.size)
        at += -(-mine.size // align) * align
        offsets.append(at)
    return tuple(torch.tensor(np.asarray(a, np.int32), device=DEV) for a in
                 (position.reshape(tuple(experts.shape)), source, offsets, counts))


def exact(case, seed):
    s = _inputs(case, seed)
    bwd = case["dir"] == "bwd"
    if case["op"] == "embedding":
        scale, ids = _scale(case), s["ids"].long()
        if not bwd:
            return torch.index_select(s["table"], 0, ids.flatten()).double().mul(scale).view(
                *ids.shape, case["H"])
        table = torch.zeros(case["V"], case["H"], dtype=torch.float64, device=DEV,
                            requires_grad=True)
        ((table[ids] * scale) * s["dy"].double()).sum().backward()
        grad = table.grad
        if _padding(case) is not None:
            grad[_padding(case)] = 0
        return grad
    T, K, E, H = case["T"], case["K"], case["E"], case["H"]
    if case["op"] == "sort":
        return _exact_sort(s["experts"], E, case["align"], _rows(case))
    R = s["source"].numel()
    position = s["position"].long()
    # choice by choice: row R is a row of nothing
    place = torch.where(position < 0, R, position)
    if case["op"] == "dispatch":
        if not bwd:
            rows = torch.zeros(R + 1, H, dtype=torch.float64, device=DEV)
            for k in range(K):
                rows[place[:, k]] = s["x"].double()
            return rows[:R]
        dx = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        rows = torch.cat((s["dy"], torch.zeros(1, H, dtype=s["dy"].dtype, device=DEV)))
        for k in range(K):
            dx += rows[place[:, k]]
        return dx
    w = s.get("weights")
    w = torch.ones(T, K, dtype=torch.float64, device=DEV) if w is None else w.double()
    out, drows = [], torch.zeros(R + 1, H, dtype=torch.float64, device=DEV) if bwd else None
    step = max(1, (1 << 26) // max(1, K * H))
    nothing = torch.zeros(1, H, dtype=s["rows"].dtype, device=DEV)
    padded = torch.cat((s["rows"], nothing))
    for i in range(0, T, step):
        p = place[i:i + step]
        mine = padded[p].double().requires_grad_(bwd)
        share = w[i:i + step].clone().requires_grad_(bwd)
        y = torch.einsum("tk,tkh->th", share, mine)
        if not bwd:
            out.append(y + s["residual"][i:i + step].double() if "residual" in s else y)
            continue
        y.backward(s["dy"][i:i + step].double())
        drows[p.flatten()] = mine.grad.flatten(0, 1)
        out.append(share.grad)
    if not bwd:
        return torch.cat(out)
    return (drows[:R], torch.cat(out)) if "weights" in s else drows[:R]


# --------------------------------------------------------------- floors
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    act, ids = size[case["act"]], 8 if case["id64"] else 4
    bwd, H = case["dir"] == "bwd", case["H"]
    if case["op"] == "embedding":
        n, V, table = case["B"] * case["T"], case["V"], size[case["table"]]
        live = n * (1 - case["pad"])
        if bwd:  # padding's rows need not be read
            return {"bytes": n * ids + live * H * act + V * H * table, "flops": live * H}
        # the rows that are hit at least once, on average
        r = np.arange(1, V + 1)
        p = np.log1p(1 / r) / math.log(V + 1)
        hit = float((1 - np.exp(live * np.log1p(-np.minimum(p, 0.999999)))).sum())
        return {"bytes": n * ids + hit * H * table + n * H * act, "flops": n * H}
    n, R, T = case["T"] * case["K"], _rows(case), case["T"]
    if case["op"] == "sort":
        return {"bytes": n * ids + 4 * (n + R + 2 * case["E"] + 1), "flops": n}
    live = n * (1 - case["pad"])
    weights = 0 if case["weight"] == "none" else n * size[case["weight"]]
    if case["op"] == "dispatch":
        if bwd:
            return {"bytes": 4 * n + (live + T) * H * act, "flops": live * H}
        return {"bytes": 4 * (n + R) + (T * (1 - case["pad"]) + R) * H * act, "flops": 0}
    if not bwd:
        rows = live + T * (2 if case["residual"] else 1)
        return {"bytes": 4 * n + weights + rows * H * act, "flops": 2 * live * H}
    if case["weight"] == "none":
        return {"bytes": 4 * (n + R) + (T * (1 - case["pad"]) + R) * H * act, "flops": 0}
    return {"bytes": 4 * (n + R) + weights + 4 * n + (T * (1 - case["pad"]) + live + R) * H * act,
            "flops": 3 * live * H}
