"""The measured calls of the image and video operators: group norm with an
activation on channels-last tensors, and the query/key norm with rotary
positions of several axes, forward and backward.

Each case is one call of a direction of one operator. `run` computes it in its
plain form (elementary torch operations in 32 bits, rounded once at the end)
or, with `own` set, through the library's entry points; `exact` computes the
definition in 64 bits, gradients by differentiating the forward.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


def _gn(name, dir, B, S, C, G, dtype, wdtype, act):
    return {"name": name, "op": "group_norm", "dir": dir, "B": B, "S": S, "C": C, "G": G,
            "dtype": dtype, "wdtype": wdtype, "act": act, "eps": 1e-5}


def _rope(name, dir, B, T, Hq, Hk, D, rot, sections, dtype, wdtype, interleaved, adjacent, norm,
          pos64):
    return {"name": name, "op": "qk_rope", "dir": dir, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D,
            "rot": rot, "sections": sections, "dtype": dtype, "wdtype": wdtype,
            "interleaved": interleaved, "adjacent": adjacent, "norm": norm, "pos64": pos64,
            "eps": 1e-6}


def listed():
    return [
        # the bottom level of an image denoiser, two samples of 8 x 8: latency counts
        _gn("gn_fwd_bottom", "fwd", 2, 64, 1280, 32, "bf16", "bf16", "silu"),
        # a top level of the same network: ten channels a group, so groups end inside 16 bytes
        _gn("gn_fwd_top", "fwd", 4, 4096, 320, 32, "f16", "f32", "silu"),
        # the last level of a latent decoder on one 1024 x 1024 image: one slab past the L2
        _gn("gn_fwd_decoder", "fwd", 1, 1024 * 1024, 128, 32, "bf16", "bf16", "silu"),
        # the training step of a middle level, 32 x 32
        _gn("gn_bwd_middle", "bwd", 8, 1024, 640, 32, "bf16", "f32", "silu"),
        # the training step of a decoder level on two 512 x 512 images: the largest here
        _gn("gn_bwd_decoder", "bwd", 2, 512 * 512, 256, 32, "bf16", "bf16", "silu"),
        # an odd picture in fp32, no activation, 20 channels a group
        _gn("gn_bwd_odd", "bwd", 3, 61 * 47, 100, 5, "f32", "f32", "none"),
        # one new token of eight requests: latency counts
        _rope("rope_fwd_decode", "fwd", 8, 1, 32, 8, 128, 128, "16,24,24", "bf16", "bf16", False,
              False, True, True),
        # a prompt of text and video, q and k as views of one projection
        _rope("rope_fwd_prompt", "fwd", 4, 4096, 32, 8, 128, 128, "16,24,24", "bf16", "bf16",
              False, False, True, True),
        # a vision encoder: no norm, two axes, heads of 80, an odd number of patches
        _rope("rope_fwd_vision", "fwd", 1, 4099, 16, 16, 80, 80, "20,20", "f16", "f16", False,
              False, False, False),
        # the training step of the QK-norm workload (8 x 4096 tokens, 32 heads of 128)
        _rope("rope_bwd_train", "bwd", 8, 4096, 32, 8, 128, 128, "24,20,20", "bf16", "f32", True,
              False, True, True),
        # a short training step in fp32, part of the head rotated, adjacent pairs
        _rope("rope_bwd_part", "bwd", 3, 341, 12, 12, 96, 64, "12,10,10", "f32", "f32", True, True,
              True, False),
        # gradients of the vision encoder's rotation
        _rope("rope_bwd_vision", "bwd", 1, 4099, 16, 16, 80, 80, "20,20", "f16", "f16", False,
              False, False, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    wdtype = rng.choice([dtype, "f32"])
    dir = rng.choice(["fwd", "bwd"])
    if rng.random() < 0.5:
        G = rng.choice([8, 16, 32])
        C = G * _log(rng, 2, 40)
        B = _log(rng, 1, 16)
        S = _log(rng, 16, max(16, min(1 << 20, (1 << 26) // (B * C))))
        act = rng.choice(["silu", "silu", "gelu", "none"])
        c = _gn("", dir, B, S, C, G, dtype, wdtype, act)
    else:
        D = rng.choice([64, 80, 96, 128, 128, 256])
        rot = D if rng.random() < 0.7 else D // 2
        half = rot // 2
        axes = rng.choice([1, 2, 3, 3])
        cuts = sorted(rng.sample(range(1, half), axes - 1))
        sections = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half]))
        Hk = rng.choice([1, 2, 4, 8, 16])
        Hq = Hk * rng.choice([1, 2, 4])
        B = _log(rng, 1, 8)
        T = _log(rng, 1, max(1, min(32768, (1 << 26) // (B * (Hq + Hk) * D))))
        c = _rope("", dir, B, T, Hq, Hk, D, rot, sections, dtype, wdtype, rng.random() < 0.5,
                  rng.random() < 0.3, rng.random() < 0.75, rng.random() < 0.5)
    del c["name"]
    return c


def _sections(case):
    return tuple(int(v) for v in case["sections"].split(","))


def _inputs(case, seed):
    """Everything a program holds before the call, made from the seed."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, wdt = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if case["op"] == "group_norm":
        B, S, C = case["B"], case["S"], case["C"]
        x = normal(B, S, C)
        # channels of a convolution's output have their own scale and offset
        x = x.mul_(1 + 0.3 * normal(C)).add_(0.5 * normal(C)).to(dt)
        s = {"x": x, "w": (1 + 0.1 * normal(C)).to(wdt), "b": (0.1 * normal(C)).to(wdt)}
        if case["dir"] == "bwd":
            s["dy"] = normal(B, S, C).to(dt)
        return s
    B, T, Hq, Hk, D = (case[k] for k in ("B", "T", "Hq", "Hk", "D"))
    qkv = normal(B, T, (Hq + 2 * Hk) * D).to(dt)
    s = {"q": qkv[..., :Hq * D].view(B, T, Hq, D),
         "k": qkv[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)}
    if case["norm"]:
        s["wq"] = (1 + 0.1 * normal(D)).to(wdt)
        s["wk"] = (1 + 0.1 * normal(D)).to(wdt)
    # text tokens count on every axis alike; then frames of pictures, row by row
    axes = len(_sections(case))
    start = torch.randint(0, 4096, (B, 1), generator=gen, device=DEV)
    i = torch.arange(T, device=DEV).expand(B, T)
    text, width = T // 4, max(1, math.isqrt(max(1, T // 4)))
    j = (i - text).clamp(min=0)
    grid = (j // (width * width), j // width % width, j % width)
    pos = torch.stack([start + torch.where(i < text, i, text + grid[a % 3])
                       for a in range(axes)])
    s["pos"] = pos.to(torch.int64 if case["pos64"] else torch.int32)
    half = case["rot"] // 2
    s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
                     ).float()
    if case["dir"] == "bwd":
        s["dq"] = normal(B, T, Hq, D).to(dt)
        s["dk"] = normal(B, T, Hk, D).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "group_norm":
        if case["dir"] == "bwd":  # the statistics that the forward returned
            x = s["x"].view(case["B"], case["S"], case["G"], -1).double()
            s["mean"] = x.mean((1, 3)).float()
            s["rstd"] = (x.var((1, 3), unbiased=False) + case["eps"]).rsqrt().float()
    else:
        s["sections"] = _sections(case)
    return s


# ------------------------------------------------------------- plain forms
def _affine(s, v):
    """A channel vector over [1, 1, G, C/G], in 32 bits."""
    c = s["case"]
    return v.float().view(1, 1, c["G"], c["C"] // c["G"])


def _gn_fwd_plain(s):
    c = s["case"]
    x = s["x"].float().view(c["B"], c["S"], c["G"], -1)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean((1, 3), keepdim=True) + c["eps"])
    z = d * rstd * _affine(s, s["w"]) + _affine(s, s["b"])
    if c["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    elif c["act"] == "gelu":
        z = 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return (z.view(s["x"].shape).to(s["x"].dtype), mean.view(c["B"], c["G"]),
            rstd.view(c["B"], c["G"]))


def _gn_bwd_plain(s):
    c = s["case"]
    shape = (c["B"], 1, c["G"], 1)
    rstd = s["rstd"].view(shape)
    xhat = (s["x"].float().view(c["B"], c["S"], c["G"], -1) - s["mean"].view(shape)) * rstd
    w = _affine(s, s["w"])
    dz = s["dy"].float().view(xhat.shape)
    if c["act"] != "none":
        z = xhat * w + _affine(s, s["b"])
        if c["act"] == "silu":
            sig = 1 / (1 + torch.exp(-z))
            dz = dz * (sig * (1 + z * (1 - sig)))
        else:
            dz = dz * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) +
                       z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    g = dz * w
    dx = (g - g.mean((1, 3), keepdim=True) - xhat * (g * xhat).mean((1, 3), keepdim=True)) * rstd
    return (dx.view(s["x"].shape).to(s["x"].dtype), (dz * xhat).sum((0, 1)).view(-1),
            dz.sum((0, 1)).view(-1))


def _angles(s):
    """cos and sin [B, T, 1, pairs] of position x inverse frequency; the
    product in 64 bits, since a far position leaves 32 too few for the angle."""
    c = s["case"]
    half, sections = c["rot"] // 2, s["sections"]
    axis = torch.repeat_interleave(torch.arange(len(sections), device=DEV),
                                   torch.tensor(sections, device=DEV), output_size=half)
    if c["interleaved"]:  # axes take pairs in turn while they have some left
        turn = torch.cat([torch.arange(n, device=DEV) for n in sections])
        axis = axis[torch.argsort(turn * len(sections) + axis)]
    p = s["pos"][axis].permute(1, 2, 0).double()
    theta = (p * s["inv_freq"].double()).unsqueeze(2)
    return torch.cos(theta).float(), torch.sin(theta).float()


def _rotate(x, cos, sin, rot, adjacent):
    r, rest = x[..., :rot], x[..., rot:]
    if adjacent:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _rope_fwd_plain(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        n = x.float()
        if c["norm"]:
            n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + c["eps"]) * w.float()
        return _rotate(n, cos, sin, c["rot"], c["adjacent"]).to(x.dtype)

    return one(s["q"], s.get("wq")), one(s["k"], s.get("wk"))


def _rope_bwd_plain(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w, dy):
        g = _rotate(dy.float(), cos, -sin, c["rot"], c["adjacent"])
        if not c["norm"]:
            return (g.to(x.dtype),)
        f = x.float()
        rstd = torch.rsqrt((f * f).mean(-1, keepdim=True) + c["eps"])
        xhat = f * rstd
        gw = g * w.float()
        dx = (gw - xhat * (gw * xhat).mean(-1, keepdim=True)) * rstd
        return dx.to(x.dtype), (g * xhat).sum((0, 1, 2))

    q, k = one(s["q"], s.get("wq"), s["dq"]), one(s["k"], s.get("wk"), s["dk"])
    return (q[0], k[0]) + q[1:] + k[1:]


def run(s):
    c = s["case"]
    if not own:
        return {("group_norm", "fwd"): _gn_fwd_plain, ("group_norm", "bwd"): _gn_bwd_plain,
                ("qk_rope", "fwd"): _rope_fwd_plain, ("qk_rope", "bwd"): _rope_bwd_plain
                }[c["op"], c["dir"]](s)
    import memory_bound_normalization_gb300 as rn

    if c["op"] == "group_norm":
        if c["dir"] == "fwd":
            return rn.group_norm_forward(s["x"], c["G"], s["w"], s["b"], eps=c["eps"],
                                         activation=c["act"])
        return rn.group_norm_backward(s["x"], c["G"], s["w"], s["b"], s["dy"], s["mean"],
                                      s["rstd"], activation=c["act"])
    style = {"interleaved": c["interleaved"], "adjacent": c["adjacent"], "eps": c["eps"]}
    if c["dir"] == "fwd":
        return rn.qk_rope_forward(s["q"], s["k"], s.get("wq"), s.get("wk"), s["pos"],
                                  s["inv_freq"], s["sections"], **style)
    out = rn.qk_rope_backward(s["q"], s["k"], s.get("wq"), s.get("wk"), s["pos"], s["inv_freq"],
                              s["sections"], s["dq"], s["dk"], **style)
    return out if c["norm"] else out[:2]


# --------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    bwd = case["dir"] == "bwd"
    if case["op"] == "group_norm":
        B, S, C, G = case["B"], case["S"], case["C"], case["G"]
        w, b = (s[k].double().requires_grad_(bwd) for k in "wb")
        ys, dxs, means, rstds = [], [], [], []
        for i in range(B):  # a sample at a time: its groups as rows
            x = s["x"][i].double().requires_grad_(bwd)
            rows = x.t().reshape(G, C // G * S)
            var, mean = torch.var_mean(rows, 1, correction=0)
            scale = (var + case["eps"]).pow(-0.5)
            normed = ((rows - mean[:, None]) * scale[:, None]).reshape(C, S)
            y = torch.addcmul(b[:, None], normed, w[:, None]).t()
            if case["act"] == "silu":
                y = torch.sigmoid(y) * y
            elif case["act"] == "gelu":
                y = y * torch.special.ndtr(y)
            if bwd:
                y.backward(s["dy"][i].double())
                dxs.append(x.grad)
            else:
                ys.append(y)
                means.append(mean)
                rstds.append(scale)
        if bwd:
            return torch.stack(dxs), w.grad, b.grad
        return torch.stack(ys), torch.stack(means), torch.stack(rstds)

    axes = list(_sections(case))
    if case["interleaved"]:
        order, left = [], list(axes)
        while any(left):
            for a in range(len(axes)):
                if left[a]:
                    order.append(a)
                    left[a] -= 1
    else:
        order = [a for a in range(len(axes)) for _ in range(axes[a])]
    pos = s["pos"].double()
    turn = torch.stack([pos[a] for a in order], -1) * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(turn), turn)[:, :, None, :]
    rot, half = case["rot"], case["rot"] // 2
    out, dws = [], []
    for name in "qk":
        x = s[name].double().requires_grad_(bwd)
        n, w = x, None
        if case["norm"]:
            w = s["w" + name].double().requires_grad_(bwd)
            n = w * x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["D"] + case["eps"])
        if case["adjacent"]:
            z = torch.view_as_complex(n[..., :rot].unflatten(-1, (half, 2)).contiguous()) * turn
            y = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(n[..., :half], n[..., half:rot]) * turn
            y = torch.cat((z.real, z.imag), -1)
        y = torch.cat((y, n[..., rot:]), -1)
        if bwd:
            y.backward(s["d" + name].double())
            out.append(x.grad)
            if w is not None:
                dws.append(w.grad)
        else:
            out.append(y)
    return tuple(out + dws)


# --------------------------------------------------------------- floors
def work(case):
    size, wsize = (4 if case[k] == "f32" else 2 for k in ("dtype", "wdtype"))
    bwd = case["dir"] == "bwd"
    if case["op"] == "group_norm":
        n, C, stats = case["B"] * case["S"] * case["C"], case["C"], 2 * case["B"] * case["G"] * 4
        act = {"none": 0, "silu": 4, "gelu": 8}[case["act"]]
        return {"bytes": n * size * (3 if bwd else 2) + 2 * C * (wsize + (4 if bwd else 0)) + stats,
                "flops": n * ((14 + 2 * act) if bwd else (7 + act))}
    rows = case["B"] * case["T"] * (case["Hq"] + case["Hk"])
    D, half = case["D"], case["rot"] // 2
    tokens = case["B"] * case["T"] * len(_sections(case)) * (8 if case["pos64"] else 4)
    norm = case["norm"]
    tensors = (3 if norm else 2) if bwd else 2
    weights = 2 * D * (wsize + (4 if bwd else 0)) if norm else 0
    return {"bytes": rows * D * size * tensors + tokens + half * 4 + weights,
            "flops": rows * (6 * half + ((12 if bwd else 4) * D if norm else 0))}
