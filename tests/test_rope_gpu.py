"""QK-norm with rotary positions of several axes against 64-bit references on
the CPU, through the tensor-level calls, the C ABI and autograd."""
from __future__ import annotations

import threading

import pytest
import torch

import image_ref as ref

pytestmark = pytest.mark.gpu

pkg = pytest.importorskip("memory_bound_normalization_gb300")

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    pkg.load_library(build_if_missing=True)
    yield


@pytest.fixture(autouse=True)
def _status():
    yield
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK


def make(lead, Hq, Hk, D, sections, dtype, w_dtype, seed=0, far=5000, pos_dtype=torch.int64):
    g = torch.Generator().manual_seed(seed + 11)
    q = torch.randn(*lead, Hq, D, generator=g).to(dtype).to(DEV)
    k = torch.randn(*lead, Hk, D, generator=g).to(dtype).to(DEV) if Hk else None
    wq = wk = None
    if w_dtype is not None:
        wq = (1 + 0.1 * torch.randn(D, generator=g)).to(w_dtype).to(DEV)
        wk = (1 + 0.1 * torch.randn(D, generator=g)).to(w_dtype).to(DEV) if Hk else None
    pos = torch.randint(0, far, (len(sections), *lead), generator=g).to(pos_dtype).to(DEV)
    half = sum(sections)
    freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEV)
    dq = torch.randn(*lead, Hq, D, generator=g).to(dtype).to(DEV)
    dk = torch.randn(*lead, Hk, D, generator=g).to(dtype).to(DEV) if Hk else None
    return dict(q=q, k=k, wq=wq, wk=wk, positions=pos, inv_freq=freq, sections=sections), dq, dk


def verify(a, dq, dk, interleaved=False, adjacent=False, eps=1e-6):
    style = dict(interleaved=interleaved, adjacent=adjacent, eps=eps)
    qo, ko = pkg.qk_rope_forward(**a, **style)
    gq, gk, gwq, gwk = pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk, **style)
    torch.cuda.synchronize()
    assert pkg.rmsnorm_get_last_device_error() == pkg.OK
    check(a, qo, ko, dq, dk, gq, gk, gwq, gwk, **style)
    return qo, ko, gq, gk, gwq, gwk


def check(a, qo, ko, dq, dk, gq, gk, gwq, gwk, interleaved, adjacent, eps):
    lead, rot = tuple(a["q"].shape[:-2]), 2 * sum(a["sections"])
    cos, sin = ref.angles(a["positions"], a["inv_freq"], a["sections"], interleaved, lead)
    for name, x, w, y, dy, dx, dw in (("q", a["q"], a["wq"], qo, dq, gq, gwq),
                                      ("k", a["k"], a["wk"], ko, dk, gk, gwk)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        ref.check_rope(x, w, cos, sin, rot, adjacent, eps, y, name)
        ref.check_rope_grads(x, w, cos, sin, rot, adjacent, eps, dy, dx, dw, name)
        assert (dw is None) == (w is None)


TYPES = [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32), (BF16, None), (F32, None)]
TYPE_IDS = ["bf16", "bf16_wf32", "f16", "f16_wf32", "f32", "bf16_rot", "f32_rot"]
# (lead, Hq, Hk, D, sections): one token, heads shared or alone, no keys, parts
# of the head rotated, widths that no 16-byte piece fits, four axes, an axis
# without pairs, the widest head
CASES = [((1,), 1, 1, 128, (16, 24, 24)), ((1, 1), 32, 8, 128, (16, 24, 24)),
         ((8, 1), 32, 8, 128, (64,)), ((3, 41), 6, 2, 64, (8, 12, 12)), ((77,), 5, 0, 128, (32, 32)),
         ((2, 19), 16, 16, 80, (20, 20)), ((50,), 3, 1, 72, (18, 18)), ((2, 33), 4, 2, 96, (12, 10, 10)),
         ((29,), 2, 1, 256, (40, 44, 44)), ((2, 9), 3, 2, 256, (1, 2, 3, 4)), ((13,), 2, 2, 2, (1,)),
         ((17,), 3, 1, 6, (0, 2)), ((11,), 2, 1, 50, (12, 11)), ((7,), 1, 1, 254, (127,)),
         ((5, 100), 12, 12, 64, (10, 0, 22)), ((600,), 8, 1, 32, (4, 4, 4, 4))]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{'x'.join(map(str, c[0]))}_{c[1]}_{c[2]}_{c[3]}_{len(c[4])}")
@pytest.mark.parametrize("dtype,w_dtype", TYPES, ids=TYPE_IDS)
def test_matches(case, dtype, w_dtype):
    a, dq, dk = make(*case, dtype, w_dtype)
    verify(a, dq, dk)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype,w_dtype", [(BF16, BF16), (F32, F32), (F16, None)],
                         ids=["bf16", "f32", "f16_rot"])
@pytest.mark.parametrize("D,sections", [(128, (24, 20, 20)), (96, (12, 10, 10)), (80, (5, 30)),
                                        (36, (3, 6)), (10, (2, 1))])
def test_pair_orders(interleaved, adjacent, dtype, w_dtype, D, sections):
    a, dq, dk = make((2, 21), 4, 2, D, sections, dtype, w_dtype, seed=3, pos_dtype=torch.int32)
    verify(a, dq, dk, interleaved, adjacent)


@pytest.mark.parametrize("pos_dtype", [torch.int32, torch.int64])
def test_far_and_negative_positions(pos_dtype):
    a, dq, dk = make((40,), 2, 1, 64, (8, 12, 12), F32, F32, pos_dtype=pos_dtype)
    far = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, (1 << 24) + 1, 123456789])
    a["positions"] = far.repeat(15).view(3, 40).to(pos_dtype).to(DEV)
    a["inv_freq"][0] = 1.5
    a["inv_freq"][1] = -0.7
    a["inv_freq"][2] = 0.0
    a["inv_freq"][3] = 1e-30
    a["inv_freq"][4] = 300.25
    verify(a, dq, dk)


def test_frequency_without_a_value():
    """An infinite or NaN frequency makes its own pairs NaN and no others."""
    a, dq, dk = make((4,), 2, 1, 16, (4, 4), F32, None)
    want, _ = pkg.qk_rope_forward(**a)
    a["inv_freq"][1] = float("inf")
    a["inv_freq"][6] = float("nan")
    got, _ = pkg.qk_rope_forward(**a)
    sick = torch.zeros(16, dtype=torch.bool, device=DEV)
    sick[[1, 9, 6, 14]] = True
    assert got[..., sick].isnan().all() and torch.equal(got[..., ~sick], want[..., ~sick])


def test_rows_with_nan_inf_or_zeros():
    a, dq, dk = make((20,), 3, 1, 128, (32, 32), F32, F32)
    want = pkg.qk_rope_forward(**a)[0]
    a["q"][3, 1, 5] = float("nan")
    a["q"][7, 2, 9] = float("inf")
    a["q"][9] = 0
    got = pkg.qk_rope_forward(**a)[0]
    keep = torch.ones(20, 3, dtype=torch.bool, device=DEV)
    keep[3, 1] = keep[7, 2] = False
    keep[9] = False
    assert torch.equal(got[keep], want[keep])
    assert got[3, 1].isnan().all() and got[7, 2].isnan().any() and not got[9].any()
    dq_, *_ = pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk)
    assert dq_[9].isfinite().all() and dq_[keep].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_views_of_one_projection(dtype):
    B, T, Hq, Hk, D = 2, 30, 4, 2, 64
    a, dq, dk = make((B, T), Hq, Hk, D, (8, 12, 12), dtype, F32)
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=g).to(dtype).to(DEV)
    a["q"] = qkv[..., :Hq * D].view(B, T, Hq, D)
    a["k"] = qkv[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)
    verify(a, dq, dk)
    # heads before tokens, a cache slice, and an odd start
    heads_first = torch.randn(B, Hq, T, D, generator=g).to(dtype).to(DEV).transpose(1, 2)
    a["q"] = heads_first
    a["k"] = torch.randn(B, 50, Hk, D + 3, generator=g).to(dtype).to(DEV)[:, 7:7 + T, :, 1:1 + D]
    strided = torch.randn(B, Hq, T, D, generator=g).to(dtype).to(DEV).transpose(1, 2)
    verify(a, strided, dk)


def test_broadcast_inputs_and_positions():
    a, dq, dk = make((3, 16), 4, 2, 64, (8, 12, 12), BF16, F32)
    a["positions"] = a["positions"][:, 0].contiguous()  # shared by the batch
    verify(a, dq, dk)
    a["positions"] = torch.arange(16, device=DEV).expand(3, 16)  # the axes alike
    verify(a, dq, dk)
    a["positions"] = torch.arange(48, device=DEV).view(16, 3).t()  # strided
    verify(a, dq, dk)
    a["q"] = a["q"][:, :, :1].expand(3, 16, 4, 64)
    verify(a, dq, dk)


@pytest.mark.parametrize("dtype,w_dtype", [(BF16, BF16), (F32, None), (F16, F32)])
def test_in_place(dtype, w_dtype):
    a, dq, dk = make((2, 70), 8, 2, 128, (16, 24, 24), dtype, w_dtype)
    want = pkg.qk_rope_forward(**a)
    q, k = a["q"].clone(), a["k"].clone()
    got = pkg.qk_rope_forward(**{**a, "q": q, "k": k}, out=(q, k))
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_keys_into_a_cache_slice():
    """k_out lands in its slots; the rows around them stay as they were."""
    a, dq, dk = make((2, 3), 4, 2, 64, (8, 12, 12), BF16, BF16)
    want = pkg.qk_rope_forward(**a)
    cache = torch.full((2, 20, 2, 64), 5.0, dtype=BF16, device=DEV)
    qo = torch.empty_like(a["q"])
    pkg.qk_rope_forward(**a, out=(qo, cache[:, 9:12]))
    assert torch.equal(cache[:, 9:12], want[1]) and torch.equal(qo, want[0])
    assert (cache[:, :9] == 5).all() and (cache[:, 12:] == 5).all()


@pytest.mark.parametrize("offset", [1, 3, 4])
def test_guard_bands_and_alignment(offset):
    a, dq, dk = make((37,), 3, 1, 64, (16, 16), BF16, BF16)
    want = pkg.qk_rope_forward(**a)
    n = a["q"].numel()
    src = torch.zeros(n + 64, dtype=BF16, device=DEV)
    src[offset:offset + n] = a["q"].flatten()
    buf = torch.full((n + 64,), 7.0, dtype=BF16, device=DEV)
    q = src[offset:offset + n].view_as(a["q"])
    out = buf[8 + offset:8 + offset + n].view_as(a["q"])
    pkg.qk_rope_forward(**{**a, "q": q}, out=(out, torch.empty_like(a["k"])))
    assert (buf[:8 + offset] == 7).all() and (buf[8 + offset + n:] == 7).all()
    cos, sin = ref.angles(a["positions"], a["inv_freq"], a["sections"], False, (37,))
    ref.check_rope(a["q"], a["wq"], cos, sin, 64, False, 1e-6, out, "q")
    assert (out.float() - want[0].float()).abs().max() < 0.05


def test_empty():
    a, dq, dk = make((0,), 3, 1, 64, (16, 16), F32, F32)
    qo, ko = pkg.qk_rope_forward(**a)
    assert qo.shape == a["q"].shape
    _, _, dwq, dwk = pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk)
    assert not dwq.any() and not dwk.any()
    a, dq, dk = make((5,), 0, 2, 64, (16, 16), F32, F32)  # keys alone
    qo, ko = pkg.qk_rope_forward(**a)
    cos, sin = ref.angles(a["positions"], a["inv_freq"], a["sections"], False, (5,))
    ref.check_rope(a["k"], a["wk"], cos, sin, 64, False, 1e-6, ko, "k")
    gq, gk, _, dwk = pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk)
    ref.check_rope_grads(a["k"], a["wk"], cos, sin, 64, False, 1e-6, dk, gk, dwk, "k")


@pytest.mark.parametrize("case", [((2, 3000), 16, 4, 128, (16, 24, 24)),
                                  ((1, 4099), 16, 16, 80, (20, 20)), ((9000,), 2, 1, 64, (32,))])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_full_size(case, dtype):
    a, dq, dk = make(*case, dtype, F32)
    verify(a, dq, dk)


def test_bitwise_repeatable():
    a, dq, dk = make((2, 1500), 16, 4, 128, (16, 24, 24), BF16, F32)
    runs = [(*pkg.qk_rope_forward(**a), *pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk))
            for _ in range(10)]
    for r in runs[1:]:
        for x, y in zip(runs[0], r):
            assert torch.equal(x, y)


def test_full_size_offsets_past_32_bits():
    """A batch stride past 2^31 elements: the far sample is read and written."""
    D, stride = 64, (1 << 31) + 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    a, dq, dk = make((2, 3), 2, 1, D, (16, 16), BF16, BF16)
    small = pkg.qk_rope_forward(**a)
    wide = torch.empty(stride + 3 * 2 * D, dtype=BF16, device=DEV)
    view = wide.as_strided((2, 3, 2, D), (stride, 2 * D, D, 1))
    view.copy_(a["q"])
    out = torch.empty_like(wide)
    ov = out.as_strided((2, 3, 2, D), (stride, 2 * D, D, 1))
    ko = torch.empty_like(a["k"])
    pkg.qk_rope_forward(**{**a, "q": view}, out=(ov, ko))
    assert torch.equal(ov, small[0]) and torch.equal(ko, small[1])
    got = pkg.qk_rope_backward(**{**a, "q": view}, dq_out=ov, dk_out=ko)
    want = pkg.qk_rope_backward(**a, dq_out=small[0], dk_out=small[1])
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_streams_and_threads():
    cases = [((8, 1), 32, 8, 128, (16, 24, 24)), ((2, 2000), 8, 2, 128, (64,)),
             ((500,), 3, 1, 72, (18, 18))]
    made = [make(*c, BF16, F32, seed=i) for i, c in enumerate(cases)]

    def step(i):
        a, dq, dk = made[i]
        return (*pkg.qk_rope_forward(**a), *pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk))

    alone = [step(i) for i in range(len(cases))]
    torch.cuda.synchronize()
    got, failed = {}, []

    def worker(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[i] = [step(i) for _ in range(8)]
            s.synchronize()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed, failed
    for i, want in enumerate(alone):
        for r in got[i]:
            for x, y in zip(want, r):
                assert torch.equal(x, y)


def test_captured_and_replayed():
    a, dq, dk = make((4, 50), 8, 2, 128, (16, 24, 24), BF16, BF16)

    def step():
        return (*pkg.qk_rope_forward(**a), *pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk))

    want = step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(s):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        for x, y in zip(want, out):
            assert torch.equal(x, y)
    a["q"].mul_(2).add_(0.5)
    a["positions"].add_(3)
    want = step()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    for x, y in zip(want, graphs[1][1]):
        assert torch.equal(x, y)


def test_autograd():
    from memory_bound_normalization_gb300.autograd import QKNormRope, qk_norm_rope

    a, dq, dk = make((2, 20), 4, 2, 64, (8, 12, 12), BF16, BF16)
    leaf = {n: a[n].clone().requires_grad_(True) for n in ("q", "k", "wq", "wk")}
    qo, ko = qk_norm_rope(**leaf, positions=a["positions"], inv_freq=a["inv_freq"],
                          sections=a["sections"], interleaved=True)
    (qo.float() * dq.float()).sum().backward(retain_graph=True)  # the keys are not used
    (ko.float() * dk.float()).sum().backward()
    want = pkg.qk_rope_forward(**a, interleaved=True)
    grads = pkg.qk_rope_backward(**a, dq_out=dq, dk_out=dk, interleaved=True)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    for n, g in zip(("q", "k", "wq", "wk"), grads):
        assert torch.equal(leaf[n].grad, g.to(BF16)), n
    layer = QKNormRope(64, (8, 12, 12), device=DEV).to(BF16)
    assert layer.inv_freq.dtype == torch.float32 and layer.q_weight.dtype == BF16
    assert torch.equal(layer.inv_freq, a["inv_freq"])
    q1, k1 = layer(a["q"], a["k"], a["positions"])
    one = torch.ones(64, dtype=BF16, device=DEV)
    w1 = pkg.qk_rope_forward(**{**a, "wq": one, "wk": one})
    assert torch.equal(q1, w1[0]) and torch.equal(k1, w1[1])
    rot = QKNormRope(64, (8, 12, 12), norm=False, device=DEV)
    x = a["q"].transpose(2, 3).contiguous().transpose(2, 3).requires_grad_(True)  # heads not dense
    q2, k2 = rot(x, None, a["positions"])
    assert k2 is None and not list(rot.parameters())
    q2.sum().backward()
    # turning back a gradient of ones
    back = pkg.qk_rope_backward(a["q"], None, None, None, a["positions"], a["inv_freq"],
                                a["sections"], torch.ones_like(a["q"]), None)
    assert torch.equal(x.grad, back[0]) and back[1:] == (None, None, None)
