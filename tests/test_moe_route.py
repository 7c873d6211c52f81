"""The expert router and its gradient against their definitions in float64."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import experts as ref
from tests.helpers import announce
from tests.linear_helpers import f64, strided

INF = float("inf")

# Weights are computed in 64 bits and rounded once to fp32: half a step, 2^-24
# of the value, and 2^-150 below the normal range; the 64-bit steps are far
# below that.  Gradients round once to the logits' type; where terms cancel the
# 64-bit error is left, 1e-13 of the terms (|g| <= 16 here).
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(T, E, dtype, seed, masked=0.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * spread
    l[torch.rand(T, E, generator=g) < masked] = -INF
    return l.to(dtype)


def check_route(lib, logits, k, pad=0, **kw):
    bias = kw.pop("bias", None)
    T, E = logits.shape
    ids = torch.full((T + 1, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), 77.0, device="cuda")
    x = strided(logits, pad) if pad else logits.cuda()
    got = lib.moe_route(x, k, ids[:T], w[:T], bias=None if bias is None else bias.cuda(), **kw)
    want_ids, want_w = ref.route(f64(logits), k, bias=None if bias is None else bias.numpy(), **kw)
    assert np.array_equal(got[0].cpu().numpy(), want_ids)
    y = f64(got[1])
    with np.errstate(invalid="ignore"):
        ok = np.abs(y - want_w) <= 1.001 * 2.0 ** -24 * np.abs(want_w) + 2.0 ** -149
    assert (ok | (np.isnan(y) & np.isnan(want_w))).all(), (y[~ok], want_w[~ok])
    assert (ids[T] == 77).all() and (w[T] == 77).all()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, torch.float32), (1, 8, 8, torch.bfloat16), (5, 63, 4, torch.float32),
                                         (33, 64, 2, torch.bfloat16), (7, 65, 7, torch.float32), (130, 160, 6, torch.float32),
                                         (3, 256, 8, torch.bfloat16), (9, 384, 10, torch.float32), (4, 1000, 64, torch.float32),
                                         (2, 1024, 32, torch.bfloat16)])
def test_route(gpu_lib, T, E, k, dtype, scoring, normalize):
    announce(f"route {T}x{E} k={k} {scoring} {dtype}")
    for seed, kw in enumerate([{}, {"bias": True}, {"scale": 2.5, "pad": 3}]):
        l = make(T, E, dtype, seed)
        if kw.pop("bias", False):
            kw["bias"] = torch.randn(E, generator=torch.Generator().manual_seed(9)) * 0.2
        check_route(gpu_lib, l, k, scoring=scoring, normalize=normalize, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (256, 8, 8, 8), (64, 64, 5, 5), (60, 3, 1, 6), (60, 4, 2, 4),
                                            (384, 12, 3, 8), (1024, 2, 1, 12), (7, 7, 2, 4), (96, 33 // 11, 2, 5)])
def test_grouped_route(gpu_lib, scoring, E, groups, top, k):
    announce(f"route E={E} groups={groups}/{top} {scoring}")
    bias = torch.randn(E, generator=torch.Generator().manual_seed(4)) * 0.1
    for seed, masked in enumerate([0.0, 0.5, 0.95]):
        l = make(41, E, torch.float32, seed, masked)
        check_route(gpu_lib, l, k, bias=bias, scoring=scoring, groups=groups, top_groups=top)
        check_route(gpu_lib, l, k, scoring=scoring, groups=groups, top_groups=top, normalize=False)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_rows_that_masks_leave_short_or_empty(gpu_lib, scoring, biased):
    announce(f"route masked {scoring} bias={biased}")
    E, k = 70, 6
    l = make(8, E, torch.float32, 0)
    l[0] = -INF
    l[1, 1:] = -INF
    l[2, :66] = -INF
    l[3, 7:] = -INF
    l[4] = torch.finfo(torch.float32).min  # the lowest value is a candidate, and equal ones go by index
    l[5, :] = 0.25
    l[6, ::2] = torch.finfo(torch.float32).min
    bias = torch.zeros(E) if biased else None
    for norm in (True, False):
        ids, w = check_route(gpu_lib, l, k, bias=bias, scoring=scoring, normalize=norm)
        assert (ids[0] == -1).all() and (w[0] == 0).all()
        assert ids[1].tolist() == [0] + [-1] * 5
        assert ids[5].tolist() == list(range(k))
        check_route(gpu_lib, l, k, bias=bias, scoring=scoring, normalize=norm, groups=7, top_groups=2)
    if biased:
        bias[3:9] = -INF
        ids, _ = check_route(gpu_lib, l, k, bias=bias, scoring=scoring)
        assert not torch.isin(ids.cpu(), torch.arange(3, 9, dtype=torch.int32)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(gpu_lib, scoring):
    announce(f"route ties {scoring}")
    for E in (64, 200, 1024):
        l = torch.randint(-2, 3, (50, E), generator=torch.Generator().manual_seed(E)).float()
        for dtype in HALF:
            check_route(gpu_lib, l.to(dtype), min(E, 40), scoring=scoring)
            check_route(gpu_lib, l.to(dtype), 8, scoring=scoring, groups=4, top_groups=2)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_of_both_signs_are_equal(gpu_lib, scoring, dtype):
    """-0 and +0 are one logit: rows that mix them, as products with a 0/1 mask do, go by index."""
    announce(f"route zeros {scoring} {dtype}")
    ids, _ = check_route(gpu_lib, torch.tensor([[-0.0, 0.0, -1.0], [0.0, -0.0, -1.0], [-1.0, -0.0, 0.0]]).to(dtype), 1, scoring=scoring)
    assert ids[:, 0].tolist() == [0, 0, 1]
    for E in (64, 100, 1024):
        g = torch.Generator().manual_seed(E)
        l = torch.randn(30, E, generator=g) * (torch.rand(30, E, generator=g) < 0.3)  # zeros of either sign
        l[::2] = -l[::2].abs()  # zeros above all others
        assert (torch.signbit(l) & (l == 0)).any() and (~torch.signbit(l) & (l == 0)).any()
        for norm in (True, False):
            check_route(gpu_lib, l.to(dtype), min(E, 40), scoring=scoring, normalize=norm)
            check_route(gpu_lib, l.to(dtype), 7, scoring=scoring, normalize=norm, bias=torch.zeros(E) * -1.0)
            check_route(gpu_lib, l.to(dtype), 7, scoring=scoring, normalize=norm, groups=2, top_groups=1)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("grouped", [False, True])
def test_values_that_are_not_finite_stay_in_their_row(gpu_lib, scoring, grouped):
    announce(f"route not finite {scoring} {grouped}")
    E, k = 80, 5
    l = make(6, E, torch.float32, 3)
    l[0, 11] = float("nan")
    l[1] = float("nan")
    l[2, 17] = INF
    l[3, 17], l[3, 18] = INF, -INF
    l[4, :78] = -INF
    l[4, 78] = float("nan")
    kw = {"groups": 4, "top_groups": 2} if grouped else {}
    for norm in (True, False):
        ids, w = check_route(gpu_lib, l, k, scoring=scoring, normalize=norm, **kw)
        assert ids[1].tolist() == list(range(k)) and torch.isnan(w[1]).all()
        assert torch.isfinite(w[5]).all()


@pytest.mark.gpu
def test_scores_next_to_each_other_in_32_bits(gpu_lib):
    """Sums s + bias that differ by less than a 32-bit step are told apart."""
    announce("route close scores")
    E = 128
    l = torch.zeros(1, E)
    l[0] = torch.arange(E).float() * 1e-6
    bias = torch.full((E,), 8.0)
    check_route(gpu_lib, l, 9, bias=bias, scoring="sigmoid")
    check_route(gpu_lib, l, 9, bias=bias, scoring="softmax")


def check_backward(lib, dw, logits, ids, pad=0, out_pad=0, **kw):
    T, E = logits.shape
    x = strided(logits, pad) if pad else logits.cuda()
    buf = torch.full((T + 1, E + out_pad), 77.0, dtype=logits.dtype, device="cuda")
    got = lib.moe_route_backward(dw.cuda(), x, ids.cuda(), buf[:T, :E], **kw)
    want = ref.route_backward(f64(dw), f64(logits), ids.numpy(), **kw)
    bound = 1.001 * HALF[logits.dtype] * np.abs(want) + 16 * 1e-13 + (2.0 ** -134 if logits.dtype is torch.bfloat16 else 2.0 ** -149)
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), (err - bound).max()
    assert (buf[T] == 77).all() and (buf[:T, E:] == 77).all()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, torch.float32), (1, 8, 8, torch.bfloat16), (5, 63, 4, torch.float32),
                                         (33, 64, 2, torch.bfloat16), (130, 160, 6, torch.float32),
                                         (3, 256, 8, torch.bfloat16), (9, 384, 10, torch.float32), (4, 1000, 64, torch.float32)])
def test_route_backward(gpu_lib, T, E, k, dtype, scoring, normalize):
    announce(f"route backward {T}x{E} k={k} {scoring} {dtype}")
    for seed, masked in enumerate([0.0, 0.6]):
        l = make(T, E, dtype, seed, masked)
        ids, _ = ref.route(f64(l), k, scoring=scoring, normalize=normalize)
        dw = torch.randn(T, k, generator=torch.Generator().manual_seed(seed + 5))
        dw[torch.from_numpy(ids) < 0] = float("nan")  # a place without an expert is not read
        check_backward(gpu_lib, dw, l, torch.from_numpy(ids), pad=3 * seed, out_pad=2 * seed, scoring=scoring,
                       normalize=normalize, scale=1.75)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [True, False])
def test_sigmoid_gradient_of_large_logits(gpu_lib, dtype, normalize):
    """s (1 - s) of logits from 20 to 80 either way, where 1 - s rounds to 0 from 37 on: bounds relative to the value alone.
    Normalised, q (g - mean) is off by a few 64-bit steps of |g|, and 1 - s multiplies that."""
    announce(f"route backward large logits {dtype} {normalize}")
    E, k = 61, 3
    l = torch.stack([torch.arange(20, 81).float(), -torch.arange(20, 81).float(), torch.arange(20, 81).float() * 1.03]).to(dtype)
    ids = torch.tensor([[0, 30, 60], [0, 30, 60], [9, 18, 55]], dtype=torch.int32)
    dw = torch.tensor([[1.0, -0.75, 0.5], [0.3, 2.0, -1.0], [-4.0, 0.1, 3.0]])
    got = f64(gpu_lib.moe_route_backward(dw.cuda(), l.cuda(), ids.cuda(), scoring="sigmoid", normalize=normalize, scale=1.5))
    x = f64(l)
    s, rest = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))
    at = ids.numpy().astype(np.int64)
    rows = np.arange(3)[:, None]
    c, g = s[rows, at], 1.5 * f64(dw)
    q = c / c.sum(1, keepdims=True)
    d = q * (g - (g * q).sum(1, keepdims=True)) if normalize else g * c
    want, slack = np.zeros_like(x), np.zeros_like(x)
    want[rows, at] = d * rest[rows, at]
    slack[rows, at] = (q if normalize else c) * 16 * 1e-15 * rest[rows, at]
    assert (np.abs(got - want) <= 1.001 * HALF[dtype] * np.abs(want) + slack + 2.0 ** -149).all()
    assert np.array_equal(got != 0, want != 0)
    oracle = ref.route_backward(f64(dw), x, ids.numpy(), scoring="sigmoid", normalize=normalize, scale=1.5)
    assert (np.abs(oracle - want) <= 1e-13 * np.abs(want) + slack).all()


@pytest.mark.gpu
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_softmax_gradient_of_rows_that_are_not_finite(gpu_lib, normalize, value):
    """One infinite or NaN logit makes every share of its row a NaN, chosen or not, and so its gradient."""
    announce(f"route backward {value} {normalize}")
    l = make(4, 70, torch.float32, 11)
    l[1, 5], l[2, 66] = value, value
    l[3, :65] = -INF
    ids = torch.tensor([[3, 8], [3, 5], [3, 8], [65, 69]], dtype=torch.int32)
    dw = torch.randn(4, 2, generator=torch.Generator().manual_seed(1))
    got = f64(gpu_lib.moe_route_backward(dw.cuda(), l.cuda(), ids.cuda(), normalize=normalize))
    with np.errstate(invalid="ignore"):
        want = ref.route_backward(f64(dw), f64(l), ids.numpy(), normalize=normalize)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got[1:3]).all() and np.isfinite(got[[0, 3]]).all()
    check_backward(gpu_lib, dw[[0, 3]], l[[0, 3]], ids[[0, 3]], normalize=normalize)


@pytest.mark.gpu
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward_of_given_ids(gpu_lib, scoring, normalize):
    """The same expert twice, ids outside the experts, a row without any."""
    announce(f"route backward ids {scoring} {normalize}")
    l = make(4, 40, torch.float32, 8)
    ids = torch.tensor([[3, 3, 5], [-1, 39, 40], [-1, -1, -1], [0, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(2))
    got = check_backward(gpu_lib, dw, l, ids, scoring=scoring, normalize=normalize)
    assert (got[2] == 0).all()


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu_lib):
    """The last tokens' logits and gradients lie past 4 GiB."""
    announce("route offsets")
    T, E, k = (1 << 21) + 70, 1024, 5
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 9 GiB of device memory")
    X = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(70, E, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    X[-70:] = last
    ids, w = gpu_lib.moe_route(X, k)
    few = gpu_lib.moe_route(last, k)
    assert torch.equal(ids[-70:], few[0]) and torch.equal(w[-70:], few[1])
    assert (ids[:1000] == torch.arange(k, device="cuda")).all() and (w[:1000] == 0.2).all()
    dw = torch.randn(T, k, device="cuda")
    dl = gpu_lib.moe_route_backward(dw, X, ids)
    assert torch.equal(dl[-70:], gpu_lib.moe_route_backward(dw[-70:].contiguous(), last, few[0]))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_oracle_gradient_is_the_difference_quotient(scoring, normalize):
    """Central differences of the oracle's own weights at fixed ids, and torch's autograd."""
    rng = np.random.default_rng(3)
    l, dw = rng.standard_normal((3, 11)) * 1.5, rng.standard_normal((3, 4))
    ids, _ = ref.route(l, 4, scoring=scoring, normalize=normalize)

    def loss(x):
        total = 0.0
        for t in range(3):
            c = ref.scores(x[t], scoring)[ids[t]]
            total += (1.3 * dw[t] * (c / c.sum() if normalize else c)).sum()
        return total

    want = ref.route_backward(dw, l, ids, scoring=scoring, normalize=normalize, scale=1.3)
    h = 1e-5
    for t in range(3):
        for e in range(11):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            # the quotient's own error: h^2 / 6 of a third derivative below 10, and 1e-16 / h of rounding
            assert abs((loss(up) - loss(down)) / (2 * h) - want[t, e]) < 1e-9
    x = torch.tensor(l, requires_grad=True)
    s = torch.softmax(x, 1) if scoring == "softmax" else torch.sigmoid(x)
    c = s.gather(1, torch.from_numpy(ids).long())
    if normalize:
        c = c / c.sum(1, keepdim=True)
    (1.3 * torch.from_numpy(dw) * c).sum().backward()
    assert np.abs(x.grad.numpy() - want).max() < 1e-13


def test_oracle_choice_is_torchs_topk():
    rng = np.random.default_rng(0)
    l, bias = rng.standard_normal((20, 48)), rng.standard_normal(48) * 0.1
    ids, w = ref.route(l, 5, bias=bias, scoring="sigmoid", scale=2.0)
    s = torch.sigmoid(torch.from_numpy(l))
    want = (s + torch.from_numpy(bias)).topk(5, dim=1).indices
    assert np.array_equal(ids, want.numpy())
    c = s.gather(1, want)
    assert np.allclose(w, (2 * c / c.sum(1, keepdim=True)).numpy(), rtol=1e-14)
    # a group's two best by hand: [3, 1 | 2.5, 2] keeps the second group alone
    ids, _ = ref.route(np.log(np.array([[0.3, 0.1, 0.26, 0.24]])), 2, groups=2, top_groups=1)
    assert ids.tolist() == [[2, 3]]


def route_call(lib, x=0x10000, ld=64, bias=None, ids=0x10000, w=0x10000, T=4, E=64, k=4, scoring=0, groups=1, top=1):
    return lib.moe_route(x, ld, bias, ids, w, T, E, k, scoring, groups, top, 1, 1.0, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), 1, "T=-1"), (dict(E=0), 1, "E=0"), (dict(k=0), 1, "k=0"), (dict(k=65), 1, "k=65 of 64"),
    (dict(scoring=2), 1, "scoring=2"), (dict(groups=3), 1, "groups=3"), (dict(groups=0), 1, "groups=0"),
    (dict(groups=4, top=5), 1, "top_groups=5"), (dict(top=0), 1, "top_groups=0"), (dict(x=None), 1, "logits is NULL"),
    (dict(ids=None), 1, "ids is NULL"), (dict(w=None), 1, "weights is NULL"), (dict(x=0x10002), 2, "logits"),
    (dict(ids=0x10002), 2, "ids"), (dict(bias=0x10001), 2, "bias"), (dict(ld=63), 1, "ld=63"),
    (dict(E=1025, ld=1025), 3, "E=1025"), (dict(E=128, ld=128, k=65), 3, "k=65"),
    (dict(E=130, ld=130, groups=65), 3, "groups=65"), (dict(T=(1 << 25) + 1), 3, "2^25"), (dict(T=0, x=None, ids=None, w=None), 0, "")])
def test_route_refusals(kw, status, needle):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    assert route_call(lib, **kw) == status
    assert needle in lib.fg_last_error().decode()


@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(E=0), 1), (dict(k=5000), 1), (dict(dw=None), 1), (dict(x=None), 1),
                                       (dict(ids=None), 1), (dict(dl=None), 1), (dict(dl=0x10001), 2), (dict(ld_dl=9), 1),
                                       (dict(ld=9), 1), (dict(scoring=-1), 1), (dict(T=0, dw=None, x=None, ids=None, dl=None), 0)])
def test_route_backward_refusals(kw, status):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    a = dict(dw=0x10000, x=0x10000, ld=64, ids=0x10000, dl=0x10000, ld_dl=64, T=4, E=64, k=4, scoring=0)
    a.update(kw)
    for fn in (lib.moe_route_backward, lib.moe_route_backward_bf16):
        assert fn(a["dw"], a["x"], a["ld"], a["ids"], a["dl"], a["ld_dl"], a["T"], a["E"], a["k"], a["scoring"], 1, 1.0,
                  None) == status, lib.fg_last_error()


def test_wrapper_refusals():
    import moe_grouped_gemm_e4m3_amd as fg

    with pytest.raises(TypeError):
        fg.moe_route(torch.zeros(2, 8), 2)  # not on the device
    with pytest.raises(ValueError):
        fg.moe_route(torch.zeros(8), 2)
    with pytest.raises(ValueError):
        fg.moe_route_backward(torch.zeros(2, 2), torch.zeros(8), torch.zeros(2, 2, dtype=torch.int32))


@pytest.mark.gpu
def test_wrapper_checks(gpu_lib):
    l = torch.zeros(3, 16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for bad in (dict(ids=torch.zeros(3, 2, device="cuda")), dict(ids=torch.zeros(2, 2, **i32)),
                dict(ids=torch.zeros(3, 4, **i32)[:, ::2]), dict(weights=torch.zeros(3, 2, dtype=torch.bfloat16, device="cuda")),
                dict(bias=torch.zeros(15, device="cuda")), dict(bias=torch.zeros(16)), dict(scoring="tanh")):
        with pytest.raises((TypeError, ValueError)):
            gpu_lib.moe_route(l, 2, **bad)
    with pytest.raises(gpu_lib.FP8GemmError):
        gpu_lib.moe_route(l, 17)
    with pytest.raises((TypeError, ValueError)):
        gpu_lib.moe_route(l.half(), 2)
    with pytest.raises((TypeError, ValueError)):
        gpu_lib.moe_route(l.t(), 2)
    ids, w = gpu_lib.moe_route(torch.zeros(0, 16, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
