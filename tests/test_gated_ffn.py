"""The gated feed-forward block (bf16 forward and backward, 8-bit-integer
forward) against its float64 definition, and the definition's gradient against
differences."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, bf16, f64, strided
from tests.test_int8_linear import codes

ACTS = ["silu", "gelu_tanh"]


def block(M, F, K, seed=0):
    """bf16 X, W, dH: products of order 1, a few large pre-activations of either sign."""
    gen = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=gen)
    X[: max(1, M // 8)] *= 6.0
    W = torch.randn(2 * F, K, generator=gen) * (K ** -0.5 if K else 1.0)
    return bf16(X), bf16(W), bf16(torch.randn(M, F, generator=gen))


# ---- the definition -------------------------------------------------------


@pytest.mark.parametrize("act", ACTS)
def test_definition_against_torch(act):
    g, u = torch.randn(200, dtype=torch.float64) * 4, torch.randn(200, dtype=torch.float64)
    a = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    assert np.allclose(ref.gated(g.numpy(), u.numpy(), act), (a * u).numpy(), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_definition_against_differences(act):
    rng = np.random.default_rng(0)
    M, F, K, eps = 3, 4, 8, 1e-5
    X, W, dH = rng.standard_normal((M, K)), rng.standard_normal((2 * F, K)), rng.standard_normal((M, F))

    def loss(X, W):
        p = X @ W.T
        return (ref.gated(p[:, :F], p[:, F:], act) * dH).sum()

    dX, dW, _, _ = ref.gated_backward(dH, X, W, act)
    for arr, grad in ((X, dX), (W, dW)):
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + eps
            up = loss(X, W)
            arr[i] = old - eps
            down = loss(X, W)
            arr[i] = old
            assert abs((up - down) / (2 * eps) - grad[i]) < 1e-7 * (1 + abs(grad[i]))


# ---- forward --------------------------------------------------------------

SHAPES = [
    (1, 1, 8), (1, 5, 16), (1, 200, 2048), (2, 33, 40), (5, 64, 1032), (16, 65, 136), (17, 48, 4096), (33, 129, 328),
    (64, 256, 512), (65, 50, 264), (100, 320, 520), (128, 1056, 256), (129, 125, 504), (200, 128, 128),
    (300, 255, 400), (513, 150, 1024), (1000, 65, 152), (700, 500, 1048), (257, 2050, 64), (2049, 33, 88),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", SHAPES)
def test_forward_matches_float64(gpu_lib, M, F, K, act):
    announce(f"gated bf16 {M}x{F}x{K} {act}")
    X, W, _ = block(M, F, K, 1)
    pad = 8 * (M % 3)
    out = Output(M, F, pad)
    P = torch.full((M, 2 * F + 3), float("nan"), device="cuda")[:, :2 * F] if M % 2 else None
    gpu_lib.gated_ffn_bf16(strided(X, pad), strided(W, 2 * pad), out.t, P=P, activation=act)
    out.check_untouched()
    g, u, eg, eu = ref.pre_activations(f64(X), f64(W))
    assert_within(out.f64(), ref.gated(g, u, act), ref.gated_bound(g, u, eg, eu, act), "H")
    if P is not None:
        assert_within(f64(P), np.concatenate([g, u], 1), np.concatenate([eg, eu], 1) + 1e-45, "P")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", [(m, f, 16 * ((k + 15) // 16)) for m, f, k in SHAPES])
def test_int8_forward_matches_float64(gpu_lib, M, F, K, act):
    announce(f"gated int8 {M}x{F}x{K} {act}")
    X, sx = codes(M, K, 3)
    W, sw = codes(2 * F, K, 4)
    sx = (sx * np.float32(2.0 ** -5)).astype(np.float32)
    pad = 16 * (M % 3)
    out = Output(M, F, pad)
    gpu_lib.gated_ffn_int8(strided(torch.from_numpy(X), pad), torch.from_numpy(sx).cuda(),
                           strided(torch.from_numpy(W), pad), torch.from_numpy(sw).cuda(), out.t, activation=act)
    out.check_untouched()
    p, _ = ref.gemm_int8(X, sx, W, sw)
    e = 4 * ref.EPS32 * np.abs(p)
    g, u, eg, eu = p[:, :F], p[:, F:], e[:, :F], e[:, F:]
    assert_within(out.f64(), ref.gated(g, u, act), ref.gated_bound(g, u, eg, eu, act), "H")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_forward_far_pre_activations(gpu_lib, M, act):
    """Gates so large or small that the sigmoid saturates and cubes overflow:
    act(g) is g or a vanishing value, never NaN."""
    g = torch.tensor([0.0, 88.0, -88.0, 120.0, -120.0, 1e4, -1e4, 1e15, -1e15, 1e30, -1e30])
    F, K = len(g), 16
    W = torch.zeros(2 * F, K)
    W[:F, 0] = g
    W[F:, 1] = 1.0
    X = torch.zeros(M, K)
    X[:, :2] = 1.0
    X, W = bf16(X), bf16(W)
    out = Output(M, F)
    gpu_lib.gated_ffn_bf16(X.cuda(), W.cuda(), out.t, activation=act)
    g = f64(W[:F, 0])
    want = np.tile(np.where(g >= 0, g, 0.0), (M, 1))
    assert_within(out.f64(), want, 2.0 ** -8 * np.abs(want) + 1e-30, "far gates")
    dH, dX, dW = bf16(torch.ones(M, F)).cuda(), Output(M, K), Output(2 * F, K)
    gpu_lib.gated_ffn_bf16_backward(dH, X.cuda(), W.cuda(), dX.t, dW.t, activation=act)
    assert np.isfinite(dX.f64()).all() and np.isfinite(dW.f64()).all()
    slope = np.where(g > 0, 1.0, np.where(g < 0, 0.0, 0.5))
    assert_within(dW.f64()[:F, 0], M * slope, 2.0 ** -7 * M * slope + 1e-25, "dW of the gates")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 300])
def test_forward_nan_and_inf_stay_in_their_rows_and_units(gpu_lib, M):
    F, K = 70, 256
    X, W, _ = block(M, F, K, 2)
    W[5, 3], W[F + 9, 0] = float("nan"), float("inf")
    if M > 4:
        X[4, 7] = float("inf")
    out = Output(M, F)
    gpu_lib.gated_ffn_bf16(X.cuda(), W.cuda(), out.t)
    got = f64(out.t)
    assert np.isnan(got[:, 5]).all() and not np.isfinite(got[:, 9]).any()
    rows = np.array([m for m in range(M) if not (M > 4 and m == 4)])
    cols = np.array([f for f in range(F) if f not in (5, 9)])
    g, u, eg, eu = ref.pre_activations(f64(X)[rows], f64(W)[np.concatenate([cols, F + cols])])
    assert_within(got[np.ix_(rows, cols)], ref.gated(g, u, "silu"), ref.gated_bound(g, u, eg, eu, "silu"), "others")


# ---- backward -------------------------------------------------------------

GRAD_SHAPES = [
    (1, 1, 8), (1, 40, 16), (2, 64, 264), (7, 33, 40), (16, 130, 136), (33, 63, 256), (64, 256, 512), (65, 100, 72),
    (128, 65, 1032), (129, 192, 128), (200, 257, 264), (300, 128, 520), (333, 96, 1528), (513, 300, 200),
    (1000, 64, 64), (700, 330, 392),
    # few outputs of dX and a long sum: split over workgroups
    (2, 2000, 64), (70, 3000, 136), (251, 1500, 264), (150, 1300, 1016),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True], ids=["recomputed", "kept"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", GRAD_SHAPES)
def test_backward_matches_float64(gpu_lib, M, F, K, act, kept):
    announce(f"gated backward {M}x{F}x{K} {act} kept={kept}")
    X, W, dH = block(M, F, K, 6)
    pad = 8 * (M % 3)
    Xd, Wd, dHd = strided(X, pad), strided(W, 2 * pad), strided(dH, pad + (M % 2))
    P = None
    if kept:
        P = torch.empty(M, 2 * F + 5, device="cuda")[:, :2 * F]
        gpu_lib.gated_ffn_bf16(Xd, Wd, torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), P=P, activation=act)
    dX, dW = Output(M, K, pad), Output(2 * F, K, pad)
    # a workspace full of NaN: nothing of it may be read before it is written
    ws = torch.full((max(gpu_lib.gated_ffn_backward_workspace_bytes(M, F, K), 1),), 255, dtype=torch.uint8, device="cuda")
    gpu_lib.gated_ffn_bf16_backward(dHd, Xd, Wd, dX.t, dW.t, P=P, activation=act, workspace=ws)
    dX.check_untouched()
    dW.check_untouched()
    wx, ww, bx, bw = ref.gated_backward(f64(dH), f64(X), f64(W), act)
    assert_within(dX.f64(), wx, bx, "dX")
    assert_within(dW.f64(), ww, bw, "dW")
    # the roundings of [dg du] and of the results are independent and each
    # spread evenly over at most +-2^-8 of its value: sqrt(2) 2^-8 / sqrt(3)
    # of the norm at most
    for got, want in ((dX.f64(), wx), (dW.f64(), ww)):
        if want.size >= 1024:
            assert np.linalg.norm(got - want) <= 3.2e-3 * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(gpu_lib, act):
    """The kernels' gradients along random directions against central
    differences of the float64 loss."""
    M, F, K = 70, 90, 72
    X, W, dH = block(M, F, K, 7)
    dX, dW = Output(M, K), Output(2 * F, K)
    gpu_lib.gated_ffn_bf16_backward(dH.cuda(), X.cuda(), W.cuda(), dX.t, dW.t, activation=act)
    x, w, d = f64(X), f64(W), f64(dH)
    _, _, bx, bw = ref.gated_backward(d, x, w, act)

    def loss(x, w):
        p = x @ w.T
        return (ref.gated(p[:, :F], p[:, F:], act) * d).sum()

    rng = np.random.default_rng(0)
    for _ in range(4):
        vx, vw, eps = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-6
        nx = (loss(x + eps * vx, w) - loss(x - eps * vx, w)) / (2 * eps)
        nw = (loss(x, w + eps * vw) - loss(x, w - eps * vw)) / (2 * eps)
        # each element's error is within its bound; along a random direction
        # independent errors add like their norm (6 standard deviations)
        assert abs((dX.f64() * vx).sum() - nx) <= 6 * np.linalg.norm(bx) + 1e-6 * abs(nx)
        assert abs((dW.f64() * vw).sum() - nw) <= 6 * np.linalg.norm(bw) + 1e-6 * abs(nw)


@pytest.mark.gpu
def test_backward_one_gradient_only(gpu_lib):
    M, F, K = 150, 70, 136
    X, W, dH = (t.cuda() for t in block(M, F, K, 8))
    both = Output(M, K), Output(2 * F, K)
    gpu_lib.gated_ffn_bf16_backward(dH, X, W, both[0].t, both[1].t)
    dX, dW = Output(M, K), Output(2 * F, K)
    assert gpu_lib.gated_ffn_bf16_backward(dH, X, W, dX.t, None)[1] is None
    assert gpu_lib.gated_ffn_bf16_backward(dH, X, W, None, dW.t)[0] is None
    assert torch.equal(dX.t, both[0].t) and torch.equal(dW.t, both[1].t)
    gpu_lib.gated_ffn_bf16_backward(dH, X, W, None, None)


@pytest.mark.gpu
def test_backward_empty_axes(gpu_lib):
    dev = dict(device="cuda", dtype=torch.bfloat16)
    dW = torch.ones(6, 16, **dev)
    gpu_lib.gated_ffn_bf16_backward(torch.empty(0, 3, **dev), torch.empty(0, 16, **dev), torch.ones(6, 16, **dev),
                                    torch.empty(0, 16, **dev), dW)
    assert not dW.any()  # no rows: a sum over nothing
    dX = torch.ones(4, 16, **dev)
    gpu_lib.gated_ffn_bf16_backward(torch.empty(4, 0, **dev), torch.ones(4, 16, **dev), torch.empty(0, 16, **dev), dX,
                                    torch.empty(0, 16, **dev))
    assert not dX.any()  # no hidden units
    H = torch.ones(4, 3, **dev)
    P = torch.ones(4, 6, device="cuda")
    gpu_lib.gated_ffn_bf16(torch.empty(4, 0, **dev), torch.empty(6, 0, **dev), H, P=P)
    assert not H.any() and not P.any()
    gpu_lib.gated_ffn_bf16(torch.empty(0, 16, **dev), torch.ones(6, 16, **dev), torch.empty(0, 3, **dev))
    gpu_lib.gated_ffn_bf16(torch.empty(4, 16, **dev), torch.ones(0, 16, **dev), torch.empty(4, 0, **dev))


@pytest.mark.gpu
def test_step_on_another_stream_and_in_a_graph(gpu_lib):
    M, F, K = 140, 100, 264
    X, W, dH = (t.cuda() for t in block(M, F, K, 9))

    def step(stream=None, ws=None, outs=None):
        H, P, dX, dW = outs or (torch.empty(M, F, dtype=torch.bfloat16, device="cuda"),
                                torch.empty(M, 2 * F, device="cuda"), torch.empty_like(X), torch.empty_like(W))
        gpu_lib.gated_ffn_bf16(X, W, H, P=P, stream=stream)
        gpu_lib.gated_ffn_bf16_backward(dH, X, W, dX, dW, P=P, stream=stream, workspace=ws)
        return H, P, dX, dW

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = tuple(torch.empty_like(t) for t in want)
    torch.cuda.synchronize()
    got = step(stream=side, outs=outs)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = tuple(torch.empty_like(t) for t in want)
    ws = torch.empty(gpu_lib.gated_ffn_backward_workspace_bytes(M, F, K), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws=ws, outs=outs)
    for _ in range(4):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        again = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))


# ---- refusals (no device) -------------------------------------------------

Q = 0x10000


@pytest.fixture(scope="module")
def lib():
    import moe_grouped_gemm_e4m3_amd as fg

    return fg.load_library()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative"), (dict(F=-2), 1, "negative"), (dict(K=12), 2, "K=12"), (dict(act=2), 1, "activation=2"),
    (dict(act=-1), 1, "activation"), (dict(X=None), 1, "X is NULL"), (dict(W=Q + 8), 2, "W is not 16-byte"),
    (dict(H=None), 1, "H is NULL"), (dict(H=Q + 1), 2, "H is not"), (dict(ldx=504), 1, "ldx=504"),
    (dict(ldw=516), 2, "ldw=516"), (dict(ldh=60), 1, "ldh=60"), (dict(ldp=100), 1, "ldp=100"),
    (dict(P=Q + 2), 2, "P is not"), (dict(ldw=(1 << 21) + 8), 3, "4 MiB"),
])
def test_forward_refusals(lib, kw, status, needle):
    a = dict(X=Q, ldx=512, W=Q, ldw=512, H=Q, ldh=64, P=Q, ldp=128, M=64, F=64, K=512, act=0)
    a.update(kw)
    st = lib.gated_ffn_bf16(a["X"], a["ldx"], a["W"], a["ldw"], a["H"], a["ldh"], a["P"], a["ldp"], a["M"], a["F"],
                            a["K"], a["act"], None)
    assert st == status, lib.fg_last_error()
    assert needle in lib.fg_last_error().decode()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative"), (dict(K=20), 2, "K=20"), (dict(act=9), 1, "activation=9"), (dict(X=None), 1, "X is NULL"),
    (dict(dH=None), 1, "dH is NULL"), (dict(dX=Q + 1), 2, "dX is not"), (dict(dW=Q + 1), 2, "dW is not"),
    (dict(lddh=63), 1, "lddh=63"), (dict(lddx=511), 1, "lddx=511"), (dict(lddw=511), 1, "lddw=511"),
    (dict(P=Q, ldp=127), 1, "ldp=127"), (dict(wsb=64), 1, "smaller"), (dict(ws=None, wsb=0), 1, "smaller"),
    (dict(ws=Q + 16), 2, "256-byte"), (dict(W=Q + 2), 2, "W is not"), (dict(ldx=(1 << 21) + 8), 3, "4 MiB"),
])
def test_backward_refusals(lib, kw, status, needle):
    a = dict(dH=Q, lddh=64, X=Q, ldx=512, W=Q, ldw=512, P=None, ldp=0, dX=Q, lddx=512, dW=Q, lddw=512, M=64, F=64, K=512,
             act=0, ws=Q, wsb=1 << 24)
    a.update(kw)
    st = lib.gated_ffn_bf16_backward(a["dH"], a["lddh"], a["X"], a["ldx"], a["W"], a["ldw"], a["P"], a["ldp"], a["dX"],
                                     a["lddx"], a["dW"], a["lddw"], a["M"], a["F"], a["K"], a["act"], a["ws"],
                                     a["wsb"], None)
    assert st == status, lib.fg_last_error()
    assert needle in lib.fg_last_error().decode()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative"), (dict(K=24), 2, "K=24"), (dict(act=5), 1, "activation=5"), (dict(sx=None), 1, "sx is NULL"),
    (dict(sw=Q + 1), 2, "sw is not"), (dict(X=Q + 8), 2, "X is not"), (dict(ldh=1), 1, "ldh=1"),
    (dict(K=131072, ldx=131072, ldw=131072), 3, "131056"),
])
def test_int8_forward_refusals(lib, kw, status, needle):
    a = dict(X=Q, ldx=512, sx=Q, W=Q, ldw=512, sw=Q, H=Q, ldh=64, M=64, F=64, K=512, act=0)
    a.update(kw)
    st = lib.gated_ffn_int8(a["X"], a["ldx"], a["sx"], a["W"], a["ldw"], a["sw"], a["H"], a["ldh"], a["M"], a["F"],
                            a["K"], a["act"], None)
    assert st == status, lib.fg_last_error()
    assert needle in lib.fg_last_error().decode()


def test_workspace_query(lib):
    assert lib.fg_gated_ffn_backward_workspace_bytes(-1, 4, 8) == -1
    assert lib.fg_gated_ffn_backward_workspace_bytes(4, 4, -8) == -1
    assert lib.fg_gated_ffn_backward_workspace_bytes(0, 4, 8) == 0
    assert lib.fg_gated_ffn_backward_workspace_bytes(3, 1, 8) >= 3 * 2 * 2
    assert lib.fg_gated_ffn_backward_workspace_bytes(1 << 30, 1 << 20, 1 << 20) > 1 << 50
    # at most 32 MiB of partials, and none where two do not fit
    pair = 2 * 64 * 2
    assert lib.fg_gated_ffn_backward_workspace_bytes(4096, 64, 8192) == 4096 * pair
    assert 0 < lib.fg_gated_ffn_backward_workspace_bytes(512, 64, 4096) - 512 * pair <= 32 << 20


def test_wrappers_reject_cpu_tensors_and_unknown_activations():
    import moe_grouped_gemm_e4m3_amd as fg

    x, w, h = bf16(torch.zeros(4, 16)), bf16(torch.zeros(12, 16)), bf16(torch.zeros(4, 6))
    with pytest.raises(TypeError):
        fg.gated_ffn_bf16(x, w, h)
    with pytest.raises(TypeError):
        fg.gated_ffn_bf16_backward(h, x, w, x.clone(), w.clone())
    with pytest.raises(ValueError):
        fg._activation("relu6")


@pytest.mark.gpu
def test_wrappers_reject_shapes(gpu_lib):
    x, w, h = (bf16(torch.zeros(s)).cuda() for s in ((4, 16), (12, 16), (4, 6)))
    for bad in (lambda: gpu_lib.gated_ffn_bf16(x, w[:10], h), lambda: gpu_lib.gated_ffn_bf16(x, w, h, activation="tanh"),
                lambda: gpu_lib.gated_ffn_bf16(x, w, h, P=torch.empty(4, 6, device="cuda")),
                lambda: gpu_lib.gated_ffn_bf16_backward(h, x, w, x[:3], w),
                lambda: gpu_lib.gated_ffn_bf16_backward(h, x, w, x, w[:, :8])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        gpu_lib.gated_ffn_bf16(x.float(), w, h)
