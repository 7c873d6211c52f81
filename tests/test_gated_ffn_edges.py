"""Edge values and sizes of the gated feed-forward block."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, bf16, f64


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True], ids=["recomputed", "kept"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_backward_of_closed_gates_under_large_gradients(gpu_lib, act, kept):
    """dH g and dH u leave fp32's range, the gradients, with the gate closed,
    do not: act and act' of a far negative value are 0.

    Every sum has one term that is not 0, so closed gates give exact zeros."""
    announce(f"closed gates {act} kept={kept}")
    big = 2.0 ** 70
    g = [-(2.0 ** 80), -(2.0 ** 64), 2.0, -(2.0 ** 100)]
    u = [2.0 ** 80, 1.0, 2.0 ** 10, -(2.0 ** 90)]
    M, F, K = 40, 4, 16
    W = torch.zeros(2 * F, K)
    W[:F, 0], W[F:, 1] = torch.tensor(g), torch.tensor(u)
    X = torch.zeros(M, K)
    X[7, :2] = 1.0
    dH = torch.zeros(M, F)
    dH[7] = torch.tensor([big, big, 1.0, big])
    X, W, dH = bf16(X).cuda(), bf16(W).cuda(), bf16(dH).cuda()
    P = None
    if kept:
        P = torch.empty(M, 2 * F, device="cuda")
        gpu_lib.gated_ffn_bf16(X, W, torch.empty_like(dH), P=P, activation=act)
    dX, dW = Output(M, K), Output(2 * F, K)
    gpu_lib.gated_ffn_bf16_backward(dH, X, W, dX.t, dW.t, P=P, activation=act)
    dg, du = ref.gated_grad(f64(dH)[7], np.array(g), np.array(u), act)
    got = dW.f64()
    assert np.isfinite(got).all() and np.isfinite(dX.f64()).all()
    assert (got[[0, 1, 3, F, F + 1, F + 3]] == 0).all()  # closed gates: nothing flows
    # the open gate: the pair and the output are rounded once each
    want, near = np.array([dg[2], du[2]]), np.array([got[2, 0], got[F + 2, 0]])
    assert_within(near, want, 2.0 ** -7 * np.abs(want), "open gate")


@pytest.mark.gpu
@pytest.mark.parametrize("plan", ["pair", "small", "w256", "kept"])
@pytest.mark.parametrize("M,F,K", [(190, 70, 1928), (40, 3, 1032)])
def test_backward_of_an_infinite_input(gpu_lib, monkeypatch, plan, M, F, K):
    """All weights and gradients positive, one input infinite: its row of dX
    is infinite, not NaN, however the pre-activations are summed, and the other
    rows do not see it."""
    announce(f"infinite input {M}x{F}x{K} {plan}")
    monkeypatch.setenv("FG_LINEAR_PLAN", "" if plan == "kept" else plan)
    gen = torch.Generator().manual_seed(1)
    X, W, dH = (bf16(torch.rand(s, generator=gen) / K + 1.0 / K) for s in ((M, K), (2 * F, K), (M, F)))
    X[7, 5] = float("inf")
    P = None
    if plan == "kept":
        P = torch.empty(M, 2 * F, device="cuda")
        gpu_lib.gated_ffn_bf16(X.cuda(), W.cuda(), bf16(torch.empty(M, F)).cuda(), P=P)
    dX, dW = Output(M, K), Output(2 * F, K)
    gpu_lib.gated_ffn_bf16_backward(dH.cuda(), X.cuda(), W.cuda(), dX.t, dW.t, P=P)
    got = f64(dX.t)
    assert np.isposinf(got[7]).all()
    rows = np.arange(M) != 7
    wx, _, bx, _ = ref.gated_backward(f64(dH)[rows], f64(X)[rows], f64(W), "silu")
    assert_within(got[rows], wx, bx, "the other rows")


def test_backward_refuses_a_workspace_of_another_device(monkeypatch):
    """Its memory is written by kernels of the operands' device."""
    import moe_grouped_gemm_e4m3_amd as fg

    class Workspace:  # a tensor of another device, as far as the wrapper looks
        dtype, is_cuda = torch.uint8, True

        def __init__(self, device):
            self.device = device

        get_device = lambda self: self.device  # noqa: E731
        is_contiguous = lambda self: True  # noqa: E731
        numel = lambda self: 1 << 20  # noqa: E731
        data_ptr = lambda self: 0x10000  # noqa: E731

    calls = []
    monkeypatch.setattr(fg, "_device", lambda: 0)
    monkeypatch.setattr(fg, "_matrix", lambda t, name, dtype, rows, cols, dev: cols)
    monkeypatch.setattr(fg, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(fg, "_call", lambda name, *args: calls.append((name, args)))
    x, w, dh = (bf16(torch.zeros(s)) for s in ((4, 16), (12, 16), (4, 6)))
    with pytest.raises(TypeError, match="workspace"):
        fg.gated_ffn_bf16_backward(dh, x, w, x.clone(), w.clone(), workspace=Workspace(1))
    assert not calls
    fg.gated_ffn_bf16_backward(dh, x, w, x.clone(), w.clone(), workspace=Workspace(0))
    assert [name for name, _ in calls] == ["gated_ffn_bf16_backward"] and 0x10000 in calls[0][1]
