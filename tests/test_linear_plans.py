"""Every tile, few-row shape and gradient plan of the 8-bit products and the
gated block, forced (FG_LINEAR_PLAN) onto shapes it would not always be chosen
for: ragged edges, one tile, and more tiles than the device has CUs."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, f64, strided
from tests.test_gated_ffn import block
from tests.test_int8_linear import codes

pytestmark = pytest.mark.gpu

FEW = [f"few{i}" for i in range(8)]
# (rows, columns, K): K ends inside a slice; 1100 x 1300 is 378 tiles of 64 x 64
SHAPES = [(5, 37, 80), (129, 300, 400), (1100, 1300, 144)]


def forced(monkeypatch, plan):
    monkeypatch.setenv("FG_LINEAR_PLAN", plan)


@pytest.mark.parametrize("plan", ["w256", "w224", "w160", "mid2", "mid", "half2", "small2", "small"] + FEW)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_int8_plans(gpu_lib, monkeypatch, plan, M, N, K):
    if plan in FEW:
        M = min(M, 640)
    announce(f"int8 plan {plan} {M}x{N}x{K}")
    forced(monkeypatch, plan)
    A, sa = codes(M, K, 1)
    B, sb = codes(N, K, 2)
    out = Output(M, N, 3)
    gpu_lib.gemm_int8_nt(strided(torch.from_numpy(A), 16), torch.from_numpy(sa).cuda(),
                         strided(torch.from_numpy(B), 32), torch.from_numpy(sb).cuda(), out.t)
    out.check_untouched()
    want, bound = ref.gemm_int8(A, sa, B, sb)
    assert_within(out.f64(), want, bound, plan)


@pytest.mark.parametrize("plan", ["w256", "w192", "mid2", "mid", "half2", "small2", "small"] + FEW)
@pytest.mark.parametrize("form", ["int8", "bf16", "kept"])
@pytest.mark.parametrize("M,F,K", [(5, 19, 80), (129, 150, 400), (1100, 650, 144)])
def test_gated_plans(gpu_lib, monkeypatch, plan, form, M, F, K):
    if plan in FEW:
        M = min(M, 640)
    act = "gelu_tanh" if M == 129 else "silu"
    announce(f"gated plan {plan} {form} {M}x{F}x{K}")
    forced(monkeypatch, plan)
    out = Output(M, F, 5)
    if form == "int8":
        X, sx = codes(M, K, 3)
        W, sw = codes(2 * F, K, 4)
        sx = (sx * np.float32(2.0 ** -5)).astype(np.float32)
        gpu_lib.gated_ffn_int8(strided(torch.from_numpy(X), 16), torch.from_numpy(sx).cuda(),
                               strided(torch.from_numpy(W), 0), torch.from_numpy(sw).cuda(), out.t, activation=act)
        p, _ = ref.gemm_int8(X, sx, W, sw)
        e = 4 * ref.EPS32 * np.abs(p)
        g, u, eg, eu = p[:, :F], p[:, F:], e[:, :F], e[:, F:]
    else:
        X, W, _ = block(M, F, K, 5)
        P = torch.full((M + 1, 2 * F + 3), float("nan"), device="cuda") if form == "kept" else None
        gpu_lib.gated_ffn_bf16(strided(X, 8), strided(W, 16), out.t, P=None if P is None else P[:M, :2 * F], activation=act)
        g, u, eg, eu = ref.pre_activations(f64(X), f64(W))
        if P is not None:
            assert_within(f64(P[:M, :2 * F]), np.concatenate([g, u], 1), np.concatenate([eg, eu], 1) + 1e-45, "P")
            assert P[:, 2 * F:].isnan().all() and P[M].isnan().all()
    out.check_untouched()
    assert_within(out.f64(), ref.gated(g, u, act), ref.gated_bound(g, u, eg, eu, act), plan)


@pytest.mark.parametrize("plan", ["w256", "w224", "w160", "mid2", "mid", "half2", "small2", "small", "split-mid",
                                  "split-small", "pair",
                                  "share-mid-mid", "share-mid-small", "share-small-mid", "share-small-small"])
@pytest.mark.parametrize("M,F,K", [(3, 11, 72), (130, 450, 136), (700, 100, 1304), (65, 700, 264),
                                   (190, 70, 1928)])
def test_gradient_plans(gpu_lib, monkeypatch, plan, M, F, K):
    announce(f"gradient plan {plan} {M}x{F}x{K}")
    forced(monkeypatch, plan)
    X, W, dH = block(M, F, K, 6)
    dX, dW = Output(M, K, 3), Output(2 * F, K, 1)
    ws = torch.full((gpu_lib.gated_ffn_backward_workspace_bytes(M, F, K),), 255, dtype=torch.uint8, device="cuda")
    gpu_lib.gated_ffn_bf16_backward(strided(dH, 1), strided(X, 8), strided(W, 0), dX.t, dW.t, workspace=ws)
    dX.check_untouched()
    dW.check_untouched()
    wx, ww, bx, bw = ref.gated_backward(f64(dH), f64(X), f64(W), "silu")
    assert_within(dX.f64(), wx, bx, f"dX {plan}")
    assert_within(dW.f64(), ww, bw, f"dW {plan}")
    # twice the same: sums have a fixed order
    again = Output(M, K, 3), Output(2 * F, K, 1)
    gpu_lib.gated_ffn_bf16_backward(strided(dH, 1), strided(X, 8), strided(W, 0), again[0].t, again[1].t, workspace=ws)
    assert torch.equal(again[0].buf, dX.buf) and torch.equal(again[1].buf, dW.buf)


def test_int8_bits_do_not_depend_on_the_plan(gpu_lib, monkeypatch):
    """The sums are exact integers."""
    M, N, K = 200, 333, 1040
    A, sa = (torch.from_numpy(t).cuda() for t in codes(M, K, 7))
    B, sb = (torch.from_numpy(t).cuda() for t in codes(N, K, 8))
    want = gpu_lib.gemm_int8_nt(A, sa, B, sb, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    for plan in ["w256", "w224", "w160", "mid2", "mid", "half2", "small2", "small"] + FEW:
        forced(monkeypatch, plan)
        got = gpu_lib.gemm_int8_nt(A, sa, B, sb, torch.empty_like(want))
        assert torch.equal(got, want), plan


def test_gradient_bits_do_not_depend_on_the_tile(gpu_lib, monkeypatch):
    """Each sum runs in the order of its slices; only a split changes it."""
    M, F, K = 200, 150, 328
    X, W, dH = (t.cuda() for t in block(M, F, K, 9))
    P = torch.empty(M, 2 * F, device="cuda")
    gpu_lib.gated_ffn_bf16(X, W, torch.empty_like(dH), P=P)
    want = None
    for plan in ["w256", "w224", "w160", "mid2", "mid", "half2", "small2", "small", "share-mid-mid", "share-mid-small",
                 "share-small-mid", "share-small-small"]:
        forced(monkeypatch, plan)
        dX, dW = torch.empty_like(X), torch.empty_like(W)
        gpu_lib.gated_ffn_bf16_backward(dH, X, W, dX, dW, P=P)
        want = (dX, dW) if want is None else want
        assert torch.equal(dW, want[1]), plan
        if not plan.startswith("share"):  # a shared launch takes dX's own split
            assert torch.equal(dX, want[0]), plan
