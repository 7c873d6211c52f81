"""float64 definitions of the 8-bit-integer product and the gated feed-forward
block, with the error bounds their fp32 kernels have to meet.

Bounds (eps32 = 2^-24 and eps16 = 2^-8, the unit roundoffs of fp32's 24 and bf16's 8 significant bits):

* a dot product of n fp32 terms is off by at most n eps32 sum |x y|;
* a result rounded to bf16 is off by eps16 |y| more (and by 2^-134 below the
  normal range);
* act(g) = g s(y) with |act'| <= 1.13 for both activations; s is computed from
  exp(-y), whose argument carries a relative error of a few eps32, so s is off
  by at most (|y| + 4) 2 eps32 s.
"""

from __future__ import annotations

import numpy as np

EPS32 = 2.0 ** -24
EPS16 = 2.0 ** -8
TINY16 = 2.0 ** -133
GELU_C = float(np.sqrt(2.0 / np.pi))
GELU_A = 0.044715


def int8_cast(x: np.ndarray):
    """Codes and scales of each row, in the fp32 steps the definition fixes."""
    x = np.asarray(x, np.float32)
    step = np.float32(1) / np.float32(127)
    s = np.maximum(np.abs(x).max(axis=1, initial=0.0), np.float32(1e-4)) * step
    return np.rint(x / s[:, None]).astype(np.int8), s


def gemm_int8(A, sa, B, sb):
    """(D, bound): sa sb A.B^T in float64 and how far a bf16 result may be from it."""
    acc = (A.astype(np.float64) @ B.astype(np.float64).T)  # exact: |sum| < 2^53
    D = acc * sa.astype(np.float64)[:, None] * sb.astype(np.float64)
    # int32 -> fp32 and the two scale products round once each, then bf16
    return D, (EPS16 + 4 * EPS32) * np.abs(D) + TINY16


def _gate(g, act):
    y = g if act == "silu" else 2 * GELU_C * (g + GELU_A * g ** 3)
    slope = np.ones_like(g) if act == "silu" else 2 * GELU_C * (1 + 3 * GELU_A * g ** 2)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-y))
        t = s / (1 + np.exp(y))  # s (1 - s) without cancellation
    return y, slope, s, t


def gated(g, u, act):
    """act(g) * u."""
    return g * _gate(g, act)[2] * u


def gated_bound(g, u, dg, du, act):
    """How far bf16(act(g') u') may be from act(g) u for |g' - g| <= dg, |u' - u| <= du."""
    y, _, s, _ = _gate(g, act)
    H = g * s * u
    return (EPS16 + (np.abs(y) + 8) * 2 * EPS32) * np.abs(H) + 1.13 * dg * (np.abs(u) + du) + np.abs(g * s) * du + TINY16


def pre_activations(X, W):
    """g, u and the bound of their fp32 sums' errors (X, W exact in float64)."""
    X, W = X.astype(np.float64), W.astype(np.float64)
    F = W.shape[0] // 2
    p, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    e = X.shape[1] * EPS32 * mag
    return p[:, :F], p[:, F:], e[:, :F], e[:, F:]


def gated_grad(dH, g, u, act):
    """dg, du."""
    _, slope, s, t = _gate(g, act)
    return dH * u * (s + g * t * slope), dH * g * s


def gated_backward(dH, X, W, act):
    """dX, dW in float64 and the bounds of the bf16 results of kernels that
    accumulate in fp32 over the pair [dg du] rounded to bf16."""
    dH, X, W = (a.astype(np.float64) for a in (dH, X, W))
    g, u, eg, eu = pre_activations(X, W)
    dg, du = gated_grad(dH, g, u, act)
    y, slope, s, t = _gate(g, act)
    # |act''| <= 1.6 for both activations; the gate's own error is relative to
    # s plus, through 1 - s, absolute at the scale of eps32
    gate_err = (np.abs(y) + 8) * 4 * EPS32
    e_dg = np.abs(dH) * (np.abs(u) * (1.6 * eg + gate_err * (s + np.abs(g) * s * slope)) + eu * 1.13) + EPS16 * np.abs(dg)
    e_du = np.abs(dH) * (1.13 * eg + gate_err * np.abs(g) * s) + EPS16 * np.abs(du)
    d, e = np.concatenate([dg, du], 1), np.concatenate([e_dg, e_du], 1) + TINY16
    dX, dW = d @ W, d.T @ X
    n_x, n_w = W.shape[0] + 128, X.shape[0] + 128
    aW, aX, ad = np.abs(W), np.abs(X), np.abs(d) + e
    b_x = e @ aW + n_x * EPS32 * (ad @ aW) + TINY16
    b_w = e.T @ aX + n_w * EPS32 * (ad.T @ aX) + TINY16
    return dX, dW, b_x + EPS16 * (np.abs(dX) + b_x), b_w + EPS16 * (np.abs(dW) + b_w)
