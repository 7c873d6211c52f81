"""float64 definitions of the expert router, 4-bit weights and the expert
layers, with the error bounds their kernels have to meet.

Bounds (eps32 = 2^-24 and eps16 = 2^-8, as in oracle/linear.py):

* a sum of n fp32 terms is off by at most n eps32 sum |x|; a few more roundings
  of each term (scales, zero points, partial sums of waves) add as many eps32;
* with a zero point z the kernel sums x q and z x apart, so the terms are
  s |x| (q + z), not s |x| |q - z|;
* a hidden unit is kept in fp32;
* the router computes in 64 bits and rounds once to its output's type.
"""

from __future__ import annotations

import numpy as np

from oracle import e4m3
from oracle.linear import EPS16, EPS32, TINY16, _gate


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp32 values to the nearest bf16, as fp32."""
    return e4m3.bf16_bits_to_f32(e4m3.bf16_rne_bits(np.asarray(x, np.float64))).astype(np.float32)


# ---------------------------------------------------------------------------
# 4-bit weights

def int4_pack(q: np.ndarray) -> np.ndarray:
    """Codes [N, K] (0..15) to the packed rows, padding codes zero."""
    N, K = q.shape
    chunks = -(-K // 128)
    out = np.zeros((N, chunks * 64), np.uint8)
    for k in range(K):
        chunk, inside = divmod(k, 128)
        m, rest = divmod(inside, 32)
        quarter, j = divmod(rest, 8)
        word = chunk * 16 + 4 * quarter + m
        out[:, word * 4 + j % 4] |= (q[:, k].astype(np.uint8) << (4 * (j // 4))).astype(np.uint8)
    return out


def int4_unpack(b: np.ndarray, K: int) -> np.ndarray:
    q = np.empty((b.shape[0], K), np.uint8)
    for k in range(K):
        chunk, inside = divmod(k, 128)
        m, rest = divmod(inside, 32)
        quarter, j = divmod(rest, 8)
        q[:, k] = (b[:, (chunk * 16 + 4 * quarter + m) * 4 + j % 4] >> (4 * (j // 4))) & 15
    return q


def int4_cast(w: np.ndarray, group: int, symmetric: bool):
    """Codes [N, K], scales (fp32 values of bf16) and zero points [N, Kg], in the fp32 steps the definition fixes."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    kg = -(-K // group)
    q = np.empty((N, K), np.uint8)
    s, z = np.empty((N, kg), np.float32), np.full((N, kg), 8, np.uint8)
    f = np.float32
    for g in range(kg):
        x = w[:, g * group:(g + 1) * group]
        lo, hi = np.minimum(x.min(axis=1), f(0)), np.maximum(x.max(axis=1), f(0))
        if symmetric:
            step = np.maximum(np.maximum(hi, -lo) / f(7), f(1e-20) / f(7))
        else:
            # of halves: the same bits, and hi - lo may pass the largest fp32
            step = np.maximum((f(0.5) * hi - f(0.5) * lo) / f(7.5), f(1e-20) / f(15))
        s[:, g] = bf16_round(step)
        if not symmetric:
            z[:, g] = np.clip(np.rint(-lo / s[:, g]), 0, 15)
        q[:, g * group:(g + 1) * group] = np.clip(np.rint(x / s[:, g, None]) + z[:, g, None].astype(f), 0, 15)
    return q, s, z


def int4_widen(q, s, z, group):
    """Weights and the magnitudes s (q + z) of their two terms, [N, K]."""
    K = q.shape[1]
    s, z = (np.repeat(np.asarray(a, np.float64), group, axis=1)[:, :K] for a in (s, z))
    q = q.astype(np.float64)
    return s * (q - z), np.abs(s) * (q + np.abs(z))


def fp8_widen(values, factors):
    """Weights [N, K] of decoded e4m3 values and 128 x 128 block factors (terms: their magnitudes)."""
    N, K = values.shape
    f = np.repeat(np.repeat(factors.astype(np.float64), 128, axis=0)[:N], 128, axis=1)[:, :K]
    w = values.astype(np.float64) * f
    return w, np.abs(w)


def product(X, W, terms):
    """(D, bound of its fp32 sums): X . W^T."""
    X = X.astype(np.float64)
    return X @ W.T, (X.shape[1] + 16) * EPS32 * (np.abs(X) @ terms.T)


def gemm_int4(A, q, s, z, group):
    D, e = product(A, *int4_widen(q, s, z, group))
    return D, e + EPS16 * (np.abs(D) + e) + TINY16


# ---------------------------------------------------------------------------
# expert layer

def layer(X, W1, W2, ids, w, act):
    """(D, bound): W1, W2: for each expert (weights, terms), ids [T, k], w [T, k]."""
    T, k = ids.shape
    X = X.astype(np.float64)
    E, K = len(W1), X.shape[1]
    D, bound, mag = np.zeros((T, K)), np.zeros((T, K)), np.zeros((T, K))
    for e in range(E):
        for t in range(T):
            js = np.flatnonzero(ids[t] == e)
            if not js.size:
                continue
            c = w[t, js].astype(np.float64).sum()
            ca = np.abs(w[t, js].astype(np.float64)).sum()
            p, ep = product(X[t:t + 1], *W1[e])
            F = p.shape[1] // 2
            g, u, dg, du = p[:, :F], p[:, F:], ep[:, :F], ep[:, F:]
            y, _, s, _ = _gate(g, act)
            h = g * s * u
            dh = (np.abs(y) + 8) * 2 * EPS32 * np.abs(h) + 1.13 * dg * (np.abs(u) + du) + np.abs(g * s) * du + TINY16
            out, _ = product(h, *W2[e])
            terms = (np.abs(h) + dh) @ W2[e][1].T
            D[t] += c * out[0]
            bound[t] += ca * (dh @ W2[e][1].T)[0]
            mag[t] += ca * terms[0]
            last = F
    if mag.any():
        bound += (last + k + 48) * EPS32 * mag
    return D, bound + EPS16 * (np.abs(D) + bound) + TINY16


# ---------------------------------------------------------------------------
# router

def scores(l, scoring):
    l = l.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = np.fmax.reduce(l)
        e = np.exp(l - (0.0 if top == -np.inf else top))
        total = e.sum()
        return np.zeros_like(e) if total == 0 else e / total


def route(logits, k, bias=None, scoring="softmax", groups=1, top_groups=1, normalize=True, scale=1.0):
    """(ids, weights) of each row, by the definition, a row at a time."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        s = scores(l, scoring)
        by = l.copy() if bias is None and groups == 1 else s + (0.0 if bias is None else bias.astype(np.float64))
        by = np.where(np.isnan(by), -1e300, by)
        candidate = (l != -np.inf) & (by != -np.inf)
        if groups > 1:
            size = E // groups
            value = []
            for g in range(groups):
                best = sorted((by[e] for e in range(g * size, (g + 1) * size) if candidate[e]), reverse=True)[:2]
                value.append(sum(best) if best else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            candidate &= np.isin(np.arange(E) // size, kept)
        order = sorted(np.flatnonzero(candidate), key=lambda e: (-by[e], e))[:k]
        ids[t, :len(order)] = order
        c = s[order]
        if normalize:
            total = c.sum()
            c = np.zeros_like(c) if total == 0 else c / total
        w[t, :len(order)] = scale * c
    return ids, w


def route_backward(dw, logits, ids, scoring="softmax", normalize=True, scale=1.0):
    """dlogits through the Jacobians of weights by scores and of scores by logits."""
    T, E = logits.shape
    dl = np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        s = scores(l, scoring)
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        c = np.array([s[ids[t, j]] for j in js])
        g = np.array([scale * float(dw[t, j]) for j in js])
        total = c.sum()
        if normalize:
            ds = np.zeros_like(c) if total == 0 else (g - (g * c).sum() / total) / total
        else:
            ds = g
        full = np.zeros(E)
        for j, d in zip(js, ds):
            full[ids[t, j]] += d
        # sigmoid: 1 - s is the sigmoid of -l, which does not cancel
        dl[t] = s * (full - (full * s).sum()) if scoring == "softmax" else full * s * scores(-l, scoring)
    return dl
