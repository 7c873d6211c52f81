"""What the 8-bit-integer linear layer and the gated feed-forward block are measured on.

Operators and their formulas (rows of every matrix are contiguous in their last dimension):

* ``cast``      q, s = int8_cast_per_row(x):  s[m] = max(max_k |x[m, k]|, 1e-4) / 127,  q = rint(x / s)
* ``gemm``      D = gemm_int8_nt(A, sa, B, sb):  D[m, n] = sa[m] sb[n] sum_k A[m, k] B[n, k]
* ``gated_int8``  H = gated_ffn_int8(X, sx, W, sw):  the two products below from 8-bit integers with a scale for each row
* ``gated``     H = gated_ffn_bf16(X, W):  g = X Wg^T, u = X Wu^T, H = act(g) u,  W = [Wg; Wu] of 2 F rows
* ``gated_grad``  dX, dW = gated_ffn_bf16_backward(dH, X, W):  the products recomputed from X and W
* ``gated_step``  H, dX, dW of one training step: the forward pass keeps g and u for the backward pass

``run`` computes them in elementary 32-bit torch operations where ``own`` is false, and through the package's
public functions where it is true.
"""

import math

import torch

own = False

#: tanh form of GELU: gelu(x) = x / (1 + exp(-2 c (x + 0.044715 x^3))), c = sqrt(2 / pi)
GELU_C = math.sqrt(2.0 / math.pi)
GELU_A = 0.044715


def listed():
    return [
        # decode: 64 sequences' hidden states, as a router or a norm leaves them in fp32, on their way into an 8-bit layer
        {"name": "cast-decode-64", "op": "cast", "M": 64, "K": 7168, "dtype": "float32", "pad": 0},
        # prefill: 4096 tokens of bf16 activations cast in front of a linear layer
        {"name": "cast-prefill-4096", "op": "cast", "M": 4096, "K": 7168, "dtype": "bfloat16", "pad": 0},
        # one token through a down projection: latency and the weight stream are all there is
        {"name": "gemm-token", "op": "gemm", "M": 1, "N": 7168, "K": 2048, "pad": 0},
        # a decode batch through a narrow projection of odd width
        {"name": "gemm-decode-128", "op": "gemm", "M": 128, "N": 2112, "K": 7168, "pad": 0},
        # a chunk of a ragged prefill, operands inside wider buffers
        {"name": "gemm-chunk-1000", "op": "gemm", "M": 1000, "N": 4096, "K": 7168, "pad": 64},
        # a long prefill through the largest projection
        {"name": "gemm-prefill-4096", "op": "gemm", "M": 4096, "N": 7168, "K": 16384, "pad": 0},
        # decode of 16 sequences through an expert's gate and up projections, weights in 8 bits
        {"name": "gated-int8-decode-16", "op": "gated_int8", "M": 16, "F": 2048, "K": 7168, "act": "silu", "pad": 0},
        # prefill through the same expert
        {"name": "gated-int8-prefill-4096", "op": "gated_int8", "M": 4096, "F": 2048, "K": 7168, "act": "silu", "pad": 0},
        # one token through the bf16 block
        {"name": "gated-token", "op": "gated", "M": 1, "F": 2048, "K": 7168, "act": "silu", "pad": 0},
        # prefill through a wide bf16 block with a short reduction
        {"name": "gated-prefill-4096", "op": "gated", "M": 4096, "F": 12288, "K": 1536, "act": "gelu_tanh", "pad": 0},
        # fine-tuning on a short, odd batch with the products recomputed (nothing kept from the forward pass)
        {"name": "gated-grad-333", "op": "gated_grad", "M": 333, "F": 1056, "K": 1528, "act": "gelu_tanh", "pad": 8},
        # a training step on 4096 tokens: forward, then both gradients
        {"name": "gated-step-4096", "op": "gated_step", "M": 4096, "F": 2048, "K": 7168, "act": "silu", "pad": 0},
    ]


#: multiply-adds of the largest drawn product (the listed ones reach 4.8e11)
MOST_MACS = 3.0e11


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cast", "gemm", "gemm", "gated_int8", "gated", "gated_grad", "gated_step"])
    pad = rng.choice([0, 0, 16, 64])
    if op == "cast":
        return {"op": op, "M": _log_int(rng, 1, 4096), "K": 16 * _log_int(rng, 4, 512),
                "dtype": rng.choice(["float32", "bfloat16"]), "pad": pad}
    # 8-bit rows are multiples of 16 columns, bf16 rows of 8
    step = 16 if op in ("gemm", "gated_int8") else 8
    K = step * _log_int(rng, 256 // step, 8192 // step)
    wide = _log_int(rng, 200, 16384)  # output rows of the weights
    M = _log_int(rng, 16, 4096) if op in ("gated_grad", "gated_step") else _log_int(rng, 1, 4096)
    while M * wide * K * (3 if op == "gated_step" else 2 if op == "gated_grad" else 1) > MOST_MACS:
        M = (M + 1) // 2
    if op == "gemm":
        return {"op": op, "M": M, "N": wide, "K": K, "pad": pad}
    return {"op": op, "M": M, "F": wide // 2, "K": K, "act": rng.choice(["silu", "gelu_tanh"]), "pad": pad}


def _buffer(rows, cols, pad, dtype):
    """A [rows, cols] view of a buffer whose rows are `pad` elements longer."""
    return torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _activations(rows, cols, pad, dtype, gen):
    """Hidden states: normal values, rows of different magnitudes, and a few channels that stand out."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x *= 0.5 + torch.rand(rows, 1, device="cuda", generator=gen)
    loud = torch.rand(cols, device="cuda", generator=gen) < 0.005
    x[:, loud] *= 6.0
    out = _buffer(rows, cols, pad, dtype)
    out.copy_(x)
    return out


def _codes(x, pad):
    """8-bit codes of x's rows and their scales, as a checkpoint or the layer before holds them."""
    s = x.abs().amax(dim=1).clamp_min(1e-4) / 127.0
    q = _buffer(x.shape[0], x.shape[1], pad, torch.int8)
    q.copy_((x / s[:, None]).round_())
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, M, K, pad = case["op"], case["M"], case["K"], case["pad"]
    st = {"op": op, "act": case.get("act")}
    if op == "cast":
        st["x"] = _activations(M, K, pad, getattr(torch, case["dtype"]), gen)
        st["q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        st["s"] = torch.empty(M, dtype=torch.float32, device="cuda")
        return st
    rows = case["N"] if op == "gemm" else 2 * case["F"]
    w = torch.randn(rows, K, device="cuda", generator=gen) / math.sqrt(K)
    if op in ("gemm", "gated_int8"):
        st["A"], st["sa"] = _codes(_activations(M, K, 0, torch.float32, gen), pad)
        st["B"], st["sb"] = _codes(w, pad)
        st["out"] = _buffer(M, case["N"] if op == "gemm" else case["F"], pad, torch.bfloat16)
        return st
    F = case["F"]
    st["X"] = _activations(M, K, pad, torch.bfloat16, gen)
    st["W"] = _buffer(rows, K, pad, torch.bfloat16)
    st["W"].copy_(w)
    if op != "gated_grad":
        st["H"] = _buffer(M, F, pad, torch.bfloat16)
    if op != "gated":
        st["dH"] = _buffer(M, F, pad, torch.bfloat16)
        st["dH"].copy_(torch.randn(M, F, device="cuda", generator=gen))
        st["dX"] = _buffer(M, K, pad, torch.bfloat16)
        st["dW"] = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    if op == "gated_step":
        st["P"] = torch.empty(M, rows, dtype=torch.float32, device="cuda")
    return st


def _run_own(st):
    import moe_grouped_gemm_e4m3_amd as fg

    op = st["op"]
    if op == "cast":
        return list(fg.int8_cast_per_row(st["x"], st["q"], st["s"]))
    if op == "gemm":
        return fg.gemm_int8_nt(st["A"], st["sa"], st["B"], st["sb"], st["out"])
    if op == "gated_int8":
        return fg.gated_ffn_int8(st["A"], st["sa"], st["B"], st["sb"], st["out"], activation=st["act"])
    if op == "gated":
        return fg.gated_ffn_bf16(st["X"], st["W"], st["H"], activation=st["act"])
    if op == "gated_grad":
        return list(fg.gated_ffn_bf16_backward(st["dH"], st["X"], st["W"], st["dX"], st["dW"], activation=st["act"]))
    fg.gated_ffn_bf16(st["X"], st["W"], st["H"], P=st["P"], activation=st["act"])
    dX, dW = fg.gated_ffn_bf16_backward(st["dH"], st["X"], st["W"], st["dX"], st["dW"], P=st["P"],
                                        activation=st["act"])
    return [st["H"], dX, dW]


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2.0 * GELU_C * (g + GELU_A * g * g * g))


def _act_grad(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1.0 + g * (1.0 - s))
    s = torch.sigmoid(2.0 * GELU_C * (g + GELU_A * g * g * g))
    return s + g * s * (1.0 - s) * (2.0 * GELU_C * (1.0 + 3.0 * GELU_A * g * g))


def run(state):
    if own:
        return _run_own(state)
    st, op = state, state["op"]
    bf16 = torch.bfloat16
    if op == "cast":
        x = st["x"].float()
        s = x.abs().amax(dim=1).clamp_min(1e-4) / 127.0
        return [(x / s[:, None]).round().to(torch.int8), s]
    if op in ("gemm", "gated_int8"):
        y = (st["A"].float() @ st["B"].float().t()) * st["sa"][:, None] * st["sb"]
        if op == "gemm":
            return y.to(bf16)
        F = y.shape[1] // 2
        return (_act(y[:, :F], st["act"]) * y[:, F:]).to(bf16)
    X, W = st["X"].float(), st["W"].float()
    F = W.shape[0] // 2
    p = X @ W.t()
    g, u = p[:, :F], p[:, F:]
    if op == "gated":
        return (_act(g, st["act"]) * u).to(bf16)
    dH = st["dH"].float()
    dP = torch.cat([dH * u * _act_grad(g, st["act"]), dH * _act(g, st["act"])], dim=1)
    grads = [(dP @ W).to(bf16), (dP.t() @ X).to(bf16)]
    return grads if op == "gated_grad" else [(_act(g, st["act"]) * u).to(bf16)] + grads


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "cast":
        item = 4 if case["dtype"] == "float32" else 2
        return {"bytes": M * K * (item + 1) + 4 * M, "flops": 2 * M * K}
    if op == "gemm":
        N = case["N"]
        return {"bytes": (M + N) * K + 4 * (M + N) + 2 * M * N, "flops": 2 * M * N * K}
    F = case["F"]
    product = 2 * M * 2 * F * K
    if op == "gated_int8":
        return {"bytes": (M + 2 * F) * K + 4 * (M + 2 * F) + 2 * M * F, "flops": product}
    forward = 2 * (M * K + 2 * F * K + M * F)
    if op == "gated":
        return {"bytes": forward, "flops": product}
    # X, W and dH read once, dX and dW written once
    backward = 2 * (2 * M * K + 4 * F * K + M * F)
    if op == "gated_grad":
        return {"bytes": backward, "flops": 3 * product}
    return {"bytes": backward + 2 * M * F, "flops": 3 * product}


def exact(case, seed):
    """The definitions in float64, a column block of the hidden units at a time."""
    st = prepare(case, seed)
    op, act = case["op"], case.get("act")
    d = torch.float64
    if op == "cast":
        top = st["x"].to(d).abs().max(dim=1).values
        return [None, torch.where(top > 1e-4, top, torch.full_like(top, 1e-4)) / 127]
    if op in ("gemm", "gated_int8"):
        a = st["A"].to(d) * st["sa"].to(d).unsqueeze(1)
        w = st["B"].to(d) * st["sb"].to(d).unsqueeze(1)
        if op == "gemm":
            return torch.mm(a, w.t())
    else:
        a, w = st["X"].to(d), st["W"].to(d)
    F = case["F"]
    H = torch.empty(case["M"], F, dtype=d, device="cuda")
    grads = op in ("gated_grad", "gated_step")
    if grads:
        dX, dW, dH = torch.zeros_like(a), torch.empty_like(w), st["dH"].to(d)
    for lo in range(0, F, 4096):
        hi = min(F, lo + 4096)
        g, u = torch.mm(a, w[lo:hi].t()), torch.mm(a, w[F + lo:F + hi].t())
        if act == "silu":
            y, slope = g, torch.ones_like(g)
        else:
            y = 2 * GELU_C * (g + GELU_A * g ** 3)
            slope = 2 * GELU_C * (1 + 3 * GELU_A * g ** 2)
        gate = 1 / (1 + torch.exp(-y))  # act(g) = g gate
        H[:, lo:hi] = g * gate * u
        if grads:
            dg = dH[:, lo:hi] * u * (gate + g * slope * gate / (1 + torch.exp(y)))
            du = dH[:, lo:hi] * g * gate
            dX += torch.mm(dg, w[lo:hi]) + torch.mm(du, w[F + lo:F + hi])
            dW[lo:hi], dW[F + lo:F + hi] = torch.mm(dg.t(), a), torch.mm(du.t(), a)
    return H if not grads else [dX, dW] if op == "gated_grad" else [H, dX, dW]
