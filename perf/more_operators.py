"""What the expert router, the product with 4-bit weights and the expert layers for a few tokens are measured on.

Operators and their formulas (rows of every matrix are contiguous in their last dimension):

* ``route``     ids, w = moe_route(logits): scores s = softmax(l) or sigmoid(l); the k experts with the largest s + bias
  (a logit of -inf is no candidate; with groups, only experts of the groups whose two best add up to most); w = s of the
  chosen, divided by their sum if normalised, times a scale.  Slots without a candidate hold id -1 and weight 0.
* ``route_step``  the same and dl = moe_route_backward(dw) of one training step
* ``int4``      D = gemm_int4_nt(A, B, s, z):  D[m, n] = sum_k A[m, k] s[n, k/g] (B[n, k] - z[n, k/g]),  4-bit codes B, z = 8
  where there are no zero points
* ``moe_fp8``   D = moe_ffn_fp8(X, W1, s1, W2, s2, ids, w):  D[t] = sum_j w[t, j] W2_e (act(g) u),  [g; u] = W1_e X[t],
  e = ids[t, j] (entries of -1 are left out), weights in e4m3 with a factor for each 128 x 128 block
* ``moe_int4``  the same on 4-bit weights with a scale (and zero point) for each group of a row

4-bit codes: columns 8 i .. 8 i + 7 of a row are one little-endian 32-bit word, column 8 i + j in its bits 8 j .. 8 j + 3
and column 8 i + 4 + j in bits 8 j + 4 .. 8 j + 7 (j < 4).  A row is padded to whole chunks of 128 columns (16 words);
columns 32 m + 8 q .. 32 m + 8 q + 7 of a chunk (m, q < 4) are its word 4 q + m.

``run`` computes them in elementary torch operations where ``own`` is false (32 bits; 64 in the router, whose choices
depend on scores next to each other), and through the package's public functions where it is true.
"""

import math

import torch

own = False


def listed():
    return [
        # one token through a wide router with grouped experts: latency alone
        {"name": "route-token", "op": "route", "T": 1, "E": 256, "k": 8, "scoring": "sigmoid", "bias": True, "groups": 8,
         "top": 4, "normalize": True, "masked": 0.0, "dtype": "float32", "pad": 0},
        # a prefill of 4096 tokens through the same router
        {"name": "route-prefill-4096", "op": "route", "T": 4096, "E": 256, "k": 8, "scoring": "sigmoid", "bias": True,
         "groups": 8, "top": 4, "normalize": True, "masked": 0.0, "dtype": "float32", "pad": 0},
        # fine-tuning on a short, odd batch; some experts switched off for some tokens
        {"name": "route-step-333", "op": "route_step", "T": 333, "E": 60, "k": 4, "scoring": "softmax", "bias": False,
         "groups": 1, "top": 1, "normalize": True, "masked": 0.3, "dtype": "bfloat16", "pad": 4},
        # a training step on 8192 tokens, weights not renormalised: the gradient reaches every logit
        {"name": "route-step-8192", "op": "route_step", "T": 8192, "E": 128, "k": 8, "scoring": "softmax", "bias": False,
         "groups": 1, "top": 1, "normalize": False, "masked": 0.0, "dtype": "float32", "pad": 0},
        # one token through a down projection
        {"name": "int4-token", "op": "int4", "M": 1, "N": 7168, "K": 2048, "group": 128, "zeros": True, "pad": 0},
        # one token through a wide up projection with a short reduction
        {"name": "int4-token-wide", "op": "int4", "M": 1, "N": 24576, "K": 1536, "group": 64, "zeros": False, "pad": 0},
        # a decode batch through a narrow projection of odd width, small groups
        {"name": "int4-decode-16", "op": "int4", "M": 16, "N": 2112, "K": 7168, "group": 32, "zeros": True, "pad": 0},
        # the largest decode batch through the largest projection, activations inside a wider buffer
        {"name": "int4-decode-64", "op": "int4", "M": 64, "N": 7168, "K": 16384, "group": 128, "zeros": True, "pad": 64},
        # one token through eight of sixteen experts: 350 MB of weights
        {"name": "moe-fp8-token", "op": "moe_fp8", "T": 1, "E": 16, "k": 8, "F": 2048, "K": 7168, "act": "silu", "away": 0.0,
         "pad": 0},
        # a decode batch on a device that holds about half of the experts each token goes to
        {"name": "moe-fp8-decode-64", "op": "moe_fp8", "T": 64, "E": 16, "k": 8, "F": 2048, "K": 7168, "act": "silu",
         "away": 0.5, "pad": 8},
        # one token through small experts in 4 bits: latency
        {"name": "moe-int4-token", "op": "moe_int4", "T": 1, "E": 64, "k": 6, "F": 704, "K": 2048, "group": 32, "zeros": False,
         "act": "silu", "away": 0.0, "pad": 0},
        # a decode batch of odd size through large experts in 4 bits
        {"name": "moe-int4-decode-23", "op": "moe_int4", "T": 23, "E": 32, "k": 4, "F": 2048, "K": 4096, "group": 128,
         "zeros": True, "act": "gelu_tanh", "away": 0.0, "pad": 0},
    ]


#: scores of the largest drawn router call, products of the largest drawn 4-bit product, weights of the largest drawn expert layer
MOST_SCORES = 1 << 20
MOST_MACS = 7.0e9
MOST_WEIGHTS = 16 * 3 * 2048 * 7168


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_step", "int4", "int4", "moe_fp8", "moe_fp8", "moe_int4", "moe_int4"])
    pad = rng.choice([0, 0, 8, 64])
    if op in ("route", "route_step"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, 4, 384 // groups)
        k = rng.randint(1, min(E // groups, 8))
        return {"op": op, "T": max(1, min(_log_int(rng, 1, 8192), MOST_SCORES // E)), "E": E, "k": k,
                "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "top": rng.randint(1, groups), "normalize": rng.random() < 0.6, "masked": rng.choice([0.0, 0.0, 0.3]),
                "dtype": rng.choice(["float32", "bfloat16"]), "pad": pad}
    group, zeros = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "int4":
        K = 32 * _log_int(rng, 8, 512)
        M, N = _log_int(rng, 1, 64), _log_int(rng, 200, 16384)
        while M * N * K > MOST_MACS:
            M = (M + 1) // 2
        return {"op": op, "M": M, "N": N, "K": K, "group": group, "zeros": zeros, "pad": pad}
    step = 16 if op == "moe_fp8" else 32
    F, K = step * _log_int(rng, 128 // step, 2048 // step), step * _log_int(rng, 256 // step, 7168 // step)
    E = _log_int(rng, 4, 64)
    while 3 * E * F * K > MOST_WEIGHTS:
        E = (E + 1) // 2
    case = {"op": op, "T": _log_int(rng, 1, 64), "E": E, "k": rng.randint(1, min(E, 8)), "F": F, "K": K,
            "act": rng.choice(["silu", "gelu_tanh"]), "away": rng.choice([0.0, 0.0, 0.5]), "pad": pad}
    return case if op == "moe_fp8" else {**case, "group": group, "zeros": zeros}


def _buffer(rows, cols, pad, dtype):
    """A [rows, cols] view of a buffer whose rows are `pad` elements longer."""
    return torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _activations(rows, cols, pad, gen):
    """Hidden states: normal values, rows of different magnitudes, and a few channels that stand out."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    x *= 0.5 + torch.rand(rows, 1, device="cuda", generator=gen)
    x[:, torch.rand(cols, device="cuda", generator=gen) < 0.005] *= 6.0
    out = _buffer(rows, cols, pad, torch.bfloat16)
    out.copy_(x)
    return out


def _fp8_weights(E, rows, cols, gen):
    """e4m3 codes and block factors of E experts' weights, as a checkpoint holds them."""
    q = torch.empty(E, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    nb, kb = -(-rows // 128), -(-cols // 128)
    s = torch.empty(E, nb, kb, device="cuda")
    for e in range(E):
        w = torch.zeros(nb * 128, kb * 128, device="cuda")
        w[:rows, :cols] = torch.randn(rows, cols, device="cuda", generator=gen) / math.sqrt(cols)
        blocks = w.view(nb, 128, kb, 128)
        s[e] = blocks.abs().amax(dim=(1, 3)).clamp_min(1e-4) / 448.0
        q[e] = (blocks / s[e][:, None, :, None]).reshape(nb * 128, kb * 128)[:rows, :cols].to(torch.float8_e4m3fn)
    return q, s


def _int4_weights(rows, cols, group, zeros, gen):
    """Packed 4-bit codes, scales and zero points of a weight matrix, as a checkpoint holds them."""
    kg, chunks = -(-cols // group), -(-cols // 128)
    w = torch.zeros(rows, kg * group, device="cuda")
    w[:, :cols] = torch.randn(rows, cols, device="cuda", generator=gen) / math.sqrt(cols)
    w = w.view(rows, kg, group)
    if zeros:
        lo, hi = w.amin(dim=2).clamp_max(0.0), w.amax(dim=2).clamp_min(0.0)
        s = ((hi - lo) / 15.0).bfloat16()
        z = (-lo / s.float()).round().clamp(0, 15)
    else:
        s = (w.abs().amax(dim=2) / 7.0).bfloat16()
        z = torch.full((rows, kg), 8.0, device="cuda")
    q = ((w / s.float()[:, :, None]).round() + z[:, :, None]).clamp(0, 15).to(torch.uint8).view(rows, kg * group)
    full = torch.zeros(rows, chunks * 128, dtype=torch.uint8, device="cuda")
    full[:, :cols] = q[:, :cols]
    parts = full.view(rows, chunks, 4, 4, 2, 4)  # chunk, m, q, half of a word, byte
    packed = (parts[:, :, :, :, 0] | (parts[:, :, :, :, 1] << 4)).transpose(2, 3).reshape(rows, chunks * 64)
    return packed.contiguous(), s, z.to(torch.uint8) if zeros else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case), "op": op}
    if op in ("route", "route_step"):
        T, E, k = case["T"], case["E"], case["k"]
        logits = torch.randn(T, E, device="cuda", generator=gen) * 1.5
        logits[torch.rand(T, E, device="cuda", generator=gen) < case["masked"]] = -math.inf
        st["logits"] = _buffer(T, E, case["pad"], getattr(torch, case["dtype"]))
        st["logits"].copy_(logits)
        st["bias"] = torch.randn(E, device="cuda", generator=gen) * 0.1 if case["bias"] else None
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(T, k, device="cuda")
        if op == "route_step":
            st["dw"] = torch.randn(T, k, device="cuda", generator=gen)
            st["dl"] = torch.empty(T, E, dtype=st["logits"].dtype, device="cuda")
        return st
    if op == "int4":
        st["A"] = _activations(case["M"], case["K"], case["pad"], gen)
        st["B"], st["s"], st["z"] = _int4_weights(case["N"], case["K"], case["group"], case["zeros"], gen)
        st["D"] = _buffer(case["M"], case["N"], case["pad"], torch.bfloat16)
        return st
    T, E, k, F, K = (case[n] for n in ("T", "E", "k", "F", "K"))
    st["X"] = _activations(T, K, case["pad"], gen)
    if op == "moe_fp8":
        st["W1"], st["s1"] = _fp8_weights(E, 2 * F, K, gen)
        st["W2"], st["s2"] = _fp8_weights(E, K, F, gen)
        st["z1"] = st["z2"] = None
    else:
        for n, rows, cols in (("1", 2 * F, K), ("2", K, F)):
            made = [_int4_weights(rows, cols, case["group"], case["zeros"], gen) for _ in range(E)]
            st["W" + n], st["s" + n] = torch.stack([m[0] for m in made]), torch.stack([m[1] for m in made])
            st["z" + n] = torch.stack([m[2] for m in made]) if case["zeros"] else None
    scores = torch.randn(T, E, device="cuda", generator=gen)
    best, ids = scores.topk(k, dim=1)
    st["w"] = torch.softmax(best, dim=1)
    away = torch.rand(T, k, device="cuda", generator=gen) < case["away"]
    st["ids"] = torch.where(away, -torch.ones_like(ids), ids).to(torch.int32)
    st["D"] = _buffer(T, K, case["pad"], torch.bfloat16)
    st["workspace"] = None
    return st


def _run_own(st):
    import moe_grouped_gemm_e4m3_amd as fg

    op, c = st["op"], st["case"]
    if op in ("route", "route_step"):
        ids, w = fg.moe_route(st["logits"], c["k"], st["ids"], st["w"], bias=st["bias"], scoring=c["scoring"],
                              groups=c["groups"], top_groups=c["top"], normalize=c["normalize"], scale=2.5)
        if op == "route":
            return [ids, w]
        return [ids, w, fg.moe_route_backward(st["dw"], st["logits"], ids, st["dl"], scoring=c["scoring"],
                                              normalize=c["normalize"], scale=2.5)]
    if op == "int4":
        return fg.gemm_int4_nt(st["A"], st["B"], st["s"], st["D"], zb=st["z"], group=c["group"])
    if st["workspace"] is None:
        # a decode loop's own, kept from call to call
        st["workspace"] = torch.empty(fg.moe_ffn_workspace_bytes(c["T"], c["k"], c["F"]), dtype=torch.uint8, device="cuda")
    if op == "moe_fp8":
        return fg.moe_ffn_fp8(st["X"], st["W1"], st["s1"], st["W2"], st["s2"], st["ids"], st["w"], st["D"],
                              activation=c["act"], workspace=st["workspace"])
    return fg.moe_ffn_int4(st["X"], st["W1"], st["s1"], st["W2"], st["s2"], st["ids"], st["w"], st["D"], z1=st["z1"],
                           z2=st["z2"], group=c["group"], activation=c["act"], workspace=st["workspace"])


def _route(st):
    """ids, weights, the chosen experts' shares and all scores, in 64 bits."""
    c = st["case"]
    l = st["logits"].double()
    T, E = l.shape
    if c["scoring"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True).clamp_min(-1e300))
        s = e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
    # without a bias and groups the scores order as the logits do
    by = l if st["bias"] is None and c["groups"] == 1 else s if st["bias"] is None else s + st["bias"].double()
    by = torch.where(l == -math.inf, l, by)
    if c["groups"] > 1:
        per = by.view(T, c["groups"], -1)
        two = per.sort(dim=2, descending=True)[0][:, :, :2]
        total = torch.where(two == -math.inf, torch.zeros_like(two), two).sum(dim=2)
        total = torch.where(two[:, :, 0] == -math.inf, two[:, :, 0], total)
        kept = torch.zeros_like(total, dtype=torch.bool)
        kept.scatter_(1, total.sort(dim=1, descending=True, stable=True)[1][:, :c["top"]], True)
        by = torch.where(kept[:, :, None], per, torch.full_like(per, -math.inf)).view(T, E)
    best, ids = by.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :c["k"]], ids[:, :c["k"]]
    there = best > -math.inf
    chosen = torch.where(there, s.gather(1, ids), torch.zeros_like(best))
    share = chosen / chosen.sum(dim=1, keepdim=True).clamp_min(1e-300) if c["normalize"] else chosen
    return torch.where(there, ids, -torch.ones_like(ids)).to(torch.int32), (2.5 * share).float(), share, s


def _route_grad(st, ids, share, s):
    c = st["case"]
    there = ids >= 0
    at = ids.clamp_min(0).long()
    g = torch.where(there, st["dw"].double(), torch.zeros_like(share)) * 2.5
    own_score = s.gather(1, at)
    if c["normalize"]:
        d = share * (g - (g * share).sum(dim=1, keepdim=True))
        if c["scoring"] == "sigmoid":
            d = d * (1.0 - own_score)
    elif c["scoring"] == "sigmoid":
        d = g * own_score * (1.0 - own_score)
    else:
        d = g * own_score
    dl = torch.zeros_like(s).scatter_add_(1, at, torch.where(there, d, torch.zeros_like(d)))
    if c["scoring"] == "softmax" and not c["normalize"]:
        dl = dl - s * (g * own_score).sum(dim=1, keepdim=True)
    return dl.to(st["logits"].dtype)


def _wide_int4(q, s, z, group, cols):
    """Packed 4-bit weights [..., rows, bytes] in 32 bits."""
    lead, chunks = q.shape[:-1], q.shape[-1] // 64
    b = q.view(*lead, chunks, 4, 4, 4).transpose(-3, -2)
    codes = torch.stack([b & 15, b >> 4], dim=-2).reshape(*lead, chunks * 128)[..., :cols].float()
    zero = 8.0 if z is None else z.float().repeat_interleave(group, dim=-1)[..., :cols]
    return (codes - zero) * s.float().repeat_interleave(group, dim=-1)[..., :cols]


def _wide_fp8(q, s):
    rows, cols = q.shape[-2:]
    wide = s.repeat_interleave(128, dim=-2)[..., :rows, :].repeat_interleave(128, dim=-1)[..., :cols]
    return q.float() * wide


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))


def _moe(st):
    c = st["case"]
    T, E, k, F, K = (c[n] for n in ("T", "E", "k", "F", "K"))
    there = st["ids"] >= 0
    w = torch.where(there, st["w"], torch.zeros_like(st["w"]))
    at = st["ids"].clamp_min(0).long()
    X = st["X"].float()
    if T * k < E:  # fewer pairs than experts: the chosen experts' weights are gathered, a pair at a time
        pick = at.view(-1)
        x = X.repeat_interleave(k, dim=0)[:, :, None]
    else:  # every expert sees every token
        pick = torch.arange(E, device=X.device)
        x = X.t()[None].expand(E, K, T).contiguous()
    if c["op"] == "moe_fp8":
        gu = torch.bmm(_wide_fp8(st["W1"].view(torch.uint8)[pick].view(torch.float8_e4m3fn), st["s1"][pick]), x)
    else:
        gu = torch.bmm(_wide_int4(st["W1"][pick], st["s1"][pick], None if st["z1"] is None else st["z1"][pick],
                                  c["group"], K), x)
    h = _act(gu[:, :F], c["act"]) * gu[:, F:]
    if c["op"] == "moe_fp8":
        y = torch.bmm(_wide_fp8(st["W2"].view(torch.uint8)[pick].view(torch.float8_e4m3fn), st["s2"][pick]), h)
    else:
        y = torch.bmm(_wide_int4(st["W2"][pick], st["s2"][pick], None if st["z2"] is None else st["z2"][pick],
                                 c["group"], F), h)
    if T * k < E:
        return (y.view(T, k, K) * w[:, :, None]).sum(dim=1).bfloat16()
    gate = torch.zeros(T, E, device=X.device).scatter_add_(1, at, w)
    return (y * gate.t()[:, None, :]).sum(dim=0).t().contiguous().bfloat16()


def run(state):
    if own:
        return _run_own(state)
    st, op = state, state["op"]
    if op in ("route", "route_step"):
        ids, w, share, s = _route(st)
        return [ids, w] if op == "route" else [ids, w, _route_grad(st, ids, share, s)]
    if op == "int4":
        c = st["case"]
        return (st["A"].float() @ _wide_int4(st["B"], st["s"], st["z"], c["group"], c["K"]).t()).bfloat16()
    return _moe(st)


def _weight_bytes(case, rows, cols):
    if case["op"] == "moe_fp8":
        return rows * cols + 4 * -(-rows // 128) * -(-cols // 128)
    return rows * cols // 2 + rows * -(-cols // case["group"]) * (3 if case["zeros"] else 2)


def work(case):
    op = case["op"]
    if op in ("route", "route_step"):
        T, E, k = case["T"], case["E"], case["k"]
        item = 4 if case["dtype"] == "float32" else 2
        forward = T * E * item + T * k * 8 + (4 * E if case["bias"] else 0)
        if op == "route":
            return {"bytes": forward, "flops": 4 * T * E}
        return {"bytes": forward + T * E * item + 4 * T * k, "flops": 8 * T * E}
    if op == "int4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * (K + N) + _weight_bytes(case, N, K), "flops": 2 * M * N * K}
    T, E, k, F, K = (case[n] for n in ("T", "E", "k", "F", "K"))
    # experts that some token goes to, on average over the ids
    active = E * (1.0 - (1.0 - (1.0 - case["away"]) * k / E) ** T)
    weights = active * (_weight_bytes(case, 2 * F, K) + _weight_bytes(case, K, F))
    return {"bytes": weights + 4 * T * K + 8 * T * k, "flops": 6 * T * k * (1.0 - case["away"]) * F * K}


def _exact_route(st):
    """Row by row, by repeated choice of the best that is left."""
    c = st["case"]
    logits = st["logits"].double().cpu()
    bias = torch.zeros(c["E"], dtype=torch.float64) if st["bias"] is None else st["bias"].double().cpu()
    T, E = logits.shape
    if c["scoring"] == "softmax":
        top = logits.max(dim=1).values
        top[top == -math.inf] = 0.0
        un = torch.exp(logits - top[:, None])
        score = un / torch.clamp(un.sum(dim=1), min=1e-300)[:, None]
    else:
        score = torch.sigmoid(logits)
    plain = st["bias"] is None and c["groups"] == 1
    left = logits.clone() if plain else score + bias
    left[logits == -math.inf] = -math.inf
    size = E // c["groups"]
    if c["groups"] > 1:
        grouped = left.reshape(T, c["groups"], size)
        first, where = grouped.max(dim=2)
        rest = grouped.scatter(2, where[:, :, None], -math.inf)
        second = rest.max(dim=2).values if size > 1 else torch.full_like(first, -math.inf)
        total = first + torch.where(torch.isinf(second), torch.zeros_like(second), second)
        allowed = torch.zeros(T, c["groups"], dtype=torch.bool)
        rows = torch.arange(T)
        for _ in range(c["top"]):
            # argmax of equal values is not the first by contract: the first is looked for
            best = total.max(dim=1, keepdim=True).values
            g = (total == best).to(torch.int8).argmax(dim=1)
            allowed[rows, g] = True
            total[rows, g] = -math.inf
        left[~allowed.repeat_interleave(size, dim=1)] = -math.inf
    rows = torch.arange(T)
    picked, w = [], []
    for _ in range(c["k"]):
        best = left.max(dim=1, keepdim=True).values
        e = (left == best).to(torch.int8).argmax(dim=1)
        gone = best[:, 0] == -math.inf
        picked.append(torch.where(gone, torch.full_like(e, -1), e))
        w.append(torch.where(gone, torch.zeros(T, dtype=torch.float64), score[rows, e]))
        left[rows, e] = -math.inf
    ids, w = torch.stack(picked, dim=1), torch.stack(w, dim=1)
    if c["normalize"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    out = [None, (w * 2.5).cuda()]
    if st["op"] == "route":
        return out
    # the gradient from the Jacobian of each weight with respect to the scores, then of the scores
    dw = st["dw"].double().cpu() * 2.5 * (ids >= 0)
    ds = torch.zeros(T, E, dtype=torch.float64)
    chosen = torch.stack([score[rows, ids[:, j].clamp(min=0)] for j in range(c["k"])], dim=1) * (ids >= 0)
    total = chosen.sum(dim=1)
    mean = (dw * w).sum(dim=1) if c["normalize"] else None
    for j in range(c["k"]):
        d = dw[:, j] if not c["normalize"] else torch.where(total > 0, (dw[:, j] - mean) / total, torch.zeros(T).double())
        ds[rows, ids[:, j].clamp(min=0)] += torch.where(ids[:, j] >= 0, d, torch.zeros(T).double())
    if c["scoring"] == "softmax":
        dl = score * (ds - (ds * score).sum(dim=1, keepdim=True))
    else:
        dl = ds * score * (1.0 - score)
    return out + [dl.cuda()]


def _exact_weights(st, name, e, rows, cols):
    """Weights of expert e (or the only ones, e None) in 64 bits."""
    c = st["case"]
    pick = (lambda t: None if t is None else t) if e is None else (lambda t: None if t is None else t[e])
    q, s = pick(st["W" + name] if e is not None else st["B"]), pick(st["s" + name])
    r = torch.arange(rows, device=q.device)[:, None]
    k = torch.arange(cols, device=q.device)[None, :]
    if c["op"] == "moe_fp8":
        return q.double() * s.double()[r // 128, k // 128]
    inside = k % 128
    m, quarter, j = inside // 32, inside % 32 // 8, inside % 8
    at = (k // 128 * 64 + (quarter * 4 + m) * 4 + j % 4).expand(rows, cols)
    code = (q.gather(1, at) >> (4 * (j // 4)).to(torch.uint8)) % 16
    z = pick(st["z" + name])
    z = torch.full_like(s, 8.0) if z is None else z
    return s.double()[r, k // c["group"]] * (code.double() - z.double()[r, k // c["group"]])


def exact(case, seed):
    """The definitions in float64, an expert at a time."""
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_step"):
        return _exact_route(st)
    if op == "int4":
        out = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        a, step = st["A"].double(), 2048
        for lo in range(0, case["N"], step):
            part = dict(st, B=st["B"][lo:lo + step], s=st["s"][lo:lo + step],
                        z=None if st["z"] is None else st["z"][lo:lo + step])
            out[:, lo:lo + step] = torch.mm(a, _exact_weights(part, "", None, part["B"].shape[0], case["K"]).t())
        return out
    T, E, F, K = (case[n] for n in ("T", "E", "F", "K"))
    out = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    X, ids, w = st["X"].double(), st["ids"], st["w"].double()
    for e in range(E):
        gate = torch.where(ids == e, w, torch.zeros_like(w)).sum(dim=1)
        rows = (ids == e).any(dim=1).nonzero()[:, 0]
        if not rows.numel():
            continue
        p = torch.mm(X[rows], _exact_weights(st, "1", e, 2 * F, K).t())
        g, u = p[:, :F], p[:, F:]
        y = g if case["act"] == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        h = g * u / (1 + torch.exp(-y))
        out[rows] += gate[rows, None] * torch.mm(h, _exact_weights(st, "2", e, K, F).t())
    return out
