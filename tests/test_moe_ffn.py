"""The expert layers for a few tokens against their definition in float64."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import e4m3, experts as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, bf16, f64, strided
from tests.test_int4 import weights as int4_weights


class Fp8:
    name = "fp8"

    def __init__(self, E, rows, cols, seed):
        rng = np.random.default_rng(seed)
        self.codes = rng.integers(0, 256, (E, rows, cols)).astype(np.uint8)
        self.codes[(self.codes & 0x7F) == 0x7F] = 0x3C  # the format's NaN
        self.s = rng.uniform(0.5, 2.0, (E, -(-rows // 128), -(-cols // 128))).astype(np.float32) * 2.0 ** -7 / np.sqrt(cols)
        self.s = self.s.astype(np.float32)

    def wide(self, e):
        return ref.fp8_widen(e4m3.decode(self.codes[e]), self.s[e])

    def gpu(self):
        return torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.s).cuda()


class Int4:
    def __init__(self, E, rows, cols, seed, group, zeros):
        made = [int4_weights(rows, cols, group, zeros, seed * 100 + e) for e in range(E)]
        self.q, self.s, self.z = (np.stack([m[i] for m in made]) for i in range(3))
        self.s = ref.bf16_round(self.s * 8 / np.sqrt(cols))
        self.group, self.zeros, self.cols = group, zeros, cols

    def wide(self, e):
        return ref.int4_widen(self.q[e], self.s[e], self.z[e], self.group)

    def gpu(self):
        return (torch.from_numpy(np.stack([ref.int4_pack(q) for q in self.q])).cuda(), torch.from_numpy(self.s).bfloat16().cuda(),
                torch.from_numpy(self.z).cuda() if self.zeros else None)


class Layer:
    """Both weight matrices of E experts; fmt "fp8" or ("int4", group, zeros)."""

    def __init__(self, fmt, E, F, K, seed=0):
        self.fmt, self.E, self.F, self.K = fmt, E, F, K
        if fmt == "fp8":
            self.W1, self.W2 = Fp8(E, 2 * F, K, seed), Fp8(E, K, F, seed + 1)
        else:
            self.W1, self.W2 = Int4(E, 2 * F, K, seed, *fmt[1:]), Int4(E, K, F, seed + 1, *fmt[1:])

    def on_gpu(self):
        if not hasattr(self, "dev"):
            self.dev = self.W1.gpu(), self.W2.gpu()
        return self.dev

    def call(self, lib, X, ids, w, D, act="silu", **kw):
        a, b = self.on_gpu()
        if self.fmt == "fp8":
            return lib.moe_ffn_fp8(X, a[0], a[1], b[0], b[1], ids, w, D, activation=act, **kw)
        return lib.moe_ffn_int4(X, a[0], a[1], b[0], b[1], ids, w, D, z1=a[2], z2=b[2], group=self.fmt[1], activation=act, **kw)

    def want(self, X, ids, w, act="silu"):
        named = set(ids.reshape(-1).tolist())
        blank = (np.zeros((0, 0)), np.zeros((0, 0)))
        W1 = [self.W1.wide(e) if e in named else blank for e in range(self.E)]
        W2 = [self.W2.wide(e) if e in named else blank for e in range(self.E)]
        return ref.layer(X, W1, W2, ids, w, act)


def tokens(T, E, k, K, seed, away=0.0):
    g = torch.Generator().manual_seed(seed)
    X = bf16(torch.randn(T, K, generator=g))
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    ids[torch.rand(T, k, generator=g) < away] = -1
    w = torch.rand(T, k, generator=g) * 2 - 0.5
    return X, ids, w


def check(lib, layer, T, k, seed=1, away=0.0, act="silu", pad=0, offset=0):
    announce(f"layer {layer.fmt} T={T} E={layer.E} k={k} F={layer.F} K={layer.K} {act}")
    X, ids, w = tokens(T, layer.E, k, layer.K, seed, away)
    w[ids < 0] = float("nan")  # not read
    D = Output(T, layer.K, pad, offset)
    layer.call(lib, strided(X, 8 * pad), ids.cuda(), w.cuda(), D.t, act)
    D.check_untouched()
    assert_within(D.f64(), *layer.want(f64(X), ids.numpy(), w.numpy(), act), f"T={T}")


FORMATS = ["fp8", ("int4", 32, True), ("int4", 64, False), ("int4", 128, True), ("int4", 256, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS, ids=str)
@pytest.mark.parametrize("T,E,k,F,K", [(1, 1, 1, 32, 32), (1, 4, 2, 64, 96), (2, 3, 3, 160, 128), (7, 8, 2, 96, 288),
                                       (16, 5, 2, 128, 160), (17, 4, 4, 224, 256), (33, 2, 1, 64, 416), (64, 6, 3, 160, 64),
                                       (65, 3, 2, 32, 192), (140, 9, 2, 96, 128)])
def test_layer(gpu_lib, fmt, T, E, k, F, K):
    check(gpu_lib, Layer(fmt, E, F, K, seed=T), T, k, away=0.3 if T % 2 else 0.0, act="silu" if T % 3 else "gelu_tanh", pad=T % 3,
          offset=T % 2)


UPS = ["up-split2", "up-split4", "up-split16", "up-wide", "up-wide-deep", "up-wide8"]
DOWNS = ["down-split1", "down-split1-two", "down-split4", "down-split4-two", "down-wide16", "down-wide16-deep", "down-wide32"]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS, ids=str)
@pytest.mark.parametrize("plan", UPS + DOWNS + ["down-wide16,one-part", "down-wide32,one-part"])
def test_every_plan(gpu_lib, monkeypatch, capfd, fmt, plan):
    """Each kernel of either half, at sizes that end inside its tiles, with experts of one token and of more than one tile."""
    monkeypatch.setenv("FG_DECODE_PLAN", plan)
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")
    sizes = [(1, 3, 2, 160, 288), (13, 3, 2, 1056, 416), (64, 2, 1, 352, 160), (70, 4, 3, 96, 544)]
    if plan == "down-split1-two":
        sizes = sizes[:2]
    for T, E, k, F, K in sizes:
        check(gpu_lib, Layer(fmt, E, F, K, seed=T), T, k, pad=T % 2)
    ran = capfd.readouterr().err
    has = {"up-split2": fmt != "fp8", "up-wide8": fmt != "fp8", "down-split4-two": fmt != "fp8", "up-wide-deep": fmt == "fp8",
           "down-wide16-deep": fmt == "fp8"}
    if has.get(plan.split(",")[0], True):
        assert ran.count(plan.split(",")[0] + " ") >= len(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,F,K", [(1, 2, 1, 16, 16), (3, 4, 2, 48, 80), (20, 3, 2, 176, 144), (64, 2, 2, 208, 336)])
def test_fp8_columns_of_16(gpu_lib, T, E, k, F, K):
    """K and F that end inside a chunk's second half, a block and a row tile."""
    check(gpu_lib, Layer("fp8", E, F, K, seed=K), T, k)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", ("int4", 128, True)], ids=str)
@pytest.mark.parametrize("T,E,k,F,K", [(1, 8, 4, 1056, 2048), (6, 4, 2, 704, 1536), (40, 2, 1, 512, 1024)])
def test_layer_of_ordinary_width(gpu_lib, fmt, T, E, k, F, K):
    check(gpu_lib, Layer(fmt, E, F, K), T, k)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", ("int4", 32, False)], ids=str)
@pytest.mark.parametrize("T,E,k", [(1, 1024, 32), (3, 1024, 5), (64, 1000, 8), (64, 1, 1), (64, 40, 32)])
def test_many_experts(gpu_lib, fmt, T, E, k):
    """Pairs fewer and more than the experts; a thousand of them."""
    check(gpu_lib, Layer(fmt, E, 32, 32), T, k)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", ("int4", 64, True)], ids=str)
def test_ids(gpu_lib, fmt):
    """An expert twice in a row, ids outside the experts, tokens without any, all tokens to one expert."""
    announce(f"layer ids {fmt}")
    layer = Layer(fmt, 3, 96, 160)
    X, _, w = tokens(6, 3, 3, 160, 4)
    ids = torch.tensor([[1, 1, 1], [0, 2, 0], [-1, -1, -1], [3, 2 ** 31 - 1, -2 ** 31], [2, -1, 2], [0, 1, 2]], dtype=torch.int32)
    w[2], w[3] = float("nan"), float("inf")
    for t in (ids, torch.ones_like(ids)):
        D = Output(6, 160)
        c = w if t is ids else torch.nan_to_num(w, nan=0.5, posinf=0.25)
        layer.call(gpu_lib, X.cuda(), t.cuda(), c.cuda(), D.t)
        clean = t.numpy().copy()
        clean[(clean < 0) | (clean >= 3)] = -1
        assert_within(D.f64(), *layer.want(f64(X), clean, c.numpy()), "ids")
        if t is ids:
            assert (D.t[2:4] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 50])
def test_values_that_are_not_finite_stay_where_they_are(gpu_lib, T):
    """NaN codes and factors of experts that nobody names, tokens with an infinity or a NaN."""
    announce(f"layer not finite T={T}")
    layer = Layer("fp8", 5, 48, 144)
    X, ids, w = tokens(T, 4, 2, 144, 6)
    X[1, 5], X[2, 143] = float("inf"), float("nan")
    layer.W1.codes[4], layer.W2.codes[4] = 0x7F, 0xFF
    layer.W1.s[4], layer.W2.s[4] = np.nan, np.inf
    D = Output(T, 144)
    layer.call(gpu_lib, X.cuda(), ids.cuda(), w.cuda(), D.t)
    Xc = np.nan_to_num(f64(X), nan=0, posinf=0)
    want, bound = layer.want(Xc, ids.numpy(), w.numpy())
    rows = [t for t in range(T) if t not in (1, 2)]
    assert_within(D.f64()[rows], want[rows], bound[rows], "finite tokens")
    assert not np.isfinite(D.f64()[1]).any() and np.isnan(D.f64()[2]).all()


@pytest.mark.gpu
def test_large_and_small_hidden_units(gpu_lib):
    """h of 1e30 and of 1e-36: the second part of h neither overflows nor makes a NaN."""
    announce("layer hidden range")
    layer = Layer("fp8", 2, 64, 64)
    X, ids, w = tokens(4, 2, 1, 64, 2)
    for scale in (1e15, 1e-18):
        Y = bf16(X.float() * scale)
        D = Output(4, 64)
        layer.call(gpu_lib, Y.cuda(), ids.cuda(), w.cuda(), D.t)
        assert_within(D.f64(), *layer.want(f64(Y), ids.numpy(), w.numpy()), f"scale {scale}")
    # h overflows: infinities, and no NaN that the exact sum does not have
    Y = bf16(X.float() * 1e25)
    D = torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")
    layer.call(gpu_lib, Y.cuda(), ids.cuda(), w.cuda(), D)
    assert not torch.isfinite(D).any()


@pytest.mark.gpu
def test_hidden_units_next_to_the_largest_number(gpu_lib):
    """A finite h that bf16 alone would round to an infinity."""
    announce("layer largest h")
    one = Layer("fp8", 1, 16, 16)
    one.W1.codes[:], one.W1.s[:] = 0, 1.0
    one.W1.codes[0, 0, 0] = one.W1.codes[0, 16, 1] = 0x38  # 1: g = x_0 and u = x_1, for the first unit
    one.W2.codes[:], one.W2.s[:] = 0x38, 2.0 ** -64
    X = torch.zeros(1, 16, dtype=torch.bfloat16)
    X[0, 0], X[0, 1] = 181 * 2.0 ** 56, 181 * 2.0 ** 57  # 32761 / 16384 2^127, for bf16's largest of 32640 / 16384
    ids, w, D = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, 1), Output(1, 16)
    one.call(gpu_lib, X.cuda(), ids.cuda(), w.cuda(), D.t)
    assert_within(D.f64(), *one.want(f64(X), ids.numpy(), w.numpy()), "largest h")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", ("int4", 32, True), ("int4", 64, True), ("int4", 128, True)], ids=str)
@pytest.mark.parametrize("T", [1, 3, 20, 64])
@pytest.mark.parametrize("plan", [""] + DOWNS)
def test_hidden_units_keep_24_bits(gpu_lib, monkeypatch, fmt, T, plan):
    """Hidden units of 64 (1 + 2^-10 + 2^-20) and 64 (1 + 2^-10), subtracted: every step of the formula is exact in fp32, and
    what is left are the 24-bit value's last bits alone.  64 and 2^-14 are bf16: the result has no tolerance."""
    if T > 16 and plan == "down-split1-two":
        pytest.skip("sums of 16 tokens at most")
    announce(f"layer 24 bits {fmt} T={T} {plan}")
    monkeypatch.setenv("FG_DECODE_PLAN", plan)
    F, K, a, b = 288, 32, 5, 261  # the hidden units: in different chunks, blocks and groups
    layer = Layer(fmt, 1, F, K)
    one = 0x38 if fmt == "fp8" else 1
    for W in (layer.W1, layer.W2):
        if fmt == "fp8":
            W.codes[:], W.s[:] = 0, 1.0
        else:
            W.q[:], W.s[:], W.z[:] = 0, 1.0, 0
    up = layer.W1.codes if fmt == "fp8" else layer.W1.q
    down = layer.W2.codes if fmt == "fp8" else layer.W2.q
    for f in (a, b):
        up[0, f, 0] = one  # g = x_0 = 64, where the gate is 1
        up[0, F + f, 1] = up[0, F + f, 2] = one
    up[0, F + a, 3] = one
    down[0, :, a] = down[0, :, b] = one
    if fmt == "fp8":
        layer.W2.codes[0, :, b] |= 0x80
    else:
        layer.W2.s[0, :, b // fmt[1]] = -1.0
    X = torch.zeros(T, K)
    X[:, 0], X[:, 1], X[:, 2], X[:, 3] = 64.0, 1.0, 2.0 ** -10, 2.0 ** -20
    X[:, 1:] *= torch.tensor([1.0, -2.0, 0.5, 2.0 ** 40])[torch.arange(T) % 4, None]
    ids, w, D = torch.zeros(T, 1, dtype=torch.int32), torch.ones(T, 1), Output(T, K)
    layer.call(gpu_lib, bf16(X).cuda(), ids.cuda(), w.cuda(), D.t)
    D.check_untouched()
    assert np.array_equal(D.f64(), np.repeat(f64(64 * X[:, 3:4]), K, axis=1))


@pytest.mark.gpu
@pytest.mark.parametrize("plan", [""] + DOWNS)
def test_infinite_hidden_units_stay_infinite(gpu_lib, monkeypatch, plan):
    """A hidden unit past fp32 is an infinity and the sum with it one too, of its sign; a NaN stays a NaN."""
    announce(f"layer infinite h {plan}")
    monkeypatch.setenv("FG_DECODE_PLAN", plan)
    layer = Layer("fp8", 1, 16, 16)
    layer.W1.codes[:], layer.W1.s[:] = 0, 1.0
    layer.W1.codes[0, 0, 0] = layer.W1.codes[0, 16, 1] = 0x38
    layer.W2.codes[:], layer.W2.s[:] = 0x38, 1.0
    X = torch.zeros(4, 16, dtype=torch.bfloat16)
    X[:, 0] = 2.0 ** 100
    X[0, 1], X[1, 1], X[2, 1], X[3, 1] = 2.0 ** 100, -2.0 ** 100, float("nan"), 2.0 ** -100
    ids, w, D = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, 1), Output(4, 16)
    layer.call(gpu_lib, X.cuda(), ids.cuda(), w.cuda(), D.t)
    got = D.f64()
    assert (got[0] == np.inf).all() and (got[1] == -np.inf).all() and np.isnan(got[2]).all() and (got[3] == 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", ("int4", 128, False)], ids=str)
def test_offsets_past_32_bits(gpu_lib, fmt):
    """The last expert's weights lie past 4 GiB."""
    announce(f"layer offsets {fmt}")
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 8 GiB of device memory")
    F, K = 1024, 4096
    E = 540 if fmt == "fp8" else 1024
    small = Layer(fmt, 1, F, K)
    a, b = small.on_gpu()
    wide = []
    for m in (a, b):
        made = []
        for t in m:
            if t is None:
                made.append(None)
                continue
            big = torch.zeros(E, *t.shape[1:], dtype=t.dtype, device="cuda")
            big[-1] = t[0]
            made.append(big)
        wide.append(tuple(made))
    layer = Layer.__new__(Layer)
    layer.fmt, layer.E, layer.F, layer.K, layer.dev = fmt, E, F, K, tuple(wide)
    X, ids, w = tokens(2, 1, 1, K, 3)
    D = Output(2, K)
    layer.call(gpu_lib, X.cuda(), (ids + E - 1).cuda(), w.cuda(), D.t)
    assert_within(D.f64(), *small.want(f64(X), ids.numpy(), w.numpy()), "last expert")


@pytest.mark.gpu
def test_empty(gpu_lib):
    announce("layer empty")
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    u8, f = dict(dtype=torch.uint8, device="cuda"), dict(device="cuda")
    D = torch.full((3, 32), float("nan"), **bf)
    ids, w = torch.zeros(3, 2, **i32), torch.ones(3, 2, **f)
    gpu_lib.moe_ffn_fp8(torch.ones(3, 32, **bf), torch.zeros(2, 0, 32, **u8), torch.zeros(2, 0, 1, **f), torch.zeros(2, 32, 0, **u8),
                        torch.zeros(2, 1, 0, **f), ids, w, D)
    assert (D == 0).all()  # no hidden units
    gpu_lib.moe_ffn_fp8(torch.ones(0, 32, **bf), torch.zeros(2, 32, 32, **u8), torch.zeros(2, 1, 1, **f),
                        torch.zeros(2, 32, 16, **u8), torch.zeros(2, 1, 1, **f), ids[:0], w[:0], D[:0])


@pytest.mark.gpu
def test_same_bits_again_and_on_another_stream(gpu_lib):
    announce("layer streams")
    layer = Layer("fp8", 6, 160, 256)
    X, ids, w = (t.cuda() for t in tokens(37, 6, 3, 256, 1))
    first = layer.call(gpu_lib, X, ids, w, torch.empty(37, 256, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    ws = torch.full((gpu_lib.moe_ffn_workspace_bytes(37, 3, 160),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    D = torch.empty_like(first)
    layer.call(gpu_lib, X, ids, w, D, stream=side, workspace=ws)
    side.synchronize()
    assert torch.equal(D.view(torch.int16), first.view(torch.int16))
    for _ in range(3):
        layer.call(gpu_lib, X, ids, w, D)
        assert torch.equal(D.view(torch.int16), first.view(torch.int16))


@pytest.mark.gpu
def test_calls_side_by_side(gpu_lib):
    """Two layers and a product with a split reduction on three streams at once, each with its own workspace, beside what
    they give one after the other."""
    announce("layers side by side")
    layers = [Layer("fp8", 6, 160, 256), Layer(("int4", 32, True), 6, 160, 256)]
    X, ids, w = (t.cuda() for t in tokens(37, 6, 3, 256, 1))
    q, s, z = int4_weights(512, 24576, 128, True, 2)
    B, sb, zb = torch.from_numpy(ref.int4_pack(q)).cuda(), torch.from_numpy(s).bfloat16().cuda(), torch.from_numpy(z).cuda()
    A = torch.randn(30, 24576, device="cuda").bfloat16()
    assert gpu_lib.int4_workspace_bytes(30, 512, 24576) > 0

    def run(i, D, stream=None):
        if i < 2:
            layers[i].call(gpu_lib, X, ids, w, D, stream=stream)
        else:
            gpu_lib.gemm_int4_nt(A, B, sb, D, zb=zb, stream=stream)

    shapes = [(37, 256), (37, 256), (30, 512)]
    want = [torch.empty(*sh, dtype=torch.bfloat16, device="cuda") for sh in shapes]
    for i, D in enumerate(want):
        run(i, D)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    got = [[torch.zeros_like(D) for D in want] for _ in range(8)]
    torch.cuda.synchronize()
    for turn in got:
        for i, st in enumerate(streams):
            run(i, turn[i], st)
    torch.cuda.synchronize()
    for turn in got:
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(turn, want))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", ("int4", 64, True)], ids=str)
def test_decode_step_in_a_graph(gpu_lib, fmt):
    """Router, expert layer and a 4-bit projection, captured once and replayed on new tokens."""
    announce(f"decode step graph {fmt}")
    T, E, k, F, K, N = 5, 16, 3, 96, 160, 70
    layer = Layer(fmt, E, F, K)
    g = torch.Generator(device="cuda").manual_seed(0)
    head = torch.randn(N, K, device="cuda", generator=g)
    B, sb, zb = gpu_lib.int4_cast_per_group(head, group=32)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros(T, E, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w, D = torch.zeros(T, k, device="cuda"), torch.zeros_like(X)
    out = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gpu_lib.moe_ffn_workspace_bytes(T, k, F), dtype=torch.uint8, device="cuda")

    def step(workspace):
        gpu_lib.moe_route(logits, k, ids, w, scoring="sigmoid", groups=4, top_groups=2)
        layer.call(gpu_lib, X, ids, w, D, workspace=workspace)
        gpu_lib.gemm_int4_nt(D, B, sb, out, zb=zb, group=32)

    step(ws)
    torch.cuda.synchronize()
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws)
    with torch.cuda.graph(other):  # the same workspace, and one from torch's allocator
        step(ws)
        step(None)
    for i in range(4):
        X.copy_(torch.randn(T, K, device="cuda", generator=g))
        logits.copy_(torch.randn(T, E, device="cuda", generator=g))
        step(None)
        want = [t.clone() for t in (ids, w, D, out)]
        for gr in (graph, other):
            for t in (ids, w, D, out):
                t.zero_()
            torch.cuda.synchronize()
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, (ids, w, D, out)))
        want_ids, want_w = ref.route(f64(logits), k, scoring="sigmoid", groups=4, top_groups=2)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert_within(f64(D), *layer.want(f64(X), want_ids, w.cpu().numpy()), "layer")
        q, s, z = ref.int4_cast(head.cpu().numpy(), 32, False)
        assert_within(f64(out), *ref.gemm_int4(f64(D), q, s, z, 32), "projection")


def call(lib, fmt="fp8", X=0x10000, ldx=64, W1=0x10000, s1=0x10000, W2=0x10000, s2=0x10000, ids=0x10000, w=0x10000, D=0x10000,
         ldd=64, T=4, k=2, E=4, F=64, K=64, act=0, ws=0x10000, nbytes=1 << 22, group=128):
    if fmt == "fp8":
        return lib.moe_ffn_fp8(X, ldx, W1, s1, W2, s2, ids, w, D, ldd, T, k, E, F, K, act, ws, nbytes, None)
    return lib.moe_ffn_int4(X, ldx, W1, s1, None, W2, s2, None, ids, w, D, ldd, T, k, E, F, K, group, act, ws, nbytes, None)


@pytest.mark.parametrize("fmt", ["fp8", "int4"])
@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), 1, "T=-1"), (dict(K=-64), 1, "K=-64"), (dict(F=-16), 1, "F=-16"), (dict(k=0), 1, "k=0"), (dict(E=0), 1, "E=0"),
    (dict(K=72), 2, "K=72"), (dict(F=72), 2, "F=72"), (dict(act=5), 1, "activation=5"), (dict(X=None), 1, "X is NULL"),
    (dict(W1=None), 1, "W1 is NULL"), (dict(W2=None), 1, "W2 is NULL"), (dict(s1=None), 1, "s1 is NULL"), (dict(s2=None), 1, "s2 is NULL"),
    (dict(ids=None), 1, "ids is NULL"), (dict(w=None), 1, "weights is NULL"), (dict(D=None), 1, "D is NULL"),
    (dict(X=0x10008), 2, "X is not"), (dict(W1=0x10008), 2, "W1 is not"), (dict(W2=0x10004), 2, "W2 is not"),
    (dict(s1=0x10001), 2, "s1"), (dict(ids=0x10002), 2, "ids"), (dict(w=0x10002), 2, "weights"), (dict(D=0x10001), 2, "D is not"),
    (dict(ldx=56), 1, "ldx=56"), (dict(ldx=68), 2, "ldx=68"), (dict(ldd=63), 1, "ldd=63"), (dict(ldx=(1 << 21) + 8), 3, "4 MiB"),
    (dict(ws=None), 1, "workspace is NULL"), (dict(ws=0x10010), 2, "workspace"), (dict(nbytes=2099199), 1, "smaller than the 2099200"),
    (dict(nbytes=-1), 1, "negative"), (dict(E=1025), 3, "E=1025"), (dict(k=33), 3, "k=33"), (dict(T=(1 << 20) + 1), 3, "T=1048577"),
    (dict(K=65568, ldx=65568, ldd=65568), 3, "K=65568"), (dict(F=65568), 3, "F=65568"),
    (dict(T=0, X=None, W1=None, W2=None, D=None, ids=None, w=None, ws=None, nbytes=0), 0, "")])
def test_refusals(fmt, kw, status, needle):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    assert call(lib, fmt, **kw) == status, lib.fg_last_error()
    assert needle in lib.fg_last_error().decode()


def test_group_refusals_and_workspace_query():
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    for group in (0, 16, 48, 192, -32):
        assert call(lib, "int4", group=group) == 1 and "group" in lib.fg_last_error().decode()
    assert call(lib, "int4", K=48) == 2
    # hidden units (two bf16 each, rounded to 256 bytes), and half a MiB of partial sums for each of up to 64 tokens
    assert fg.moe_ffn_workspace_bytes(1, 3, 16) == 256
    assert fg.moe_ffn_workspace_bytes(3, 2, 64) == 3 * 2 * 64 * 4 + (3 << 19)
    assert fg.moe_ffn_workspace_bytes(1 << 20, 32, 1 << 16) == (1 << 43) + (64 << 19)
    for bad in ((-1, 2, 64), (1, -1, 64), (1, 2, -64), ((1 << 20) + 1, 1, 64), (1, 33, 64), (1, 1, (1 << 16) + 16)):
        with pytest.raises(ValueError):
            fg.moe_ffn_workspace_bytes(*bad)


@pytest.mark.parametrize("T,k,F", [(4, 0, 64), (0, 0, 64), (4, 2, 24), (4, 2, 8), (-1, 2, 64), (4, 33, 64), (4, 2, (1 << 16) + 16)])
def test_workspace_query_refuses_what_both_layers_refuse(T, k, F):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    assert lib.fg_moe_ffn_workspace_bytes(T, k, F) == -1
    for fmt in ("fp8", "int4"):
        assert call(lib, fmt, T=T, k=k, F=F, nbytes=1 << 40) != 0
    with pytest.raises(ValueError):
        fg.moe_ffn_workspace_bytes(T, k, F)


def test_wrapper_refusals():
    import moe_grouped_gemm_e4m3_amd as fg

    bf = torch.bfloat16
    args = [torch.zeros(2, 32, dtype=bf), torch.zeros(3, 64, 32, dtype=torch.uint8), torch.zeros(3, 1, 1),
            torch.zeros(3, 32, 32, dtype=torch.uint8), torch.zeros(3, 1, 1), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2),
            torch.zeros(2, 32, dtype=bf)]
    for fn in (fg.moe_ffn_fp8, fg.moe_ffn_int4):
        with pytest.raises(TypeError):  # not on the device
            fn(*args)
        with pytest.raises(ValueError):
            fn(args[0][0], *args[1:])


@pytest.mark.gpu
def test_wrapper_leaves_sizes_to_the_library(gpu_lib):
    bf, u8, f = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.uint8, device="cuda"), dict(device="cuda")
    for k, F, message in ((0, 32, "k=0"), (33, 32, "k=33"), (2, 24, "F=24")):
        with pytest.raises(gpu_lib.FP8GemmError, match=message):
            gpu_lib.moe_ffn_fp8(torch.zeros(2, 32, **bf), torch.zeros(3, 2 * F, 32, **u8), torch.zeros(3, 1, 1, **f), torch.zeros(3, 32, F, **u8),
                                torch.zeros(3, 1, 1, **f), torch.zeros(2, k, dtype=torch.int32, device="cuda"), torch.zeros(2, k, **f),
                                torch.zeros(2, 32, **bf))


@pytest.mark.gpu
def test_wrapper_checks(gpu_lib):
    bf, u8, f = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.uint8, device="cuda"), dict(device="cuda")
    a = dict(X=torch.zeros(2, 32, **bf), W1=torch.zeros(3, 64, 32, **u8), s1=torch.zeros(3, 1, 1, **f), W2=torch.zeros(3, 32, 32, **u8),
             s2=torch.zeros(3, 1, 1, **f), ids=torch.zeros(2, 2, dtype=torch.int32, device="cuda"), weights=torch.zeros(2, 2, **f),
             D=torch.zeros(2, 32, **bf))
    gpu_lib.moe_ffn_fp8(**a)
    gpu_lib.moe_ffn_fp8(**{**a, "W1": a["W1"].view(torch.float8_e4m3fn)})
    for bad in (dict(W1=torch.zeros(3, 62, 32, **u8)), dict(W1=torch.zeros(2, 64, 32, **u8)), dict(s1=torch.zeros(3, 2, 1, **f)),
                dict(s2=torch.zeros(3, 1, 1, **bf)), dict(ids=a["ids"].long()), dict(ids=a["ids"][:1]), dict(weights=torch.zeros(2, 2, **bf)),
                dict(weights=torch.zeros(2, 3, **f)), dict(D=torch.zeros(3, 32, **bf)), dict(X=torch.zeros(2, 48, **bf)),
                dict(activation="relu"), dict(workspace=torch.zeros(64, **f)), dict(W2=a["W2"].transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            gpu_lib.moe_ffn_fp8(**{**a, **bad})
    with pytest.raises(gpu_lib.FP8GemmError, match="smaller"):
        gpu_lib.moe_ffn_fp8(**a, workspace=torch.zeros(16, **u8))
