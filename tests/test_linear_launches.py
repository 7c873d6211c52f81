"""Which kernels the calls of the 8-bit-integer products and the gated block
launch (the lines of FG_PRINT_CONFIGS), and the gradients of every kind of
launch that their own plans choose."""

from __future__ import annotations

import re

import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, f64, strided
from tests.test_gated_ffn import block

pytestmark = pytest.mark.gpu

# tile and threads of each plan; "small" is 64x64 in 512 threads for every operand order
TILES = {"w256": (256, 256, 512), "w224": (256, 224, 512), "w192": (256, 192, 512), "w160": (256, 160, 512),
         "mid2": (128, 128, 256), "mid": (128, 128, 512), "half2": (128, 64, 512), "small2": (64, 64, 256),
         "small": (64, 64, 512)}
FEW = [(16, 16, 4), (16, 16, 8), (16, 32, 4), (32, 16, 4), (32, 32, 4), (64, 16, 4), (64, 32, 4), (64, 64, 4)]


@pytest.fixture
def launches(monkeypatch, capfd):
    """launches(plan, call): runs call() with that plan forced ("": none) and
    returns its launches' lines as dictionaries."""
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")

    def run(plan, call):
        monkeypatch.setenv("FG_LINEAR_PLAN", plan)
        capfd.readouterr()
        call()
        torch.cuda.synchronize()
        found = []
        for line in capfd.readouterr().err.splitlines():
            m = re.match(r"\[fp8gemm\] (\w+) ((?:shared )?\w+) (.*)", line)
            if m:
                words = dict(w.split("=") for w in m[3].split() if "=" in w)
                found.append({"what": m[1], "launch": m[2], "few": "few-row" in m[3], **words})
        return found

    return run


def tile(line):
    return tuple(int(v) for v in line["tile"].split("x")) + (int(line["threads"]),)


@pytest.mark.parametrize("plan", ["w256", "w224", "w160", "mid2", "mid", "half2", "small2", "small"]
                         + [f"few{i}" for i in range(8)])
def test_forced_forward_plans_run(gpu_lib, launches, plan):
    M, N, K = 40, 96, 256
    announce(f"launch of int8 {plan}")
    q = torch.ones(2 * N, K, dtype=torch.int8, device="cuda")
    s = torch.ones(2 * N, device="cuda")
    h = torch.ones(2 * N, K, dtype=torch.bfloat16, device="cuda")
    D = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    P = torch.empty(M, 2 * N, device="cuda")
    calls = [lambda: gpu_lib.gemm_int8_nt(q[:M], s[:M], q[:N], s[:N], D)]
    if plan not in ("w224", "w160"):
        calls += [lambda: gpu_lib.gated_ffn_int8(q[:M], s[:M], q, s, D), lambda: gpu_lib.gated_ffn_bf16(h[:M], h, D),
                  lambda: gpu_lib.gated_ffn_bf16(h[:M], h, D, P=P)]
    for call in calls:
        line, = launches(plan, call)
        assert line["launch"] == "product"
        if plan.startswith("few"):
            assert line["few"] and tuple(int(line[k]) for k in ("rows", "cols", "waves")) == FEW[int(plan[3])]
        else:
            assert not line["few"] and tile(line) == TILES[plan]


def gradients(gpu_lib, M, F, K, kept=False, seed=6):
    """A call of the backward pass with odd strides: (call, check)."""
    X, W, dH = block(M, F, K, seed)
    Xd, Wd, dHd = strided(X, 8), strided(W, 16), strided(dH, 1)
    P = None
    if kept:
        P = torch.empty(M, 2 * F + 1, device="cuda")[:, :2 * F]
        gpu_lib.gated_ffn_bf16(Xd, Wd, torch.empty(M, F, dtype=torch.bfloat16, device="cuda"), P=P)
    dX, dW = Output(M, K, 3), Output(2 * F, K, 1)
    ws = torch.full((gpu_lib.gated_ffn_backward_workspace_bytes(M, F, K),), 255, dtype=torch.uint8, device="cuda")

    def call():
        gpu_lib.gated_ffn_bf16_backward(dHd, Xd, Wd, dX.t, dW.t, P=P, workspace=ws)

    def check(what):
        dX.check_untouched()
        dW.check_untouched()
        wx, ww, bx, bw = ref.gated_backward(f64(dH), f64(X), f64(W), "silu")
        assert_within(dX.f64(), wx, bx, f"dX {what}")
        assert_within(dW.f64(), ww, bw, f"dW {what}")

    return call, check


# a shape that has the plan, for each: dX and dW of a launch of their own, dX's
# sum split, and the shared launches with dX whole and split on either tile
FORCED = [(p, (130, 450, 136)) for p in ("w256", "w224", "w160", "mid2", "mid", "half2", "small2")]
FORCED += [("split-mid", (65, 700, 264)), ("split-small", (65, 700, 264)), ("pair", (190, 70, 1928))]
FORCED += [(f"share-{a}-{b}", s) for a in ("mid", "small") for b in ("mid", "small")
           for s in ((260, 69, 520), (65, 2695, 1096) if a == "mid" else (5, 1025, 136))]


@pytest.mark.parametrize("plan,shape", FORCED)
def test_forced_gradient_plans_run(gpu_lib, launches, plan, shape):
    announce(f"launch of gradients {plan} {shape}")
    call, check = gradients(gpu_lib, *shape)
    lines = {x["launch"]: x for x in launches(plan, call)}
    if plan in TILES:
        assert tile(lines["dX"]) == tile(lines["dW"]) == TILES[plan] and lines["dX"]["splits"] == "1"
    elif plan == "pair":
        assert tile(lines["pair"]) == TILES["small"] and int(lines["pair"]["splits"]) > 1
    elif plan.startswith("split"):
        assert tile(lines["dX"]) == TILES[plan.split("-")[1]] and int(lines["dX"]["splits"]) > 1 and "dW" in lines
    else:
        x, w = plan.split("-")[1:]
        assert tile(lines["shared dX"]) == TILES[x] and tile(lines["shared dW"]) == TILES[w]
        assert (int(lines["shared dX"]["splits"]) > 1) == (shape[1] > 500)
    check(plan)


# (M, F, K), launches on 256 CUs: tiles of dX and dW, whether they share a
# launch, whether dX's sum is split
OWN = [
    ((260, 69, 3152), "mid", "mid", True, False), ((321, 5, 72), "mid", "small", True, False),
    ((37, 130, 72), "small", "mid", True, False), ((5, 33, 8), "small", "small", True, False),
    ((65, 2695, 1096), "mid", "mid", True, True), ((1860, 2706, 8), "mid", "small", True, True),
    ((5, 1025, 136), "small", "mid", True, True), ((33, 385, 136), "small", "small", True, True),
    ((593, 3229, 352), "mid", "mid", True, True),
    ((1, 769, 2352), "mid", "mid2", False, True), ((1, 899, 1544), "small", "mid2", False, True),
]


@pytest.mark.parametrize("kept", [False, True], ids=["recomputed", "kept"])
@pytest.mark.parametrize("shape,x,w,shared,split", OWN)
def test_gradients_of_every_kind_of_launch(gpu_lib, launches, shape, x, w, shared, split, kept):
    announce(f"gradients {shape} kept={kept}")
    call, check = gradients(gpu_lib, *shape, kept=kept)
    lines = {v["launch"]: v for v in launches("", call)}
    check(str(shape))
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        return  # another plan
    pre = "shared " if shared else ""
    assert tile(lines[pre + "dX"]) == TILES[x] and (int(lines[pre + "dX"]["splits"]) > 1) == split
    assert tile(lines[pre + "dW"]) == TILES[w]


def test_plans_that_a_call_does_not_have(gpu_lib, launches):
    """The call's own plan runs: "small" has no gradient tile of its own
    launch, "w192" no plain product, and no call knows the others."""
    call, check = gradients(gpu_lib, 130, 450, 136)
    own = launches("", call)
    for plan in ("few3", "share-mid", "none"):
        assert launches(plan, call) == own, plan
    for plan in ("small", "w192"):  # these are plans of the recomputed pair
        assert [x for x in launches(plan, call) if x["launch"] != "pair"] == [x for x in own if x["launch"] != "pair"]
    check("own")
