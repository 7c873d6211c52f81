"""examples/gated_block.py end to end: training through the gated block's
gradients, serving through the 8-bit cast, gated block and product."""

from __future__ import annotations

import pytest
import torch

from tests.helpers import announce

pytestmark = pytest.mark.gpu


def test_autograd_function_matches_torch(gpu_lib):
    from examples.gated_block import GatedFFN

    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(37, 72, device="cuda", generator=g).bfloat16().requires_grad_()
    W = (torch.randn(2 * 45, 72, device="cuda", generator=g) / 8).bfloat16().requires_grad_()
    dH = torch.randn(37, 45, device="cuda", generator=g).bfloat16()
    H = GatedFFN.apply(X, W, "gelu_tanh")
    H.backward(dH)
    Xd, Wd = X.detach().double().requires_grad_(), W.detach().double().requires_grad_()
    p = Xd @ Wd.t()
    Hd = torch.nn.functional.gelu(p[:, :45], approximate="tanh") * p[:, 45:]
    Hd.backward(dH.double())
    # one bf16 rounding of H; of the gradient pair and of each gradient:
    # relative to the norm at most 2^-8 each
    for got, want, roundings in ((H, Hd, 1), (X.grad, Xd.grad, 2), (W.grad, Wd.grad, 2)):
        assert (got.double() - want).norm() <= roundings * 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("argv", [["--width", "256", "--hidden", "704", "--batch", "512"],
                                  ["--width", "208", "--hidden", "336", "--batch", "333", "--activation", "gelu_tanh"]])
def test_example(gpu_lib, argv):
    from examples.gated_block import main

    announce("example " + " ".join(argv))
    r = main(argv + ["--steps", "40"])
    assert r["losses"][-1] < 0.7 * r["losses"][0]
    # each cast rounds to 127 steps of its row's largest value: for Gaussian
    # rows of some hundred values (largest about 3.5 deviations) a relative
    # error of 3.5 / 127 / sqrt(12) = 0.8 %; four casts and a gated product of
    # two such factors stay under six times that
    assert r["prefill"] < 0.05
    # the plan differs, the integer sums do not
    assert r["decode"] == 0.0
