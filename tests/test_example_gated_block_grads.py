"""Second derivatives through the example's autograd function."""

from __future__ import annotations

import pytest
import torch

from tests.helpers import announce

pytestmark = pytest.mark.gpu


def test_gradients_of_gradients_raise(gpu_lib):
    """The block's part of a second derivative is refused, not left out."""
    from examples.gated_block import GatedFFN

    announce("gradients of the example's gradients")
    X = torch.randn(9, 16, device="cuda").bfloat16().requires_grad_()
    W = torch.randn(12, 16, device="cuda").bfloat16().requires_grad_()
    scale = torch.ones((), device="cuda", requires_grad=True)
    loss = (GatedFFN.apply(X, W, "silu").float() * scale).square().sum()
    dX, = torch.autograd.grad(loss, X, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dX.float().square().sum().backward()
    # first derivatives alone are as before
    GatedFFN.apply(X, W, "silu").float().sum().backward()
    assert X.grad is not None and W.grad is not None
