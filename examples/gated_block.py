"""A gated feed-forward block, trained in BF16 and served on 8-bit integers.

    python examples/gated_block.py [--width 1024] [--hidden 2816] [--steps 60]

Training: ``GatedFFN`` is an autograd function over ``gated_ffn_bf16`` (which
keeps the pre-activations) and ``gated_ffn_bf16_backward``; a student block
learns the outputs of a teacher block of a quarter of its units, its fp32
weights copied to BF16 for each step.

Serving: the learnt weights are cast once, a scale per output channel
(``int8_cast_per_row``).  A call casts the tokens, runs ``gated_ffn_int8``,
casts the hidden units and runs ``gemm_int8_nt`` for the down projection;
single tokens replay it as a HIP graph.  Everything runs on the current stream.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_grouped_gemm_e4m3_amd as fg  # noqa: E402


class GatedFFN(torch.autograd.Function):
    """H = act(X W[:F]^T) * (X W[F:]^T) for bf16 X [M, K] and W [2F, K]."""

    @staticmethod
    def forward(ctx, X, W, activation):
        M, F = X.shape[0], W.shape[0] // 2
        H = torch.empty(M, F, dtype=torch.bfloat16, device=X.device)
        P = torch.empty(M, 2 * F, dtype=torch.float32, device=X.device)
        fg.gated_ffn_bf16(X, W, H, P=P, activation=activation)
        ctx.save_for_backward(X, W, P)
        ctx.activation = activation
        return H

    # a gradient of the gradients raises: the kernels have none to give
    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dH):
        X, W, P = ctx.saved_tensors
        dX = torch.empty_like(X) if ctx.needs_input_grad[0] else None
        dW = torch.empty_like(W) if ctx.needs_input_grad[1] else None
        fg.gated_ffn_bf16_backward(dH.contiguous(), X, W, dX, dW, P=P, activation=ctx.activation)
        return dX, dW, None


class Block(torch.nn.Module):
    """down(GatedFFN(x)) with fp32 master weights."""

    def __init__(self, width: int, hidden: int, activation: str = "silu", seed: int = 0):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.gate_up = torch.nn.Parameter(rand(2 * hidden, width) * width ** -0.5)
        self.down = torch.nn.Parameter(rand(width, hidden) * hidden ** -0.5)
        self.activation = activation

    def forward(self, x):
        h = GatedFFN.apply(x, self.gate_up.bfloat16(), self.activation)
        return torch.nn.functional.linear(h, self.down.bfloat16())


class Int8Block:
    """A trained Block on 8-bit integers, for up to ``rows`` tokens a call.
    Weights are cast once; buffers are the block's own."""

    def __init__(self, block: Block, rows: int):
        width, hidden = block.down.shape
        self.activation = block.activation
        self.W, self.sw = fg.int8_cast_per_row(block.gate_up.detach())
        self.Wd, self.sd = fg.int8_cast_per_row(block.down.detach())
        dev = "cuda"
        self.q = torch.empty(rows, width, dtype=torch.int8, device=dev)
        self.s = torch.empty(rows, dtype=torch.float32, device=dev)
        self.H = torch.empty(rows, hidden, dtype=torch.bfloat16, device=dev)
        self.qh = torch.empty(rows, hidden, dtype=torch.int8, device=dev)
        self.sh = torch.empty(rows, dtype=torch.float32, device=dev)

    def __call__(self, x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
        m = x.shape[0]
        q, s, H, qh, sh = self.q[:m], self.s[:m], self.H[:m], self.qh[:m], self.sh[:m]
        fg.int8_cast_per_row(x, q, s)
        fg.gated_ffn_int8(q, s, self.W, self.sw, H, activation=self.activation)
        fg.int8_cast_per_row(H, qh, sh)
        return fg.gemm_int8_nt(qh, sh, self.Wd, self.sd, y)


def tokens(n: int, width: int, seed: int) -> torch.Tensor:
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, width, device="cuda", generator=g).bfloat16()


def train(block: Block, teacher: Block, steps: int, batch: int) -> list[float]:
    width = block.down.shape[0]
    opt = torch.optim.Adam(block.parameters(), lr=2e-3)
    losses = []
    for step in range(steps):
        x = tokens(batch, width, 1000 + step)
        with torch.no_grad():
            want = teacher(x).float()
        loss = (block(x).float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def relative(got: torch.Tensor, want: torch.Tensor) -> float:
    return float((got.float() - want.float()).norm() / want.float().norm())


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--batch", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--activation", choices=sorted(fg.ACTIVATIONS), default="silu")
    a = ap.parse_args(argv)

    block = Block(a.width, a.hidden, a.activation, seed=1)
    teacher = Block(a.width, max(a.hidden // 4, 8), a.activation, seed=2)
    losses = train(block, teacher, a.steps, a.batch)
    print(f"training: {a.batch} tokens a step, loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    served = Int8Block(block, a.batch)
    x = tokens(a.batch, a.width, 7)
    with torch.no_grad():
        want = block(x)
    y = served(x, torch.empty_like(want))
    prefill = relative(y, want)
    print(f"serving {a.batch} tokens on 8-bit integers: relative difference {prefill:.4f}")

    # single tokens: one graph, replayed on new inputs
    x1, y1 = x[:1].clone(), torch.empty_like(want[:1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        served(x1, y1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        served(x1, y1)
    decode = 0.0
    for i in range(8):
        x1.copy_(x[i:i + 1])
        graph.replay()
        decode = max(decode, relative(y1, y[i:i + 1]))
    print(f"serving single tokens: relative difference to the batch {decode:.2e}")
    return {"losses": losses, "prefill": prefill, "decode": decode}


if __name__ == "__main__":
    main()
