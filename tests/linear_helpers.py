"""Inputs and comparisons shared by the tests of the 8-bit-integer products
and the gated feed-forward block."""

from __future__ import annotations

import numpy as np
import torch

from tests.helpers import SENTINEL_BF16, bf16_to_f64


def strided(a: torch.Tensor, pad: int, fill=None) -> torch.Tensor:
    """a on the GPU as a view of a buffer whose rows are `pad` elements longer
    (poisoned: NaN, or -128 for bytes), followed by one more poisoned row."""
    rows, cols = a.shape
    if fill is None:
        fill = -128 if a.dtype == torch.int8 else float("nan")
    buf = torch.full((rows + 1, cols + pad), fill, dtype=a.dtype, device="cuda")
    buf[:rows, :cols] = a.cuda()
    return buf[:rows, :cols]


class Output:
    """A [rows, cols] bf16 output inside a sentinel-filled buffer."""

    def __init__(self, rows: int, cols: int, pad: int = 0, offset: int = 0):
        ld = cols + pad
        self.buf = torch.full(((rows + 2) * ld + offset,), SENTINEL_BF16, dtype=torch.int16, device="cuda")
        self.rows, self.cols, self.ld = rows, cols, ld
        body = self.buf[offset:offset + rows * ld].view(torch.bfloat16)
        self.t = body.view(rows, ld)[:, :cols]

    def check_untouched(self):
        torch.cuda.synchronize()
        written = (self.buf != SENTINEL_BF16).sum().item()
        inside = (self.t.contiguous().view(torch.int16) != SENTINEL_BF16).sum().item()
        assert written == inside, f"{written - inside} values written outside the output"
        assert inside == self.rows * self.cols, f"{self.rows * self.cols - inside} outputs not written"

    def f64(self) -> np.ndarray:
        return bf16_to_f64(self.t.contiguous())


def assert_within(got: np.ndarray, want: np.ndarray, bound: np.ndarray, what: str):
    assert got.shape == want.shape
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    over = np.abs(got - want) - bound
    if over.size and over.max() > 0:
        i = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{what}: {np.count_nonzero(over > 0)} of {over.size} out of bounds, worst at {i}: "
                             f"{got[i]} for {want[i]} (bound {bound[i]:.3g})")


def bf16(a) -> torch.Tensor:
    return torch.as_tensor(a).to(torch.bfloat16)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to(torch.float64).cpu().numpy()
