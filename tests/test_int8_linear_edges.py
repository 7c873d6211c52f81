"""Edge sizes of the per-row 8-bit cast and the 8-bit-integer product."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 3, 300])
def test_cast_of_empty_rows(gpu_lib, dtype, M):
    """K = 0: the scale of an empty row is the floor's, and a product on the
    codes is zero."""
    announce(f"int8 cast {M}x0 {dtype}")
    buf = torch.full((M + 1,), float("nan"), device="cuda")
    x = torch.empty(M, 0, dtype=dtype, device="cuda")
    q, s = gpu_lib.int8_cast_per_row(x, s=buf[:M])
    want_q, want_s = ref.int8_cast(np.zeros((M, 0), np.float32))
    assert q.shape == want_q.shape and np.array_equal(s.cpu().numpy(), want_s)
    assert torch.isnan(buf[M])
    w, sw = gpu_lib.int8_cast_per_row(torch.empty(5, 0, device="cuda"))
    D = torch.full((M, 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    gpu_lib.gemm_int8_nt(q, s, w, sw, D)
    assert (D == 0).all()


def test_cast_of_empty_rows_needs_the_scales_alone():
    """Refused without s; x and q are not looked at."""
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    for fn in (lib.int8_cast_per_row, lib.int8_cast_per_row_bf16):
        assert fn(None, 0, None, None, 4, 0, None) == 1
        assert "s is NULL" in lib.fg_last_error().decode()
        assert fn(None, 0, None, 0x10002, 4, 0, None) == 2
