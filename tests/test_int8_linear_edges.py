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


@pytest.mark.gpu
def test_cast_of_the_most_rows(gpu_lib):
    """2^31 - 1 rows: the row count plus one turn of the grid passes 2^31."""
    M, K = (1 << 31) - 1, 16
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 104 GiB of device memory")
    announce(f"int8 cast {M}x{K} bf16")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    ends = [slice(0, 3), slice((1 << 30) - 1, (1 << 30) + 2), slice(M - (1 << 20) - 2, M - (1 << 20) + 2),
            slice(M - 3, M)]
    some = torch.randn(4, K, generator=torch.Generator().manual_seed(0)).bfloat16()
    for e in ends:
        x[e] = some[:e.stop - e.start].cuda()
    q, s = gpu_lib.int8_cast_per_row(x)
    for e in ends:
        want_q, want_s = ref.int8_cast(some[:e.stop - e.start].float().numpy())
        assert np.array_equal(s[e].cpu().numpy(), want_s), e
        assert np.array_equal(q[e].cpu().numpy(), want_q), e
    zero = ref.int8_cast(np.zeros((1, K), np.float32))[1][0]
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    for e in ends:
        rest[e] = False
    step = 1 << 23
    for i in range(0, M, step):
        j = slice(i, min(i + step, M))
        assert bool(((s[j] == float(zero)) | ~rest[j]).all()), i
        assert not (q[j].view(torch.int64).any(dim=1) & rest[j]).any(), i
    del x, q, s, rest
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("ld", [-16, -(1 << 40), 1 << 60, 7])
@pytest.mark.parametrize("M,N", [(5, 40), (700, 300)])
def test_no_reduction_looks_at_no_operand(gpu_lib, M, N, ld):
    """K = 0: outputs are zero whatever the operands' pointers and strides."""
    announce(f"K=0 {M}x{N} ld={ld}")
    lib = gpu_lib.load_library()
    one = torch.ones(max(M, 2 * N), device="cuda")
    D = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    P = torch.full((M, 2 * N), float("nan"), device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    calls = [
        lambda: lib.gemm_int8_nt(None, ld, one.data_ptr(), None, ld, one.data_ptr(), D.data_ptr(), N, M, N, 0, s),
        lambda: lib.gated_ffn_int8(None, ld, one.data_ptr(), None, ld, one.data_ptr(), D.data_ptr(), N, M, N, 0, 0, s),
        lambda: lib.gated_ffn_bf16(None, ld, None, ld, D.data_ptr(), N, None, 0, M, N, 0, 1, s),
        lambda: lib.gated_ffn_bf16(None, ld, None, ld, D.data_ptr(), N, P.data_ptr(), 2 * N, M, N, 0, 0, s),
    ]
    for call in calls:
        D.fill_(float("nan"))
        assert call() == 0, lib.fg_last_error()
        assert (D == 0).all()
    assert (P == 0).all()


@pytest.mark.parametrize("M,N,needle", [((1 << 30) + 1, 64, "M=1073741825: more than 2^30"),
                                        (64, (1 << 29) + 1, "536870913 output columns, more than 2^29")])
def test_size_limits_are_named(M, N, needle):
    import moe_grouped_gemm_e4m3_amd as fg

    lib, q = fg.load_library(), 0x10000
    for st in (lib.gemm_int8_nt(q, 16, q, q, 16, q, q, N, M, N, 16, None),
               lib.gated_ffn_int8(q, 16, q, q, 16, q, q, N, M, N, 16, 0, None),
               lib.gated_ffn_bf16(q, 16, q, 16, q, N, None, 0, M, N, 16, 0, None)):
        assert st == 3 and needle in lib.fg_last_error().decode()
    F = min(N, (1 << 28) + 1)
    st = lib.gated_ffn_bf16_backward(q, F, q, 16, q, 16, None, 0, q, 16, q, 16, M, F, 16, 0, q, 1 << 62, None)
    assert st == 3 and ("M=1073741825" if M > 64 else "F=268435457: more than 2^28") in lib.fg_last_error().decode()
