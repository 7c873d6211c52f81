"""The 4-bit cast and product against their definitions in float64."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import experts as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, bf16, f64, strided


def weights(N, K, group, zeros, seed):
    """Codes, scales (bf16 values) and zero points, the whole range of codes."""
    rng = np.random.default_rng(seed)
    kg = -(-K // group)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    s = ref.bf16_round(rng.uniform(0.002, 0.05, (N, kg)) * rng.choice([-1, 1], (N, kg)))
    z = rng.integers(0, 16, (N, kg)).astype(np.uint8) if zeros else np.full((N, kg), 8, np.uint8)
    return q, s, z


def to_gpu(q, s, z, zeros):
    return (torch.from_numpy(ref.int4_pack(q)).cuda(), torch.from_numpy(s).bfloat16().cuda(),
            torch.from_numpy(z).cuda() if zeros else None)


def check_product(lib, M, N, K, group, zeros, seed=0, pad=0, offset=0):
    announce(f"int4 {M}x{N}x{K} group={group} zeros={zeros}")
    q, s, z = weights(N, K, group, zeros, seed)
    A = bf16(torch.randn(M, K, generator=torch.Generator().manual_seed(seed + 1)))
    D = Output(M, N, pad, offset)
    B, sb, zb = to_gpu(q, s, z, zeros)
    lib.gemm_int4_nt(strided(A, 8 * pad), B, sb, D.t, zb=zb, group=group)
    D.check_untouched()
    assert_within(D.f64(), *ref.gemm_int4(f64(A), q, s, z, group), f"{M}x{N}x{K}")


@pytest.mark.parametrize("K", [32, 96, 128, 160, 1056])
def test_packing_round_trip(K):
    rng = np.random.default_rng(K)
    q = rng.integers(0, 16, (3, K)).astype(np.uint8)
    b = ref.int4_pack(q)
    assert b.shape == (3, -(-K // 128) * 64) and np.array_equal(ref.int4_unpack(b, K), q)


def test_packing_by_hand():
    """Column 0 alone is bit 0 of byte 0; column 4 its high half; column 8 the fifth word; column 32 the second."""
    for col, byte, shift in [(0, 0, 0), (3, 3, 0), (4, 0, 4), (7, 3, 4), (8, 16, 0), (13, 17, 4), (32, 4, 0), (127, 63, 4), (128, 64, 0)]:
        q = np.zeros((1, 256), np.uint8)
        q[0, col] = 9
        b = ref.int4_pack(q)
        assert b[0, byte] == 9 << shift and np.count_nonzero(b) == 1


@pytest.mark.parametrize("symmetric", [True, False])
def test_oracle_cast_is_near(symmetric):
    """Every weight is within half a step of its code's value, where the code is not clamped by the rounded scale."""
    rng = np.random.default_rng(1)
    w = rng.standard_normal((20, 192)).astype(np.float32)
    q, s, z = ref.int4_cast(w, 64, symmetric)
    back, _ = ref.int4_widen(q, s, z, 64)
    step = np.repeat(s, 64, axis=1)
    # the bf16 scale is off by 2^-8 of itself, 15 codes wide, and the zero point by half a step
    assert (np.abs(back - w) <= (0.5 + 15 * 2.0 ** -8 + (0.0 if symmetric else 0.5)) * step).all()


@pytest.mark.gpu
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (3, 96, 64), (7, 160, 128), (33, 1056, 32), (130, 1536, 64), (5, 2112, 128),
                                       (2, 640, 256), (3, 1696, 384), (1, 4128, 4096), (9, 32, 128)])
def test_cast(gpu_lib, N, K, group, dtype, symmetric):
    announce(f"int4 cast {N}x{K} group={group} {dtype} symmetric={symmetric}")
    g = torch.Generator().manual_seed(N + K)
    w = (torch.randn(N, K, generator=g) * torch.rand(N, 1, generator=g)).to(dtype)
    w[0, :32] = 0  # a group of zeros where groups are 32
    if N > 2:
        w[1] = w[1].abs()  # one sign only
        w[2] = 0
    pad = 16
    kg, width = -(-K // group), -(-K // 128) * 64
    q = torch.full((N + 1, width), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((N + 1, kg), 77.0, dtype=torch.bfloat16, device="cuda")
    z = None if symmetric else torch.full((N + 1, kg), 77, dtype=torch.uint8, device="cuda")
    got = gpu_lib.int4_cast_per_group(strided(w, pad), group, symmetric, q[:N], s[:N], None if symmetric else z[:N])
    want_q, want_s, want_z = ref.int4_cast(w.float().numpy(), group, symmetric)
    assert np.array_equal(got[1].float().cpu().numpy(), want_s)
    assert np.array_equal(got[0].cpu().numpy(), ref.int4_pack(want_q))  # padding codes are zero
    assert (q[N] == 0xAA).all() and (s[N] == 77).all()
    if symmetric:
        assert got[2] is None
    else:
        assert np.array_equal(got[2].cpu().numpy(), want_z) and (z[N] == 77).all()
    again = gpu_lib.int4_cast_per_group(w.cuda(), group, symmetric)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("group", [32, 128, 256])
def test_cast_of_the_largest_weights(gpu_lib, dtype, symmetric, group):
    """hi - lo past the largest fp32: scales and codes stay those of the definition, whose span is taken of halves."""
    announce(f"int4 cast largest {dtype} {symmetric} {group}")
    top = torch.finfo(dtype).max
    w = torch.rand(5, 288, generator=torch.Generator().manual_seed(3)).sub(0.5).mul(2.0).double()
    w[0] *= top
    w[1] *= 2.0 ** 127
    w[2, :40] = top
    w[2, 40:] = -top
    w[3, 0], w[3, 1] = top, -top
    w = w.to(dtype)
    assert torch.isfinite(w).all()
    q, s, z = gpu_lib.int4_cast_per_group(w.cuda(), group, symmetric)
    want_q, want_s, want_z = ref.int4_cast(w.float().numpy(), group, symmetric)
    assert np.isfinite(want_s).all() and np.array_equal(s.float().cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), ref.int4_pack(want_q)) and (symmetric or np.array_equal(z.cpu().numpy(), want_z))
    # a code's value is within the steps of test_oracle_cast_is_near of its weight
    back, _ = ref.int4_widen(want_q, want_s, want_z, group)
    step = np.repeat(want_s.astype(np.float64), group, axis=1)[:, :288]
    assert (np.abs(back - w.double().numpy()) <= (0.5 + 15 * 2.0 ** -8 + (0.0 if symmetric else 0.5)) * step).all()


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128, 384])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 40, 96), (2, 17, 128), (15, 33, 160), (16, 100, 1056), (17, 48, 544),
                                   (32, 31, 256), (33, 65, 1184), (64, 130, 416), (65, 20, 288), (130, 50, 2080)])
def test_product(gpu_lib, M, N, K, group, zeros):
    check_product(gpu_lib, M, N, K, group, zeros, seed=M, pad=M % 3, offset=M % 2)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M,N,K", [(1, 40, 1056), (7, 130, 416), (40, 50, 2080)])
def test_zero_points_up_to_255(gpu_lib, M, N, K, group):
    """Any uint8 zero point, far outside the codes too."""
    announce(f"int4 zero points {M}x{N}x{K} group={group}")
    q, s, z = weights(N, K, group, True, 12)
    z = np.random.default_rng(M).integers(0, 256, z.shape).astype(np.uint8)
    z[0, 0], z[-1, -1] = 255, 16
    A = bf16(torch.randn(M, K, generator=torch.Generator().manual_seed(4)))
    D = Output(M, N)
    B, sb, zb = to_gpu(q, s, z, True)
    gpu_lib.gemm_int4_nt(A.cuda(), B, sb, D.t, zb=zb, group=group)
    assert_within(D.f64(), *ref.gemm_int4(f64(A), q, s, z, group), f"{M}x{N}x{K}")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,group", [(1, 2112, 7168, 128), (4, 1024, 2048, 32), (16, 600, 8192, 64), (64, 300, 4096, 128)])
def test_product_of_whole_layers(gpu_lib, M, N, K, group):
    check_product(gpu_lib, M, N, K, group, True, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("plan", ["split2", "split2deep", "split8", "split8deep", "split16", "split16deep", "wide16", "wide32", "wide64",
                                  "wide16,kparts3", "wide32,kparts2", "wide64,kparts5", "wide16,kparts8"])
def test_every_plan(gpu_lib, monkeypatch, capfd, plan, group, zeros):
    monkeypatch.setenv("FG_DECODE_PLAN", plan)
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")
    for M, N, K in ((1, 40, 96), (7, 130, 2208), (37, 131, 4128), (70, 33, 1056)):
        check_product(gpu_lib, M, N, K, group, zeros, seed=M, pad=M % 2)
    assert capfd.readouterr().err.count(" " + plan.split(",")[0] + " ") == 4


@pytest.mark.gpu
@pytest.mark.parametrize("plan", ["wide16", "wide32", "wide64", "wide16,kparts3", "split2", "split16deep"])
@pytest.mark.parametrize("M", [1, 2])
def test_forced_plans_of_one_and_two_rows(gpu_lib, monkeypatch, plan, M):
    """Many chunks, few tiles: a plan that would split the reduction does without for rows that have no workspace."""
    monkeypatch.setenv("FG_DECODE_PLAN", plan)
    assert gpu_lib.int4_workspace_bytes(M, 200, 7168) == 0
    check_product(gpu_lib, M, 200, 7168, 128, True, seed=8)


@pytest.mark.gpu
def test_workspace(gpu_lib):
    """A product whose reduction is split: with a workspace, with one that holds NaN, with torch's, on another stream;
    one that is too small or misaligned is refused."""
    announce("int4 workspace")
    M, N, K = 30, 512, 24576
    need = gpu_lib.int4_workspace_bytes(M, N, K)
    assert need >= 2 * M * N * 4 and gpu_lib.int4_workspace_bytes(1, N, K) == 0
    q, s, z = weights(N, K, 128, True, 1)
    B, sb, zb = to_gpu(q, s, z, True)
    A = bf16(torch.randn(M, K, generator=torch.Generator().manual_seed(3))).cuda()
    D = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    gpu_lib.gemm_int4_nt(A, B, sb, D[0], zb=zb)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    gpu_lib.gemm_int4_nt(A, B, sb, D[1], zb=zb, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gpu_lib.gemm_int4_nt(A, B, sb, D[2], zb=zb, stream=side)
    side.synchronize()
    assert_within(f64(D[0]), *ref.gemm_int4(f64(A), q, s, z, 128), "split reduction")
    assert torch.equal(D[0].view(torch.int16), D[1].view(torch.int16)) and torch.equal(D[0].view(torch.int16), D[2].view(torch.int16))
    for bad in (ws[:need - 256], ws[16:]):
        with pytest.raises(gpu_lib.FP8GemmError):
            gpu_lib.gemm_int4_nt(A, B, sb, D[0], zb=zb, workspace=bad)


@pytest.mark.gpu
def test_empty_and_no_reduction(gpu_lib):
    announce("int4 empty")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    D = torch.full((3, 5), float("nan"), **bf)
    gpu_lib.gemm_int4_nt(torch.empty(3, 0, **bf), torch.empty(5, 0, **u8), torch.empty(5, 0, **bf), D)
    assert (D == 0).all()
    gpu_lib.gemm_int4_nt(torch.empty(0, 64, **bf), torch.empty(5, 64, **u8), torch.empty(5, 1, **bf), D[:0])
    gpu_lib.gemm_int4_nt(torch.empty(3, 64, **bf), torch.empty(0, 64, **u8), torch.empty(0, 1, **bf), D[:, :0])
    q, s, z = gpu_lib.int4_cast_per_group(torch.empty(4, 0, device="cuda"))
    assert q.shape == (4, 0) and s.shape == (4, 0) and z.shape == (4, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 40])
def test_values_that_are_not_finite_stay_in_their_row(gpu_lib, M):
    """A row of A with an infinity or NaN; scales of a weight row that are NaN; what lies behind a partial
    last group (the next row's scales) and in padding codes is not used."""
    announce(f"int4 not finite M={M}")
    N, K = 24, 160
    q, s, z = weights(N, K, 32, True, 3)
    A = bf16(torch.randn(M, K, generator=torch.Generator().manual_seed(0)))
    A[1, 3], A[2, 150] = float("inf"), float("nan")
    s[7, 0] = np.nan  # directly behind row 6's last group
    B, sb, zb = to_gpu(q, s, z, True)
    B.view(N, 2, 4, 4, 4)[:, 1, :, 1:] = 0xEE  # codes behind column 160
    D = Output(M, N)
    gpu_lib.gemm_int4_nt(A.cuda(), B, sb, D.t, zb=zb, group=32)
    got = D.f64()
    want, bound = ref.gemm_int4(np.nan_to_num(f64(A), posinf=1, neginf=1, nan=1), q, np.nan_to_num(s), z, 32)
    rows, cols = [r for r in range(M) if r not in (1, 2)], [c for c in range(N) if c != 7]
    at = np.ix_(rows, cols)
    assert_within(got[at], want[at], bound[at], "finite rows")
    assert np.isnan(got[:, 7]).all() and not np.isfinite(got[1]).any() and np.isnan(got[2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(1 << 18, 16384)])
def test_offsets_past_32_bits(gpu_lib, N, K):
    """2 GiB of codes: the last rows are those of a small matrix."""
    announce(f"int4 {N}x{K}")
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 3 GiB of device memory")
    q, s, z = weights(48, K, 128, True, 2)
    B, sb, zb = to_gpu(q, s, z, True)
    wide = torch.zeros(N + 48, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(N + 48, K // 128, dtype=torch.bfloat16, device="cuda")
    wz = torch.zeros(N + 48, K // 128, dtype=torch.uint8, device="cuda")
    wide[-48:], ws[-48:], wz[-48:] = B, sb, zb
    A = bf16(torch.randn(2, K, generator=torch.Generator().manual_seed(7)))
    D = torch.empty(2, N + 48, dtype=torch.bfloat16, device="cuda")
    gpu_lib.gemm_int4_nt(A.cuda(), wide, ws, D, zb=wz)
    assert_within(f64(D[:, -48:]), *ref.gemm_int4(f64(A), q, s, z, 128), "last rows")
    assert (D[:, :-48] == 0).all()


@pytest.mark.parametrize("M,N,K", [(-1, 8, 64), (8, -1, 64), (8, 8, -32), ((1 << 20) + 1, 8, 64), (8, (1 << 26) + 1, 64),
                                   (8, 8, (1 << 20) + 32), (30, 512, 24576 + 16), (1, 64, 48)])
def test_workspace_query_refuses_what_the_product_refuses(M, N, K):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    assert lib.fg_int4_workspace_bytes(M, N, K) == -1
    assert product_call(lib, M=M, N=N, K=K, lda=1 << 20, ldd=1 << 27, ws=0x10000, nbytes=1 << 40) != 0
    with pytest.raises(ValueError):
        fg.int4_workspace_bytes(M, N, K)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8])
def test_wrapper_leaves_sizes_to_the_library(gpu_lib, M):
    bf, u8 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.uint8, device="cuda")
    with pytest.raises(gpu_lib.FP8GemmError, match="K=48"):
        gpu_lib.gemm_int4_nt(torch.zeros(M, 48, **bf), torch.zeros(8, 64, **u8), torch.zeros(8, 1, **bf), torch.zeros(M, 8, **bf))


def product_call(lib, A=0x10000, lda=512, B=0x10000, s=0x10000, z=None, D=0x10000, ldd=64, M=4, N=64, K=512, group=128, ws=None,
                 nbytes=0):
    return lib.gemm_int4_nt(A, lda, B, s, z, D, ldd, M, N, K, group, ws, nbytes, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative"), (dict(N=-1), 1, "negative"), (dict(K=-32), 1, "negative"), (dict(K=48), 2, "K=48"),
    (dict(group=16), 1, "group=16"), (dict(group=96), 1, "group=96"), (dict(group=0), 1, "group=0"), (dict(group=-128), 1, "group"),
    (dict(A=None), 1, "A is NULL"), (dict(B=None), 1, "B is NULL"), (dict(s=None), 1, "sb is NULL"), (dict(D=None), 1, "D is NULL"),
    (dict(A=0x10008), 2, "A is not"), (dict(B=0x10008), 2, "B is not"), (dict(s=0x10001), 2, "sb"), (dict(D=0x10001), 2, "D"),
    (dict(lda=511), 1, "lda=511"), (dict(lda=516), 2, "lda=516"), (dict(ldd=63), 1, "ldd=63"),
    (dict(lda=(1 << 21) + 8), 3, "4 MiB"), (dict(K=(1 << 20) + 32, lda=1 << 21), 3, "K="), (dict(M=(1 << 20) + 1), 3, "2^20 rows"), (dict(N=(1 << 26) + 1, ldd=1 << 27), 3, "2^26 columns"),
    (dict(nbytes=-1), 1, "negative"), (dict(nbytes=64), 1, "workspace is NULL"), (dict(ws=0x10010, nbytes=64), 2, "256-byte"),
    (dict(M=32, N=512, ldd=512, K=24576, lda=24576), 1, "smaller than the"),
    (dict(M=0, A=None, B=None, s=None, D=None), 0, ""), (dict(N=0, A=None, B=None, s=None, D=None), 0, "")])
def test_product_refusals(kw, status, needle):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    assert product_call(lib, **kw) == status
    assert needle in lib.fg_last_error().decode()


@pytest.mark.parametrize("kw,status", [(dict(N=-1), 1), (dict(K=100), 2), (dict(group=8), 1), (dict(x=None), 1), (dict(q=None), 1),
                                       (dict(s=None), 1), (dict(x=0x10004), 2), (dict(q=0x10008), 2), (dict(s=0x10001), 2),
                                       (dict(ld=500), 1), (dict(ld=513), 2), (dict(K=(1 << 20) + 32, ld=1 << 21), 3),
                                       (dict(N=0, x=None, q=None, s=None), 0), (dict(K=0, x=None, q=None, s=None), 0)])
def test_cast_refusals(kw, status):
    import moe_grouped_gemm_e4m3_amd as fg

    lib = fg.load_library()
    a = dict(x=0x10000, ld=512, q=0x10000, s=0x10000, N=4, K=512, group=128)
    a.update(kw)
    for fn in (lib.int4_cast_per_group, lib.int4_cast_per_group_bf16):
        assert fn(a["x"], a["ld"], a["q"], a["s"], None, a["N"], a["K"], a["group"], None) == status, lib.fg_last_error()


def test_wrapper_refusals():
    import moe_grouped_gemm_e4m3_amd as fg

    bf = torch.bfloat16
    with pytest.raises(TypeError):
        fg.int4_cast_per_group(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        fg.int4_cast_per_group(torch.zeros(4, 64), group=48)
    with pytest.raises(ValueError):
        fg.int4_cast_per_group(torch.zeros(4, 64), symmetric=True, z=torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        fg.gemm_int4_nt(torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1, dtype=bf),
                        torch.zeros(4, 8, dtype=bf))


@pytest.mark.gpu
def test_wrapper_checks(gpu_lib):
    bf, u8 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.uint8, device="cuda")
    a = dict(A=torch.zeros(4, 160, **bf), B=torch.zeros(8, 128, **u8), sb=torch.zeros(8, 2, **bf), D=torch.zeros(4, 8, **bf))
    gpu_lib.gemm_int4_nt(**a)
    for bad in (dict(B=torch.zeros(8, 80, **u8)), dict(B=torch.zeros(7, 128, **u8)), dict(sb=torch.zeros(8, 2, device="cuda")),
                dict(sb=torch.zeros(8, 1, **bf)), dict(zb=torch.zeros(8, 3, **u8)), dict(zb=torch.zeros(8, 2, **bf)),
                dict(D=torch.zeros(5, 8, **bf)), dict(A=torch.zeros(160, 4, **bf).t()), dict(B=torch.zeros(8, 256, **u8)[:, ::2]),
                dict(group=17)):
        with pytest.raises((TypeError, ValueError)):
            gpu_lib.gemm_int4_nt(**{**a, **bad})
