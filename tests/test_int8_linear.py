"""Per-row 8-bit cast and the 8-bit-integer product, against float64."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, f64, strided


def codes(rows, cols, seed):
    rng = np.random.default_rng(seed)
    q = rng.integers(-127, 128, (rows, cols), dtype=np.int8)
    s = rng.uniform(0.5, 2.0, rows).astype(np.float32) * np.float32(2.0 ** -7)
    return q, s


# ---- cast -----------------------------------------------------------------


def test_cast_definition_against_brute_force():
    """The vectorised definition against one written value by value."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 32)).astype(np.float32)
    x[1] = 0
    x[2] *= 1e-6
    q, s = ref.int8_cast(x)
    for m in range(5):
        top = max(max(abs(float(v)) for v in x[m]), float(np.float32(1e-4)))
        assert s[m] == np.float32(np.float32(top) * np.float32(1 / 127))
        for k in range(32):
            assert q[m, k] == int(np.rint(np.float32(x[m, k] / s[m])))
    assert np.abs(q.astype(int)).max() <= 127


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 7168), (3, 2048), (5, 48), (64, 4096), (257, 1040), (2, 65536),
                                 (1000, 128), (7, 16400)])
def test_cast_is_bit_exact(gpu_lib, dtype, M, K):
    announce(f"int8 cast {M}x{K} {dtype}")
    gen = torch.Generator().manual_seed(M * 7 + K)
    x = (torch.randn(M, K, generator=gen) * torch.logspace(-6, 4, M)[:, None]).to(dtype)
    if M > 2:
        x[1] = 0.0
        x[2] = 1e-7  # below the floor of the scale
    q, s = gpu_lib.int8_cast_per_row(strided(x, 8))
    want_q, want_s = ref.int8_cast(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.gpu
def test_cast_ties_go_to_even(gpu_lib):
    """With amax = 127 the scale is 1 and halves are exact."""
    x = torch.zeros(2, 64)
    x[:, 0] = 127.0
    x[0, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5])
    x[1, 63] = -127.0
    q, s = gpu_lib.int8_cast_per_row(x.cuda())
    assert s.tolist() == [1.0, 1.0]
    assert q[0, :9].tolist() == [127, 0, 2, 2, 0, -2, -2, 126, -126]
    assert q[1, 63].item() == -127


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_cast_near_ties(gpu_lib, dtype):
    """Values a few units in the last place around every half step of many
    scales: the rounding is that of the fp32 quotient, exactly."""
    rows, K = 400, 512
    gen = torch.Generator().manual_seed(0)
    amax = (torch.rand(rows, generator=gen) * 4 + 0.01).to(dtype).float()
    half = torch.arange(K) % 254 - 126.5
    x = half[None, :] * (amax / 127)[:, None]
    ulps = torch.randint(-3, 4, (rows, K), generator=gen, dtype=torch.int32)
    x = (x.view(torch.int32) + ulps).view(torch.float32)
    x = x.to(dtype).float().clamp(-amax[:, None], amax[:, None])
    x[:, 7] = amax
    q, s = gpu_lib.int8_cast_per_row(x.to(dtype).cuda())
    want_q, want_s = ref.int8_cast(x.numpy())
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.gpu
def test_cast_writes_only_its_outputs(gpu_lib):
    x = torch.randn(3, 48, device="cuda")
    q = torch.full((4, 48), 99, dtype=torch.int8, device="cuda")
    s = torch.full((4,), 7.0, device="cuda")
    gpu_lib.int8_cast_per_row(x, q[:3], s[:3])
    assert (q[3] == 99).all() and s[3] == 7.0
    empty_q, empty_s = gpu_lib.int8_cast_per_row(torch.empty(0, 48, device="cuda"))
    assert empty_q.shape == (0, 48) and empty_s.shape == (0,)


# ---- product --------------------------------------------------------------

SHAPES = [
    # few rows, widths and reductions that end inside a tile or a slice
    (1, 1, 16), (1, 7, 16), (1, 300, 2048), (2, 33, 48), (5, 64, 1040), (16, 129, 144), (17, 96, 4096),
    (31, 257, 320), (64, 512, 1024), (65, 100, 272), (100, 640, 528), (128, 2112, 512), (129, 250, 1008),
    # many rows
    (200, 256, 256), (256, 256, 128), (300, 511, 400), (513, 300, 1024), (1000, 130, 160), (700, 1000, 2064),
    (257, 4100, 64), (2049, 65, 96),
]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("pads", [(0, 0), (16, 3)], ids=["packed", "strided"])
def test_gemm_matches_float64(gpu_lib, M, N, K, pads):
    announce(f"int8 gemm {M}x{N}x{K} {pads}")
    A, sa = codes(M, K, 1)
    B, sb = codes(N, K, 2)
    out = Output(M, N, pads[1])
    gpu_lib.gemm_int8_nt(strided(torch.from_numpy(A), pads[0]), torch.from_numpy(sa).cuda(),
                         strided(torch.from_numpy(B), 2 * pads[0]), torch.from_numpy(sb).cuda(), out.t)
    out.check_untouched()
    want, bound = ref.gemm_int8(A, sa, B, sb)
    assert_within(out.f64(), want, bound, f"{M}x{N}x{K}")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 33, 260])
def test_gemm_extreme_codes_do_not_overflow(gpu_lib, M):
    """The largest sums K allows: every product 128 * 128, or of alternating sign."""
    K, N = 131056, 33
    A = np.full((M, K), -128, np.int8)
    B = np.full((N, K), -128, np.int8)
    B[1::2, ::2] = 127
    one = np.ones(max(M, N), np.float32)
    out = Output(M, N)
    gpu_lib.gemm_int8_nt(torch.from_numpy(A).cuda(), torch.from_numpy(one[:M]).cuda(), torch.from_numpy(B).cuda(),
                         torch.from_numpy(one[:N]).cuda(), out.t)
    out.check_untouched()
    want, bound = ref.gemm_int8(A[:1], one[:1], B, one[:N])
    assert_within(out.f64(), np.repeat(want, M, 0), np.repeat(bound, M, 0), "extreme codes")


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_gemm_output_alignment(gpu_lib, offset):
    """Outputs that are 2-, 4- or 8-byte aligned, with odd and even strides."""
    M, N, K = 40, 72, 256
    A, sa = codes(M, K, 5)
    B, sb = codes(N, K, 6)
    for pad in (0, 1, 4):
        out = Output(M, N, pad, offset)
        gpu_lib.gemm_int8_nt(torch.from_numpy(A).cuda(), torch.from_numpy(sa).cuda(), torch.from_numpy(B).cuda(),
                             torch.from_numpy(sb).cuda(), out.t)
        out.check_untouched()
        want, bound = ref.gemm_int8(A, sa, B, sb)
        assert_within(out.f64(), want, bound, f"offset {offset} pad {pad}")


@pytest.mark.gpu
def test_gemm_empty_and_zero_reduction(gpu_lib):
    dev = dict(device="cuda")
    out = Output(3, 5)
    gpu_lib.gemm_int8_nt(torch.empty(3, 0, dtype=torch.int8, **dev), torch.ones(3, **dev),
                         torch.empty(5, 0, dtype=torch.int8, **dev), torch.ones(5, **dev), out.t)
    out.check_untouched()
    assert (out.t == 0).all()
    for M, N in ((0, 5), (3, 0)):
        gpu_lib.gemm_int8_nt(torch.empty(M, 16, dtype=torch.int8, **dev), torch.ones(M, **dev),
                             torch.empty(N, 16, dtype=torch.int8, **dev), torch.ones(N, **dev),
                             torch.empty(M, N, dtype=torch.bfloat16, **dev))


@pytest.mark.gpu
def test_gemm_infinite_and_nan_scales_stay_in_their_rows(gpu_lib):
    M, N, K = 20, 40, 64
    A, sa = codes(M, K, 7)
    B, sb = codes(N, K, 8)
    sa[3], sb[5] = np.nan, np.inf
    out = Output(M, N)
    gpu_lib.gemm_int8_nt(torch.from_numpy(A).cuda(), torch.from_numpy(sa).cuda(), torch.from_numpy(B).cuda(),
                         torch.from_numpy(sb).cuda(), out.t)
    got = f64(out.t)
    assert np.isnan(got[3]).all() and not np.isfinite(got[:, 5]).any()
    rows, cols = np.delete(np.arange(M), 3), np.delete(np.arange(N), 5)
    want, bound = ref.gemm_int8(A[rows], sa[rows], B[cols], sb[cols])
    assert_within(got[np.ix_(rows, cols)], want, bound, "other rows and columns")


@pytest.mark.gpu
def test_gemm_on_another_stream_and_in_a_graph(gpu_lib):
    """A call on a stream of its own, and replays of a captured call, each
    checked against the eager result with eager work between the replays."""
    for M, N, K in ((1, 520, 4096), (300, 264, 512)):
        A, sa = (torch.from_numpy(t).cuda() for t in codes(M, K, 9))
        B, sb = (torch.from_numpy(t).cuda() for t in codes(N, K, 10))
        want = gpu_lib.gemm_int8_nt(A, sa, B, sb, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = gpu_lib.gemm_int8_nt(A, sa, B, sb, torch.empty_like(want), stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        out = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.gemm_int8_nt(A, sa, B, sb, out)
        for _ in range(4):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            again = gpu_lib.gemm_int8_nt(A, sa, B, sb, torch.empty_like(want))
            torch.cuda.synchronize()
            assert torch.equal(again, want)


@pytest.mark.gpu
def test_gemm_on_weights_past_32_bit_offsets(gpu_lib):
    """Weight rows that lie more than 2^31 bytes into their buffer."""
    K, N = 4096, (1 << 19) + 4096
    B = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    tail = torch.randint(-127, 128, (300, K), dtype=torch.int8, generator=torch.Generator().manual_seed(0))
    B[-300:] = tail.cuda()
    sb = torch.ones(N, device="cuda")
    for M in (2, 200):
        A, sa = codes(M, K, 11)
        D = gpu_lib.gemm_int8_nt(torch.from_numpy(A).cuda(), torch.from_numpy(sa).cuda(), B, sb,
                                 torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
        want, bound = ref.gemm_int8(A, sa, tail.numpy(), np.ones(300, np.float32))
        assert_within(f64(D[:, -300:]), want, bound, f"last rows, M={M}")
        assert not D[:, :-300].any()


@pytest.mark.gpu
def test_cast_and_gemm_run_as_one_layer(gpu_lib):
    """x W^T through both casts stays within the quantisation step of each operand."""
    gen = torch.Generator().manual_seed(1)
    x, w = torch.randn(77, 512, generator=gen), torch.randn(200, 512, generator=gen)
    qx, sx = gpu_lib.int8_cast_per_row(x.cuda())
    qw, sw = gpu_lib.int8_cast_per_row(w.to(torch.bfloat16).cuda())
    D = gpu_lib.gemm_int8_nt(qx, sx, qw, sw, torch.empty(77, 200, dtype=torch.bfloat16, device="cuda"))
    w = f64(w.to(torch.bfloat16))
    want = f64(x) @ w.T
    # each code is off by at most half a step (and the fp32 division's rounding)
    ex, ew = 0.501 * f64(sx)[:, None], 0.501 * f64(sw)[:, None]
    bound = ex * np.abs(w).sum(1) + np.abs(f64(x)).sum(1)[:, None] * ew.T + 512 * ex * ew.T
    assert_within(f64(D), want, bound + 2.0 ** -8 * (np.abs(want) + bound), "layer")


# ---- refusals (no device) -------------------------------------------------

P = 0x10000


@pytest.fixture(scope="module")
def lib():
    import moe_grouped_gemm_e4m3_amd as fg

    return fg.load_library()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative"), (dict(N=-1), 1, "negative"), (dict(K=-16), 1, "negative"),
    (dict(K=40), 2, "K=40"), (dict(K=131072, lda=131072, ldb=131072), 3, "131056"),
    (dict(A=None), 1, "A is NULL"), (dict(B=None), 1, "B is NULL"), (dict(D=None), 1, "D is NULL"),
    (dict(sa=None), 1, "sa is NULL"), (dict(sb=None), 1, "sb is NULL"), (dict(A=P + 8), 2, "A is not 16-byte"),
    (dict(B=P + 4), 2, "B is not 16-byte"), (dict(D=P + 1), 2, "D is not 2-byte"), (dict(sa=P + 2), 2, "sa is not"),
    (dict(lda=500), 1, "lda=500"), (dict(ldb=520), 2, "ldb=520"), (dict(ldd=100), 1, "ldd=100"),
    (dict(lda=(1 << 22) + 16), 3, "4 MiB"),
    (dict(M=(1 << 30) + 1), 3, "2^30"),
])
def test_gemm_refusals(lib, kw, status, needle):
    a = dict(A=P, lda=512, sa=P, B=P, ldb=512, sb=P, D=P, ldd=256, M=64, N=256, K=512)
    a.update(kw)
    st = lib.gemm_int8_nt(a["A"], a["lda"], a["sa"], a["B"], a["ldb"], a["sb"], a["D"], a["ldd"], a["M"], a["N"],
                          a["K"], None)
    assert st == status, lib.fg_last_error()
    assert needle in lib.fg_last_error().decode()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative"), (dict(K=24), 2, "K=24"), (dict(x=None), 1, "x is NULL"),
    (dict(q=P + 8), 2, "q is not 16-byte"), (dict(s=P + 2), 2, "s is not"), (dict(x=P + 8), 2, "x is not"),
    (dict(ldx=500), 1, "ldx=500"), (dict(ldx=513), 2, "ldx=513"),
])
def test_cast_refusals(lib, kw, status, needle):
    a = dict(x=P, ldx=512, q=P, s=P, M=4, K=512)
    a.update(kw)
    for fn in (lib.int8_cast_per_row, lib.int8_cast_per_row_bf16):
        assert fn(a["x"], a["ldx"], a["q"], a["s"], a["M"], a["K"], None) == status
        assert needle in lib.fg_last_error().decode()


def test_empty_calls_need_no_pointers(lib):
    assert lib.gemm_int8_nt(None, 0, None, None, 0, None, None, 0, 0, 256, 512, None) == 0
    assert lib.gemm_int8_nt(None, 0, None, None, 0, None, None, 0, 64, 0, 512, None) == 0
    assert lib.int8_cast_per_row(None, 0, None, None, 0, 512, None) == 0


def test_wrappers_reject_what_the_kernels_cannot_take():
    import moe_grouped_gemm_e4m3_amd as fg

    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    d = torch.zeros(4, 4, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fg.gemm_int8_nt(q, s, q, s, d)  # not on the GPU
    with pytest.raises(TypeError):
        fg.int8_cast_per_row(torch.zeros(4, 32))
    with pytest.raises(ValueError):
        fg.gemm_int8_nt(q[0], s, q, s, d)
    with pytest.raises(ValueError):
        fg.int8_cast_per_row(torch.zeros(32))


@pytest.mark.gpu
def test_wrappers_reject_shapes_and_strides(gpu_lib):
    q, s = torch.zeros(4, 32, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    d = torch.zeros(4, 4, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: gpu_lib.gemm_int8_nt(q, s[:3], q, s, d), lambda: gpu_lib.gemm_int8_nt(q, s, q[:, :16], s, d),
                lambda: gpu_lib.gemm_int8_nt(q, s, q, s, d.t()[:, :3]), lambda: gpu_lib.gemm_int8_nt(q, s, q, s, d[:3]),
                lambda: gpu_lib.gemm_int8_nt(q.t(), s, q, s, d)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gpu_lib.gemm_int8_nt(q.float(), s, q, s, d), lambda: gpu_lib.gemm_int8_nt(q, s, q, s, d.float()),
                lambda: gpu_lib.gemm_int8_nt(q, s.double(), q, s, d)):
        with pytest.raises(TypeError):
            bad()
