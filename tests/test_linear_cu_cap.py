"""The 8-bit-integer product and the gated block under a cap on the CUs: the
persistent launches keep to it, integer bits do not change, BF16 results stay
within their bounds."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import linear as ref
from tests.helpers import announce
from tests.linear_helpers import Output, assert_within, f64
from tests.test_gated_ffn import block
from tests.test_int8_linear import codes
from tests.test_linear_launches import gradients, launches, tile  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 7, 64])
def cap(gpu_lib, request):
    gpu_lib.set_num_cus(request.param)
    yield request.param
    gpu_lib.set_num_cus(0)


def within(lines, cap):
    """Every launch has at most two workgroups (of the tiles that share a CU:
    those of 256 threads, and 128 x 64) for each CU of the cap."""
    for x in lines:
        if not x["few"]:
            pairs = tile(x)[2] == 256 or tile(x)[:2] == (128, 64)
            assert int(x["grid"]) <= cap * (2 if pairs else 1), x


@pytest.mark.parametrize("M,N,K", [(3, 300, 2048), (100, 640, 528), (700, 1000, 528)])
def test_int8_under_a_cap(gpu_lib, launches, cap, M, N, K):  # noqa: F811
    announce(f"int8 {M}x{N}x{K} on {cap} CUs")
    A, sa = (torch.from_numpy(t).cuda() for t in codes(M, K, 1))
    B, sb = (torch.from_numpy(t).cuda() for t in codes(2 * N, K, 2))
    got = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    within(launches("", lambda: gpu_lib.gemm_int8_nt(A, sa, B[:N], sb[:N], got[0])), cap)
    within(launches("", lambda: gpu_lib.gated_ffn_int8(A, sa, B, sb, got[1])), cap)
    gpu_lib.set_num_cus(0)
    gpu_lib.gemm_int8_nt(A, sa, B[:N], sb[:N], got[2])
    gpu_lib.gated_ffn_int8(A, sa, B, sb, got[3])
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


@pytest.mark.parametrize("M,F,K", [(20, 130, 264), (300, 150, 136), (700, 500, 264)])
def test_gated_forward_under_a_cap(gpu_lib, launches, cap, M, F, K):  # noqa: F811
    announce(f"gated {M}x{F}x{K} on {cap} CUs")
    X, W, _ = block(M, F, K, 3)
    out, P = Output(M, F, 3), torch.empty(M, 2 * F, device="cuda")
    within(launches("", lambda: gpu_lib.gated_ffn_bf16(X.cuda(), W.cuda(), out.t, P=P)), cap)
    out.check_untouched()
    g, u, eg, eu = ref.pre_activations(f64(X), f64(W))
    assert_within(out.f64(), ref.gated(g, u, "silu"), ref.gated_bound(g, u, eg, eu, "silu"), "H")
    assert_within(f64(P), np.concatenate([g, u], 1), np.concatenate([eg, eu], 1) + 1e-45, "P")


# (5, 1025, 136) and (300, 128, 520) share a launch on the whole device, the
# first with dX's sum split
@pytest.mark.parametrize("kept", [False, True], ids=["recomputed", "kept"])
@pytest.mark.parametrize("M,F,K", [(5, 1025, 136), (300, 128, 520), (190, 70, 1928), (33, 63, 256)])
def test_gradients_under_a_cap(gpu_lib, launches, cap, M, F, K, kept):  # noqa: F811
    announce(f"gradients {M}x{F}x{K} kept={kept} on {cap} CUs")
    call, check = gradients(gpu_lib, M, F, K, kept)
    lines = launches("", call)
    assert {"dX", "dW"} <= {x["launch"] for x in lines}
    within(lines, cap)
    check("under a cap")
    # a forced plan keeps to it as well
    within(launches("share-small-small", call), cap)
    check("under a cap, forced")
