"""Calls whose launch would have 2^32 threads or more are refused before it: the
runtime keeps the low 32 bits of the count and runs a part of the grid."""
import ctypes as C

import pytest

from token_routed_expert_amd import _native as N
from token_routed_expert_amd import make_shape

P = C.c_void_p(16)      # non-null and aligned; no call below may use it
UNS = N.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("d,T", [(4096, 1 << 23), (256, 1 << 26)])     # 512 and 64 threads a token
def test_unpermute(d, T):
    sh = make_shape(T, d, 8, 1, 128)
    assert N.lib().moe_unpermute(C.byref(sh), P, P, P, None, P, None) == UNS


def test_combine_bwd():
    sh = make_shape(1 << 24, 256, 8, 1, 128)
    assert N.lib().moe_combine_bwd(C.byref(sh), P, P, P, P, P, P, None) == UNS


@pytest.mark.parametrize("E,T", [(256, 1 << 26), (16, 1 << 28), (8, 1 << 29)])
def test_route(E, T):
    assert N.lib().moe_route(P, T, E, 2, P, P, None) == UNS


def test_rows_of_fp8():
    for fn in (N.lib().moe_quantize_rows, N.lib().moe_quantize_rows_mx):
        assert fn(P, N.MOE_BF16, 1 << 28, 8192, P, P, None) == UNS


def test_products():
    lib = N.lib()
    sh = make_shape(1, 4, 256, 1, 1 << 22, dtype="f32")
    assert lib.moe_grouped_gemm_fwd(C.byref(sh), *[P] * 8, None, 0, None) == UNS
    f = (1 << 24) - 128
    w = N.moe_mx4_weights(16, 16, 16, 16)
    for dtype in ("mxfp4", "mxfp4_a8"):
        sh = make_shape(32, 128, 256, 1, f, dtype=dtype)
        assert lib.moe_grouped_gemm_fwd_mx4(C.byref(sh), P, None, P, P, C.byref(w), P, P, 1 << 40, None) == UNS
    sh = make_shape(32, 128, 256, 1, f)
    assert lib.moe_grouped_gemm_fwd_ckpt8(C.byref(sh), P, None, *[P] * 9, None) == UNS
