"""Argument checks of the norm and of the rows' reading back, before anything
touches a device."""
import ctypes as C

import pytest

from token_routed_expert_amd import _native as N
from token_routed_expert_amd import make_shape, moe_workspace_bytes

P = C.c_void_p(16)  # a non-null dummy: the calls below must fail before any use
ODD = C.c_void_p(8)
INV, UNS, WS = N.MOE_ERR_INVALID, N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_WORKSPACE


def norm(x=P, residual=P, gamma=P, dtype=N.MOE_BF16, T=4, d=256, eps=1e-6, sum_=P, y=P, rstd=P, q=N.MOE_E4M3,
         codes=P, scales=P):
    return N.lib().moe_add_rms_norm(x, residual, gamma, dtype, T, d, eps, sum_, y, rstd, q, codes, scales, None)


def bwd(dy=P, sum_=P, rstd=P, gamma=P, dsum=P, dtype=N.MOE_BF16, T=4, d=256, dx=P, dgamma=P, ws=P, nb=1 << 40):
    return N.lib().moe_add_rms_norm_bwd(dy, sum_, rstd, gamma, dsum, dtype, T, d, dx, dgamma, ws, nb, None)


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), INV), (dict(gamma=None), INV), (dict(codes=None), INV), (dict(scales=None), INV),
    (dict(sum_=None, y=None, rstd=None, codes=None, scales=None), INV), (dict(T=-1), INV), (dict(d=0), INV),
    (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(dtype=N.MOE_E4M3), UNS), (dict(d=260), UNS), (dict(d=192), UNS), (dict(d=40, q=N.MOE_MXFP8), UNS),
    (dict(d=48, q=N.MOE_MXFP4), UNS), (dict(q=N.MOE_BF16), UNS), (dict(d=32896), UNS), (dict(T=1 << 31), UNS),
    (dict(T=1 << 30, d=64, codes=None, scales=None), UNS), (dict(x=ODD), UNS), (dict(residual=ODD), UNS),
    (dict(gamma=ODD), UNS), (dict(sum_=ODD), UNS), (dict(y=ODD), UNS), (dict(codes=ODD), UNS),
    (dict(scales=C.c_void_p(18)), UNS), (dict(rstd=C.c_void_p(18)), UNS),
    (dict(T=0), 0), (dict(T=0, residual=None, sum_=None, codes=None, scales=None, q=99), 0),
    (dict(T=0, scales=C.c_void_p(17), q=N.MOE_MXFP8), 0)])
def test_norm(change, expect):
    assert norm(**change) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(dy=None), INV), (dict(sum_=None), INV), (dict(rstd=None), INV), (dict(gamma=None), INV),
    (dict(dx=None), INV), (dict(dgamma=None), INV), (dict(T=-1), INV), (dict(d=0), INV), (dict(dtype=N.MOE_MXFP8), UNS),
    (dict(d=20), UNS), (dict(d=32776), UNS), (dict(T=1 << 31), UNS), (dict(ws=None), WS), (dict(nb=4 * 256 * 4 - 1), WS),
    (dict(dy=ODD), UNS), (dict(sum_=ODD), UNS), (dict(gamma=ODD), UNS), (dict(dsum=ODD), UNS), (dict(dx=ODD), UNS),
    (dict(ws=ODD), UNS), (dict(rstd=C.c_void_p(18)), UNS)])
def test_bwd(change, expect):
    assert bwd(**change) == expect


@pytest.mark.parametrize("T,d,teams", [(4, 256, 4), (2048, 1024, 2048), (2049, 1024, 1025), (16384, 7168, 512),
                                       (1000, 8192, 500), (300, 16384, 150), (1, 32768, 1)])
def test_workspace(T, d, teams):
    for dtype in ("bf16", "f32", "mxfp8"):
        assert moe_workspace_bytes(make_shape(T, d, 1, 1, 128, dtype=dtype), N.MOE_WS_NORM_BWD) == teams * d * 4
    assert bwd(T=T, d=d, nb=teams * d * 4 - 1) == WS


@pytest.mark.parametrize("q,rows,cols,dst,expect", [
    (N.MOE_E4M3, 4, 64, N.MOE_BF16, UNS), (N.MOE_MXFP8, 4, 48, N.MOE_BF16, UNS), (N.MOE_BF16, 4, 128, N.MOE_BF16, UNS),
    (N.MOE_MXFP8, 4, 64, N.MOE_E4M3, UNS), (N.MOE_MXFP8, -1, 64, N.MOE_F32, INV), (N.MOE_MXFP8, 1, -64, N.MOE_F32, INV),
    (N.MOE_MXFP4, 1 << 36, 64, N.MOE_F32, UNS), (N.MOE_MXFP4, 0, 64, N.MOE_F32, 0), (N.MOE_E4M3, 5, 0, N.MOE_BF16, 0)])
def test_dequantize_rows(q, rows, cols, dst, expect):
    lib = N.lib()
    assert lib.moe_dequantize_rows(P, P, q, rows, cols, P, dst, None) == expect
    for i in range(3):
        a = [P, P, P]
        a[i] = None
        assert lib.moe_dequantize_rows(a[0], a[1], q, rows, cols, a[2], dst, None) == INV
    if expect == 0:
        assert lib.moe_dequantize_rows(ODD, P, q, rows, cols, P, dst, None) == UNS


@pytest.mark.parametrize("dtype", ["mxfp4", "mxfp4_a8", "mxfp8", "e4m3"])
def test_layer_without_x(dtype):
    """x may be missing where its rows are there already; the rows may not."""
    sh = make_shape(64, 256, 8, 2, 384, dtype=dtype)
    io = N.moe_layer_io()
    for n in ("logits", "topk_idx", "topk_prob", "counts", "offsets", "row_of", "token_of", "xq", "xs", "xpq", "xps",
              "ab", "h", "o", "y"):
        setattr(io, n, 16)
    w = (N.moe_mx4_weights(*[16] * 4), N.moe_mx_weights(*[16] * 12), N.moe_e4m3_weights(*[16] * 9))
    io.wmx4, io.wmx, io.wq = (C.cast(C.pointer(i), C.c_void_p).value for i in w)
    call = N.lib().moe_layer_fwd
    assert call(C.byref(sh), C.byref(io), P, 0, None) == INV
    io.x_quantized = 1
    assert call(C.byref(sh), C.byref(io), P, 0, None) == WS
    for n in ("xq", "xs"):
        setattr(io, n, None)
        assert call(C.byref(sh), C.byref(io), P, 0, None) == INV
        setattr(io, n, 16)
