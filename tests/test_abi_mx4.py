"""Argument checks of the MXFP4 calls, before anything touches a device."""
import ctypes as C

import pytest

from token_routed_expert_amd import _native as N
from token_routed_expert_amd import make_shape, moe_workspace_bytes

P = C.c_void_p(16)  # a non-null dummy: the calls below must fail before any use
INV, UNS, WS = N.MOE_ERR_INVALID, N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_WORKSPACE
OK_SHAPE = dict(T=64, d=256, E=8, k=2, f=384, dtype="mxfp4")


def weights(**null):
    return N.moe_mx4_weights(*[None if null.get(n) else 16 for n in ("W13", "W2", "W13s", "W2s")])


@pytest.mark.parametrize("rows,cols,dtype,expect", [
    (4, 33, N.MOE_BF16, UNS), (-1, 32, N.MOE_BF16, INV), (4, -32, N.MOE_F32, INV),
    (4, 64, N.MOE_E4M3, UNS), (1 << 41, 32, N.MOE_BF16, UNS), (1 << 36, 64, N.MOE_F32, UNS),
    (0, 64, N.MOE_BF16, 0), (5, 0, N.MOE_F32, 0)])
def test_quantize_rows(rows, cols, dtype, expect):
    assert N.lib().moe_quantize_rows_mx4(P, dtype, rows, cols, P, P, None) == expect


def test_null_pointers():
    lib = N.lib()
    for i in range(3):
        a = [P, P, P]
        a[i] = None
        assert lib.moe_quantize_rows_mx4(a[0], N.MOE_BF16, 4, 64, a[1], a[2], None) == INV
        assert lib.moe_quantize_weights_mx4(a[0], None, N.MOE_F32, 1, 128, 128, a[1], a[2], None) == INV
        assert lib.moe_dequantize_weights_mx4(a[0], a[1], 1, 128, 128, a[2], None, None) == INV


@pytest.mark.parametrize("E,R,C_,pair,expect", [
    (1, 100, 128, None, UNS), (1, 128, 64, None, UNS), (-1, 128, 128, None, INV),
    (65536, 128, 128, None, UNS), (32768, 128, 128, P, UNS), (1, 128 * 65536, 128, None, UNS),
    (1, 128, 1 << 30, None, UNS), (0, 128, 128, None, 0), (1, 0, 128, P, 0)])
def test_quantize_weights(E, R, C_, pair, expect):
    lib = N.lib()
    assert lib.moe_quantize_weights_mx4(P, pair, N.MOE_F32, E, R, C_, P, P, None) == expect
    assert lib.moe_dequantize_weights_mx4(P, P, E, R, C_, P, pair, None) == expect
    if expect == 0:
        assert lib.moe_quantize_weights_mx4(P, pair, N.MOE_MXFP8, E, R, C_, P, P, None) == UNS


@pytest.mark.parametrize("change,expect", [
    (dict(dtype="mxfp8"), INV), (dict(dtype="bf16"), INV), (dict(d=320), UNS), (dict(f=192), UNS),
    (dict(f_shared=128), UNS), (dict(E=257), UNS), (dict(k=9), INV), (dict(T=0), INV),
    (dict(T=1 << 20, d=1024), UNS), (dict(T=1 << 20, f=1024), UNS), (dict(d=65536, f=32768), UNS),
    ({}, WS)])
def test_grouped_gemm_shapes(change, expect):
    sh = make_shape(**{**OK_SHAPE, **change})
    assert N.lib().moe_grouped_gemm_fwd_mx4(C.byref(sh), P, None, P, P, C.byref(weights()), P, None,
                                            1 << 40, None) == expect


@pytest.mark.parametrize("dtype", ["mxfp4", "mxfp4_a8"])
def test_grouped_gemm_arguments(dtype):
    lib = N.lib()
    sh = make_shape(**{**OK_SHAPE, "dtype": dtype})
    need = moe_workspace_bytes(sh, N.MOE_WS_GEMM_FWD)
    rows = 64 * 2
    assert need == rows * (384 // (2 if dtype == "mxfp4" else 1)) + rows * 384 // 32

    def call(offsets=P, xq=P, xs=P, w=weights(), o=P, ws=P, nb=need - 1):
        return lib.moe_grouped_gemm_fwd_mx4(C.byref(sh), offsets, P, xq, xs, C.byref(w), o, ws, nb, None)
    for bad in (dict(offsets=None), dict(xq=None), dict(xs=None), dict(o=None), dict(w=weights(W13=1)),
                dict(w=weights(W2=1)), dict(w=weights(W13s=1)), dict(w=weights(W2s=1))):
        assert call(**bad) == INV
    assert call() == WS
    assert lib.moe_grouped_gemm_fwd_mx4(C.byref(sh), P, P, P, P, None, P, P, need, None) == INV


@pytest.mark.parametrize("dtype", ["mxfp4", "mxfp4_a8"])
def test_other_calls_refuse_the_forward_only_types(dtype):
    lib = N.lib()
    sh = make_shape(**{**OK_SHAPE, "dtype": dtype})
    io = N.moe_layer_io()
    assert lib.moe_layer_bwd(C.byref(sh), C.byref(io), P, 1 << 40, None) == UNS
    assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, 1 << 40, None) == INV
    assert lib.moe_layer_fwd(C.byref(sh), None, P, 1 << 40, None) == INV
    assert lib.moe_grouped_gemm_fwd(C.byref(sh), P, P, P, P, P, P, P, P, None, 0, None) == UNS
    assert lib.moe_grouped_gemm_bwd(C.byref(sh), P, P, P, P, P, P, P, P, P, P, P, P, P, None, 0,
                                    None) == UNS
    assert lib.moe_grouped_gemm_fwd_gather(C.byref(sh), P, P, P, P, P, P, P, P, P, None, 0, None) == UNS
    assert lib.moe_grouped_gemm_fwd_rowscaled(C.byref(sh), P, P, P, P, P, P, P, P, P, None) == UNS
    w = N.moe_e4m3_weights()
    assert lib.moe_grouped_gemm_fwd_e4m3(C.byref(sh), P, P, P, C.byref(w), P, P, P, P, 1 << 40,
                                         None) == INV
    for kind in (N.MOE_WS_GEMM_BWD, N.MOE_WS_LAYER_BWD, N.MOE_WS_LAYER_BWD_ROWSCALED):
        assert moe_workspace_bytes(sh, kind) == 0


def test_layer_refuses_before_enqueuing():
    lib = N.lib()
    sh = make_shape(**OK_SHAPE)
    w = weights()
    io = N.moe_layer_io()
    for n in ("logits", "x", "topk_idx", "topk_prob", "counts", "offsets", "row_of", "token_of", "xq",
              "xs", "o", "y"):
        setattr(io, n, 16)
    assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, 1 << 40, None) == INV      # no weights
    io.wmx4 = C.cast(C.pointer(w), C.c_void_p).value
    need = moe_workspace_bytes(sh, N.MOE_WS_LAYER_FWD)
    assert need == moe_workspace_bytes(sh, N.MOE_WS_PERMUTE) + moe_workspace_bytes(sh, N.MOE_WS_GEMM_FWD)
    assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, need - 1, None) == WS
    io.memory_efficient = 1
    assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, need, None) == UNS
    io.memory_efficient = 0
    for n in ("xq", "xs", "o", "token_of"):
        setattr(io, n, None)
        assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, need, None) == INV
        setattr(io, n, 16)
    io.aux_loss = 16
    assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, need, None) == WS


def test_layer_refuses_misaligned_buffers_before_enqueuing():
    lib = N.lib()
    sh = make_shape(**OK_SHAPE)
    need = moe_workspace_bytes(sh, N.MOE_WS_LAYER_FWD)
    names = ("logits", "x", "topk_idx", "topk_prob", "counts", "offsets", "row_of", "token_of", "xq",
             "xs", "o", "y")
    for odd, value in (("x", 24), ("xq", 24), ("o", 24), ("y", 24), ("xs", 18), ("W13", 24), ("W2s", 18)):
        w = weights()
        io = N.moe_layer_io()
        for n in names:
            setattr(io, n, 16)
        setattr(io if odd in names else w, odd, value)
        io.wmx4 = C.cast(C.pointer(w), C.c_void_p).value
        assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, need, None) == UNS, odd


def test_python_refuses_a_stream_of_another_device():
    from token_routed_expert_amd.ops import _Bufs

    class Stream:
        device_index, cuda_stream = 7, 64

    b = _Bufs("call")
    with pytest.raises(ValueError, match="stream is not on the current device"):
        b.stream(Stream)
    b.dev = 7
    assert b.stream(Stream) == 64


ODD = C.c_void_p(24)  # 8-byte aligned only


def test_misaligned_pointers():
    lib = N.lib()
    for a in ((ODD, P), (P, ODD)):
        assert lib.moe_quantize_rows_mx4(a[0], N.MOE_BF16, 4, 64, a[1], P, None) == UNS
        assert lib.moe_quantize_weights_mx4(a[0], None, N.MOE_F32, 1, 128, 128, a[1], P, None) == UNS
        assert lib.moe_dequantize_weights_mx4(a[0], P, 1, 128, 128, a[1], None, None) == UNS
    assert lib.moe_quantize_weights_mx4(P, ODD, N.MOE_F32, 1, 128, 128, P, P, None) == UNS
    sh = make_shape(**OK_SHAPE)
    for i in (2, 4, 5):                                   # xq, o, ws
        a = [P, None, P, P, P, P]
        a[i] = ODD
        assert lib.moe_grouped_gemm_fwd_mx4(C.byref(sh), a[0], a[1], a[2], a[3], C.byref(weights()), a[4],
                                            a[5], 1 << 40, None) == UNS, i
    half = C.c_void_p(18)
    assert lib.moe_grouped_gemm_fwd_mx4(C.byref(sh), P, None, P, half, C.byref(weights()), P, P, 1 << 40,
                                        None) == UNS


def test_python_refuses_what_the_kernels_cannot_take():
    """Host tensors, wrong types, short buffers and foreign layouts stop before the library."""
    import torch

    import token_routed_expert_amd as tre
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        tre.moe_quantize_rows_mx4(x, q, s)
    with pytest.raises(TypeError):
        tre.moe_quantize_rows_mx4(x.half(), q, s)
    with pytest.raises(ValueError, match="contiguous"):
        tre.moe_quantize_rows_mx4(x.t(), q, s)
    W = torch.zeros(1, 128, 128)
    with pytest.raises(ValueError, match="shape"):
        tre.moe_quantize_weights_mx4(W, W[:, :, :64], q, s)
    with pytest.raises(ValueError, match="shape"):
        tre.moe_dequantize_weights_mx4(q, s, W.bfloat16(), W[:, :64].bfloat16())
