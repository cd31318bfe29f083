"""Argument checks of the 8-bit checkpoint calls, before anything touches a device."""
import ctypes as C

import pytest

from token_routed_expert_amd import _native as N
from token_routed_expert_amd import make_shape, moe_workspace_bytes

P = C.c_void_p(16)
INV, UNS, WS = N.MOE_ERR_INVALID, N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_WORKSPACE
SHAPE = dict(T=64, d=256, E=8, k=2, f=384, dtype="bf16")


def fwd(sh, null=None, token_of=P):
    a = [P, token_of] + [P] * 9 + [None]
    if null is not None:
        a[null] = None
    return N.lib().moe_grouped_gemm_fwd_ckpt8(C.byref(sh), *a)


def bwd(sh, null=None, token_of=P, ws=P, nb=1 << 40):
    a = [P, token_of] + [P] * 14 + [None, None]
    if null is not None:
        a[null] = None
    return N.lib().moe_grouped_gemm_bwd_ckpt8(C.byref(sh), *a, ws, nb, None)


@pytest.mark.parametrize("change,expect", [
    (dict(dtype="f32"), UNS), (dict(dtype="mxfp8"), UNS), (dict(dtype="mxfp4"), UNS), (dict(f=200), UNS),
    (dict(d=320), UNS), (dict(k=9), INV), (dict(T=1 << 19, d=512, k=8, f=128), UNS)])
def test_shapes(change, expect):
    sh = make_shape(**{**SHAPE, **change})
    assert fwd(sh, null=0) == expect and bwd(sh, null=0) == expect


def test_gathered_rows_have_their_own_limit():
    sh = make_shape(**{**SHAPE, "T": 1 << 20, "d": 1024, "k": 1, "f": 128, "E": 1})   # x: 2^31 bytes
    assert fwd(sh, null=0) == UNS and bwd(sh, null=0) == UNS
    assert fwd(sh, null=0, token_of=None) == INV and bwd(sh, null=0, token_of=None) == INV


def test_null_pointers_and_workspace():
    sh = make_shape(**SHAPE)
    for i in [0] + list(range(2, 11)):
        assert fwd(sh, null=i) == INV, i
    for i in [0] + list(range(2, 16)):
        assert bwd(sh, null=i) == INV, i
    need = moe_workspace_bytes(sh, N.MOE_WS_GEMM_BWD_ROWSCALED)
    assert need > 0
    assert bwd(sh, ws=None) == WS and bwd(sh, nb=need - 1) == WS


@pytest.mark.parametrize("call", ["moe_layer_fwd", "moe_layer_bwd"])
def test_layer_mode(call):
    lib = N.lib()
    sh = make_shape(**SHAPE)
    io = N.moe_layer_io()
    for n in N.IO_FIELDS:
        if n not in ("ab_q", "ab_s", "ab", "aux_loss", "dlogits"):
            setattr(io, n, 16)
    io.memory_efficient = 3
    fn = getattr(lib, call)
    assert fn(C.byref(sh), C.byref(io), P, 16, None) == INV         # no checkpoint buffers
    io.ab_q = 16
    assert fn(C.byref(sh), C.byref(io), P, 16, None) == INV
    io.ab_s = 16
    assert fn(C.byref(sh), C.byref(io), P, 16, None) == WS
    io.memory_efficient = 2                                         # (mode 2 still needs ab)
    assert fn(C.byref(sh), C.byref(io), P, 16, None) == INV
    io.memory_efficient = 3
    w8, wmx = N.moe_e4m3_weights(*[16] * 9), N.moe_mx_weights(*[16] * 12)
    io.wq, io.wmx = (C.cast(C.pointer(w), C.c_void_p).value for w in (w8, wmx))
    for dtype in ("e4m3", "mxfp8", "f32"):
        s8 = make_shape(**{**SHAPE, "dtype": dtype})
        assert fn(C.byref(s8), C.byref(io), P, 16, None) == UNS


@pytest.mark.parametrize("call,names", [("moe_layer_fwd", ("x", "xp", "W1", "ab_q", "h", "o")),
                                        ("moe_layer_bwd", ("xp", "ab_q", "dO", "dab", "dXp", "dW2"))])
def test_layer_refuses_misaligned_buffers_before_enqueuing(call, names):
    sh = make_shape(**SHAPE)
    for odd in names:
        io = N.moe_layer_io()
        for n in N.IO_FIELDS:
            if n not in ("ab", "aux_loss", "dlogits"):
                setattr(io, n, 24 if n == odd else 16)
        io.memory_efficient = 3
        assert getattr(N.lib(), call)(C.byref(sh), C.byref(io), P, 1 << 40, None) == UNS, odd


def test_misaligned_pointers():
    sh = make_shape(**SHAPE)
    odd = C.c_void_p(24)
    for i in (2, 3, 4, 5, 7, 9, 10):
        a = [P, P] + [P] * 9 + [None]
        a[i] = odd
        assert N.lib().moe_grouped_gemm_fwd_ckpt8(C.byref(sh), *a) == UNS, i
    for i in (2, 3, 5, 6, 7, 8, 10, 11, 12, 13, 14, 15):
        a = [P, P] + [P] * 14 + [None, None]
        a[i] = odd
        assert N.lib().moe_grouped_gemm_bwd_ckpt8(C.byref(sh), *a, P, 1 << 40, None) == UNS, i
    half = C.c_void_p(18)
    for i in (0, 1, 6):
        a = [P, P] + [P] * 9 + [None]
        a[i] = half
        assert N.lib().moe_grouped_gemm_fwd_ckpt8(C.byref(sh), *a) == UNS, i
