"""Workspaces that a program allocates once, for its largest batch: on the CPU, before
anything touches a device."""
import ctypes as C

import pytest
import torch

from token_routed_expert_amd import _native as N
from token_routed_expert_amd import make_shape, moe_workspace_bytes

P = C.c_void_p(16)  # a non-null dummy: the calls below must fail before any use
WS = N.MOE_ERR_WORKSPACE

# d, E, k, f and the T around which the sums over parts of K come and go
INT4 = [(7168, 2, 1, 2048, 2300), (4096, 8, 2, 14336, 1500), (2048, 1, 1, 8192, 3000), (384, 4, 1, 2560, 7000),
        (1024, 2, 1, 2048, 2000), (4096, 16, 2, 512, 2300), (5120, 32, 4, 512, 1500)]


def least_i4(sh):
    return sh.T * sh.k * sh.f * 2


@pytest.mark.parametrize("d,E,k,f,top", INT4)
def test_int4_least_workspace(d, E, k, f, top):
    """What a call and a layer refuse goes up with T alone, and nothing that moe_workspace_bytes gives for a larger T is
    refused for a smaller one."""
    lib = N.lib()
    w = N.moe_i4_weights(16, 16, 16, 16, 64)
    io = N.moe_layer_io()
    for n in ("logits", "x", "topk_idx", "topk_prob", "counts", "offsets", "row_of", "token_of", "o", "y"):
        setattr(io, n, 16)
    io.wi4 = C.cast(C.pointer(w), C.c_void_p).value
    parts, smaller, last = False, False, [0, 0, 0, 0]
    for T in [*range(1, 40), *range(40, top, 7), top]:
        sh = make_shape(T, d, E, k, f, dtype="int4")
        gemm, layer = (moe_workspace_bytes(sh, n) for n in (N.MOE_WS_GEMM_FWD, N.MOE_WS_LAYER_FWD))
        aux = moe_workspace_bytes(sh, N.MOE_WS_AUX_LOSS)
        least = least_i4(sh)
        fixed = moe_workspace_bytes(sh, N.MOE_WS_PERMUTE) + 256
        assert layer == fixed + gemm and gemm >= least
        parts, smaller = parts or gemm > least, smaller or gemm < last[0]
        now = [gemm, least, fixed, aux]
        assert all(a <= b for a, b in zip(last[1:], now[1:]))      # the least, the permutation's, the loss's
        last = now
        assert lib.moe_grouped_gemm_fwd_i4(C.byref(sh), P, None, P, C.byref(w), P, P, least - 1, None) == WS
        io.aux_loss = None
        assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, fixed + least - 1, None) == WS
        io.aux_loss = 16
        assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, fixed + least + aux - 1, None) == WS
    assert parts and smaller       # the sums do come, and go again as T grows


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="takes calls up to their launch, which only fails without a GPU")
@pytest.mark.parametrize("d,E,k,f,top", INT4)
def test_int4_workspace_of_a_larger_batch(d, E, k, f, top):
    """The least workspace of the largest T, for every smaller one: no call refuses it."""
    lib = N.lib()
    w = N.moe_i4_weights(16, 16, 16, 16, 64)
    nb = least_i4(make_shape(top, d, E, k, f, dtype="int4"))
    for T in [1, 2, 40, *range(101, top, 101), top - 1, top]:
        sh = make_shape(T, d, E, k, f, dtype="int4")
        assert lib.moe_grouped_gemm_fwd_i4(C.byref(sh), P, None, P, C.byref(w), P, P, nb, None) == N.MOE_ERR_HIP


@pytest.mark.parametrize("d", [8, 512, 1024, 1032, 4096, 8192, 8200, 32768])
def test_norm_backward_workspace_of_a_larger_batch(d):
    """MOE_WS_NORM_BWD_MAX grows with T and holds what every smaller T needs; MOE_WS_NORM_BWD alone does not."""
    lib = N.lib()
    need = most = 0
    fell = False
    for T in [*range(1, 4200), 16384, 16385, 100000, (1 << 31) - 1]:
        sh = make_shape(T, d, 1, 1, 128, dtype="f32")
        now, top = (moe_workspace_bytes(sh, k) for k in (N.MOE_WS_NORM_BWD, N.MOE_WS_NORM_BWD_MAX))
        fell = fell or now < need
        need = max(need, now)
        assert top == need and top >= most
        most = top
    assert fell
    for T in (1, 7, 255, 256, 257, 511, 512, 513, 2047, 2048, 2049, 4100):
        assert lib.moe_add_rms_norm_bwd(*[P] * 5, N.MOE_F32, T, d, P, P, P,
                                        moe_workspace_bytes(make_shape(T, d, 1, 1, 128), N.MOE_WS_NORM_BWD) - 1, None) == WS


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="takes calls up to their launch, which only fails without a GPU")
@pytest.mark.parametrize("d,top", [(512, 5000), (1024, 2049), (4096, 513), (7168, 16384), (16384, 300)])
def test_norm_backward_takes_the_larger_workspace(d, top):
    nb = moe_workspace_bytes(make_shape(top, d, 1, 1, 128), N.MOE_WS_NORM_BWD_MAX)
    for T in sorted({1, 2, 100, 256, 257, 512, 513, 1024, 2048, top - 1, top} & set(range(top + 1))):
        assert N.lib().moe_add_rms_norm_bwd(*[P] * 5, N.MOE_BF16, T, d, P, P, P, nb, None) == N.MOE_ERR_HIP
