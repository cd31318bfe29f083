"""Argument checks of the integer-weight calls, before anything touches a device."""
import ctypes as C

import pytest

from token_routed_expert_amd import _native as N
from token_routed_expert_amd import make_shape, moe_workspace_bytes

P = C.c_void_p(16)  # a non-null dummy: the calls below must fail before any use
ODD = C.c_void_p(8)
INV, UNS, WS = N.MOE_ERR_INVALID, N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_WORKSPACE
OK_SHAPE = dict(T=64, d=256, E=8, k=2, f=384, dtype="int4")
NAMES = ("W13", "W2", "W13s", "W2s")


def weights(group=64, **set_):
    return N.moe_i4_weights(*[set_.get(n, 16) for n in NAMES], group)


@pytest.mark.parametrize("E,R,C_,pair,group,expect", [
    (1, 100, 128, None, 64, UNS), (1, 128, 64, None, 64, UNS), (-1, 128, 128, None, 64, INV),
    (65536, 128, 128, None, 64, UNS), (32768, 128, 128, P, 64, UNS), (1, 128 * 65536, 128, None, 64, UNS),
    (1, 128, 1 << 30, None, 64, UNS), (1, 128, 128, None, 16, UNS), (1, 128, 128, None, 0, UNS),
    (1, 256, 128, None, 256, UNS), (0, 128, 128, None, 32, 0), (1, 0, 128, P, 128, 0)])
def test_weights(E, R, C_, pair, group, expect):
    lib = N.lib()
    assert lib.moe_quantize_weights_i4(P, pair, N.MOE_F32, 1, group, E, R, C_, P, P, None) == expect
    assert lib.moe_pack_weights_i4(P, P, P, pair, pair, None, group, E, R, C_, P, P, None) == expect
    assert lib.moe_dequantize_weights_i4(P, P, group, E, R, C_, P, pair, None) == expect
    if expect == 0:
        assert lib.moe_quantize_weights_i4(P, pair, N.MOE_MXFP8, 0, group, E, R, C_, P, P, None) == UNS
        assert lib.moe_pack_weights_i4(P, P, None, None, None, P, group, E, R, C_, P, P, None) == INV
        assert lib.moe_pack_weights_i4(P, P, None, P, None, None, group, E, R, C_, P, P, None) == INV
        assert lib.moe_pack_weights_i4(P, P, None, None, P, None, group, E, R, C_, P, P, None) == INV
        for i in range(3):
            a = [P, P, P]
            a[i] = None
            assert lib.moe_quantize_weights_i4(a[0], pair, N.MOE_F32, 0, group, E, R, C_, a[1], a[2], None) == INV
            assert lib.moe_dequantize_weights_i4(a[0], a[1], group, E, R, C_, a[2], pair, None) == INV
            a[i] = ODD
            assert lib.moe_quantize_weights_i4(a[0], pair, N.MOE_F32, 0, group, E, R, C_, a[1], a[2], None) == UNS
            assert lib.moe_dequantize_weights_i4(a[0], a[1], group, E, R, C_, a[2], pair, None) == UNS
        for i in range(4):
            for bad, st in ((None, INV), (ODD, UNS)):
                a = [P] * 4
                a[i] = bad
                assert lib.moe_pack_weights_i4(a[0], a[1], None, None, None, None, group, E, R, C_, a[2], a[3],
                                               None) == st


@pytest.mark.parametrize("change,expect", [
    (dict(dtype="mxfp4"), INV), (dict(dtype="bf16"), INV), (dict(d=320), UNS), (dict(f=192), UNS),
    (dict(E=257), UNS), (dict(k=9), INV), (dict(T=0), INV), (dict(T=1 << 19, d=1024), UNS),
    (dict(T=1 << 19, f=1024), UNS), (dict(d=65536, f=32768), UNS), ({}, WS)])
def test_grouped_gemm_shapes(change, expect):
    sh = make_shape(**{**OK_SHAPE, **change})
    assert N.lib().moe_grouped_gemm_fwd_i4(C.byref(sh), P, None, P, C.byref(weights()), P, None, 1 << 40,
                                           None) == expect


def test_grouped_gemm_arguments():
    lib = N.lib()
    sh = make_shape(**OK_SHAPE)
    need = moe_workspace_bytes(sh, N.MOE_WS_GEMM_FWD)
    assert need == 64 * 2 * 384 * 2

    def call(offsets=P, token_of=P, x=P, w=weights(), o=P, ws=P, nb=need - 1):
        return lib.moe_grouped_gemm_fwd_i4(C.byref(sh), offsets, token_of, x, C.byref(w), o, ws, nb, None)
    for n in ("offsets", "x", "o"):
        assert call(**{n: None}) == INV
    for n in NAMES:
        assert call(w=weights(**{n: None})) == INV
        assert call(w=weights(**{n: 24})) == UNS
    for g in (0, 16, 96, 256, -32):
        assert call(w=weights(group=g)) == UNS
    for n in ("x", "o", "ws"):
        assert call(**{n: ODD}) == UNS
    for n in ("offsets", "token_of"):
        assert call(**{n: C.c_void_p(18)}) == UNS
    assert call() == WS
    assert lib.moe_grouped_gemm_fwd_i4(C.byref(sh), P, P, P, None, P, P, need, None) == INV


def test_other_calls_refuse_the_forward_only_type():
    lib = N.lib()
    sh = make_shape(**OK_SHAPE)
    io = N.moe_layer_io()
    assert lib.moe_layer_bwd(C.byref(sh), C.byref(io), P, 1 << 40, None) == UNS
    assert lib.moe_layer_fwd(C.byref(sh), C.byref(io), P, 1 << 40, None) == INV
    assert lib.moe_layer_fwd(C.byref(sh), None, P, 1 << 40, None) == INV
    assert lib.moe_grouped_gemm_fwd(C.byref(sh), P, P, P, P, P, P, P, P, None, 0, None) == UNS
    assert lib.moe_grouped_gemm_bwd(C.byref(sh), *[P] * 13, None, 0, None) == UNS
    assert lib.moe_grouped_gemm_fwd_gather(C.byref(sh), *[P] * 9, None, 0, None) == UNS
    assert lib.moe_grouped_gemm_bwd_gather(C.byref(sh), *[P] * 15, 0, None) == UNS
    assert lib.moe_grouped_gemm_fwd_rowscaled(C.byref(sh), *[P] * 9, None) == UNS
    assert lib.moe_grouped_gemm_fwd_ckpt8(C.byref(sh), *[P] * 11, None) == UNS
    w = N.moe_mx4_weights(16, 16, 16, 16)
    assert lib.moe_grouped_gemm_fwd_mx4(C.byref(sh), P, None, P, P, C.byref(w), P, P, 1 << 40, None) == INV
    for kind in (N.MOE_WS_GEMM_BWD, N.MOE_WS_LAYER_BWD, N.MOE_WS_LAYER_BWD_ROWSCALED, N.MOE_WS_GEMM_BWD_ROWSCALED):
        assert moe_workspace_bytes(sh, kind) == 0


def test_layer_refuses_before_enqueuing():
    lib = N.lib()
    sh = make_shape(**OK_SHAPE)
    w = weights()
    io = N.moe_layer_io()
    names = ("logits", "x", "topk_idx", "topk_prob", "counts", "offsets", "row_of", "token_of", "o", "y")
    for n in names:
        setattr(io, n, 16)

    def call(nb=1 << 40, shape=sh):
        return lib.moe_layer_fwd(C.byref(shape), C.byref(io), P, nb, None)
    assert call() == INV      # no weights
    io.wi4 = C.cast(C.pointer(w), C.c_void_p).value
    need = moe_workspace_bytes(sh, N.MOE_WS_LAYER_FWD)
    assert need == (moe_workspace_bytes(sh, N.MOE_WS_PERMUTE) + 256 + moe_workspace_bytes(sh, N.MOE_WS_GEMM_FWD))
    assert call(need - 1) == WS
    io.memory_efficient = 1
    assert call(need) == UNS
    io.memory_efficient = 0
    for n in names:
        setattr(io, n, None)
        assert call(need) == INV
        setattr(io, n, 16)
    for n in ("x", "o", "y"):
        setattr(io, n, 24)
        assert call(need) == UNS
        setattr(io, n, 16)
    w.group = 48
    assert call(need) == UNS
    w.group = 32
    io.aux_loss = 16
    assert call(need) == WS
    io.aux_loss = None
    shared = make_shape(**OK_SHAPE, f_shared=256)
    assert call(need - 1, shared) == INV
    for n in ("Ws1", "Ws3", "Ws2", "s_ab", "s_h", "ys"):
        assert call(need - 1, shared) == INV
        setattr(io, n, 16)
    assert call(need - 1, shared) == WS
    assert call(need, make_shape(**OK_SHAPE, f_shared=200)) == UNS


def test_gpu_cases_reach_every_kernel():
    """The counts that the GPU tests use: few rows alone, many with the added expert, each form of the few-row kernel."""
    import test_gpu_i4 as G
    for name, counts in G.COUNTS.items():
        d, f = G.WIDTHS.get(name, (256, 128))
        assert G.few(sum(counts), len(counts), d, f)
        many = G.with_many(counts, d, f)
        assert not G.few(sum(many), len(many), d, f) and sum(many) < 40000
    forms = {n: G.blocks(*c) for n, c in G.FORMS.items()}
    assert all(G.few(sum(c[0]), len(c[0]), *c[1:]) for c in G.FORMS.values())
    assert max(forms["eight"]) <= 128 < min(forms["four"]) and max(forms["four"]) < 1024 <= min(forms["wide"])


def test_few_rows_rule():
    """Where the two kernels take about as long (few experts: later), and shapes that are refused."""
    def few(P, E, d, f, **kw):
        return bool(N.lib().moe_few_rows(C.byref(make_shape(**{**dict(T=P, d=d, E=E, k=1, f=f, dtype="int4"), **kw}))))
    assert few(20 * 128, 128, 4096, 1536) and not few(32 * 128, 128, 4096, 1536)
    assert few(20 * 8, 8, 4096, 14336) and not few(28 * 8, 8, 4096, 14336)
    assert few(128 * 8, 8, 1024, 1024) and not few(512 * 8, 8, 1024, 1024)
    assert few(1, 8, 128, 128) and not few(1, 8, 200, 128)


def test_parts_of_k():
    """The workspace of calls with many rows: h, and the larger of the two products' sums over parts of K; one part
    where the tiles fill the chip, and no sums with few rows."""
    import test_gpu_i4 as G

    def ws(P, E, d, f):
        return N.lib().moe_workspace_bytes(C.byref(make_shape(P, d, E, 1, f, dtype="int4")), N.MOE_WS_GEMM_FWD)

    def want(P, d, f, fc1, fc2):
        up = lambda n: (n + 255) // 256 * 256
        return up(2 * P * f) + up(max(4 * fc1 * P * 2 * f * (fc1 > 1), 4 * fc2 * P * d * (fc2 > 1)))
    for counts, d, f, fc1, fc2 in G.PARTS.values():
        assert not G.few(sum(counts), len(counts), d, f)
        assert ws(sum(counts), len(counts), d, f) == want(sum(counts), d, f, fc1, fc2)
    for P, E, d, f in ((8192 * 8, 128, 4096, 1536), (4096 * 2, 8, 4096, 14336), (8, 128, 4096, 1536), (1, 1, 8192, 128)):
        assert ws(P, E, d, f) == want(P, d, f, 1, 1)


def test_launches_of_two_to_the_32_threads():
    f = (1 << 24) - 128
    sh = make_shape(32, 128, 256, 1, f, dtype="int4")
    assert N.lib().moe_grouped_gemm_fwd_i4(C.byref(sh), P, None, P, C.byref(weights()), P, P, 1 << 40, None) == UNS
