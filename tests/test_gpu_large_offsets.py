"""Norm rows and integer weights whose element or byte offsets pass 32 bits: rows and
experts at both ends against the oracle.  Tolerances as in test_gpu_norm.py and
test_gpu_i4.py."""
import numpy as np
import pytest
import torch

import oracle
from moe_workloads import to_f64

from gpu_common import announce, need_gpu
from test_gpu_i4 import I32, U8, expected
from test_gpu_norm import BF16, EPS, H, U, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d", [((1 << 18) + 3, 16384), ((1 << 20) + 5, 4224)])
def test_norm_forward_backward_and_back(T, d):
    import token_routed_expert_amd as tre
    assert T * d > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, d, dtype=BF16, device="cuda")
    for r in range(0, T, 1 << 16):
        x[r:r + (1 << 16)].normal_(generator=g)
    gamma = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF16)
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    codes = torch.empty(T, d, dtype=U8, device="cuda")
    scales = torch.empty(T, d // 32, dtype=U8, device="cuda")
    tre.moe_add_rms_norm(x, None, gamma, EPS, None, y, rstd, "mxfp8", codes, scales)
    ends = [0, 1, (1 << 32) // d - 1, (1 << 32) // d, (1 << 32) // d + 1, T - 2, T - 1]
    want, wr = oracle.rms_norm(f64(x[ends]), f64(gamma), EPS)
    assert (np.abs(f64(rstd[ends]) - wr) <= (d / 2 + 5) * U * wr).all()
    e = (d / 2 + 7) * U
    assert (np.abs(f64(y[ends]) - want) <= (e + H[BF16] * (1 + e)) * np.abs(want)).all()
    back = torch.empty_like(x)
    tre.moe_dequantize_rows(codes, scales, "mxfp8", back)
    sc = np.repeat(np.exp2(f64(scales[ends]) - 127), 32, axis=1)
    tol = (2.0 ** -4 + (d + 20) * U) * np.abs(want) + 2.0 ** -10 * sc
    assert (np.abs(f64(back[ends]) - want) <= tol).all()    # (codes of E4M3 times a power of two are bf16 numbers)
    del back, codes, scales
    # the backward with dy = y, in place of it; dgamma is linear in dy: with dy zero but in the last rows, theirs
    dx, dg = y, torch.empty_like(gamma)
    y[:T - 8] = 0
    keep = y[T - 8:].clone()
    ws = torch.empty(tre.moe_workspace_bytes(tre.make_shape(T, d, 1, 1, 128), tre.MOE_WS_NORM_BWD), dtype=U8, device="cuda")
    tre.moe_add_rms_norm_bwd(y, x, rstd, gamma, None, dx, dg, ws)
    s, dyn, gn, rn = f64(x[T - 8:]), f64(keep), f64(gamma), f64(rstd[T - 8:])[:, None]
    wx, wg = oracle.rms_norm_bwd(dyn, s, rn[:, 0], gn)
    gs, xh = np.abs(dyn * gn), np.abs(s * rn)
    mean = (gs * xh).mean(1, keepdims=True)
    size = rn * (gs + xh * mean)
    tol = H[BF16] * (np.abs(wx) + 1e-6 * size) + 8 * U * size + (d + 4) * U * rn * xh * mean
    assert (np.abs(f64(dx[T - 8:]) - wx) <= tol).all()
    assert (dx[[r for r in ends if r < T - 8]] == 0).all()
    size = np.abs(dyn * s * rn).sum(0)
    assert (np.abs(f64(dg) - wg) <= H[BF16] * (np.abs(wg) + 1e-3 * size) + 16 * U * size).all()


def test_weights_there_and_back():
    """17 GB of bf16 weights; experts at both ends and around 2^32 bytes of source, codes and values."""
    import token_routed_expert_amd as tre
    E, R, C, group = 260, 4096, 8192, 64
    assert E * R * C // 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(2)
    W = torch.empty(E, R, C, dtype=BF16, device="cuda")
    for e in range(E):
        W[e].normal_(generator=g)
    codes = torch.empty(E, C // 16, R // 128, 4, 16, 16, dtype=U8, device="cuda")
    words = torch.empty(E, C // 64, R // 128, 128 // group, 16, 4, dtype=I32, device="cuda")
    tre.moe_quantize_weights_i4(W, None, group, True, codes, words)
    back = torch.empty_like(W)
    tre.moe_dequantize_weights_i4(codes, words, group, back)
    for e in (0, 63, 64, 127, 255, 256, E - 1):
        c2, w2 = torch.empty_like(codes[:1]), torch.empty_like(words[:1])
        tre.moe_quantize_weights_i4(W[e:e + 1], None, group, True, c2, w2)
        assert torch.equal(c2[0], codes[e]) and torch.equal(w2[0], words[e])
        v = torch.empty_like(W[:1])
        tre.moe_dequantize_weights_i4(c2, w2, group, v)
        assert torch.equal(v[0], back[e])
    # one expert's corner against the oracle
    q, s, z = oracle.quant_i4(to_f64(W[E - 1:, :128, :128].contiguous()), group, True)
    assert np.array_equal(to_f64(back[E - 1:, :128, :128].contiguous()), oracle.dequant_i4(q, s, z))


@pytest.mark.parametrize("rows", [(1, 3), (17, 30), (300, 1500)])
def test_product_on_more_than_4_gb_of_codes(rows):
    """256 experts of which the first and the last have rows; codes and scales at random."""
    import token_routed_expert_amd as tre
    E, d, f, group = 256, 4096, 4224, 128
    assert E * d * f > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(3)
    w = {}
    for name, n in (("W13", E * d * f), ("W2", E * d * f // 2)):
        w[name] = torch.randint(0, 256, (n,), generator=g, dtype=U8, device="cuda")
        w[name + "s"] = torch.randint(119 << 23, 120 << 23, (2 * n // group,), generator=g, dtype=I32, device="cuda")
    off = np.zeros(E + 1, np.int32)
    off[1:] = rows[0]
    off[E] = sum(rows)
    T = sum(rows)
    x = torch.randn(T, d, generator=g, device="cuda").to(BF16)
    tok = torch.randint(0, T, (T,), generator=g, dtype=I32, device="cuda")
    sh = tre.make_shape(T, d, E, 1, f, dtype="int4")
    o = torch.full((T, d), 7.0, dtype=BF16, device="cuda")
    ws = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=U8, device="cuda")
    tre.moe_grouped_gemm_fwd_i4(sh, torch.from_numpy(off).cuda(), tok, x, tre.I4Weights(w, group), o, ws)
    # the two experts' own tiles, their rows alone
    for e, r in ((0, slice(0, rows[0])), (E - 1, slice(rows[0], T))):
        own = tre.I4Weights({n: t.view(E, -1)[e].clone() for n, t in w.items()}, group)
        pick = np.unique(np.r_[0, 15, 16, 31, 32, 127, 128, r.stop - r.start - 1])
        pick = pick[pick < r.stop - r.start]
        tokens = tok[r].cpu().numpy()[pick]
        ref, tol = expected((x.cpu(), tokens, own, np.array([0, len(pick)], np.int32)), 1, d, f)
        assert (np.abs(to_f64(o[r][torch.from_numpy(pick).cuda()]) - ref) <= tol).all()
