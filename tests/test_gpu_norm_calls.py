"""Calls of the norm and of layers on its rows that the header allows and that stand in
no other test: y written over sum, a layer's backward behind a forward on rows that were
there already, training from the residual stream to the layer and back on such rows,
one backward workspace for several batches."""
import numpy as np
import pytest
import torch

import oracle
from moe_workloads import Workload

from gpu_common import announce, need_gpu
from test_gpu_norm import BF16, EPS, F32, f64, layer_of, rows_buffers, stream_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", [None, "e4m3", "mxfp4"])
@pytest.mark.parametrize("T,d", [(6, 512), (40000, 512), (5000, 4096), (4100, 7168), (300, 7168), (20, 16384)])
def test_y_over_sum(T, d, fmt, dtype):
    """sum and y the same memory: y stands there afterwards, with the bits of the call that has both."""
    import token_routed_expert_amd as tre
    x, r, gamma = stream_rows(T, d, dtype, 21)
    both, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    rows = (None, None) if fmt is None else rows_buffers(T, d, fmt)
    rows2 = (None, None) if fmt is None else rows_buffers(T, d, fmt)
    tre.moe_add_rms_norm(x, r, gamma, EPS, torch.empty_like(x), y, rstd, fmt, *rows)
    tre.moe_add_rms_norm(x, r, gamma, EPS, both, both, None, fmt, *rows2)
    assert torch.equal(both, y)
    if fmt:
        assert torch.equal(rows[0], rows2[0]) and torch.equal(rows[1], rows2[1])
    for over in (x, r):                              # all three in one place
        keep = over.clone()
        tre.moe_add_rms_norm(x, r, gamma, EPS, over, over, None)
        assert torch.equal(over, y)
        over.copy_(keep)


GRADS = ("dX", "dW1", "dW3", "dW2", "dprob", "dlogits")


@pytest.mark.parametrize("me", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["e4m3", "mxfp8"])
def test_backward_behind_a_forward_on_rows_that_are_there(dtype, me):
    """The same codes, made by the layer and handed to it: the same gradients, bit for bit; a backward without x is
    refused."""
    import token_routed_expert_amd as tre
    wl = Workload("norm_bwd", T=150, d=256, E=8, k=2, f=384, dtype=dtype)
    sh, b, wsf, wsb = layer_of(wl, seed=2, router_grad=True, **({"memory_efficient": me} if me else {}))
    tre.moe_layer_fwd(sh, b, wsf)
    tre.moe_layer_bwd(sh, b, wsb)
    want = {n: b[n].clone() for n in GRADS + ("y", "aux_loss")}
    assert all(torch.isfinite(t).all() for t in want.values())
    for n in ("y", "o", "ab", "h", "dO", "dab", "dXp", "aux_loss") + GRADS:
        b[n].fill_(float("nan"))
    x = b.pop("x")
    b["x_quantized"] = 1
    tre.moe_layer_fwd(sh, b, wsf)
    with pytest.raises(tre.MoeError, match="INVALID"):
        tre.moe_layer_bwd(sh, b, wsb)
    b["x"] = x
    tre.moe_layer_bwd(sh, b, wsb)
    assert all(torch.equal(b[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype", ["e4m3", "mxfp8"])
def test_training_on_quantised_rows(dtype):
    """Residual addition, norm with the layer's rows, the layer on them, and back to the residual stream.  The layer's
    gradients are those of its own calls on the same codes (bit for bit); the norm's, the 64-bit formula's on the
    device's dX."""
    import token_routed_expert_amd as tre
    wl = Workload("norm_train8", T=130, d=256, E=8, k=2, f=256, dtype=dtype)
    sh, b, wsf, wsb = layer_of(wl, seed=4)
    x, r, gamma = stream_rows(wl.T, wl.d, BF16, 8, special=False)
    sum_, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(wl.T, device="cuda")
    tre.moe_add_rms_norm(x, r, gamma, EPS, sum_, y, rstd, dtype, b["xq"], b["xs"])
    rows = b["xq"].clone(), b["xs"].clone()
    b["x"], b["x_quantized"] = y, 1
    tre.moe_layer_fwd(sh, b, wsf)
    tre.moe_layer_bwd(sh, b, wsb)
    assert torch.equal(b["xq"], rows[0]) and torch.equal(b["xs"], rows[1])       # the rows are read alone
    dx, dg = torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.empty(tre.moe_workspace_bytes(tre.make_shape(5000, wl.d, 1, 1, 128), tre.MOE_WS_NORM_BWD_MAX),
                     dtype=torch.uint8, device="cuda")
    tre.moe_add_rms_norm_bwd(b["dX"], sum_, rstd, gamma, b["dY"], dx, dg, ws)
    # the products once more, call by call, on these rows
    w = b["wq"] if dtype == "e4m3" else b["wmx"]
    fwd, bwd = ((tre.moe_grouped_gemm_fwd_e4m3, tre.moe_grouped_gemm_bwd_e4m3) if dtype == "e4m3" else
                (tre.moe_grouped_gemm_fwd_mx, tre.moe_grouped_gemm_bwd_mx))
    tok = b["token_of"].long()
    xpq, xps = b["xq"][tok].contiguous(), b["xs"].view(wl.T, -1)[tok].contiguous()
    ab, h, o = (torch.empty_like(b[n]) for n in ("ab", "h", "o"))
    ws_g = torch.empty(max(256, tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD)), dtype=torch.uint8, device="cuda")
    fwd(sh, b["offsets"], xpq, xps, w, ab, h, o, ws_g)
    assert torch.equal(ab, b["ab"]) and torch.equal(h, b["h"]) and torch.equal(o, b["o"])
    got = {n: torch.empty_like(b[n]) for n in ("dab", "dXp", "dW1", "dW3", "dW2")}
    ws_g = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_BWD), dtype=torch.uint8, device="cuda")
    bwd(sh, b["offsets"], b["token_of"], y, ab, h, b["dO"], w, *got.values(), ws_g)
    assert all(torch.equal(t, b[n]) for n, t in got.items())
    # (half a step of bf16 per element of a row, and the fp32 terms' error far below it)
    wx, wg = oracle.rms_norm_bwd(f64(b["dX"]), f64(sum_), f64(rstd), f64(gamma), f64(b["dY"]))
    assert oracle.row_rel_err(f64(dx), wx) <= 2.0 ** -8 + 1e-4
    size = np.abs(f64(b["dX"]) * f64(sum_) * f64(rstd)[:, None]).sum(0)
    assert (np.abs(f64(dg) - wg) <= 2.0 ** -8 * np.abs(wg) + 1e-4 * size).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_backward_workspace_for_several_batches(dtype):
    """MOE_WS_NORM_BWD_MAX of the largest: the bits of calls with workspaces of their own, nothing behind it touched."""
    import token_routed_expert_amd as tre
    d, top = 1024, 2049
    nb = tre.moe_workspace_bytes(tre.make_shape(top, d, 1, 1, 128), tre.MOE_WS_NORM_BWD_MAX)
    assert nb == 2048 * d * 4
    room = torch.full((nb + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    for T in (top, 2048, 1025, 700, 1):
        x, dy, gamma = stream_rows(T, d, dtype, T, special=False)
        rstd = torch.empty(T, device="cuda")
        tre.moe_add_rms_norm(x, None, gamma, EPS, None, None, rstd)
        res = []
        for ws in (room[:nb], torch.full((tre.moe_workspace_bytes(tre.make_shape(T, d, 1, 1, 128), tre.MOE_WS_NORM_BWD),),
                                         0xFF, dtype=torch.uint8, device="cuda")):
            dx, dg = torch.full_like(x, float("nan")), torch.full_like(gamma, float("nan"))
            tre.moe_add_rms_norm_bwd(dy, x, rstd, gamma, None, dx, dg, ws)
            res.append((dx, dg))
        assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
        assert torch.isfinite(res[0][0]).all() and torch.isfinite(res[0][1]).all()
    assert (room[nb:] == 0xFF).all()
