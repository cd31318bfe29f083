"""NaNs and infinities in MXFP8 operands on the GPU: a block that holds one has
scale byte 255 in every quantiser, and the products it enters are NaN, in the
experts with 4-bit weights (MXFP8 rows) and in the MXFP8 layer."""
import numpy as np
import pytest
import torch

import device_layout
import oracle
from moe_workloads import Workload, make_inputs

from gpu_common import announce, need_gpu, run_layer
from test_gpu_mx4 import edge_rows, expected, product_case, run_product, u8

pytestmark = pytest.mark.gpu
BAD = {"nan": np.nan, "inf": np.inf, "-inf": -np.inf}


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


def with_bad_blocks(rows, cols, rng):
    """edge_rows, with blocks of nothing but NaN, of a NaN among zeros and among numbers."""
    X = edge_rows(rows, cols, rng)
    blocks = [np.full(32, np.nan), np.r_[np.zeros(31), np.nan], np.r_[np.nan, np.zeros(31)],
              np.r_[np.zeros(7), np.inf, np.zeros(24)], np.full(32, -np.inf), np.r_[np.nan, np.inf, np.ones(30)],
              np.r_[np.full(31, 1e-41), np.nan], np.r_[np.full(31, 3.3e38), -np.nan]]
    for i, b in enumerate(blocks):
        r, c = (i * 11 + 4) % rows, ((i * 3 + 1) % (cols // 32)) * 32
        X[r, c:c + 32] = b
    return X


def same(codes, sb, ref, ref_sb, per):
    """Equal bytes, and equal codes wherever they mean something."""
    assert np.array_equal(sb, ref_sb)
    fine = np.repeat(ref_sb != 255, per, axis=-1)
    assert (ref_sb == 255).any() and np.array_equal(codes[fine], ref[fine])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (37, 384), (300, 1152)])
def test_rows(dtype, rows, cols):
    import token_routed_expert_amd as tre
    X = torch.from_numpy(with_bad_blocks(rows, cols, np.random.default_rng(rows))).to(dtype)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    sb = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    tre.moe_quantize_rows_mx(X.cuda(), codes, sb)
    rq, rs = oracle.quant_mx_rows(X.float().numpy())
    same(u8(codes), u8(sb), rq, rs, 32)


def test_weights():
    import token_routed_expert_amd as tre
    E, R, C = 2, 256, 384
    rng = np.random.default_rng(8)
    W = np.stack([with_bad_blocks(R, C, rng), with_bad_blocks(C, R, rng).T])
    t = {n: torch.empty(*shape, dtype=torch.uint8, device="cuda") for n, shape in
         (("q", (E, R, C)), ("s", (E, R, C // 32)), ("qt", (E, C, R)), ("st", (E, C, R // 32)))}
    tre.moe_quantize_weights_mx(torch.from_numpy(W).cuda(), t["q"], t["s"], t["qt"], t["st"])
    rq, rs, rqt, rst = oracle.quant_mx_weights(W)
    same(u8(t["q"]), u8(t["s"]), rq, rs, 32)
    same(u8(t["qt"]), u8(t["st"]), rqt, rst, 32)


def test_token_blocks():
    import token_routed_expert_amd as tre
    off = np.concatenate([[0], np.cumsum([300, 0, 128, 77, 1, 33])]).astype(np.int32)
    E, P, C = len(off) - 1, int(off[-1]), 384
    X = torch.from_numpy(with_bad_blocks(P, C, np.random.default_rng(2))).bfloat16()
    cap = tre.moe_token_block_capacity(P, E)
    z = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")
    blk = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    codes, sbt, rcodes, rsb = z(P, C), z(cap, C, 4), z(P, C), z(P, C // 32)
    tre.moe_quantize_token_blocks_with_rows_mx(torch.from_numpy(off).cuda(), E, P, X.cuda(), None, blk,
                                               codes, sbt, rcodes, rsb)
    x = X.float().numpy()
    rq, rs = oracle.quant_mx_token_blocks(x, off)
    NB = int(oracle.token_block_offsets(off)[-1])
    got = device_layout.mx_token_block_scales(u8(sbt)[:NB], off)
    assert np.array_equal(got, rs) and (rs == 255).any()
    fine = np.isfinite(oracle.dequant_mx_token_blocks(rq, rs, off))
    assert np.array_equal(u8(codes)[fine], rq[fine])
    same(u8(rcodes), u8(rsb), *oracle.quant_mx_rows(x), 32)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("rows", [5, 300, 4200])   # the kernel for few rows, then tiles
def test_mxfp4_a8_product(rows, bad):
    """The row of x that holds it, and no other, is NaN throughout."""
    case = product_case([rows], 256, 256, True, 4, False)
    ref, _ = run_product(case, True, 1, 1, rows, 256)
    at = min(3, rows - 1)
    case[0][at, 70] = BAD[bad]
    case[0][rows - 1, 32:64] = float("nan")        # a block of nothing else
    o, _ = run_product(case, True, 1, 1, rows, 256)
    gone = torch.isnan(o).cpu()
    keep = torch.ones(rows, dtype=torch.bool)
    keep[[at, rows - 1]] = False
    assert gone[~keep].all() and torch.equal(o.cpu()[keep], ref.cpu()[keep])


@pytest.mark.parametrize("dtype", ["mxfp4", "mxfp4_a8", "mxfp8"])
def test_layer_forward(dtype):
    """A token with a NaN has a NaN y; the other tokens keep their bits."""
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers
    wl = Workload("nan", T=301, d=256, E=8, k=2, f=384, dtype="mxfp8")
    inp = make_inputs(wl, seed=1, device="cuda")
    got = []
    for bad in (False, True):
        if bad:
            inp["x"][7, 3], inp["x"][40, 250] = float("nan"), float("-inf")
        sh, b, ws, _ = layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, 0, dtype, "cuda", inp)
        tre.moe_layer_fwd(sh, b, ws)
        got.append(b["y"].cpu())
    keep = torch.ones(wl.T, dtype=torch.bool)
    keep[[7, 40]] = False
    assert torch.isnan(got[1][~keep]).all() and torch.equal(got[0][keep], got[1][keep])


def test_mxfp8_layer_backward():
    """A NaN in dY reaches the token's dX and the weight gradients it enters: of its
    experts, dW2's column of it (all rows of it) and every dW1 and dW3 column."""
    wl = Workload("nan_bwd", T=301, d=256, E=8, k=2, f=384, dtype="mxfp8")
    inp = make_inputs(wl, seed=1, device="cuda")
    ref = run_layer(wl, inp)
    inp["dY"][9, 100] = float("nan")
    b = run_layer(wl, inp)
    idx = b["topk_idx"][9].cpu().tolist()
    keep = torch.arange(wl.T) != 9
    assert torch.isnan(b["dX"][9]).all() and torch.equal(b["dX"].cpu()[keep], ref["dX"].cpu()[keep])
    for e in range(wl.E):
        nan2 = torch.isnan(b["dW2"][e]).cpu()
        if e in idx:
            assert nan2[:, 100].all() and torch.isnan(b["dW1"][e]).all() and torch.isnan(b["dW3"][e]).all()
            nan2[:, 100] = False
        assert not nan2.any()
        if e not in idx:
            for n in ("dW1", "dW3", "dW2"):
                assert torch.equal(b[n][e], ref[n][e])


def test_the_oracle_layer_and_the_products_quantise_x_alike():
    """oracle.layer_fwd_mx4's o against the device's, x with a NaN and with a block of
    tiny values (scale byte 0, the MXFP8 rows' own clamp)."""
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers
    wl = Workload("x_rule", T=65, d=256, E=8, k=2, f=256)
    inp = make_inputs(wl, seed=3, device="cuda")
    inp["x"][5, 64:96] = 2.0 ** -128
    inp["x"][6, 1] = float("nan")
    sh, b, ws, _ = layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, 0, "mxfp4_a8", "cuda", inp)
    tre.moe_layer_fwd(sh, b, ws)
    h = {n: v.double().cpu().numpy() for n, v in inp.items() if n != "logits"}
    st = oracle.layer_fwd_mx4(inp["logits"].cpu().numpy(), h["x"], h["W1"], h["W3"], h["W2"], wl.k, True)
    xq, xs = oracle.quant_mx_rows(h["x"])
    assert np.array_equal(u8(b["xs"]), xs) and xs[5, 2] == 0 and xs[6, 0] == 255
    assert np.array_equal(np.isnan(b["o"].float().cpu().numpy()), np.isnan(st["o"]))
    case = (inp["x"].cpu(), st["token_of"].astype(np.int32), None, None, None, st["offsets"])
    ref, tol = expected(case, b["wmx4"], True)
    fine = ~np.isnan(st["o"])
    assert np.array_equal(ref[fine], st["o"][fine])
    assert (np.abs(b["o"].double().cpu().numpy() - ref)[fine] <= tol[fine]).all()
