"""An MXFP4 layer with a shared expert, from the library's calls one by one (the
layer call refuses one): the shared expert is a product of one expert on the same
quantised rows, added by the combine."""
import numpy as np
import pytest
import torch

import oracle
from moe_workloads import Workload, make_inputs, to_f64

from gpu_common import announce, need_gpu
from test_gpu_mx4 import expected

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
@pytest.mark.parametrize("T", [3, 300])
def test_layer_with_a_shared_expert(T, a8, request):
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers, quantized_weights_mx4
    need_gpu()
    announce(request.node.nodeid)
    dtype, fs = "mxfp4_a8" if a8 else "mxfp4", 384
    wl = Workload(f"mx4_shared_{T}", T=T, d=256, E=8, k=2, f=256, f_shared=fs)
    inp = make_inputs(wl, seed=5, device="cuda")
    refused = tre.make_shape(T, wl.d, wl.E, wl.k, wl.f, fs, dtype)
    sh, b, ws, _ = layer_buffers(T, wl.d, wl.E, wl.k, wl.f, 0, dtype, "cuda", inp)
    with pytest.raises(tre.MoeError):
        tre.moe_layer_fwd(refused, b, ws)
    w = quantized_weights_mx4(inp["W1"], inp["W3"], inp["W2"])
    wsh = quantized_weights_mx4(*(inp[n][None] for n in ("Ws1", "Ws3", "Ws2")))
    one = tre.make_shape(T, wl.d, 1, 1, fs, dtype=dtype)
    ys = torch.empty(T, wl.d, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ws1 = torch.empty(tre.moe_workspace_bytes(one, tre.MOE_WS_GEMM_FWD), dtype=torch.uint8, device="cuda")
    wsg = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=torch.uint8, device="cuda")
    tre.moe_route(inp["logits"], wl.k, b["topk_idx"], b["topk_prob"])
    tre.moe_permute(sh, None, b["topk_idx"], None, 1, b["counts"], b["offsets"], b["row_of"], b["token_of"],
                    None, ws)
    (tre.moe_quantize_rows_mx if a8 else tre.moe_quantize_rows_mx4)(inp["x"], b["xq"], b["xs"])
    tre.moe_grouped_gemm_fwd_mx4(one, off, None, b["xq"], b["xs"], wsh, ys, ws1)
    tre.moe_grouped_gemm_fwd_mx4(sh, b["offsets"], b["token_of"], b["xq"], b["xs"], w, b["o"], wsg)
    tre.moe_unpermute(sh, b["o"], b["row_of"], b["topk_prob"], ys, b["y"])
    torch.cuda.synchronize()
    x = inp["x"].cpu()
    ref, tol = expected((x, None, None, None, None, np.array([0, T], np.int32)), wsh, a8)
    assert (np.abs(to_f64(ys) - ref) <= tol).all()
    ref, tol = expected((x, b["token_of"].cpu().numpy(), None, None, None, b["offsets"].cpu().numpy()), w, a8)
    assert (np.abs(to_f64(b["o"]) - ref) <= tol).all()
    p, rows, o = (b[n].cpu().numpy().astype(np.float64) if n == "topk_prob" else b[n].cpu().numpy() if n == "row_of"
                  else to_f64(b[n]) for n in ("topk_prob", "row_of", "o"))
    y = oracle.combine(o, rows, p) + to_f64(ys)
    mag = oracle.combine(np.abs(o), rows, p) + np.abs(to_f64(ys))
    # the sum of k + 1 terms in fp32, then bf16
    assert (np.abs(to_f64(b["y"]) - y) <= 2.0 ** -8 * np.abs(y) + (wl.k + 1) * 2.0 ** -23 * mag).all()
