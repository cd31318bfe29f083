"""Integer-weight experts with less workspace than the sums over all parts of K take:
as many parts as fit, nothing outside the workspace, and the same element-by-element
tolerance (it holds for any order of the sums)."""
import numpy as np
import pytest
import torch

from moe_workloads import Workload, make_inputs, to_f64

from gpu_common import announce, need_gpu
from test_gpu_i4 import BF16, PARTS, U8, expected, few, product_case

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


def run_with(case, E, T, d, f, ws_bytes):
    """o with a workspace of ws_bytes and canaries behind it."""
    import token_routed_expert_amd as tre
    X, tok, w, off = case
    sh = tre.make_shape(T, d, E, 1, f, dtype="int4")
    room = torch.full((ws_bytes + GUARD,), 0xFF, dtype=U8, device="cuda")
    o = torch.full((T, d), 7.0, dtype=BF16, device="cuda")
    tre.moe_grouped_gemm_fwd_i4(sh, torch.from_numpy(off).cuda(), None if tok is None else torch.from_numpy(tok).cuda(),
                                X.cuda(), w, o, room[:ws_bytes])
    torch.cuda.synchronize()
    assert (room[ws_bytes:] == 0xFF).all()
    return o


@pytest.mark.parametrize("name", PARTS)
def test_as_many_parts_as_fit(name):
    counts, d, f, fc1, fc2 = PARTS[name]
    E, P = len(counts), sum(counts)
    case = product_case(counts, d, f, 64, True, 5, True)
    ref, tol = expected(case, E, d, f)
    h = 2 * P * f
    one = [4 * P * 2 * f * (fc1 > 1), 4 * P * d * (fc2 > 1)]             # a part's sums of the two products
    full = max(one[0] * fc1, one[1] * fc2)
    sizes = sorted({0, 256, full} | {p * n + e for n, top in zip(one, (fc1, fc2)) for p in range(2, top + 1) if n
                                     for e in (-256, 0)})
    outs = []
    for extra in sizes:
        o = run_with(case, E, P, d, f, h + extra)
        assert (np.abs(to_f64(o) - ref) <= tol).all(), extra
        outs.append(o)
    again = run_with(case, E, P, d, f, h + sizes[0])
    assert torch.equal(again, outs[0])                                   # the same workspace: the same bits
    more = run_with(case, E, P, d, f, h + full + (1 << 20))
    assert torch.equal(more, outs[-1])                                   # more room than is needed changes nothing


def test_a_workspace_of_a_larger_batch_serves_the_smaller_ones():
    """The sizes where a larger T has the smaller moe_workspace_bytes."""
    import token_routed_expert_amd as tre
    d, E, f = 1024, 2, 2048

    def size(T):
        return tre.moe_workspace_bytes(tre.make_shape(T, d, E, 1, f, dtype="int4"), tre.MOE_WS_GEMM_FWD)
    top = next(T for T in range(300, 60000) if size(T) < size(T - 1) and size(T) == 2 * T * f)
    for T in (top, top - 1, top // 2, 301, 3):
        counts = [T - T // 3, T // 3]
        case = product_case(counts, d, f, 128, False, T, True)
        ref, tol = expected(case, E, d, f)
        o = run_with(case, E, T, d, f, size(top))
        assert (np.abs(to_f64(o) - ref) <= tol).all()


@pytest.mark.parametrize("f_shared", [0, 256])
def test_layer_with_the_least_workspace(f_shared):
    """A layer with its aux loss whose K would be taken in parts: in the least workspace, in the reported one, and the
    loss (whose partial sums lie where the products' sums go afterwards) the same."""
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers
    wl = Workload("i4_least", T=1200, d=1536, E=2, k=1, f=2304, f_shared=f_shared, skew=False)
    sh, b, wsf, _ = layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, wl.f_shared, "int4", "cuda",
                                  make_inputs(wl, seed=1, device="cuda"), router_grad=True, group=64)
    b.pop("dlogits")
    assert not few(wl.T, wl.E, wl.d, wl.f)
    assert tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD) > 2 * wl.T * wl.f
    least = (tre.moe_workspace_bytes(sh, tre.MOE_WS_PERMUTE) + 256 + 2 * wl.T * wl.f +
             tre.moe_workspace_bytes(sh, tre.MOE_WS_AUX_LOSS))
    assert least < wsf.numel()
    res = []
    for n in (wsf.numel(), least):
        room = torch.full((n + GUARD,), 0xFF, dtype=U8, device="cuda")
        for name in ("y", "o", "aux_loss"):
            b[name].fill_(float("nan"))
        tre.moe_layer_fwd(sh, b, room[:n])
        torch.cuda.synchronize()
        assert (room[n:] == 0xFF).all()
        tok, off = b["token_of"].cpu().numpy(), b["offsets"].cpu().numpy()
        ref, tol = expected((b["x"].cpu(), tok, b["wi4"], off), wl.E, wl.d, wl.f)
        assert (np.abs(to_f64(b["o"]) - ref) <= tol).all()
        res.append((b["aux_loss"].clone(), b["topk_idx"].clone(), b["y"].clone()))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert torch.isfinite(res[0][0]).all() and torch.isfinite(res[1][2]).all()
    with pytest.raises(tre.MoeError, match="WORKSPACE"):
        tre.moe_layer_fwd(sh, b, room[:least - 1])
