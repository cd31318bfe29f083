"""The MXFP4 quantiser of rows beyond the threads of one launch."""
import numpy as np
import pytest
import torch

import oracle

from gpu_common import announce, need_gpu

pytestmark = pytest.mark.gpu


def test_rows_of_more_than_one_launch(request):
    import token_routed_expert_amd as tre
    need_gpu()
    announce(request.node.nodeid)
    rows, cols = (1 << 23) + 3, 4096                       # 2^35 values and a little more
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 23) - 1, 1 << 23, rows - 1]
    some = torch.from_numpy(np.random.default_rng(1).standard_normal((len(at), cols)).astype(np.float32)).bfloat16()
    x[at] = some.cuda()
    codes = torch.full((rows, cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((rows, cols // 32), 0xA5, dtype=torch.uint8, device="cuda")
    tre.moe_quantize_rows_mx4(x, codes, sb)
    rq, rs = oracle.quant_mx4_rows(some.double().numpy())
    assert np.array_equal(codes[at].cpu().numpy(), rq) and np.array_equal(sb[at].cpu().numpy(), rs)
    codes[at] = 0
    sb[at] = 127
    assert not codes.view(torch.int64).any() and int(sb.min()) == 127 and int(sb.max()) == 127
    del x, codes, sb
    torch.cuda.empty_cache()


def free(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
@pytest.mark.parametrize("few", [True, False], ids=["few", "many"])
def test_product_at_full_widths(a8, few, request):
    """d 4096, f 14336, rows read through token_of: the tile kernel with as many rows
    as the call takes (the quantised h ends just below 2^31 bytes), the kernel for
    few rows with as many weight bytes; sampled rows, among them the first and the
    last of each expert."""
    import token_routed_expert_amd as tre
    from test_gpu_mx4 import expected
    need_gpu()
    announce(request.node.nodeid)
    free(16)
    d, f, E = 4096, 14336, 2
    P = 39 if few else (2 ** 31 - 4096 - 1) // f
    T = P
    counts = [P - 14, 14] if few else [P // 2 + 77, P - P // 2 - 77]
    sh = tre.make_shape(T, d, E, 1, f, dtype="mxfp4_a8" if a8 else "mxfp4")
    assert tre.moe_few_rows(sh) == few
    if not few:                                   # one row more is refused
        assert (P + 1) * f >= 2 ** 31 - 4096
    g = torch.Generator(device="cuda").manual_seed(4)
    rnd = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, dtype=torch.uint8, device="cuda")
    # (scales of 2^-10 to 2^-7: a, b and o of order one)
    w = tre.MX4Weights({"W13": rnd(0, 256, E, 2 * f // 16, d // 128, 4, 16, 16),
                        "W2": rnd(0, 256, E, d // 16, f // 128, 4, 16, 16),
                        "W13s": rnd(117, 121, E, 2 * f // 64, d // 128, 4, 16, 4),
                        "W2s": rnd(117, 121, E, d // 64, f // 128, 4, 16, 4)})
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    tok = torch.randint(0, T, (P,), generator=g, device="cuda", dtype=torch.int32)
    tok[-1], tok[0] = T - 1, T - 1
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xq = torch.empty(T, d if a8 else d // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(T, d // 32, dtype=torch.uint8, device="cuda")
    (tre.moe_quantize_rows_mx if a8 else tre.moe_quantize_rows_mx4)(x, xq, xs)
    o = torch.full((P, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=torch.uint8, device="cuda")
    tre.moe_grouped_gemm_fwd_mx4(sh, torch.from_numpy(off).cuda(), tok, xq, xs, w, o, ws)
    assert torch.isfinite(o).all()
    at = sorted({0, 1, off[1] - 1, off[1], P - 2, P - 1, off[1] // 3, off[1] + (P - off[1]) // 2})
    at = torch.tensor([int(i) for i in at])
    rows = x[tok[at.cuda()].long()].cpu()
    n0 = int((at < int(off[1])).sum())
    case = (rows, None, None, None, None, np.array([0, n0, len(at)], np.int32))
    ref, tol = expected(case, w, a8)
    got = o[at.cuda()].double().cpu().numpy()
    over = np.abs(got - ref) / np.maximum(tol, 1e-300)
    assert (over <= 1).all(), f"worst {over.max():.3f} of the tolerance"


def test_checkpoint_calls_at_full_widths(request):
    """The bf16 kernels for few rows at d 4096, f 14336: h and o of every row in fp64
    from the stored operands, tolerances as in test_gpu_ckpt8."""
    import token_routed_expert_amd as tre
    need_gpu()
    announce(request.node.nodeid)
    free(8)
    d, f, E, counts = 4096, 14336, 2, [37, 20]
    P = sum(counts)
    sh = tre.make_shape(P, d, E, 1, f)
    assert tre.moe_few_rows(sh)
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()
    x, W1, W3 = rnd(P, d), rnd(E, d, f, std=d ** -0.5), rnd(E, d, f, std=d ** -0.5)
    W2, p = rnd(E, f, d, std=f ** -0.5), torch.rand(P, generator=g, device="cuda")
    off = torch.tensor([0, counts[0], P], dtype=torch.int32, device="cuda")
    q = torch.empty(P, 2 * f, dtype=torch.uint8, device="cuda")
    s = torch.empty(P, 2 * f // 32, dtype=torch.uint8, device="cuda")
    h, o = (torch.empty(P, n, dtype=torch.bfloat16, device="cuda") for n in (f, d))
    tre.moe_grouped_gemm_fwd_ckpt8(sh, off, None, x, W1, W3, W2, p, q, s, h, o)
    U = 2.0 ** -23
    for e, r in enumerate((slice(0, counts[0]), slice(counts[0], P))):
        xd, pd = x[r].double(), p[r].double()[:, None]
        a, b = xd @ W1[e].double(), xd @ W3[e].double()
        ea, eb = ((d + 16) * U * (xd.abs() @ W[e].double().abs()) for W in (W1, W3))
        silu = a * torch.sigmoid(a)
        ref = pd * silu * b
        tol = (2.0 ** -8 + 2.0 ** -20) * ref.abs() + 1.01 * pd * (1.1 * ea * (b.abs() + eb) + silu.abs() * eb)
        assert ((h[r].double() - ref).abs() <= tol).all()
        hd, w2 = h[r].double(), W2[e].double()
        ref = hd @ w2
        assert ((o[r].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (f + 16) * U * 1.01 * (hd.abs() @ w2.abs())).all()
