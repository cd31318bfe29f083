"""Entries of token_of outside [0, T) on the GPU: the calls that read x through
the map take them as rows of zeros, forward and weight gradients alike, whichever
kernels run.  Every output has the bits of the same call on permuted rows that
hold those zeros."""
import copy

import numpy as np
import pytest
import torch

from gpu_common import announce, need_gpu
from test_gpu_ckpt8 import COUNTS, Case, backward, checkpoint, few_rows, forward
from test_gpu_mx4 import product_case, run_product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


def unknown(tok, T, row_bytes):
    """tok with entries outside [0, T), among them those whose byte offset is a little
    more than 2^32; and tok with T (a row of zeros behind x's last) in their place."""
    wrap = -(-2 ** 32 // row_bytes)
    bad = tok.copy()
    for i, v in enumerate((T, -1, wrap, wrap + 1, 2 ** 31 - 1, -2 ** 31, wrap + T - 1)):
        bad[(i * 37 + 5) % len(tok)] = v
    zeros = np.where((bad >= 0) & (bad < T), bad, T).astype(np.int32)
    assert (bad != zeros).sum() >= 5
    return bad, zeros


@pytest.mark.parametrize("name", ["edges", "few", "tiles", "many"])
def test_checkpoint_calls(name):
    c = Case(*COUNTS[name], seed=5)
    assert few_rows(c.T, c.E, c.d, c.f) == (name != "many")
    rows = copy.copy(c)
    c.tok, rows.tok = unknown(c.tok, c.T, 2 * c.d)
    rows.x = torch.cat([c.x, torch.zeros(1, c.d, dtype=torch.bfloat16)])
    got, want = forward(c, True), forward(rows, False)
    for a, b, n in zip(got, want, ("abq", "abs", "h", "o")):
        assert torch.equal(a, b), n
    q, s = checkpoint(c, 7)                        # (kept values of their own: no row of zeros)
    (a, dp, _), (b, dq, _) = backward(c, q, s, True), backward(rows, q, s, False)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert torch.equal(dp, dq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("counts,d,f", [([40, 0, 300, 7], 256, 128), ([900], 128, 384)])
def test_gathered_products(dtype, counts, d, f):
    import token_routed_expert_amd as tre
    E, T = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    x, dO = rnd(T, d), rnd(T, d)
    W1, W3, W2 = rnd(E, d, f) * d ** -0.5, rnd(E, d, f) * d ** -0.5, rnd(E, f, d) * f ** -0.5
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    bad, zeros = unknown(np.random.default_rng(3).permutation(T).astype(np.int32), T, x.element_size() * d)
    tok = torch.from_numpy(bad).cuda()
    xp = torch.cat([x, x.new_zeros(1, d)])[torch.from_numpy(zeros).long().cuda()].contiguous()
    sh = tre.make_shape(T, d, E, 1, f, dtype="bf16" if dtype == torch.bfloat16 else "f32")
    outs = []
    for gather in (False, True):
        o = {n: torch.full(s, 7.0, dtype=dtype, device="cuda") for n, s in
             dict(ab=(T, 2 * f), h=(T, f), o=(T, d), dab=(T, 2 * f), dXp=(T, d), dW1=(E, d, f), dW3=(E, d, f),
                  dW2=(E, f, d)).items()}
        src = (tok, x) if gather else (xp,)
        fwd = tre.moe_grouped_gemm_fwd_gather if gather else tre.moe_grouped_gemm_fwd
        bwd = tre.moe_grouped_gemm_bwd_gather if gather else tre.moe_grouped_gemm_bwd
        fwd(sh, off, *src, W1, W3, W2, o["ab"], o["h"], o["o"])
        bwd(sh, off, *src, o["ab"], o["h"], dO, W1, W3, W2, o["dab"], o["dXp"], o["dW1"], o["dW3"], o["dW2"])
        outs.append(o)
    for n in outs[0]:
        assert torch.equal(outs[0][n], outs[1][n]), n


@pytest.mark.parametrize("rows", [5, 21, 300, 3700])     # one and two fragments of the few-row kernel, tiles
@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
def test_mxfp4_product_on_weights_with_a_nan(a8, rows):
    """A row of zeros is no row of zero results where a block of the weights is NaN."""
    counts = [rows, 0, 0, 2]
    X, tok, W1, W3, W2, off = product_case(counts, 384, 256, a8, rows, True)
    T = sum(counts)
    bad, zeros = unknown(tok, T, 384)
    W1[0, 5, 40] = np.nan
    W2[3, 7, 100] = np.inf
    Xz = torch.cat([X, torch.zeros(1, 384, dtype=torch.bfloat16)])[torch.from_numpy(zeros).long()].contiguous()
    X[0, 3] = float("nan")     # (the row whose place a token that there is not takes in the loads)
    keep = torch.from_numpy(zeros != 0)
    got, _ = run_product((X, bad, W1, W3, W2, off), a8, 4, 1, T, 256)
    want, _ = run_product((Xz, None, W1, W3, W2, off), a8, 4, 1, T, 256)
    got, want = got.float().cpu()[keep], want.float().cpu()[keep]
    assert torch.isnan(got[: rows // 2]).all() and not torch.isnan(got[-1, :100]).any()
    assert torch.equal(got.nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))
