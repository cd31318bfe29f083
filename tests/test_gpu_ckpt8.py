"""8-bit checkpoints of the bf16 experts' pre-activations on the GPU, through the
C ABI, each output against the fp64 formula of the inputs it is made from.

Tolerances.  A bf16 output rounds by 2^-8 of itself.  A sum of n products on the
matrix cores carries at most (n + 16) 2^-23 of the sum of the magnitudes (each
fp32 addition may cut one unit).  The exponential, reciprocal and products of the
SwiGLU add 2^-20 of the result.  The codes: where e, the bound on a's (b's) own
error, carries a value over a rounding border, the neighbouring code is right too.
"""
import numpy as np
import pytest
import torch

import oracle
from moe_workloads import Workload, make_inputs, to_f64

from gpu_common import announce, need_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
COUNTS = {
    "one": ([1], 128, 128),
    "edges": ([16, 0, 15, 17, 1, 31, 32, 33, 0], 256, 128),
    "tiles": ([255, 256, 0, 257, 127], 128, 384),
    "hot": ([600, 1, 0, 40], 384, 256),
    # few rows an expert, more than one tile of 64; many rows (256 x 256 tiles)
    "few": ([63, 64, 65, 0, 128, 1, 2, 3] + [0] * 40, 384, 640),
    "many": ([300, 0, 24700], 128, 640),
    # one expert has most of the rows: another order of the weight gradients' tiles
    "uneven": ([9] * 11 + [400, 0] + [9] * 11, 768, 768),
}


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).bfloat16()


class Case:
    def __init__(self, counts, d, f, seed, extra_rows=0):
        rng = np.random.default_rng(seed)
        self.E, self.rows, self.d, self.f = len(counts), int(sum(counts)), d, f
        self.T = self.rows + extra_rows
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.x = bf16(rng, self.T, d)
        self.tok = rng.permutation(self.T).astype(np.int32)
        self.W1, self.W3 = (bf16(rng, self.E, d, f, std=d ** -0.5) for _ in range(2))
        self.W2 = bf16(rng, self.E, f, d, std=f ** -0.5)
        self.p = rng.uniform(0.01, 1, self.T).astype(np.float32)
        self.dO = bf16(rng, self.T, d)

    def shape(self):
        import token_routed_expert_amd as tre
        return tre.make_shape(self.T, self.d, self.E, 1, self.f, dtype="bf16")

    def dev(self, *names):
        return [torch.from_numpy(v).cuda() if isinstance(v := getattr(self, n), np.ndarray) else v.cuda()
                for n in names]

    def segments(self):
        return [(e, slice(self.off[e], self.off[e + 1])) for e in range(self.E)
                if self.off[e + 1] > self.off[e]]


def z(*shape, dtype=torch.bfloat16, fill=7.0):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


def forward(c, gather):
    import token_routed_expert_amd as tre
    off, tok, x, W1, W3, W2, p = c.dev("off", "tok", "x", "W1", "W3", "W2", "p")
    xin = x if gather else x[tok.long()].contiguous()
    q = z(c.T, 2 * c.f, dtype=torch.uint8, fill=0x55)
    s = z(c.T, 2 * c.f // 32, dtype=torch.uint8, fill=0x55)
    h, o = z(c.T, c.f), z(c.T, c.d)
    tre.moe_grouped_gemm_fwd_ckpt8(c.shape(), off, tok if gather else None, xin, W1, W3, W2, p, q, s, h, o)
    torch.cuda.synchronize()
    return q, s, h, o


def plain_forward(c):
    """The row-scaled forward that keeps [a|b] in bf16."""
    import token_routed_expert_amd as tre
    off, tok, x, W1, W3, W2, p = c.dev("off", "tok", "x", "W1", "W3", "W2", "p")
    ab, h, o = z(c.T, 2 * c.f), z(c.T, c.f), z(c.T, c.d)
    tre.moe_grouped_gemm_fwd_rowscaled(c.shape(), off, x[tok.long()].contiguous(), W1, W3, W2, p, ab, h, o)
    torch.cuda.synchronize()
    return h, o


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("name", COUNTS)
def test_forward(name, gather):
    c = Case(*COUNTS[name], seed=5, extra_rows=3)
    q, s, h, o = forward(c, gather)
    n = c.rows
    assert (q[n:] == 0x55).all() and (s[n:] == 0x55).all() and (o[n:] == 7.0).all()
    xp = c.x.double().numpy()[c.tok]
    W1, W3 = c.W1.double().numpy(), c.W3.double().numpy()
    got = oracle.dequant_mx8_rows(q[:n].cpu().numpy(), s[:n].cpu().numpy())
    back = lambda v: oracle.dequant_mx8_rows(*oracle.quant_mx8_rows(v))  # noqa: E731
    hd, od, W2 = to_f64(h), to_f64(o), c.W2.double().numpy()
    for e, r in c.segments():
        ab, errs = [], []
        for v, W in ((got[r, :c.f], W1), (got[r, c.f:], W3)):
            a = xp[r] @ W[e]
            err = (c.d + 16) * U * (np.abs(xp[r]) @ np.abs(W[e]))
            base = back(a)
            delta = np.maximum(*(np.abs(back(a + t * np.sign(a) * err) - base) for t in (-1, 1)))
            assert (np.abs(v - base) <= delta).all()
            ab.append(a)
            errs.append(err)
        # h = p silu(a) b of the unrounded a and b (|silu'| < 1.1), o from the h that was stored
        (a, b), (ea, eb), p = ab, errs, c.p[r].astype(np.float64)[:, None]
        href = p * oracle.moe.silu(a) * b
        near("h", hd[r], href, (2.0 ** -8 + 2.0 ** -20) * np.abs(href)
             + 1.01 * p * (1.1 * ea * (np.abs(b) + eb) + np.abs(oracle.moe.silu(a)) * eb))
        oref = hd[r] @ W2[e]
        near("o", od[r], oref, 2.0 ** -8 * np.abs(oref) + (c.f + 16) * U * 1.01 * (np.abs(hd[r]) @ np.abs(W2[e])))


def test_forward_is_the_rowscaled_one():
    """Enough rows for the same kernels: the forward's results keep their bits."""
    c = Case([70, 0, 24700], 128, 640, seed=9)
    assert not few_rows(c.T, c.E, c.d, c.f)
    h, o = plain_forward(c)
    for gather in (False, True):
        got = forward(c, gather)
        assert torch.equal(got[2], h) and torch.equal(got[3], o)


def few_rows(P, E, d, f):
    """The calls that take the kernels for few rows (they split the contraction)."""
    if P * (f // 128) * 4 > E * f * d * 2:
        return False

    def steps(bm, bn):
        tiles = P / bm + 0.5 * min(P, E)
        return sum(max(1.0, tiles * ((n + bn - 1) // bn) / 256) * k
                   for n, k in ((2 * f, d), (d, f), (f, d), (d, 2 * f)))
    return P <= 32 * E or steps(64, 128) <= 2.75 * steps(256, 256)


def checkpoint(c, seed):
    """Kept codes of normal values, with blocks of zeros, of tiny and of large ones."""
    rng = np.random.default_rng(seed)
    ab = rng.standard_normal((c.T, 2 * c.f)) * 1.5
    ab[0, :32] = 0.0
    ab[-1, 32:64] = -0.0
    ab[0, 64:96] *= 2.0 ** -40
    ab[-1, :32] *= 8.0
    q, s = oracle.quant_mx8_rows(ab)
    return q, s


def backward(c, q, s, gather, dprob=True, row_of=False):
    import token_routed_expert_amd as tre
    off, tok, x, W1, W3, W2, p, dO = c.dev("off", "tok", "x", "W1", "W3", "W2", "p", "dO")
    xin = x if gather else x[tok.long()].contiguous()
    sh = c.shape()
    ws = z(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_BWD_ROWSCALED), dtype=torch.uint8, fill=0xFF)
    out = dict(h=z(c.T, c.f), dab=z(c.T, 2 * c.f), dXp=z(c.T, c.d), dW1=z(c.E, c.d, c.f),
               dW3=z(c.E, c.d, c.f), dW2=z(c.E, c.f, c.d))
    dp = z(c.T, dtype=torch.float32) if dprob else None
    perm = torch.randperm(c.T, generator=torch.Generator().manual_seed(1)).int().cuda() if row_of else None
    tre.moe_grouped_gemm_bwd_ckpt8(sh, off, tok if gather else None, xin, torch.from_numpy(q).cuda(),
                                   torch.from_numpy(s).cuda(), dO, W1, W3, W2, p, *out.values(), perm, dp,
                                   ws)
    torch.cuda.synchronize()
    return out, dp, perm


def near(name, got, ref, tol):
    over = np.abs(got - ref) / np.maximum(tol, 1e-300)
    assert (over <= 1).all(), f"{name}: worst {over.max():.3f} of the tolerance"


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("name", COUNTS)
def test_backward(name, gather):
    c = Case(*COUNTS[name], seed=6, extra_rows=2)
    q, s = checkpoint(c, 7)
    out, dp, _ = backward(c, q, s, gather)
    g = {n: to_f64(t) for n, t in out.items()}
    n, f = c.rows, c.f
    for k in ("h", "dab", "dXp"):
        assert (g[k][n:] == 7.0).all(), k
    ab = oracle.dequant_mx8_rows(q, s)
    x, dO = c.x.double().numpy()[c.tok], c.dO.double().numpy()
    W1, W3, W2 = (getattr(c, m).double().numpy() for m in ("W1", "W3", "W2"))
    dpn = dp.cpu().numpy().astype(np.float64)
    for e in range(c.E):
        r = slice(c.off[e], c.off[e + 1])
        if r.stop == r.start:
            assert not any(g[k][e].any() for k in ("dW1", "dW3", "dW2"))
            continue
        a, b, p = ab[r, :f], ab[r, f:], c.p[r].astype(np.float64)
        dh = dO[r] @ W2[e].T
        edh = (c.d + 16) * U * (np.abs(dO[r]) @ np.abs(W2[e]).T)
        da, db, h, dprob = oracle.swiglu_bwd_rowscaled(a, b, p, dh)
        ga, gb, _, _ = oracle.swiglu_bwd_rowscaled(a, b, p, np.ones_like(dh))  # d(da)/d(dh)
        # da = p dh b s (1 + a (1 - s)): its last factor is a sum whose terms may cancel
        sg = 1 / (1 + np.exp(-a))
        mag = p[:, None] * np.abs(dh * b) * sg * (1 + np.abs(a) * (1 - sg))
        near("da", g["dab"][r, :f], da, 2.0 ** -8 * np.abs(da) + 1.01 * np.abs(ga) * edh + 2.0 ** -20 * mag)
        near("db", g["dab"][r, f:], db, 2.0 ** -8 * np.abs(db) + 1.01 * np.abs(gb) * edh
             + 2.0 ** -20 * np.abs(db))
        near("h", g["h"][r], h, (2.0 ** -8 + 2.0 ** -20) * np.abs(h))
        gh = np.abs(h / p[:, None])
        near("dprob", dpn[r], dprob, (gh * edh).sum(1) + ((f + 16) * U + 2.0 ** -20) * (gh * np.abs(dh)).sum(1))
        # the products, from the dab and h that the call wrote
        da, db, h = g["dab"][r, :f], g["dab"][r, f:], g["h"][r]

        def product(name, got, A, B, A2=None, B2=None):
            ref, m = A @ B, np.abs(A) @ np.abs(B)
            k = A.shape[1]
            if A2 is not None:
                ref, m, k = ref + A2 @ B2, m + np.abs(A2) @ np.abs(B2), k + A2.shape[1]
            near(name, got, ref, 2.0 ** -8 * np.abs(ref) + (k + 16) * U * 1.01 * m)
        product("dXp", g["dXp"][r], da, W1[e].T, db, W3[e].T)
        product("dW1", g["dW1"][e], x[r].T, da)
        product("dW3", g["dW3"][e], x[r].T, db)
        product("dW2", g["dW2"][e], h.T, dO[r])


def test_backward_is_the_rowscaled_one_on_the_kept_values():
    """E4M3 times a power of two fits bf16: the bf16 backward on the values that the
    codes stand for must give the same bits, gathered or not."""
    import token_routed_expert_amd as tre
    c = Case([70, 0, 300, 5, 41000], 128, 384, seed=9)
    assert not few_rows(c.T, c.E, c.d, c.f)
    q, s = checkpoint(c, 3)
    a, dpa, _ = backward(c, q, s, True)
    b, dpb, _ = backward(c, q, s, False)
    off, tok, x, W1, W3, W2, p, dO = c.dev("off", "tok", "x", "W1", "W3", "W2", "p", "dO")
    ab = torch.from_numpy(oracle.dequant_mx8_rows(q, s)).bfloat16().cuda()
    sh = c.shape()
    ws = z(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_BWD_ROWSCALED), dtype=torch.uint8)
    h, dab, dXp = z(c.T, c.f), z(c.T, 2 * c.f), z(c.T, c.d)
    dW1, dW3, dW2 = z(c.E, c.d, c.f), z(c.E, c.d, c.f), z(c.E, c.f, c.d)
    dp = z(c.T, dtype=torch.float32)
    tre.moe_grouped_gemm_bwd_rowscaled(sh, off, x[tok.long()].contiguous(), ab, h, dO, W1, W3, W2, p, dab,
                                       dXp, dW1, dW3, dW2, None, dp, ws, recompute_h=True)
    torch.cuda.synchronize()
    for n, t in dict(h=h, dab=dab, dXp=dXp, dW1=dW1, dW3=dW3, dW2=dW2).items():
        assert torch.equal(a[n], t) and torch.equal(b[n], t), n
    assert torch.equal(dpa, dp) and torch.equal(dpb, dp)


@pytest.mark.parametrize("counts,d,f", [([70] * 16, 384, 640), ([300, 0, 24700], 128, 640)], ids=["few", "many"])
def test_repeated_calls_give_the_same_bits(counts, d, f):
    c = Case(counts, d, f, seed=11)
    q, s = checkpoint(c, 4)
    ref, (out, dp, _) = forward(c, True), backward(c, q, s, True)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(ref, forward(c, True)))
        again, dq, _ = backward(c, q, s, True)
        assert torch.equal(dp, dq) and all(torch.equal(out[n], again[n]) for n in out)


def test_dprob_order_and_absence():
    c = Case([40, 9], 128, 128, seed=1)
    q, s = checkpoint(c, 2)
    a, dp, _ = backward(c, q, s, True)
    b, dq, perm = backward(c, q, s, True, row_of=True)
    n, none, _ = backward(c, q, s, True, dprob=False)
    assert none is None and torch.equal(dq, dp[perm.long()])
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], n[k])


def test_a_nan_row_stays_its_own():
    """A NaN or an infinity in one token: its blocks read back as NaN, its gradients
    and its expert's weight gradients are NaN, everything else keeps its bits."""
    import token_routed_expert_amd as tre
    c = Case([30, 40], 128, 128, seed=2)
    ref = forward(c, True)
    r0, _, _ = backward(c, ref[0].cpu().numpy(), ref[1].cpu().numpy(), True)
    c.x[c.tok[33], 5] = float("inf")
    q, s, h, o = forward(c, True)
    assert (s[33] == 255).all() and (s[:33] != 255).all() and (s[34:] != 255).all()
    keep = torch.arange(70) != 33
    assert torch.equal(q.cpu()[keep], ref[0].cpu()[keep]) and torch.equal(o.cpu()[keep], ref[3].cpu()[keep])
    got, _, _ = backward(c, q.cpu().numpy(), s.cpu().numpy(), True)
    assert torch.isnan(got["dXp"][33]).all() and torch.isnan(got["dW1"][1]).all()
    assert torch.equal(got["dXp"].cpu()[keep], r0["dXp"].cpu()[keep])
    for n in ("dW1", "dW3", "dW2"):
        assert torch.equal(got[n][0], r0[n][0])


LAYERS = [(Workload("ck", T=333, d=256, E=16, k=4, f=384), dict(router_grad=True)),
          (Workload("ck_fused", T=333, d=256, E=16, k=4, f=384), dict(router_grad=True, fused_permute=True)),
          (Workload("ck_shared", T=200, d=256, E=8, k=2, f=256, f_shared=128), {}),
          (Workload("ck_skew", T=500, d=128, E=24, k=3, f=128, skew=True), dict(fused_permute=True)),
          (Workload("ck_many", T=8200, d=128, E=4, k=4, f=256), dict(router_grad=True)),
          (Workload("ck_many_fused", T=8200, d=128, E=4, k=4, f=256), dict(fused_permute=True))]
GRADS = ("dX", "dW1", "dW3", "dW2", "dWs1", "dWs3", "dWs2", "dprob", "dlogits")


@pytest.mark.parametrize("wl,kw", LAYERS, ids=lambda c: c.name if isinstance(c, Workload) else "")
def test_layer(wl, kw):
    """moe_layer_fwd / _bwd with memory_efficient = 3 are the calls in sequence, bit
    for bit; the backward reads neither h nor o nor ab.  Where both take the same
    kernels (many rows), the forward is mode 2's and the backward is mode 2's on the
    values that were kept, bit for bit."""
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers
    inp = make_inputs(wl, seed=3, device="cuda")

    def buffers(mode):
        return layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, wl.f_shared, "bf16", "cuda", inp,
                             memory_efficient=mode, **kw)
    sh, b, wsf, wsb = buffers(3)
    assert "ab" not in b
    tre.moe_layer_fwd(sh, b, wsf)
    y, P = b["y"].clone(), wl.T * wl.k
    x = (b["token_of"], b["x"]) if "xp" not in b else (None, b["xp"])
    W = (b["W1"], b["W3"], b["W2"], b["row_prob"])
    q, s = torch.empty_like(b["ab_q"]), torch.empty_like(b["ab_s"])
    h, o = torch.empty_like(b["h"]), torch.empty_like(b["o"])
    plain = tre.make_shape(wl.T, wl.d, wl.E, wl.k, wl.f)
    tre.moe_grouped_gemm_fwd_ckpt8(plain, b["offsets"], *x, *W, q, s, h, o)
    assert torch.equal(q, b["ab_q"]) and torch.equal(s, b["ab_s"]) and torch.equal(o, b["o"])
    for n in ("h", "o"):
        b[n].fill_(float("nan"))
    tre.moe_layer_bwd(sh, b, wsb)
    out = [torch.empty_like(b[n]) for n in ("h", "dab", "dXp", "dW1", "dW3", "dW2")]
    dp = torch.empty(wl.T, wl.k, device="cuda")
    ws = torch.empty(tre.moe_workspace_bytes(plain, tre.MOE_WS_GEMM_BWD_ROWSCALED), dtype=torch.uint8,
                     device="cuda")
    tre.moe_grouped_gemm_bwd_ckpt8(plain, b["offsets"], *x, q, s, b["dO"], *W, *out, b["row_of"], dp, ws)
    for n, t in zip(("h", "dab", "dXp", "dW1", "dW3", "dW2"), out):
        assert torch.equal(b[n], t), n
    if "dprob" in b:
        assert torch.equal(b["dprob"], dp)
    for n in GRADS:
        assert n not in b or torch.isfinite(b[n]).all(), n
    # mode 2 on the kept values
    _, m, wf, wb = buffers(2)
    tre.moe_layer_fwd(sh, m, wf)
    kept = oracle.dequant_mx8_rows(b["ab_q"].cpu().numpy(), b["ab_s"].cpu().numpy())
    exact = to_f64(m["ab"])
    step = 2.0 ** -4 * np.abs(exact) + 2.0 ** -8 * np.abs(exact) + 1e-3 * np.abs(exact).max(1, keepdims=True)
    assert (np.abs(kept - exact) <= step).all()
    if few_rows(P, wl.E, wl.d, wl.f):
        return
    assert torch.equal(m["y"], y)
    m["ab"].copy_(torch.from_numpy(kept).bfloat16())
    tre.moe_layer_bwd(sh, m, wb)
    torch.cuda.synchronize()
    for n in GRADS:
        if n in b:
            assert torch.equal(b[n], m[n]), n


def test_layer_graph_replays_on_new_inputs():
    """Forward and backward captured, replayed on changed inputs with eager layers of
    the same buffers between the replays."""
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers
    wl = Workload("ck_graph", T=300, d=256, E=8, k=2, f=256)
    inp = make_inputs(wl, seed=2, device="cuda")
    sh, b, wsf, wsb = layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, 0, "bf16", "cuda", inp,
                                    router_grad=True, memory_efficient=3, fused_permute=True)

    def step():
        tre.moe_layer_fwd(sh, b, wsf)
        tre.moe_layer_bwd(sh, b, wsb)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    names = ("y", "dX", "dW1", "dW3", "dW2", "dlogits", "ab_q", "ab_s")
    for rep in range(4):
        new = make_inputs(wl, seed=20 + rep, device="cuda")
        for n in ("logits", "x", "dY"):
            b[n].copy_(new[n])
        for n in names:
            b[n].fill_(float("nan") if b[n].is_floating_point() else 0xAA)
        g.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in names}
        step()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(got[n], b[n]), (rep, n)
