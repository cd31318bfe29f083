"""MXFP4 on the GPU against the oracle, through the C ABI: quantisers bit-exact,
the experts' product element by element, the layer, streams, graphs.

Tolerance of the product, for one element of o = Q(h) W2:
* h comes from fp32 sums: an element may differ from the exact one by
  e = 1.1 |b| g_a + |silu(a)| g_b + 2^-20 |h|, g = (d + 16) 2^-24 sum |x w| (the
  worst rounding of d fp32 additions; |silu'| < 1.1; the last term covers the
  exponential and the reciprocal).  Where that carries h across a rounding
  border its code moves: delta = max |Q(h +- e) - Q(h)|, and o by sum delta |W2|;
* with E4M3 rows (a8) the matrix instruction cuts the products of each 8
  consecutive k, toward zero, to multiples of 2^-13 of the largest one's binade
  (read from single products next to a large one), so each of the 7 others loses
  less than 2^-13 of it: g and the sum over f grow by 7 * 2^-13 * the sum over
  groups of 8 of the largest |product|;
* the sum over f rounds by at most (f + 16) 2^-24 sum |Q(h) W2|;
* o is stored in bf16: 2^-8 |o|.
"""
import numpy as np
import pytest
import torch

import oracle
from moe_workloads import Workload, make_inputs, to_f64
from oracle.moe import silu

from gpu_common import announce, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


def u8(t):
    return t.cpu().numpy()


def edge_rows(rows, cols, rng):
    """Rows with every special block: zeros of both signs, subnormals, borders of
    the scale rule, all midpoints, large and small magnitudes, NaN, infinities."""
    X = rng.standard_normal((rows, cols)).astype(np.float32)
    X *= np.exp2(rng.integers(-30, 30, (rows, cols // 32))).repeat(32, 1).astype(np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    special = [np.zeros(32), -np.zeros(32), np.full(32, 1e-41), np.tile(mids, 4),
               -np.tile(np.nextafter(mids, 0, dtype=np.float32), 4), np.full(32, 6.0 * 2.0 ** 100),
               np.tile(np.nextafter(mids, 7, dtype=np.float32), 4), np.full(32, 3.3e38),
               np.r_[np.nan, np.ones(31)], np.r_[np.ones(31), np.inf], np.r_[np.ones(31), -np.inf],
               np.r_[2.0 ** -126, np.zeros(31)], np.r_[-1.5 * 2.0 ** -124, np.full(31, 1e-38)]]
    for i, blk in enumerate(special):
        r, c = (i * 7) % rows, ((i * 5) % (cols // 32)) * 32
        X[r, c:c + 32] = blk
    return X


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (37, 384), (1000, 4096)])
def test_quantize_rows_bit_exact(dtype, rows, cols):
    import token_routed_expert_amd as tre
    X = torch.from_numpy(edge_rows(rows, cols, np.random.default_rng(rows + cols))).to(dtype)
    guard = 64
    codes = torch.full((rows * cols // 2 + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((rows * cols // 32 + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    tre.moe_quantize_rows_mx4(X.cuda(), codes, sb)
    rq, rs = oracle.quant_mx4_rows(X.double().numpy())
    got = u8(codes[:-guard]).reshape(rows, -1)
    assert np.array_equal(u8(sb[:-guard]).reshape(rows, -1), rs)
    fine = np.repeat(rs != 255, 16, axis=1)
    assert np.array_equal(got[fine], rq[fine])
    assert (codes[-guard:] == 0xA5).all() and (sb[-guard:] == 0xA5).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("E,R,C", [(1, 128, 128), (2, 384, 256), (3, 128, 384)])
def test_quantize_weights_bit_exact_and_back(dtype, pair, E, R, C):
    import token_routed_expert_amd as tre
    rng = np.random.default_rng(E + R + C)
    Ws = [torch.from_numpy(np.stack([edge_rows(C, R, rng).T for _ in range(E)]).copy()).to(dtype)
          for _ in range(1 + pair)]
    n = len(Ws)
    codes = torch.empty(E, n * C // 16, R // 128, 4, 16, 16, dtype=torch.uint8, device="cuda")
    sb = torch.empty(E, n * C // 64, R // 128, 4, 16, 4, dtype=torch.uint8, device="cuda")
    dev = [w.cuda() for w in Ws] + [None]
    tre.moe_quantize_weights_mx4(dev[0], dev[1], codes, sb)
    rq, rs = oracle.quant_mx4_weights(*[w.double().numpy() for w in Ws])
    assert np.array_equal(u8(sb), rs)
    # the scale byte of every code byte: [E][N/64][KT][4][16][4 tiles] -> [E][N/16][KT][4][16]
    of = rs.transpose(0, 1, 5, 2, 3, 4).reshape(rq.shape[:-1])
    fine = of != 255
    assert np.array_equal(u8(codes)[fine], rq[fine])
    out = [torch.empty(E, R, C, dtype=torch.bfloat16, device="cuda") for _ in range(n)] + [None]
    tre.moe_dequantize_weights_mx4(codes, sb, out[0], out[1])
    want = oracle.dequant_mx4_weights(rq, rs)
    parts = oracle.mx4.split_pair(want) if pair else (want,)
    for o, w in zip(out, parts):
        assert np.array_equal(to_f64(o), torch.from_numpy(w).to(torch.bfloat16).double().numpy(),
                              equal_nan=True)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def product_case(counts, d, f, a8, seed, gather, T=None):
    """Random quantised rows and weights for given rows per expert."""
    rng = np.random.default_rng(seed)
    E, P = len(counts), int(sum(counts))
    T = P if T is None else T
    X = torch.from_numpy(rng.standard_normal((T if gather else P, d)).astype(np.float32)).bfloat16()
    tok = rng.integers(0, T, T).astype(np.int32) if gather else None   # (entries past the last expert: unused)
    W1, W3 = (rng.standard_normal((E, d, f)).astype(np.float32) * d ** -0.5 for _ in range(2))
    W2 = rng.standard_normal((E, f, d)).astype(np.float32) * f ** -0.5
    return X, tok, W1, W3, W2, offsets_of(counts)


def run_product(case, a8, E, k, T, f):
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import quantized_weights_mx4
    X, tok, W1, W3, W2, off = case
    d = X.shape[1]
    sh = tre.make_shape(T, d, E, k, f, dtype="mxfp4_a8" if a8 else "mxfp4")
    w = quantized_weights_mx4(*[torch.from_numpy(m).cuda() for m in (W1, W3, W2)])
    rows = X.shape[0]
    xq = torch.empty(rows, d if a8 else d // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(rows, d // 32, dtype=torch.uint8, device="cuda")
    (tre.moe_quantize_rows_mx if a8 else tre.moe_quantize_rows_mx4)(X.cuda(), xq, xs)
    o = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    tre.moe_grouped_gemm_fwd_mx4(sh, torch.from_numpy(off).cuda(),
                                 None if tok is None else torch.from_numpy(tok).cuda(), xq, xs, w, o, ws)
    torch.cuda.synchronize()
    return o, w


def cut(X, W):
    """7 * 2^-13 * sum over groups of 8 k of max |X[:, k] W[k, :]| (float64)."""
    X, W = (torch.from_numpy(np.abs(v)).cuda() for v in (X, W))
    out = torch.zeros(X.shape[0], W.shape[1], dtype=torch.float64, device="cuda")
    for k in range(0, X.shape[1], 8):
        out += (X[:, k:k + 8, None] * W[None, k:k + 8]).amax(1)
    return 7 * 2.0 ** -13 * out.cpu().numpy()


def expected(case, w, a8):
    X, tok, W1, W3, W2, off = case
    x = X.double().numpy()
    xd = oracle.dequant_mx8_rows(*oracle.quant_mx_rows(x)) if a8 else \
        oracle.dequant_mx4_rows(*oracle.quant_mx4_rows(x))
    xd = xd if tok is None else xd[tok]
    W13d = oracle.dequant_mx4_weights(u8(w["W13"]), u8(w["W13s"]))
    W2d = oracle.dequant_mx4_weights(u8(w["W2"]), u8(w["W2s"]))
    a, b, h, o = oracle.experts_mx4(xd, off, W13d, W2d, a8)
    q = (lambda v: oracle.dequant_mx8_rows(*oracle.quant_mx8_rows(v))) if a8 else \
        (lambda v: oracle.dequant_mx4_rows(*oracle.quant_mx4_rows(v)))
    tol = 2.0 ** -8 * np.abs(o)
    d, f = xd.shape[1], h.shape[1]
    for e in range(len(off) - 1):
        r = slice(off[e], off[e + 1])
        if r.stop == r.start:
            continue
        mag = oracle.mx4.split_pair(np.abs(xd[r]) @ np.abs(W13d[e]))
        ga, gb = ((d + 16) * 2.0 ** -24 * m for m in mag)
        if a8:
            ga, gb = (g + c for g, c in zip((ga, gb), oracle.mx4.split_pair(cut(xd[r], W13d[e]))))
        err = 1.1 * np.abs(b[r]) * ga + np.abs(silu(a[r])) * gb + 2.0 ** -20 * np.abs(h[r])
        base = q(h[r])
        delta = np.maximum(*(np.abs(q(h[r] + s * np.sign(h[r]) * err) - base) for s in (-1, 1)))
        tol[r] += delta @ np.abs(W2d[e]) + (f + 16) * 2.0 ** -24 * (np.abs(base) @ np.abs(W2d[e]))
        if a8:
            tol[r] += cut(np.abs(base) + delta, W2d[e])
    return o, tol


def check(case, a8, E, k, T, f):
    o, w = run_product(case, a8, E, k, T, f)
    ref, tol = expected(case, w, a8)
    P = int(case[-1][-1])
    got = to_f64(o)
    over = np.abs(got[:P] - ref[:P]) / np.maximum(tol[:P], 1e-300)
    assert not P or (over <= 1).all(), f"worst {over.max():.3f} of the tolerance"
    assert (got[P:] == 7.0).all(), "rows behind the last expert were written"


# rows per expert around every fragment, tile and choice of kernel
COUNTS = {
    "one_row": [1],
    "one_row_of_many": [0, 0, 0, 1, 0, 0, 0, 0],
    "edges16": [16, 0, 15, 17, 1, 31, 32, 33],
    "edges64": [63, 64, 0, 65, 128],
    "edges128": [127, 129, 0, 200, 1],
    "edges256": [255, 256, 257],
    "hot": [700, 3, 0, 1],
    "wide": [0, 5] * 100,
    "tail": [513],
    # few rows on average: one expert holds many, and the passes of 16 and 32 rows end inside them
    "few_edges": [16, 17, 0, 31, 32, 33, 48, 64, 65] + [0] * 30,
    "few_hot": [0] * 40 + [300, 1],
}


def few_rows(P, E, d, f):
    """The calls that take the kernel for few rows."""
    pieces = P / 32 + 0.5 * min(P, E)
    steps = max(1.0, pieces * (2 * f // 64) / 512) * d + max(1.0, pieces * (d // 64) / 512) * f
    return P <= 20 * E or steps <= 1.5 * (d + f)


def with_many(counts, d, f):
    """An expert more, with enough rows for the kernel for many rows."""
    n = 65
    while few_rows(sum(counts) + n, len(counts) + 1, d, f):
        n += 64
    return counts + [n]


@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("name", COUNTS)
def test_product(name, gather, a8, many):
    counts = COUNTS[name]
    d, f = {"edges64": (384, 256), "edges128": (128, 640), "hot": (640, 128), "tail": (256, 384),
            "edges256": (512, 256)}.get(name, (256, 128))
    if many:
        counts = with_many(counts, d, f)
    P = sum(counts)
    case = product_case(counts, d, f, a8, 3 + P, gather)
    check(case, a8, len(counts), 1, P, f)


@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
@pytest.mark.parametrize("d,f", [(128, 128), (128, 1152), (1152, 128), (896, 384)])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_product_widths(d, f, a8, many):
    counts = with_many([40, 0, 1, 90], d, f) if many else [40, 0, 1, 90]
    case = product_case(counts, d, f, a8, d + f, True)
    check(case, a8, len(counts), 1, sum(counts), f)


@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
def test_rows_past_the_last_expert_stay(a8):
    """offsets[E] below P (assignments that the map skipped)."""
    case = product_case([20, 0, 300], 256, 256, a8, 9, True, T=400)
    check(case, a8, 3, 1, 400, 256)
    counts = with_many([20, 0], 256, 256)
    case = product_case(counts, 256, 256, a8, 9, True, T=sum(counts) + 90)
    check(case, a8, 3, 1, sum(counts) + 90, 256)
    empty = product_case([0, 0], 256, 256, a8, 9, False, T=4)
    case = (torch.ones(8, 256).bfloat16(), None) + empty[2:]
    check(case, a8, 2, 2, 4, 256)


@pytest.mark.parametrize("per_expert", [8, 100])
@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
def test_repeated_calls_give_the_same_bits(a8, per_expert):
    """Many tiles with few K steps, over and over: a load that is read before it has
    landed (its slot then holds what an earlier call left) shows as another result."""
    import token_routed_expert_amd as tre
    E, k, d, f = 96, 8, 384, 1152
    T = E * per_expert // k
    g = torch.Generator(device="cuda").manual_seed(5)
    dev = dict(dtype=torch.uint8, device="cuda")
    sh = tre.make_shape(T, d, E, k, f, dtype="mxfp4_a8" if a8 else "mxfp4")
    rnd = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, **dev)
    # (scales that differ from block to block, around 2^-4)
    w = tre.MX4Weights({"W13": rnd(0, 256, E, d * f), "W2": rnd(0, 256, E, d * f // 2),
                        "W13s": rnd(121, 126, E, d * f // 16), "W2s": rnd(121, 126, E, d * f // 32)})
    off = torch.arange(0, E + 1, dtype=torch.int32, device="cuda") * per_expert
    ws = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), **dev)
    xs = rnd(121, 126, T, d // 32)
    tok = torch.randint(0, T, (T * k,), generator=g, device="cuda", dtype=torch.int32)
    xq = [rnd(0, 120 if a8 else 256, T, d if a8 else d // 2) for _ in range(2)]
    o = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda")
    first = [None, None]
    for i in range(400):
        tre.moe_grouped_gemm_fwd_mx4(sh, off, tok, xq[i & 1], xs, w, o, ws)
        if i < 2:
            first[i] = o.clone()
            assert torch.isfinite(o).all()
        else:
            assert torch.equal(o, first[i & 1]), f"call {i}"


@pytest.mark.parametrize("rows", [21, 300, 3700])
@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
def test_a_token_that_there_is_not_reads_zeros(a8, rows):
    """Entries of token_of outside [0, T): rows of zeros, their neighbours untouched."""
    counts = [rows] if rows > 32 else [rows, 0, 0, 2]
    E, T = len(counts), sum(counts)
    case = product_case(counts, 384, 256, a8, rows, True)
    o, w = run_product(case, a8, E, 1, T, 256)
    tok = case[1].copy()
    bad = {0: -1, 3: T, rows // 2: 2 ** 31 - 1, rows - 1: -2 ** 31}
    for at, v in bad.items():
        tok[at] = v
    got, _ = run_product((case[0], tok) + case[2:], a8, E, 1, T, 256)
    got, want = to_f64(got), to_f64(o)
    want[list(bad)] = 0
    assert np.array_equal(got, want)


@pytest.mark.parametrize("rows", [5, 300, 4200])
@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
def test_a_nan_stays_in_its_row(a8, rows):
    """A NaN in x (4-bit rows), or one that arises in h (a scale of 255 in a
    weight block), gives NaN outputs where the formula has them and nowhere else."""
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import quantized_weights_mx4
    case = product_case([rows], 256, 256, a8, 4, False)
    X = case[0]
    ref, w = run_product(case, a8, 1, 1, rows, 256)
    if not a8:
        X[3, 70] = float("nan")
        o, _ = run_product(case, a8, 1, 1, rows, 256)
        bad = torch.isnan(o).cpu()
        assert bad[3].all() and not bad[:3].any() and not bad[4:].any()
        keep = torch.arange(rows) != 3
        assert torch.equal(o.cpu()[keep], ref.cpu()[keep])
        X[3, 70] = 0.5
    W2 = case[4].copy()
    W2[0, 5, 9] = np.inf                      # one 32-row block of output column 9
    o, _ = run_product(case[:4] + (W2, case[5]), a8, 1, 1, rows, 256)
    bad = torch.isnan(o).cpu()
    assert bad[:, 9].all() and bad.sum() == rows
    W1 = case[2].copy()
    W1[0, 5, 40] = np.nan                     # h column 40, so its whole block and every output
    o, _ = run_product(case[:2] + (W1,) + case[3:], a8, 1, 1, rows, 256)
    assert torch.isnan(o).all()


def layer(wl, a8, inp, **kw):
    import token_routed_expert_amd as tre
    from token_routed_expert_amd.buffers import layer_buffers
    sh, b, ws, _ = layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, 0, "mxfp4_a8" if a8 else "mxfp4", "cuda",
                                 inp, **kw)
    return tre, sh, b, ws


@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (3, 16, 4), (257, 8, 2), (301, 64, 8), (2300, 8, 2)])
def test_layer_forward(T, E, k, a8):
    """Route, map, quantise, experts, combine: the parts' own results put
    together in fp64 give y within bf16's rounding of o and of y."""
    wl = Workload(f"mx4_{T}_{E}", T=T, d=256, E=E, k=k, f=384)
    inp = {n: v for n, v in make_inputs(wl, seed=1, device="cuda").items()}
    tre, sh, b, ws = layer(wl, a8, inp, router_grad=True)
    tre.moe_layer_fwd(sh, b, ws)
    torch.cuda.synchronize()
    h = {n: to_f64(v) for n, v in inp.items() if n != "logits"}
    st = oracle.layer_fwd_mx4(inp["logits"].cpu().numpy(), h["x"], h["W1"], h["W3"], h["W2"], k, a8)
    assert np.array_equal(b["topk_idx"].cpu().numpy(), st["idx"])
    assert np.array_equal(b["row_of"].cpu().numpy(), st["row_of"])
    case = (inp["x"].cpu(), st["token_of"].astype(np.int32), None, None, None, st["offsets"])
    ref, tol = expected(case, b["wmx4"], a8)
    assert (np.abs(to_f64(b["o"]) - ref) <= tol).all()
    p = b["topk_prob"].cpu().numpy().astype(np.float64)
    o = to_f64(b["o"])
    y = oracle.combine(o, st["row_of"], p)
    bound = 2.0 ** -8 * np.abs(y) + k * 2.0 ** -23 * oracle.combine(np.abs(o), st["row_of"], p)
    assert (np.abs(to_f64(b["y"]) - y) <= bound).all()
    loss = oracle.aux_loss(inp["logits"].cpu().numpy().astype(np.float64), st["counts"], k, 0.01)[0]
    assert abs(float(b["aux_loss"].item()) - loss) <= 5e-5 * loss
    with pytest.raises(tre.MoeError):
        tre.moe_layer_bwd(sh, b, ws)


@pytest.mark.parametrize("a8", [False, True], ids=["a4", "a8"])
@pytest.mark.parametrize("T", [2, 400, 2500])
def test_layer_graph_replays_on_new_inputs(T, a8):
    """One captured graph, replayed on changed inputs with eager work between the
    replays, against eager calls; a second graph shares the workspace."""
    wl = Workload(f"mx4_graph_{T}", T=T, d=256, E=8, k=2, f=256)
    inp = make_inputs(wl, seed=2, device="cuda")
    tre, sh, b, ws = layer(wl, a8, inp)
    side = torch.cuda.Stream()
    tre.moe_layer_fwd(sh, b, ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            tre.moe_layer_fwd(sh, b, ws)
    for rep in range(4):
        new = make_inputs(wl, seed=10 + rep, device="cuda")
        for n in ("logits", "x"):
            b[n].copy_(new[n])
        b["y"].fill_(float("nan"))
        ws.fill_(0xFF)
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        got = b["y"].clone()
        tre.moe_layer_fwd(sh, b, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, b["y"])
        assert torch.isfinite(got).all()


def test_a_call_on_another_stream():
    """Calls go to the stream they are given: work queued there first is seen."""
    import token_routed_expert_amd as tre
    X = torch.zeros(512, 4096, device="cuda", dtype=torch.bfloat16)
    codes = torch.empty(512, 2048, dtype=torch.uint8, device="cuda")
    sb = torch.empty(512, 128, dtype=torch.uint8, device="cuda")
    src = torch.randn(512, 4096, device="cuda").bfloat16()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):
            X.copy_(src)
            X.mul_(1.0)
        tre.moe_quantize_rows_mx4(X, codes, sb, stream=s)
    s.synchronize()
    rq, rs = oracle.quant_mx4_rows(src.double().cpu().numpy())
    assert np.array_equal(u8(codes), rq) and np.array_equal(u8(sb), rs)


def test_python_refuses_short_and_misaligned_tensors():
    import token_routed_expert_amd as tre
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(8 * 32, dtype=torch.uint8, device="cuda"), torch.zeros(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="elements"):
        tre.moe_quantize_rows_mx4(x, q[:-1], s)
    with pytest.raises(ValueError, match="elements"):
        tre.moe_quantize_rows_mx4(x, q, s[:-1])
    with pytest.raises(ValueError, match="aligned"):
        tre.moe_quantize_rows_mx4(x.flatten()[4:4 + 7 * 64].view(7, 64), q, s)
    with pytest.raises(ValueError, match="device"):
        tre.moe_quantize_rows_mx4(x, q.cpu(), s)
    case = product_case([3], 128, 128, False, 1, False)
    o, w = run_product(case, False, 1, 1, 3, 128)
    sh = tre.make_shape(3, 128, 1, 1, 128, dtype="mxfp4")
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    xq, xs = torch.zeros(3, 64, dtype=torch.uint8, device="cuda"), torch.zeros(3, 4, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    tre.moe_grouped_gemm_fwd_mx4(sh, off, None, xq, xs, w, o, ws)
    for bad in (dict(xq=xq[:2]), dict(xs=xs[:2]), dict(o=o[:2]), dict(off=off[:1]), dict(off=off.long())):
        a = {**dict(off=off, xq=xq, xs=xs, o=o), **bad}
        with pytest.raises((ValueError, TypeError)):
            tre.moe_grouped_gemm_fwd_mx4(sh, a["off"], None, a["xq"], a["xs"], w, a["o"], ws)
    with pytest.raises(tre.MoeError):
        tre.moe_grouped_gemm_fwd_mx4(sh, off, None, xq, xs, w, o, None)
    for name in w.NAMES:
        short = tre.MX4Weights({**w.tensors, name: w[name].flatten()[:-16]})
        with pytest.raises(ValueError, match="elements"):
            tre.moe_grouped_gemm_fwd_mx4(sh, off, None, xq, xs, short, o, ws)
        host = tre.MX4Weights({**w.tensors, name: w[name].cpu()})
        with pytest.raises(ValueError, match="device"):
            tre.moe_grouped_gemm_fwd_mx4(sh, off, None, xq, xs, host, o, ws)
    torch.cuda.synchronize()
    assert not o.float().abs().max()          # zero rows give zeros
