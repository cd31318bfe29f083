"""Integer expert weights on the GPU against the oracle, through the C ABI: the
quantiser, the packing and the reading back bit-exact, the experts' product element
by element, the layer, streams, graphs.

Tolerance of the product, for one element of o = bf16(h) W2 (weights are exact bf16
numbers on both sides):
* an addition in the matrix unit is off by at most one unit in the last place,
  2^-23: a and b by g = (d + 16) 2^-23 sum |x w|; so an element of h may differ from
  the exact one by e = 1.1 |b| g_a + |silu(a)| g_b + 2^-20 |h| (|silu'| < 1.1; the
  last term covers the exponential and the reciprocal).  Where that carries h across
  a rounding border it moves: delta = max |bf16(h +- e) - bf16(h)|, and o by sum
  delta |W2|;
* the sum over f is off by (f + 16) 2^-23 sum |h W2|;
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
U8, I32, BF16, F32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu(request):
    need_gpu()
    announce(request.node.nodeid)
    yield
    torch.cuda.synchronize()


def tile_buffers(E, R, N, group, guard=0):
    codes = torch.full((E * N * R // 2 + guard,), 0xA5, dtype=U8, device="cuda")
    words = torch.full((E * N * R // group + guard,), -7, dtype=I32, device="cuda")
    return codes, words


def shaped(codes, words, E, R, N, group):
    return (codes[:E * N * R // 2].view(E, N // 16, R // 128, 4, 16, 16).cpu().numpy(),
            words[:E * N * R // group].view(E, N // 64, R // 128, 128 // group, 16, 4).cpu().numpy().view(np.uint32))


def edge_weights(E, R, C, rng):
    """Groups of every kind: zeros of both signs, one sign only, ties, borders of the scale, subnormals, the largest
    numbers, NaN and infinities."""
    W = rng.standard_normal((E, R, C)).astype(np.float32)
    W *= np.exp2(rng.integers(-30, 30, (E, 1, C))).astype(np.float32)
    n = min(R, 128)
    ties = np.resize(np.r_[7.0, np.arange(-13, 14) / 2], n)
    near = np.nextafter(np.resize(np.r_[7.0, np.arange(-13, 14) / 2], n).astype(np.float32), np.float32(9))
    special = [np.zeros(n), -np.zeros(n), np.abs(W[0, :n, 0]), -np.abs(W[0, :n, 1]), ties, ties * 2.0 ** -60,
               near, np.full(n, 1e-41), np.resize([3.4e38, -3.4e38, 1e38], n), np.full(n, 2.0 ** -126),
               np.r_[np.nan, np.ones(n - 1)], np.r_[np.ones(n - 1), np.inf], np.r_[np.ones(n - 1), -np.inf],
               np.resize([1.48e38, -1.48e38], n), np.resize([1.5e38, 0], n),
               np.full(n, 7 * (1 + 2.0 ** -20)), np.resize([15.0, 7.5, 0.0, 1.0], n), np.resize([1.0, 1e-30], n)]
    for i, col in enumerate(special):
        W[i % E, :n, (i * 7) % C] = col
    return W


def same_groups(codes, words, rc, rw):
    """Scale words equal, and the codes where the scale is a number."""
    assert np.array_equal(words, rw)
    bad = np.isnan((rw & np.uint32(0xfffffff0)).view(np.float32))              # [E][N/64][KT][U][16][4]
    E, NB, KT, U = bad.shape[:4]
    cols = bad.transpose(0, 1, 5, 2, 3, 4).reshape(E, NB * 4, KT, U, 16)       # [E][N/16][KT][U][c]
    cols = np.repeat(cols, 4 // U, axis=3)                                     # [..][j][c]
    mask = np.repeat(cols.transpose(0, 1, 2, 4, 3)[:, :, :, None], 4, axis=3)  # [..][g][c][j]
    mask = np.repeat(mask, 4, axis=5)
    assert np.array_equal(codes[~mask], rc[~mask])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("E,R,C", [(1, 128, 128), (2, 384, 256), (3, 128, 384)])
def test_quantize_bit_exact_and_back(E, R, C, pair, dtype, asym, group):
    import token_routed_expert_amd as tre
    rng = np.random.default_rng(E + R + group)
    W = [torch.from_numpy(edge_weights(E, R, C, rng)).to(dtype) for _ in range(2 if pair else 1)]
    N = C * len(W)
    codes, words = tile_buffers(E, R, N, group, 16)
    tre.moe_quantize_weights_i4(W[0].cuda(), W[1].cuda() if pair else None, group, asym, codes, words)
    q = [oracle.quant_i4(w.double().numpy(), group, asym) for w in W]
    got = shaped(codes, words, E, R, N, group)
    same_groups(*got, *oracle.i4_tiles(*q[0], q[1] if pair else None))
    assert (codes[-16:] == 0xA5).all() and (words[-16:] == -7).all()
    out = [torch.full((E * R * C + 16,), 5.0, dtype=BF16, device="cuda") for _ in W]
    tre.moe_dequantize_weights_i4(codes, words, group, out[0][:-16].view(E, R, C),
                                  out[1][:-16].view(E, R, C) if pair else None)
    for o, (c, s, z) in zip(out, q):
        assert (o[-16:] == 5.0).all()
        want = torch.from_numpy(oracle.dequant_i4(c, s, z)).to(BF16)
        assert torch.equal(torch.nan_to_num(o[:-16].view(E, R, C).cpu(), nan=1e30), torch.nan_to_num(want, nan=1e30))


def test_quantize_random_against_the_oracle():
    """Many values, with quotients next to halves: every code."""
    import token_routed_expert_amd as tre
    g = torch.Generator().manual_seed(0)
    W = torch.randn(2, 1024, 512, generator=g)
    W[1] = (torch.randint(-27, 28, (1024, 512), generator=g) / 2) * (1 + 2.0 ** -23 * torch.randint(-2, 3, (1024, 512), generator=g))
    for asym in (False, True):
        codes, words = tile_buffers(2, 1024, 512, 64)
        tre.moe_quantize_weights_i4(W.cuda(), None, 64, asym, codes, words)
        same_groups(*shaped(codes, words, 2, 1024, 512, 64), *oracle.i4_tiles(*oracle.quant_i4(W.double().numpy(), 64, asym)))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("E,R,C", [(1, 128, 128), (2, 256, 384)])
def test_pack(E, R, C, pair, zeros, group):
    import token_routed_expert_amd as tre
    rng = np.random.default_rng(group + E)
    srcs = []
    for i in range(2 if pair else 1):
        q = rng.integers(0, 16, (E, R, C)).astype(np.uint8)
        s = (rng.standard_normal((E, R // group, C)) * 2.0 ** rng.integers(-12, 12, (E, R // group, C))).astype(
            np.float16 if i else np.float32).astype(np.float32)
        s[0, 0, :6] = [np.nan, np.inf, 2.0 ** 124, 0.0, 1 + 2.0 ** -20, 1 + 3 * 2.0 ** -20]   # two ties
        srcs.append((q, s, rng.integers(0, 16, (E, R // group, C)).astype(np.uint8) if zeros else None))
    N = C * len(srcs)
    codes, words = tile_buffers(E, R, N, group, 16)
    dev = [tuple(None if t is None else torch.from_numpy(t).cuda() for t in x) for x in srcs]
    tre.moe_pack_weights_i4(*dev[0], dev[1] if pair else None, group, codes, words)
    ref = []
    for q, s, z in srcs:
        m, e = np.frexp(s.astype(np.float64))
        with np.errstate(invalid="ignore", over="ignore"):
            r = np.ldexp(np.rint(np.ldexp(m, 20)), e - 20).astype(np.float32).astype(np.float64)   # to 20 bits, ties to even
        ref.append((q, np.where(np.abs(r) < 2.0 ** 124, r, np.nan), np.full(s.shape, 8, np.uint8) if z is None else z))
    got = shaped(codes, words, E, R, N, group)
    want = oracle.i4_tiles(*ref[0], ref[1] if pair else None)
    assert np.array_equal(got[0], want[0])
    nan = np.isnan((want[1] & np.uint32(0xfffffff0)).view(np.float32))
    assert np.array_equal(got[1][~nan], want[1][~nan])
    assert np.isnan((got[1][nan] & np.uint32(0xfffffff0)).view(np.float32)).all()
    assert (codes[-16:] == 0xA5).all() and (words[-16:] == -7).all()
    # fp16 scales are kept exactly
    if pair:
        s16 = srcs[1][1]
        fin = np.isfinite(s16) & (np.abs(s16) < 65504) & (np.abs(s16) != 1 + 2.0 ** -20) & (np.abs(s16) != 1 + 3 * 2.0 ** -20)
        assert np.array_equal(ref[1][1][fin], s16[fin].astype(np.float64))


def test_every_code_and_zero_point():
    """All 16 codes with all 16 zero points and scales of 20 bits, read back exactly."""
    import token_routed_expert_amd as tre
    rng = np.random.default_rng(8)
    R, C = 256, 256
    q = np.tile(np.arange(16, dtype=np.uint8), R * C // 16).reshape(1, R, C)
    q = rng.permuted(q, axis=1)
    z = np.resize(np.arange(16, dtype=np.uint8), (1, R // 32, C))
    s = ((rng.integers(2 ** 19, 2 ** 20, (1, R // 32, C)) * 2.0 ** -30) * np.exp2(rng.integers(-60, 60, (1, R // 32, C)))).astype(np.float32)
    codes, words = tile_buffers(1, R, C, 32)
    tre.moe_pack_weights_i4(*(torch.from_numpy(t).cuda() for t in (q, s, z)), None, 32, codes, words)
    out = torch.empty(1, R, C, dtype=BF16, device="cuda")
    tre.moe_dequantize_weights_i4(codes, words, 32, out)
    assert np.array_equal(to_f64(out), oracle.dequant_i4(q, s, z))


# ---------------------------------------------------------------------------------------------------- products
def product_case(counts, d, f, group, asym, seed, gather, T=None):
    """Rows with outliers, weights through the quantiser, offsets of the given rows per expert."""
    from token_routed_expert_amd.buffers import quantized_weights_i4
    rng = np.random.default_rng(seed)
    P, E = sum(counts), len(counts)
    rows = max(1, (T or max(1, P)) if gather else P)
    X = rng.standard_normal((rows, d)) * np.where(rng.random((rows, d)) < 0.01, 20, 1)
    tok = rng.integers(0, rows, T or P).astype(np.int32) if gather else None
    W = [torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[1])).astype(np.float32)).cuda()
         for s in ((E, d, f), (E, d, f), (E, f, d))]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return torch.from_numpy(X).to(BF16), tok, quantized_weights_i4(*W, group, asym), off


def run_product(case, E, k, T, d, f):
    import token_routed_expert_amd as tre
    X, tok, w, off = case
    sh = tre.make_shape(T, d, E, k, f, dtype="int4")
    o = torch.full((T * k, d), 7.0, dtype=BF16, device="cuda")
    ws = torch.full((tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD),), 0xFF, dtype=U8, device="cuda")
    tre.moe_grouped_gemm_fwd_i4(sh, torch.from_numpy(off).cuda(), None if tok is None else torch.from_numpy(tok).cuda(),
                                X.cuda(), w, o, ws)
    torch.cuda.synchronize()
    return o


def weights_of(w, E, d, f):
    import token_routed_expert_amd as tre
    W1, W3 = (torch.empty(E, d, f, dtype=BF16, device="cuda") for _ in range(2))
    W2 = torch.empty(E, f, d, dtype=BF16, device="cuda")
    tre.moe_dequantize_weights_i4(w["W13"], w["W13s"], w.group, W1, W3)
    tre.moe_dequantize_weights_i4(w["W2"], w["W2s"], w.group, W2)
    return W1, W3, W2


def expected(case, E, d, f):
    X, tok, w, off = case
    x = X.double().numpy()
    x = x if tok is None else x[tok]
    W1, W3, W2 = (to_f64(t) for t in weights_of(w, E, d, f))
    o, h, a, b = oracle.experts_fwd_i4(x, off, W1, W3, W2)
    tol = 2.0 ** -8 * np.abs(o)
    u = 2.0 ** -23
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if r.stop == r.start:
            continue
        ga, gb = ((d + 16) * u * (np.abs(x[r]) @ np.abs(W[e])) for W in (W1, W3))
        err = 1.1 * np.abs(b[r]) * ga + np.abs(silu(a[r])) * gb + 2.0 ** -20 * np.abs(h[r])
        base = oracle.bf16_round(h[r])
        delta = np.maximum(*(np.abs(oracle.bf16_round(h[r] + s * err) - base) for s in (-1, 1)))
        tol[r] += delta @ np.abs(W2[e]) + (f + 16) * u * ((np.abs(base) + delta) @ np.abs(W2[e]))
    return o, tol


def check(case, E, k, T, d, f):
    o = run_product(case, E, k, T, d, f)
    ref, tol = expected(case, E, d, f)
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
    "few_edges": [16, 17, 0, 31, 32, 33, 48, 64, 65] + [0] * 30,
    "few_hot": [0] * 40 + [300, 1],
}
WIDTHS = {"edges64": (384, 256), "edges128": (128, 640), "hot": (640, 128), "tail": (256, 384), "edges256": (512, 256)}


def few(P, E, d, f):
    import token_routed_expert_amd as tre
    return tre.moe_few_rows(tre.make_shape(P, d, E, 1, f, dtype="int4"))


def with_many(counts, d, f):
    """An expert more, with enough rows for the kernel for many rows."""
    n = 65
    while few(sum(counts) + n, len(counts) + 1, d, f):
        n += 64
    return counts + [n]


@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
@pytest.mark.parametrize("group,asym", [(32, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("name", COUNTS)
def test_product(name, gather, group, asym, many):
    counts = COUNTS[name]
    d, f = WIDTHS.get(name, (256, 128))
    if many:
        counts = with_many(counts, d, f)
    P = sum(counts)
    case = product_case(counts, d, f, group, asym, 3 + P, gather)
    check(case, len(counts), 1, P, d, f)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("d,f", [(128, 128), (128, 1152), (1152, 128), (896, 384)])
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_product_widths(d, f, group, many):
    counts = with_many([40, 0, 1, 90], d, f) if many else [40, 0, 1, 90]
    case = product_case(counts, d, f, group, True, d + f, True)
    check(case, len(counts), 1, sum(counts), d, f)


# (counts, d, f) whose two products take blocks of 32 columns with eight wavefronts, with four, and of 64 columns
FORMS = {"eight": ([16, 3, 17], 128, 128), "four": ([7, 16, 0, 17, 32, 33, 1] * 4, 256, 384),
         "wide": ([7, 16, 0, 17, 32, 33, 1] * 20, 1152, 1152)}


def blocks(counts, d, f):
    """Blocks of 64 columns that the two products of a call with few rows have at most."""
    P, E = sum(counts), len(counts)
    return [n // 64 * (P // 32 + min(P, E)) for n in (2 * f, d)]


@pytest.mark.parametrize("group,asym", [(32, False), (64, True), (128, True)])
@pytest.mark.parametrize("form", FORMS)
def test_product_every_form_of_the_rows_kernel(form, group, asym):
    counts, d, f = FORMS[form]
    case = product_case(counts, d, f, group, asym, 7, True)
    check(case, len(counts), 1, sum(counts), d, f)


# (counts, d, f) with too few tiles for the chip, and the parts of K of the two products
PARTS = {"four_one": ([700, 0, 590], 4096, 512, 4, 1), "one_four": ([1, 1299], 256, 4096, 1, 4),
         "three_one": ([400, 33, 857], 3200, 896, 3, 1), "one_three": ([128, 1162, 0], 896, 2304, 1, 3),
         "two_four": ([390, 0], 3200, 4096, 2, 4), "one_two": ([0, 1300], 1536, 2304, 1, 2)}


@pytest.mark.parametrize("group,asym", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("name", PARTS)
def test_product_in_parts_of_k(name, group, asym):
    counts, d, f = PARTS[name][:3]
    case = product_case(counts, d, f, group, asym, 5, group != 64)
    check(case, len(counts), 1, sum(counts), d, f)


def test_parts_of_k_leave_the_other_rows():
    """Rows behind the last expert; a NaN in one row; the same bits again, and from a replayed graph on other inputs."""
    import token_routed_expert_amd as tre
    counts, d, f = PARTS["two_four"][:3]
    T = sum(counts)
    short = product_case([200, 60], d, f, 64, True, 8, True, T=T)
    check(short, 2, 1, T, d, f)
    case = product_case(counts, d, f, 32, True, 6, False)
    o = run_product(case, 2, 1, T, d, f)
    xs = [case[0].clone().cuda(), case[0].clone().cuda()]
    xs[1][7, 40] = float("nan")
    bad = run_product((xs[1].cpu(),) + case[1:], 2, 1, T, d, f)
    keep = torch.arange(T) != 7
    assert torch.equal(bad.cpu()[keep], o.cpu()[keep]) and torch.isnan(bad[7]).all()
    sh = tre.make_shape(T, d, 2, 1, f, dtype="int4")
    x, out, off = xs[0].clone(), torch.empty_like(o), torch.from_numpy(case[3]).cuda()
    ws = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=U8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tre.moe_grouped_gemm_fwd_i4(sh, off, None, x, case[2], out, ws)
    for i in (0, 1, 0, 1):
        x.copy_(xs[i])
        out.fill_(7.0)
        ws.fill_(0xEE)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), (o, bad)[i].view(torch.int16))
    del graph


def test_rows_past_the_last_expert_stay():
    """offsets[E] below P (assignments that the map skipped)."""
    case = product_case([20, 0, 300], 256, 256, 64, True, 9, True, T=400)
    check(case, 3, 1, 400, 256, 256)
    counts = with_many([20, 0], 256, 256)
    case = product_case(counts, 256, 256, 64, True, 9, True, T=sum(counts) + 90)
    check(case, 3, 1, sum(counts) + 90, 256, 256)
    empty = product_case([0, 0], 256, 256, 64, True, 9, False, T=4)
    case = (torch.ones(8, 256).bfloat16(), None) + empty[2:]
    check(case, 2, 2, 4, 256, 256)


@pytest.mark.parametrize("per_expert", [8, 100, 400])
@pytest.mark.parametrize("group", [32, 128])
def test_repeated_calls_give_the_same_bits(group, per_expert):
    """Many tiles with few K steps, over and over: a load that is read before it has landed (its slot then holds what an
    earlier call left) shows as another result."""
    import token_routed_expert_amd as tre
    E, k, d, f = 96, 8, 384, 1152
    T = E * per_expert // k
    g = torch.Generator(device="cuda").manual_seed(5)
    sh = tre.make_shape(T, d, E, k, f, dtype="int4")

    def codes(n):
        return torch.randint(0, 256, (n,), generator=g, dtype=U8, device="cuda")

    def words(n):   # scales around 2^-6, each its own, with every zero point
        return torch.randint(121 << 23, 122 << 23, (n,), generator=g, dtype=I32, device="cuda")
    w = tre.I4Weights({"W13": codes(E * d * f), "W2": codes(E * d * f // 2), "W13s": words(2 * E * d * f // group),
                       "W2s": words(E * d * f // group)}, group)
    off = torch.arange(0, E + 1, dtype=I32, device="cuda") * per_expert
    ws = torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=U8, device="cuda")
    tok = torch.randint(0, T, (T * k,), generator=g, device="cuda", dtype=I32)
    x = [torch.randn(T, d, generator=g, device="cuda").to(BF16) for _ in range(2)]
    o = torch.empty(T * k, d, dtype=BF16, device="cuda")
    first = [None, None]
    for i in range(400):
        tre.moe_grouped_gemm_fwd_i4(sh, off, tok, x[i & 1], w, o, ws)
        if i < 2:
            first[i] = o.clone()
            assert torch.isfinite(o).all()
        else:
            assert torch.equal(o, first[i & 1]), f"call {i}"


@pytest.mark.parametrize("rows", [21, 300, 3700])
def test_a_token_that_there_is_not_reads_zeros(rows):
    """Entries of token_of outside [0, T): rows of zeros, their neighbours untouched; with a NaN group in the weights
    such a row is NaN where the others are (0 times a NaN)."""
    from token_routed_expert_amd.buffers import quantized_weights_i4
    counts = [rows] if rows > 32 else [rows, 0, 0, 2]
    E, T, d, f = len(counts), sum(counts), 384, 256
    case = product_case(counts, d, f, 64, True, rows, True)
    o = run_product(case, E, 1, T, d, f)
    tok = case[1].copy()
    bad = {0: -1, 3: T, rows // 2: 2 ** 31 - 1, rows - 1: -2 ** 31}
    for at, v in bad.items():
        tok[at] = v
    got, want = to_f64(run_product((case[0], tok) + case[2:], E, 1, T, d, f)), to_f64(o)
    want[list(bad)] = 0
    assert np.array_equal(got, want)
    g = torch.Generator(device="cuda").manual_seed(1)
    W = [torch.randn(*s, generator=g, device="cuda") / 16 for s in ((E, d, f), (E, d, f), (E, f, d))]
    W[2][0, 5, 9] = float("nan")
    o = run_product((case[0], tok, quantized_weights_i4(*W, 64, True), case[3]), E, 1, T, d, f)
    assert torch.isnan(o[:rows, 9]).all() and torch.isfinite(o[:rows, :9]).all() and torch.isfinite(o[:, 10:]).all()


@pytest.mark.parametrize("rows", [5, 300, 4200])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_nan_stays_in_its_row(bad, rows):
    case = product_case([rows], 256, 256, 128, False, 4, False)
    ref = run_product(case, 1, 1, rows, 256, 256)
    case[0][3, 70] = bad
    o = run_product(case, 1, 1, rows, 256, 256)
    keep = torch.arange(rows) != 3
    assert torch.equal(o.cpu()[keep], ref.cpu()[keep])
    assert torch.isnan(o[3]).all()      # (an infinity: some product of it and of h with both signs or a zero)


@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_same_as_the_bf16_layer_on_the_dequantised_weights(many):
    """The weights that moe_dequantize_weights_i4 writes are those of the product: the bf16 experts on them agree up to
    the order of the fp32 sums, so their backward belongs to this forward."""
    import token_routed_expert_amd as tre
    d, f = 384, 256
    counts = with_many([40, 0, 7], d, f) if many else [40, 0, 7]
    E, P = len(counts), sum(counts)
    case = product_case(counts, d, f, 64, True, 2, True)
    o = run_product(case, E, 1, P, d, f)
    W = weights_of(case[2], E, d, f)
    sh = tre.make_shape(P, d, E, 1, f, dtype="bf16")
    ab, h, ob = (torch.empty(P, n, dtype=BF16, device="cuda") for n in (2 * f, f, d))
    tre.moe_grouped_gemm_fwd_gather(sh, torch.from_numpy(case[3]).cuda(), torch.from_numpy(case[1]).cuda(), case[0].cuda(),
                                    *W, ab, h, ob)
    _, tol = expected(case, E, d, f)
    assert (np.abs(to_f64(o) - to_f64(ob)) <= 2 * tol).all()


# ------------------------------------------------------------------------------------------------------- layers
LAYERS = [Workload("i4_one", T=1, d=256, E=8, k=2, f=256), Workload("i4_small", T=37, d=384, E=16, k=4, f=256),
          Workload("i4_prompt", T=700, d=256, E=8, k=2, f=384, skew=False),
          Workload("i4_shared", T=130, d=256, E=8, k=2, f=256, f_shared=384)]


def layer(wl, seed=0, **kw):
    from token_routed_expert_amd.buffers import layer_buffers
    return layer_buffers(wl.T, wl.d, wl.E, wl.k, wl.f, wl.f_shared, "int4", "cuda", make_inputs(wl, seed=seed, device="cuda"),
                         **kw)


@pytest.mark.parametrize("group,asym", [(32, True), (128, False)])
@pytest.mark.parametrize("wl", LAYERS, ids=lambda w: w.name)
def test_layer(wl, group, asym):
    import token_routed_expert_amd as tre
    sh, b, wsf, _ = layer(wl, group=group, asymmetric=asym, router_grad=True)
    b.pop("dlogits")
    tre.moe_layer_fwd(sh, b, wsf)
    idx, p, counts = oracle.route(b["logits"].cpu().numpy(), wl.k)[0], None, None
    assert np.array_equal(b["topk_idx"].cpu().numpy(), idx)
    tok, off = b["token_of"].cpu().numpy(), b["offsets"].cpu().numpy()
    ref, tol = expected((b["x"].cpu(), tok, b["wi4"], off), wl.E, wl.d, wl.f)
    assert (np.abs(to_f64(b["o"]) - ref) <= tol).all()
    prob, row_of = to_f64(b["topk_prob"]), b["row_of"].cpu().numpy()
    terms = to_f64(b["o"])[row_of] * prob[..., None]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    if wl.f_shared:
        ys = to_f64(b["ys"])
        sh_ref = oracle.experts_fwd(to_f64(b["x"]), np.array([0, wl.T]), *(to_f64(b[n])[None] for n in ("Ws1", "Ws3", "Ws2")))[3]
        assert oracle.row_rel_err(ys, sh_ref) <= 2e-2
        want, size = want + ys, size + np.abs(ys)
    assert (np.abs(to_f64(b["y"]) - want) <= 2.0 ** -8 * np.abs(want) + 16 * 2.0 ** -24 * size).all()
    assert torch.isfinite(b["aux_loss"]).all()


def test_norm_into_layer():
    """Residual addition and norm, router logits, the layer on its bf16 rows: a block of a serving program, one token and
    many, against the same calls made one by one."""
    import token_routed_expert_amd as tre
    for wl in (LAYERS[0], LAYERS[2]):
        sh, b, wsf, _ = layer(wl, group=64)
        g = torch.Generator().manual_seed(7)
        stream, delta = (torch.randn(wl.T, wl.d, generator=g).to(BF16).cuda() for _ in range(2))
        gamma = (1 + 0.2 * torch.randn(wl.d, generator=g)).to(BF16).cuda()
        gate = torch.randn(wl.d, wl.E, generator=g).cuda()
        y, sum_ = torch.empty_like(stream), torch.empty_like(stream)
        tre.moe_add_rms_norm(delta, stream, gamma, 1e-6, sum_, y, None)
        b["x"], b["logits"] = y, y.float() @ gate
        tre.moe_layer_fwd(sh, b, wsf)
        want, _ = oracle.rms_norm(to_f64(sum_), to_f64(gamma), 1e-6)
        assert (np.abs(to_f64(y) - want) <= (2.0 ** -8 + 1e-4) * np.abs(want)).all()
        tok, off = b["token_of"].cpu().numpy(), b["offsets"].cpu().numpy()
        ref, tol = expected((y.cpu(), tok, b["wi4"], off), wl.E, wl.d, wl.f)
        assert (np.abs(to_f64(b["o"]) - ref) <= tol).all()


def test_layer_graph_replay():
    """A captured layer, replayed on other inputs with the outputs overwritten between: the eager bits every time."""
    import token_routed_expert_amd as tre
    wl = LAYERS[3]
    sh, b, wsf, _ = layer(wl, group=32, asymmetric=True)
    xs = [b["x"].clone(), torch.randn_like(b["x"])]
    eager = []
    for x in xs:
        b["x"].copy_(x)
        tre.moe_layer_fwd(sh, b, wsf)
        eager.append((b["y"].clone(), b["o"].clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        tre.moe_layer_fwd(sh, b, wsf)
    for i in (0, 1, 0, 1):
        b["x"].copy_(xs[i])
        for n in ("y", "o", "ys"):
            b[n].fill_(float("nan"))
        wsf.fill_(0xEE)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["y"], eager[i][0]) and torch.equal(b["o"], eager[i][1])
    del graph


def test_two_streams():
    """Two calls at once on two streams, each with its own workspace and outputs."""
    import token_routed_expert_amd as tre
    cases = [product_case(c, 256, 256, 64, True, i, True) for i, c in enumerate(([200, 3, 700], [1, 0, 2]))]
    alone = [run_product(c, 3, 1, int(c[-1][-1]), 256, 256) for c in cases]
    args = []
    for X, tok, w, off in cases:
        P = int(off[-1])
        sh = tre.make_shape(P, 256, 3, 1, 256, dtype="int4")
        args.append((sh, torch.from_numpy(off).cuda(), torch.from_numpy(tok).cuda(), X.cuda(), w,
                     torch.zeros(P, 256, dtype=BF16, device="cuda"),
                     torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=U8, device="cuda")))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for a, s in zip(args, streams):
            tre.moe_grouped_gemm_fwd_i4(*a, stream=s)
    torch.cuda.synchronize()
    for a, ref in zip(args, alone):
        assert torch.equal(a[5], ref)


def test_python_calls_check_their_tensors():
    import token_routed_expert_amd as tre
    E, d, f, T = 2, 128, 256, 6
    case = product_case([4, 2], d, f, 64, False, 1, True)
    X, tok, w, off = case
    sh = tre.make_shape(T, d, E, 1, f, dtype="int4")
    good = dict(sh=sh, offsets=torch.from_numpy(off).cuda(), token_of=torch.from_numpy(tok).cuda(), x=X.cuda(), w=w,
                o=torch.empty(T, d, dtype=BF16, device="cuda"),
                ws=torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=U8, device="cuda"))
    tre.moe_grouped_gemm_fwd_i4(**good)
    short = tre.I4Weights({n: (w[n].flatten()[:-1].contiguous() if n == "W2s" else w[n]) for n in w.NAMES}, 64)
    as32 = tre.I4Weights({n: w[n] for n in w.NAMES}, 32)
    for bad, text in ((dict(offsets=good["offsets"][:2]), "offsets has"), (dict(token_of=good["token_of"][:5]), "token_of has"),
                      (dict(x=good["x"][:5]), "x has"), (dict(x=good["x"].float()), "x: expected"),
                      (dict(o=good["o"][:5]), "o has"), (dict(o=good["o"].float()), "o: expected"), (dict(w=short), "are needed"),
                      (dict(w=as32), "are needed"), (dict(ws=good["ws"][:-1]), "WORKSPACE"), (dict(ws=None), "WORKSPACE"),
                      (dict(x=good["x"].cpu()), "device")):
        with pytest.raises((TypeError, ValueError, tre.MoeError), match=text):
            tre.moe_grouped_gemm_fwd_i4(**{**good, **bad})
    with pytest.raises(ValueError, match="32, 64 or 128"):
        tre.I4Weights(w.tensors, 48)
    with pytest.raises(TypeError):
        tre.I4Weights({**w.tensors, "W2s": w["W2s"].float()}, 64)
    W = torch.zeros(1, 128, 128, device="cuda")
    codes, words = tile_buffers(1, 128, 128, 32)
    q, s = W.to(U8), torch.ones(1, 4, 128, device="cuda")
    for call, text in ((lambda: tre.moe_quantize_weights_i4(W, None, 32, False, codes[:-1], words), "codes has"),
                       (lambda: tre.moe_quantize_weights_i4(W, None, 32, False, codes, words[:-1]), "scales has"),
                       (lambda: tre.moe_quantize_weights_i4(W, W, 32, False, codes, words), "codes has"),
                       (lambda: tre.moe_quantize_weights_i4(W, W[:, :64], 32, False, codes, words), "shape"),
                       (lambda: tre.moe_quantize_weights_i4(W.half(), None, 32, False, codes, words), "bfloat16 or float32"),
                       (lambda: tre.moe_quantize_weights_i4(W, None, 16, False, codes, words), "32, 64 or 128"),
                       (lambda: tre.moe_pack_weights_i4(q, s[:, :3], None, None, 32, codes, words), "s has"),
                       (lambda: tre.moe_pack_weights_i4(q, s, q[0], None, 32, codes, words[:-1]), "scales has"),
                       (lambda: tre.moe_pack_weights_i4(q, s, s, None, 32, codes, words), "z: expected"),
                       (lambda: tre.moe_pack_weights_i4(q, s, None, (q[:, :64], s, None), 32, codes, words), "q "),
                       (lambda: tre.moe_dequantize_weights_i4(codes, words[:-1], 32, W.to(BF16)), "scales has"),
                       (lambda: tre.moe_dequantize_weights_i4(codes, words, 32, W), "W: expected")):
        with pytest.raises((TypeError, ValueError), match=text):
            call()
