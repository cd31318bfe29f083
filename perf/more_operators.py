"""Operators around the routed experts: what is measured, on which inputs, and their plain forms.

* ``norm``: the root-mean-square norm in front of a layer, with the residual's addition, and the rows that the layer
  reads quantised on the way (E4M3 blocks of 128 or MXFP8 blocks of 32); the values that the codes stand for are read
  back.
* ``norm_bwd``: its gradients: of x (and of the residual, the same tensor) and of the gains.
* ``weights``: 4-bit integer quantisation of expert weights with a scale and a zero point for each group of rows, and
  the bf16 values that the codes stand for.
* ``experts``: the experts' forward on such weights and bf16 activations, as a serving program runs it on the rows of
  one layer, from one token on.

Integer weights: ``group`` consecutive rows of a column (along the contraction) share a scale s and a zero point z; the
weight of code q (0 .. 15) is s (q - z), rounded to bf16.  s is the smallest number of 20 significant bits (at least
2^-126; 1 for a group of zeros) with max|w| <= 7 s and z = 8 (symmetric), or hi - lo <= 15 s with lo = min(w, 0),
hi = max(w, 0) and z = round(-lo / s) (asymmetric); q = round(w / s) + z, held to 0 .. 15; ties to even.
E4M3 blocks: scale = amax / 448 (1 for zeros), codes E4M3(v / scale).  MXFP8 blocks: scale 2^s with s the smallest integer such that
amax <= 448 * 2^s (0 for zeros, at least -126), codes E4M3(v * 2^-s).
"""
import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------------------- cases
def _norm(name, T, d, src, fmt, res, y):
    return {"name": name, "kind": "norm", "T": T, "d": d, "src": src, "fmt": fmt, "res": res, "y": y}


def _bwd(name, T, d, src, res):
    return {"name": name, "kind": "norm_bwd", "T": T, "d": d, "src": src, "res": res}


def _weights(name, E, R, C, pair, src, group, asym):
    return {"name": name, "kind": "weights", "E": E, "R": R, "C": C, "pair": pair, "src": src, "group": group, "asym": asym}


def _experts(name, T, d, E, k, f, group, asym, skew=False):
    return {"name": name, "kind": "experts", "T": T, "d": d, "E": E, "k": k, "f": f, "group": group, "asym": asym,
            "skew": skew}


def listed():
    return [
        # one token of one request in front of a layer with MXFP8 rows: latency alone
        _norm("norm decode 1 mxfp8", 1, 4096, "bf16", "mxfp8", True, True),
        # a decode step of a large batch in front of a layer of e4m3 blocks
        _norm("norm decode 177 e4m3", 177, 7168, "bf16", "e4m3", True, False),
        # fp32 residual stream of a training step, T off any grid
        _norm("norm train 8200 f32", 8200, 4096, "f32", "e4m3", True, True),
        # the largest batch
        _norm("norm 16384 mxfp8", 16384, 7168, "bf16", "mxfp8", True, True),
        # the backward of a small model's norm, no gradient on the residual stream
        _bwd("norm bwd 257 f32", 257, 512, "f32", False),
        # the backward of the largest batch, joined with the residual stream's gradient
        _bwd("norm bwd 16384", 16384, 7168, "bf16", True),
        # W1 and W3 of a large layer from the fp32 masters
        _weights("weights pair f32", 64, 4096, 1536, True, "f32", 128, False),
        # a small model's W2 from a bf16 checkpoint, fine groups
        _weights("weights small bf16", 8, 384, 512, False, "bf16", 32, True),
        # one token of one request: eight experts' weights are read for one row each
        _experts("experts decode 1", 1, 4096, 128, 8, 1536, 128, False),
        # a decode step of a large batch: every expert active, about eleven rows each
        _experts("experts decode 177", 177, 4096, 128, 8, 1536, 64, True),
        # an ordinary prompt of odd length through few wide experts
        _experts("experts prompt 1037", 1037, 4096, 8, 2, 14336, 32, True),
        # the largest prefill batch off the tile grid, with hot, cold and empty experts
        _experts("experts prompt 8200 skewed", 8200, 4096, 128, 8, 1536, 128, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["norm", "norm", "norm_bwd", "weights", "experts", "experts", "experts"])
    if kind in ("norm", "norm_bwd"):
        d, src = 128 * _log(rng, 1, 64), rng.choice(["bf16", "bf16", "f32"])
        T = max(1, min(_log(rng, 1, 16384), int(1.1e8 // d) // (2 if src == "f32" else 1)))
        case = {"kind": kind, "T": T, "d": d, "src": src, "res": rng.random() < 0.7}
        return case if kind == "norm_bwd" else {**case, "fmt": rng.choice(["e4m3", "mxfp8"]), "y": rng.random() < 0.6}
    E = rng.choice([4, 8, 16, 24, 32, 64, 96, 128])
    k = rng.randint(1, min(8, E))
    d, f = 128 * _log(rng, 2, 32), 128 * _log(rng, 1, 40)
    group, asym = rng.choice([32, 64, 128]), rng.random() < 0.5
    if kind == "weights":
        E = min(E, max(1, int(4e8 // (d * f))))
        return {"kind": kind, "E": E, "R": d, "C": f, "pair": rng.random() < 0.5, "src": rng.choice(["f32", "bf16"]),
                "group": group, "asym": asym}
    E = min(E, max(k, int(8e8 // (d * f))))
    T = max(1, min(_log(rng, 1, 8192), int(4.1e11 // (k * d * f))))
    skew = T * k >= 8 * E and E >= 16 and rng.random() < 0.4
    return {"kind": kind, "T": T, "d": d, "E": E, "k": min(k, E - E // 12) if skew else k, "f": f, "group": group,
            "asym": asym, "skew": skew}


# ------------------------------------------------------------------------------------------- pieces of the plain forms
def _pow2(e):
    """2^e exactly (e in [-126, 127]), from the bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _e4m3(v):
    """v (fp32, magnitude at most 448) rounded to E4M3's nearest value, ties to even."""
    _, e = torch.frexp(v)
    e = torch.clamp(e - 1, min=-6) - 3
    return torch.round(v * _pow2(-e)) * _pow2(e)


def _rows_read_back(v, fmt):
    """v [T][d] with every block of a row replaced by the values that its 8-bit codes stand for."""
    b = v.unflatten(1, (-1, 128 if fmt == "e4m3" else 32))
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "e4m3":
        scale = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
        return (_e4m3(torch.clamp(b / scale, -448, 448)) * scale).flatten(1)
    n, g = torch.frexp(amax)                                             # amax = n 2^g, 448 = 0.875 * 2^9
    s = g - 9 + (n > 0.875).to(torch.int32)
    s = torch.where(amax == 0, torch.zeros_like(s), torch.clamp(s, min=-126))
    return (_e4m3(b * _pow2(-s)) * _pow2(s)).flatten(1)


def _i4_groups(W, group, asym):
    """Codes, scales (fp32) and zero points of W [E][R][C]: [E][R/group][group][C], [E][R/group][1][C] (twice).  Scales
    and quotients in 64 bits: in 32 a quotient next to a half would round to it."""
    w = W.unflatten(1, (-1, group)).double()
    if asym:
        lo, hi = torch.clamp(w.amin(2, keepdim=True), max=0), torch.clamp(w.amax(2, keepdim=True), min=0)
        span, n = hi - lo, 15
    else:
        span, n = w.abs().amax(2, keepdim=True), 7
    bits = torch.clamp((span / n).float().view(torch.int32) & ~15, min=0x00800000)
    bits = torch.where(bits.view(torch.float32).double() * n < span, bits + 16, bits)
    s = torch.where(span == 0, torch.ones_like(span, dtype=torch.float32), bits.view(torch.float32))
    z = torch.clamp(torch.round(-lo / s.double()), 0, 15) if asym else torch.full_like(span, 8)
    q = torch.clamp(torch.round(w / s.double()) + z, 0, 15)
    return q.to(torch.uint8), s, z.to(torch.int32)


def _i4_tiles(W, pair, group, asym):
    """The stored form: codes [E][N/16][K/128][4][16][16] (k group g, column, byte 4 j + b: rows 32 j + 8 g + b in the
    low and + 4 in the high nibble of a tile's 128) and scale words [E][N/64][K/128][128/group][16][4] (column & 15, column
    / 16 & 3: the fp32 scale, whose low four bits are the zero point).  `pair`: a second matrix whose 16-column groups alternate with W's."""
    if pair is not None:
        W = torch.stack([W.unflatten(2, (-1, 16)), pair.unflatten(2, (-1, 16))], 3).flatten(2)
    E, K, N = W.shape
    q, s, z = _i4_groups(W, group, asym)
    n = q.view(E, K // 128, 4, 4, 2, 4, N // 16, 16)                     # kt, j, g, half, b, nt, c
    codes = (n[:, :, :, :, 0] | (n[:, :, :, :, 1] << 4)).permute(0, 5, 1, 3, 6, 2, 4).reshape(E, N // 16, K // 128, 4, 16, 16)
    words = (s.view(torch.int32) | z).view(E, K // 128, 128 // group, N // 64, 4, 16).permute(0, 3, 1, 2, 5, 4)
    return codes.contiguous(), words.contiguous()


def _i4_values(codes, words):
    """The weights [E][K][N] that tiles stand for, as fp32 (each a bf16 value)."""
    E, NT, KT = codes.shape[:3]
    U = words.shape[3]
    c = codes.view(E, NT, KT, 4, 16, 4, 4)                               # nt, kt, g, c, j, b
    q = torch.stack([c & 15, c >> 4], 6).permute(0, 2, 5, 3, 6, 7, 1, 4)   # kt, j, g, half, b, nt, c
    q = q.reshape(E, KT * U, 128 // U, NT * 16).float()
    w = words.permute(0, 2, 3, 1, 5, 4).reshape(E, KT * U, 1, NT * 16)
    v = (w & ~15).view(torch.float32) * (q - (w & 15).float())
    return v.to(torch.bfloat16).float().reshape(E, KT * 128, NT * 16)


# ------------------------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)


def _routing(case, g):
    """A routed batch: offsets [E+1], the source token of every permuted row, and where each row sits in a padded
    [active experts][most rows] layout."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device=DEV)
    if case["skew"]:
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        logits += torch.where(rank > E - E // 12, torch.full_like(rank, -64.0), 3.0 * rank ** -1.2)
    expert, order = torch.sort(torch.topk(logits, k, dim=1)[1].flatten(), stable=True)
    counts = torch.bincount(expert, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    active = torch.nonzero(counts).flatten()
    rank = torch.zeros(E, dtype=torch.int64, device=DEV)
    rank[active] = torch.arange(len(active), device=DEV)
    cap = int(counts.max())
    slot = rank[expert] * cap + torch.arange(T * k, device=DEV) - offsets[expert]
    return {"offsets": offsets.to(torch.int32), "token_of": (order // k).to(torch.int32), "active": active, "cap": cap,
            "slot": slot}


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    kind = case["kind"]
    if kind in ("norm", "norm_bwd"):
        T, d, dt = case["T"], case["d"], DTYPES[case["src"]]
        # a residual stream: rows of different size, a few large channels
        size = torch.exp(0.5 * _randn(g, T, 1))
        chan = torch.where(torch.rand(d, generator=g, device=DEV) < 0.004, 30.0, 1.0)
        stream = _randn(g, T, d).mul_(size).mul_(chan)
        s["gamma"] = (1 + _randn(g, d, std=0.2)).to(dt)
        if kind == "norm":
            s["x"] = _randn(g, T, d, dtype=dt)
            s["res"] = stream.to(dt) if case["res"] else None
            if s["res"] is None:
                s["x"] = stream.to(dt)
            return s
        s["sum"] = stream.to(dt)
        s["rstd"] = torch.rsqrt(s["sum"].double().square().mean(1) + EPS).float()
        s["dy"] = _randn(g, T, d, dtype=dt)
        s["dsum"] = _randn(g, T, d, dtype=dt) if case["res"] else None
        return s
    if kind == "weights":
        dt, (E, R, C) = DTYPES[case["src"]], (case["E"], case["R"], case["C"])
        s["W"] = _randn(g, E, R, C, std=R ** -0.5, dtype=dt)
        s["pair"] = _randn(g, E, R, C, std=R ** -0.5, dtype=dt) if case["pair"] else None
        return s
    T, d, E, f, group, asym = (case[n] for n in ("T", "d", "E", "f", "group", "asym"))
    s.update(_routing(case, g))
    s["x"] = _randn(g, T, d, dtype=torch.bfloat16)
    parts = []
    for e in range(0, E, 8):
        n = min(8, E - e)
        W1, W3 = _randn(g, n, d, f, std=d ** -0.5), _randn(g, n, d, f, std=d ** -0.5)
        parts.append(_i4_tiles(W1, W3, group, asym) + _i4_tiles(_randn(g, n, f, d, std=f ** -0.5), None, group, asym))
    s["W13"], s["W13s"], s["W2"], s["W2s"] = (torch.cat(p) for p in zip(*parts))
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _plain_norm(s):
    case, x = s["case"], s["x"]
    out = {}
    if s["res"] is not None:
        x = out["sum"] = (x.float() + s["res"].float()).to(x.dtype)
    v = x.float()
    rstd = 1 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
    y = v * rstd * s["gamma"].float()
    out["rstd"] = rstd.squeeze(1)
    if case["y"]:
        out["y"] = y.to(x.dtype)
    out["values"] = _rows_read_back(y, case["fmt"]).to(torch.bfloat16)
    return out


def _plain_bwd(s):
    v, dy, rstd = s["sum"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = v * rstd
    gy = s["gamma"].float() * dy
    dx = rstd * (gy - xhat * (gy * xhat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["sum"].dtype), "dgamma": (dy * xhat).sum(0).to(s["gamma"].dtype)}


def _plain_one_matrix(W, group, asym):
    q, s, z = _i4_groups(W, group, asym)
    return (s * (q.float() - z.float())).flatten(1, 2).to(torch.bfloat16)


def _plain_weights(s):
    group, asym = s["case"]["group"], s["case"]["asym"]
    first = _plain_one_matrix(s["W"], group, asym)
    return [first] if s["pair"] is None else [first, _plain_one_matrix(s["pair"], group, asym)]


def _padded(s, rows):
    """Permuted rows [P][n] as [active experts][most rows][n]."""
    out = rows.new_zeros(len(s["active"]) * s["cap"], rows.shape[1])
    out[s["slot"]] = rows
    return out.view(len(s["active"]), s["cap"], rows.shape[1])


def _plain_experts(s):
    f, act = s["case"]["f"], s["active"]
    x = s["x"].float()[s["token_of"].long()]
    ab = torch.bmm(_padded(s, x), _i4_values(s["W13"][act], s["W13s"][act]))
    a, b = ab.unflatten(2, (f // 16, 2, 16)).unbind(3)
    h = (a / (1 + torch.exp(-a)) * b).flatten(2)
    o = torch.bmm(h, _i4_values(s["W2"][act], s["W2s"][act]))
    return o.flatten(0, 1)[s["slot"]].to(torch.bfloat16)


# ------------------------------------------------------------------------------------------- the framework's calls
def _own_norm(tre, s):
    case, x = s["case"], s["x"]
    if "buf" not in s:
        T, d = x.shape
        per = 128 if case["fmt"] == "e4m3" else 32
        s["buf"] = (torch.empty_like(x) if case["res"] else None, torch.empty_like(x) if case["y"] else None,
                    torch.empty(T, dtype=torch.float32, device=DEV), torch.empty(T, d, dtype=torch.uint8, device=DEV),
                    torch.empty(T, d // per, dtype=torch.float32 if per == 128 else torch.uint8, device=DEV),
                    torch.empty(T, d, dtype=torch.bfloat16, device=DEV))
    sum_, y, rstd, codes, scales, values = s["buf"]
    tre.moe_add_rms_norm(x, s["res"], s["gamma"], EPS, sum_, y, rstd, case["fmt"], codes, scales)
    tre.moe_dequantize_rows(codes, scales, case["fmt"], values)
    out = {"rstd": rstd, "values": values}
    if sum_ is not None:
        out["sum"] = sum_
    if y is not None:
        out["y"] = y
    return out


def _own_bwd(tre, s):
    if "buf" not in s:
        T, d = s["dy"].shape
        ws = tre.moe_workspace_bytes(tre.make_shape(T, d, 1, 1, 128, dtype=s["case"]["src"]), tre.MOE_WS_NORM_BWD)
        s["buf"] = (torch.empty_like(s["dy"]), torch.empty_like(s["gamma"]), torch.empty(ws, dtype=torch.uint8, device=DEV))
    dx, dgamma, ws = s["buf"]
    tre.moe_add_rms_norm_bwd(s["dy"], s["sum"], s["rstd"], s["gamma"], s["dsum"], dx, dgamma, ws)
    return {"dx": dx, "dgamma": dgamma}


def _own_weights(tre, s):
    W, pair, group = s["W"], s["pair"], s["case"]["group"]
    if "buf" not in s:
        E, R, C = W.shape
        N = C if pair is None else 2 * C
        s["buf"] = (torch.empty(E, N // 16, R // 128, 4, 16, 16, dtype=torch.uint8, device=DEV),
                    torch.empty(E, N // 64, R // 128, 128 // group, 16, 4, dtype=torch.int32, device=DEV),
                    [torch.empty(E, R, C, dtype=torch.bfloat16, device=DEV) for m in (W, pair) if m is not None])
    codes, scales, out = s["buf"]
    tre.moe_quantize_weights_i4(W, pair, group, s["case"]["asym"], codes, scales)
    tre.moe_dequantize_weights_i4(codes, scales, group, out[0], None if pair is None else out[1])
    return out


def _own_experts(tre, s):
    case, x = s["case"], s["x"]
    if "buf" not in s:
        T, d, E, k, f = (case[n] for n in "TdEkf")
        sh = tre.make_shape(T, d, E, k, f, dtype="int4")
        s["buf"] = (sh, tre.I4Weights({n: s[n] for n in ("W13", "W13s", "W2", "W2s")}, case["group"]),
                    torch.empty(T * k, d, dtype=torch.bfloat16, device=DEV),
                    torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), dtype=torch.uint8, device=DEV))
    sh, w, o, ws = s["buf"]
    tre.moe_grouped_gemm_fwd_i4(sh, s["offsets"], s["token_of"], x, w, o, ws)
    return o


def run(s):
    kind = s["case"]["kind"]
    if own:
        import token_routed_expert_amd as tre
        return {"norm": _own_norm, "norm_bwd": _own_bwd, "weights": _own_weights, "experts": _own_experts}[kind](tre, s)
    return {"norm": _plain_norm, "norm_bwd": _plain_bwd, "weights": _plain_weights, "experts": _plain_experts}[kind](s)


def work(case):
    kind = case["kind"]
    if kind == "weights":
        n = case["E"] * case["R"] * case["C"] * (2 if case["pair"] else 1)
        # the source once, the codes and scale words once, the bf16 values once (4 operations a value)
        return {"bytes": n * ((4 if case["src"] == "f32" else 2) + 0.5 + 4 / case["group"] + 2), "flops": 4 * n}
    if kind == "experts":
        T, d, E, k, f = (case[n] for n in "TdEkf")
        P = T * k
        live = E - E // 12 if case["skew"] else E * (1 - (1 - k / E) ** T)   # experts with rows
        return {"bytes": T * d * 2 + live * 3 * d * f * (0.5 + 4 / case["group"]) + P * d * 2, "flops": 6 * P * d * f}
    T, d, b = case["T"], case["d"], 4 if case["src"] == "f32" else 2
    n = T * d
    if kind == "norm_bwd":
        # sum, dy (and the stream's gradient) once, dx once; gains and their gradient, rstd
        return {"bytes": n * b * (4 if case["res"] else 3) + 2 * d * b + 4 * T, "flops": 10 * n}
    per = 4 / 128 if case["fmt"] == "e4m3" else 1 / 32
    # x (and the residual) once, the sum, y, codes with scales and their values once
    return {"bytes": n * b * (1 + 2 * case["res"] + case["y"]) + n * (1 + per) + 2 * n + d * b + 4 * T, "flops": 8 * n}


# ------------------------------------------------------------------------------------ the definition, in 64 bits
def _exact_grid():
    v = sorted({m * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(16) if m * 2.0 ** (e - 3) <= 448})
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_blocks(v, fmt):
    """Blocks of v (fp64) as the nearest representable multiples of their scales, found in the list of E4M3's values."""
    grid = _exact_grid()
    b = v.reshape(-1, 128 if fmt == "e4m3" else 32)
    out = torch.empty_like(b)
    for i in range(0, len(b), 1 << 19):
        c = b[i:i + (1 << 19)]
        amax = c.abs().amax(1, keepdim=True)
        if fmt == "e4m3":
            sc = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
        else:
            sc = torch.pow(2.0, torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 448)))
            sc = torch.where(amax > 448 * sc, 2 * sc, sc)
            sc = torch.where(amax <= 224 * sc, sc / 2, sc)
            sc = torch.where(amax == 0, torch.ones_like(sc), torch.clamp(sc, min=2.0 ** -126))
        m = c.abs() / sc
        hi = torch.clamp(torch.searchsorted(grid, m), 1, len(grid) - 1)
        mid = (grid[hi] + grid[hi - 1]) / 2
        up = (m > mid) | ((m == mid) & (hi % 2 == 0))
        out[i:i + (1 << 19)] = torch.where(up, grid[hi], grid[hi - 1]) * torch.copysign(sc, c)
    return out.view(v.shape)


def _exact_column_groups(W, group, asym):
    """One expert's matrix [R][C] through the definition, a row of `group` weights at a time: its bf16 values."""
    w = W.double().t().reshape(-1, group)
    lo, hi = w.min(1, keepdim=True)[0], w.max(1, keepdim=True)[0]
    zero = torch.zeros_like(lo)
    lo, hi = torch.minimum(lo, zero), torch.maximum(hi, zero)
    need = (hi - lo) / 15 if asym else torch.maximum(hi, -lo) / 7
    m, e = torch.frexp(torch.clamp(need, min=2.0 ** -126))
    s = torch.ldexp(torch.ceil(torch.ldexp(m, torch.full_like(e, 20))), e - 20)
    s = torch.where(need == 0, torch.ones_like(s), s)
    z = torch.clamp(torch.round(-lo / s), 0, 15) if asym else torch.full_like(s, 8)
    q = torch.clamp(torch.round(w / s) + z, 0, 15)
    return (s * (q - z)).reshape(W.shape[1], W.shape[0]).t().to(torch.bfloat16)


def _exact_matrix(codes, words):
    """One expert's tiles [N/16][K/128][4][16][16] and words [N/64][K/128][U][16][4] -> its weights [N][K], fp64."""
    NT, KT = codes.shape[:2]
    U = words.shape[2]
    q = torch.empty(NT, 16, KT, 128, dtype=torch.float64, device=codes.device)
    for k in range(128):
        j, g, half, b = k // 32, k // 8 % 4, k // 4 % 2, k % 4
        q[:, :, :, k] = ((codes[:, :, g, :, 4 * j + b] >> (4 * half)) & 15).permute(0, 2, 1).double()
    w = words.permute(0, 4, 3, 1, 2).reshape(NT, 16, KT, U).repeat_interleave(128 // U, dim=3)
    z = w % 16
    s = (w - z).view(torch.float32).double()
    return (s * (q - z)).to(torch.bfloat16).double().reshape(NT * 16, KT * 128)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "weights":
        return [torch.stack([_exact_column_groups(m, case["group"], case["asym"]) for m in W])
                for W in (s["W"], s["pair"]) if W is not None]
    if kind == "norm":
        v, out = s["x"].double(), {}
        if s["res"] is not None:
            out["sum"] = (v + s["res"].double()).to(s["x"].dtype)
            v = out["sum"].double()
        out["rstd"] = ((v * v).sum(1) / case["d"] + EPS) ** -0.5
        y = v * out["rstd"][:, None] * s["gamma"].double()
        if case["y"]:
            out["y"] = y
        out["values"] = _exact_blocks(y, case["fmt"])
        return out
    if kind == "norm_bwd":
        v, dy, r = s["sum"].double(), s["dy"].double(), s["rstd"].double()[:, None]
        gy = dy * s["gamma"].double()
        dx = r * gy - r ** 3 * v * (gy * v).sum(1, keepdim=True) / case["d"]
        return {"dx": dx if s["dsum"] is None else dx + s["dsum"].double(), "dgamma": (dy * v * r).sum(0)}
    f, off, tok = case["f"], s["offsets"].tolist(), s["token_of"].long()
    o = torch.empty(len(tok), case["d"], dtype=torch.float64, device=DEV)
    x = s["x"].double()
    for e in range(case["E"]):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            ab = (x[tok[r]] @ _exact_matrix(s["W13"][e], s["W13s"][e]).t()).view(-1, f // 16, 2, 16)
            a, b = ab[:, :, 0].reshape(-1, f), ab[:, :, 1].reshape(-1, f)
            o[r] = (a * torch.sigmoid(a) * b) @ _exact_matrix(s["W2"][e], s["W2s"][e]).t()
    return o
