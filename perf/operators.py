"""The microscaled operators of the routed experts: what is measured, on which inputs, and their plain forms.

* ``experts``: the experts' forward with 4-bit weights, as a serving program runs it on the rows of one layer: the
  activations' quantisation (MXFP4, or MXFP8 with ``act`` = "a8"), fc1 with SwiGLU, the quantisation of h, fc2.
* ``weights``: 4-bit quantisation of expert weights from fp32 masters or bf16 checkpoints, and the bf16 values that
  the codes stand for.
* ``train``: the bf16 experts' forward and backward with the pre-activations [a|b] kept in 8 bits between the two.
* ``bwd``: that backward alone, from a kept checkpoint, with the routing probabilities' gradient.

Block formats: 32 consecutive values along the contraction share a scale 2^s with s the smallest integer such that no
value saturates (amax <= 6 * 2^s for E2M1, 448 * 2^s for E4M3), stored as the byte s + 127; an all-zero block has s = 0.
Codes are round-to-nearest-even.
"""
import torch

own = False

DEV = "cuda"
FP4 = (1, 0, 6.0)     # mantissa bits, smallest normal exponent, largest value of E2M1
FP8 = (3, -6, 448.0)  # E4M3
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------- cases
def _experts(name, T, d, E, k, f, act, skew=False):
    return {"name": name, "kind": "experts", "T": T, "d": d, "E": E, "k": k, "f": f, "act": act, "skew": skew}


def _weights(name, E, R, C, pair, src):
    return {"name": name, "kind": "weights", "E": E, "R": R, "C": C, "pair": pair, "src": src}


def _train(name, kind, T, d, E, k, f, skew=False):
    return {"name": name, "kind": kind, "T": T, "d": d, "E": E, "k": k, "f": f, "skew": skew}


def listed():
    return [
        # one token of one request: eight experts' weights are read for one row each
        _experts("experts decode 1 a8", 1, 4096, 128, 8, 1536, "a8"),
        # a decode step of a small batch, most experts with one or two rows
        _experts("experts decode 23 a4", 23, 4096, 128, 8, 1536, "a4"),
        # a decode step of a large batch: every expert active, about eleven rows each
        _experts("experts decode 177 a8", 177, 4096, 128, 8, 1536, "a8"),
        # an ordinary prompt of odd length through few wide experts
        _experts("experts prompt 1037 a8", 1037, 4096, 8, 2, 14336, "a8"),
        # the largest prefill batch, 4-bit activations
        _experts("experts prompt 8192 a4", 8192, 4096, 128, 8, 1536, "a4"),
        # prefill off the tile grid with hot, cold and empty experts
        _experts("experts prompt skewed a8", 8200, 4096, 128, 8, 1536, "a8", True),
        # a small model's W2, bf16 checkpoint
        _weights("weights small bf16", 8, 384, 512, False, "bf16"),
        # W1 and W3 of a large layer from the fp32 masters
        _weights("weights pair f32", 128, 4096, 1536, True, "f32"),
        # a small training batch, ragged experts, latency of the eight launches
        _train("train small", "train", 257, 512, 16, 4, 384),
        # the training step's experts at full size
        _train("train 8192", "train", 8192, 4096, 128, 8, 1536),
        # the backward alone, skewed routing with empty experts, a router gradient
        _train("bwd skewed", "bwd", 2051, 2048, 64, 6, 1408, True),
        # the backward of few wide experts
        _train("bwd wide", "bwd", 4096, 4096, 8, 2, 14336),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["experts", "experts", "experts", "weights", "train", "bwd"])
    E = rng.choice([4, 8, 16, 24, 32, 64, 96, 128])
    k = rng.randint(1, min(8, E))
    d, f = 128 * _log(rng, 2, 32), 128 * _log(rng, 1, 40)
    if kind == "weights":
        E = min(E, max(1, int(8e8 // (d * f))))
        return {"kind": kind, "E": E, "R": d, "C": f, "pair": rng.random() < 0.5, "src": rng.choice(["f32", "bf16"])}
    E = min(E, max(k, int(8e8 // (d * f))))
    T = _log(rng, 1, 8192) if kind == "experts" else _log(rng, 16, 8192)
    T = max(1, min(T, int(4.1e11 // (k * d * f))))
    skew = T * k >= 8 * E and E >= 16 and rng.random() < 0.4
    case = {"kind": kind, "T": T, "d": d, "E": E, "k": min(k, E - E // 12) if skew else k, "f": f, "skew": skew}
    return {**case, "act": rng.choice(["a4", "a8"])} if kind == "experts" else case


# ------------------------------------------------------------------------------------------------ the plain pieces
def _pow2(e):
    """2^e exactly (e in [-126, 127]), from the bits: the power function may be off in the last place."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _round_to(v, fmt):
    """v (fp32, within the format's range) rounded to the format's nearest value, ties to even."""
    mant, emin, _ = fmt
    _, e = torch.frexp(v)
    e = torch.clamp(e - 1, min=emin) - mant
    return torch.round(v * _pow2(-e)) * _pow2(e)


def _scale_exp(amax, fmt):
    """Smallest s with amax <= max * 2^s, 0 for amax = 0, at least -126: max = m * 2^e, amax = n * 2^g, m, n in [0.5, 1)."""
    top, e = {6.0: 0.75, 448.0: 0.875}[fmt[2]], {6.0: 3, 448.0: 9}[fmt[2]]
    n, g = torch.frexp(amax)
    s = g - e + (n > top).to(torch.int32)
    return torch.where(amax == 0, torch.zeros_like(s), torch.clamp(s, min=-126))


def _blocks(v, fmt):
    """v [..., K] in blocks of 32 along K: the code values [..., K/32, 32] and the exponents s [..., K/32, 1]."""
    v = v.unflatten(-1, (-1, 32))
    s = _scale_exp(v.abs().amax(-1, keepdim=True), fmt)
    return _round_to(v * _pow2(-s), fmt), s


def _rounded(v, fmt):
    """v with every block of 32 along the last axis replaced by the values that its codes stand for."""
    c, s = _blocks(v, fmt)
    return (c * _pow2(s)).flatten(-2)


def _nibbles(c):
    """E2M1 code values -> 4-bit codes (sign in bit 3)."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=c.device)
    return torch.bucketize(c.abs().contiguous(), mids).to(torch.uint8) | (torch.signbit(c).to(torch.uint8) << 3)


def _tiles(W, pair=None):
    """Expert matrices W [E][K][N] (blocks along K) in the layout of the 4-bit weights: codes
    [E][N/16][K/128][4][16][16] (16 columns x 128 k; 32-value group g, column, byte: two k each, low nibble first) and
    scale bytes [E][N/64][K/128][4][16][4] (group g, column & 15, column / 16 & 3).  `pair`: a second matrix whose
    16-column groups alternate with W's."""
    if pair is not None:
        W = torch.stack([W.unflatten(2, (-1, 16)), pair.unflatten(2, (-1, 16))], 3).flatten(2)
    E, K, N = W.shape
    c, s = _blocks(W.float().transpose(1, 2), FP4)                        # [E][N][K/32][32], [E][N][K/32][1]
    n = _nibbles(c).view(E, N // 16, 16, K // 128, 4, 16, 2)
    codes = (n[..., 0] | (n[..., 1] << 4)).permute(0, 1, 3, 4, 2, 5).contiguous()
    scales = (s + 127).to(torch.uint8).view(E, N // 64, 4, 16, K // 128, 4).permute(0, 1, 4, 5, 3, 2).contiguous()
    return codes, scales


def _untiled(codes, scales):
    """The values [E][K][N] that tiled codes and scales stand for, fp32."""
    E, NT, KT = codes.shape[:3]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = codes.permute(0, 2, 3, 5, 1, 4)                                   # [E][K/128][4][16 bytes][N/16][16]
    v = table[torch.stack([c & 15, c >> 4], 4).to(torch.int32)]           # [E][K/128][4][16][2][N/16][16]
    s = scales.permute(0, 2, 3, 1, 5, 4).reshape(E, KT, 4, 1, 1, NT, 16).to(torch.int32) - 127
    return (v * _pow2(s)).reshape(E, KT * 128, NT * 16)


def _routing(case, g):
    """A routed batch: offsets [E+1], source token and probability of every permuted row, and where each row sits in
    a padded [active experts][most rows] layout."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device=DEV)
    if case["skew"]:
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        logits += torch.where(rank > E - E // 12, torch.full_like(rank, -64.0), 3.0 * rank ** -1.2)
    top, idx = torch.topk(logits, k, dim=1)
    prob = torch.softmax(top, 1)
    expert, order = torch.sort(idx.flatten(), stable=True)
    counts = torch.bincount(expert, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    active = torch.nonzero(counts).flatten()
    rank = torch.zeros(E, dtype=torch.int64, device=DEV)
    rank[active] = torch.arange(len(active), device=DEV)
    cap = int(counts.max())
    slot = rank[expert] * cap + torch.arange(T * k, device=DEV) - offsets[expert]
    return {"offsets": offsets.to(torch.int32), "token_of": (order // k).to(torch.int32),
            "row_prob": prob.flatten()[order].contiguous(), "active": active, "cap": cap, "slot": slot}


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    if case["kind"] == "weights":
        dt = torch.float32 if case["src"] == "f32" else torch.bfloat16
        E, R, C = case["E"], case["R"], case["C"]
        s["W"] = _randn(g, E, R, C, std=R ** -0.5, dtype=dt)
        s["pair"] = _randn(g, E, R, C, std=R ** -0.5, dtype=dt) if case["pair"] else None
        return s
    T, d, E, k, f = (case[n] for n in "TdEkf")
    s.update(_routing(case, g))
    s["x"] = _randn(g, T, d, dtype=torch.bfloat16)
    if case["kind"] == "experts":
        parts = []
        for e in range(0, E, 8):
            n = min(8, E - e)
            W1, W3 = _randn(g, n, d, f, std=d ** -0.5), _randn(g, n, d, f, std=d ** -0.5)
            parts.append(_tiles(W1, W3) + _tiles(_randn(g, n, f, d, std=f ** -0.5)))
        s["W13"], s["W13s"], s["W2"], s["W2s"] = (torch.cat(p) for p in zip(*parts))
        return s
    s["W1"], s["W3"] = (_randn(g, E, d, f, std=d ** -0.5, dtype=torch.bfloat16) for _ in range(2))
    s["W2"] = _randn(g, E, f, d, std=f ** -0.5, dtype=torch.bfloat16)
    s["dO"] = _randn(g, T, d, dtype=torch.bfloat16)[s["token_of"].long()]
    if case["kind"] == "bwd":
        # a kept checkpoint: blocks of normal pre-activations
        c, e = _blocks(_randn(g, T * k, 2 * f), FP8)
        s["abq"] = c.flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8)
        s["abs"] = (e.squeeze(-1) + 127).to(torch.uint8)
    return s


# ------------------------------------------------------------------------------------------------ the plain forms
def _padded(s, rows):
    """Permuted rows [P][n] as [active experts][most rows][n]."""
    out = rows.new_zeros(len(s["active"]) * s["cap"], rows.shape[1])
    out[s["slot"]] = rows
    return out.view(len(s["active"]), s["cap"], rows.shape[1])


def _rows(s, padded):
    return padded.flatten(0, 1)[s["slot"]]


def _silu(a):
    return a / (1 + torch.exp(-a))


def _plain_experts(s):
    case = s["case"]
    fmt = FP4 if case["act"] == "a4" else FP8
    act = s["active"]
    x = _rounded(s["x"].float(), fmt)[s["token_of"].long()]
    ab = _rows(s, torch.bmm(_padded(s, x), _untiled(s["W13"][act], s["W13s"][act])))
    a, b = ab.view(-1, case["f"] // 16, 2, 16).unbind(2)
    h = _rounded((_silu(a) * b).flatten(1), fmt)
    return _rows(s, torch.bmm(_padded(s, h), _untiled(s["W2"][act], s["W2s"][act]))).to(torch.bfloat16)


def _plain_weights(s):
    return [_rounded(W.float().transpose(1, 2), FP4).transpose(1, 2).to(torch.bfloat16).contiguous()
            for W in (s["W"], s["pair"]) if W is not None]


def _plain_fwd(s):
    """o with the probabilities applied before W2, and the kept [a|b] in 8 bits (as values)."""
    act = s["active"]
    x = _padded(s, s["x"].float()[s["token_of"].long()])
    a, b = (_rows(s, torch.bmm(x, W[act].float())) for W in (s["W1"], s["W3"]))
    h = s["row_prob"][:, None] * _silu(a) * b
    o = _rows(s, torch.bmm(_padded(s, h), s["W2"][act].float()))
    return o.to(torch.bfloat16), torch.cat([_rounded(a, FP8), _rounded(b, FP8)], 1)


def _grown(s, dW):
    """Gradients of the active experts among all experts' (zeros for the others), bf16."""
    out = torch.zeros(s["case"]["E"], *dW.shape[1:], dtype=torch.bfloat16, device=dW.device)
    out[s["active"]] = dW.to(torch.bfloat16)
    return out


def _plain_bwd(s, ab):
    """Gradients from [a|b] as kept: (dXp, dW1, dW3, dW2, the probabilities' gradient of every row)."""
    act, f, p = s["active"], s["case"]["f"], s["row_prob"][:, None]
    a, b = ab[:, :f], ab[:, f:]
    W1, W3, W2 = (s[n][act].float() for n in ("W1", "W3", "W2"))
    dO = _padded(s, s["dO"].float())
    dh = _rows(s, torch.bmm(dO, W2.transpose(1, 2).contiguous()))
    sg = 1 / (1 + torch.exp(-a))
    h = a * sg * b
    dprob = (h * dh).sum(1)
    da = _padded(s, p * dh * b * sg * (1 + a * (1 - sg)))
    db = _padded(s, p * dh * a * sg)
    dXp = _rows(s, torch.bmm(da, W1.transpose(1, 2).contiguous()) + torch.bmm(db, W3.transpose(1, 2).contiguous()))
    xt = _padded(s, s["x"].float()[s["token_of"].long()]).transpose(1, 2).contiguous()
    dW2 = torch.bmm(_padded(s, p * h).transpose(1, 2).contiguous(), dO)
    return (dXp.to(torch.bfloat16), _grown(s, torch.bmm(xt, da)), _grown(s, torch.bmm(xt, db)), _grown(s, dW2), dprob)


def _plain_kept(s):
    """The values of the checkpoint that prepare() made."""
    c = s["abq"].view(torch.float8_e4m3fn).float().unflatten(1, (-1, 32))
    return (c * _pow2(s["abs"].to(torch.int32)[..., None] - 127)).flatten(1)


# ------------------------------------------------------------------------------------------- the framework's calls
def _own_experts(tre, s):
    case, x = s["case"], s["x"]
    a4 = case["act"] == "a4"
    if "buf" not in s:
        T, d, E, k, f = (case[n] for n in "TdEkf")
        sh = tre.make_shape(T, d, E, k, f, dtype="mxfp4" if a4 else "mxfp4_a8")
        u8 = {"dtype": torch.uint8, "device": DEV}
        s["buf"] = (sh, tre.MX4Weights({n: s[n] for n in ("W13", "W13s", "W2", "W2s")}),
                    torch.empty(T, d // 2 if a4 else d, **u8), torch.empty(T, d // 32, **u8),
                    torch.empty(T * k, d, dtype=torch.bfloat16, device=DEV),
                    torch.empty(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_FWD), **u8))
    sh, w, xq, xs, o, ws = s["buf"]
    (tre.moe_quantize_rows_mx4 if a4 else tre.moe_quantize_rows_mx)(x, xq, xs)
    tre.moe_grouped_gemm_fwd_mx4(sh, s["offsets"], s["token_of"], xq, xs, w, o, ws)
    return o


def _own_weights(tre, s):
    W, pair = s["W"], s["pair"]
    if "buf" not in s:
        E, R, C = W.shape
        N = C if pair is None else 2 * C
        s["buf"] = (torch.empty(E, N // 16, R // 128, 4, 16, 16, dtype=torch.uint8, device=DEV),
                    torch.empty(E, N // 64, R // 128, 4, 16, 4, dtype=torch.uint8, device=DEV),
                    [torch.empty(E, R, C, dtype=torch.bfloat16, device=DEV) for m in (W, pair) if m is not None])
    codes, scales, out = s["buf"]
    tre.moe_quantize_weights_mx4(W, pair, codes, scales)
    tre.moe_dequantize_weights_mx4(codes, scales, out[0], None if pair is None else out[1])
    return out


def _own_train(tre, s):
    case = s["case"]
    fwd = case["kind"] == "train"
    if "buf" not in s:
        T, d, E, k, f = (case[n] for n in "TdEkf")
        P = T * k
        sh = tre.make_shape(T, d, E, k, f, dtype="bf16")

        def z(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=DEV)

        s["buf"] = (sh, z(P, 2 * f, dtype=torch.uint8) if fwd else s["abq"],
                    z(P, 2 * f // 32, dtype=torch.uint8) if fwd else s["abs"], z(P, f), z(P, d), z(P, 2 * f), z(P, d),
                    z(E, d, f), z(E, d, f), z(E, f, d), None if fwd else z(P, dtype=torch.float32),
                    z(tre.moe_workspace_bytes(sh, tre.MOE_WS_GEMM_BWD_ROWSCALED), dtype=torch.uint8))
    sh, abq, abs_, h, o, dab, dXp, dW1, dW3, dW2, dprob, ws = s["buf"]
    W = (s["W1"], s["W3"], s["W2"], s["row_prob"])
    if fwd:
        tre.moe_grouped_gemm_fwd_ckpt8(sh, s["offsets"], s["token_of"], s["x"], *W, abq, abs_, h, o)
    tre.moe_grouped_gemm_bwd_ckpt8(sh, s["offsets"], s["token_of"], s["x"], abq, abs_, s["dO"], *W, h, dab, dXp, dW1,
                                   dW3, dW2, None, dprob, ws)
    return {"o": o, "dXp": dXp, "dW1": dW1, "dW3": dW3, "dW2": dW2} if fwd else {
        "dXp": dXp, "dW1": dW1, "dW3": dW3, "dW2": dW2, "dprob": dprob}


def run(s):
    kind = s["case"]["kind"]
    if own:
        import token_routed_expert_amd as tre
        return {"experts": _own_experts, "weights": _own_weights, "train": _own_train, "bwd": _own_train}[kind](tre, s)
    if kind == "experts":
        return _plain_experts(s)
    if kind == "weights":
        return _plain_weights(s)
    if kind == "train":
        o, ab = _plain_fwd(s)
        return {"o": o, **dict(zip(("dXp", "dW1", "dW3", "dW2"), _plain_bwd(s, ab)))}
    return dict(zip(("dXp", "dW1", "dW3", "dW2", "dprob"), _plain_bwd(s, _plain_kept(s))))


def work(case):
    if case["kind"] == "weights":
        n = case["E"] * case["R"] * case["C"] * (2 if case["pair"] else 1)
        # the source once, the codes and scales once, the bf16 values once (4 operations a value)
        return {"bytes": n * ((4 if case["src"] == "f32" else 2) + 0.5 + 1 / 32 + 2), "flops": 4 * n}
    T, d, E, k, f = (case[n] for n in "TdEkf")
    P = T * k
    live = E - E // 12 if case["skew"] else E * (1 - (1 - k / E) ** T)   # experts with rows
    if case["kind"] == "experts":
        return {"bytes": T * d * 2 + live * 3 * d * f * (0.5 + 1 / 32) + P * d * 2, "flops": 6 * P * d * f}
    bwd = T * d * 2 + live * 3 * d * f * 2 + P * d * 2 + P * 4 + P * d * 2 + E * 3 * d * f * 2
    if case["kind"] == "bwd":
        return {"bytes": bwd + P * 2 * f * 33 / 32 + P * 4, "flops": 12 * P * d * f}
    return {"bytes": bwd + P * d * 2, "flops": 18 * P * d * f}


# ------------------------------------------------------------------------------------ the definition, in 64 bits
def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(fmt):
    mant, emin, top = fmt
    v = sorted({m * 2.0 ** (e - mant) for e in range(emin, 10) for m in range(2 ** (mant + 1))
                if m * 2.0 ** (e - mant) <= top})
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _exact_rounded(v, fmt):
    """Blocks of 32 of v (fp64) as the nearest representable multiples of their scales, by searching the format's
    values; a tie goes to the value with the even code (codes count the values from zero)."""
    values = _exact_values(fmt)
    b = v.reshape(-1, 32)
    amax = b.abs().amax(1, keepdim=True)
    s = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / fmt[2]))
    s = torch.where(amax > fmt[2] * _exact_pow2(s), s + 1, s)
    s = torch.where(amax <= fmt[2] * _exact_pow2(s - 1), s - 1, s)
    s = torch.where(amax == 0, torch.zeros_like(s), torch.clamp(s, min=-126))
    out = torch.empty_like(b)
    for i in range(0, len(b), 1 << 22):
        c, sc = b[i:i + (1 << 22)], _exact_pow2(s[i:i + (1 << 22)])
        m = c.abs() / sc
        hi = torch.clamp(torch.searchsorted(values, m), 1, len(values) - 1)
        mid = (values[hi] + values[hi - 1]) / 2
        up = (m > mid) | ((m == mid) & (hi % 2 == 0))
        out[i:i + (1 << 22)] = torch.where(up, values[hi], values[hi - 1]) * torch.copysign(sc, c)
    return out.view(v.shape)


def _exact_matrix(codes, scales):
    """One expert's tiled codes [N/16][K/128][4][16][16] and scales [N/64][K/128][4][16][4] -> values [N][K], fp64."""
    NT, KT = codes.shape[:2]
    value = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    out = torch.empty(NT, 16, KT, 4, 16, 2, dtype=torch.float64, device=codes.device)
    for half in range(2):
        c = ((codes >> (4 * half)) & 15).long()
        out[..., half] = (value[c & 7] * (1 - 2 * (c >> 3))).permute(0, 3, 1, 2, 4)
    sc = _exact_pow2(scales.long() - 127)                       # [N/64][K/128][4][16][4]
    sc = sc.permute(0, 4, 3, 1, 2).reshape(NT, 16, KT, 4)
    return (out * sc[..., None, None]).reshape(NT * 16, KT * 128)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "weights":
        return [torch.stack([_exact_rounded(m.double().t().contiguous(), FP4).t().contiguous() for m in W])
                for W in (s["W"], s["pair"]) if W is not None]
    E, d, f = case["E"], case["d"], case["f"]
    off = s["offsets"].tolist()
    tok = s["token_of"].long()
    spans = [(e, slice(off[e], off[e + 1])) for e in range(E) if off[e + 1] > off[e]]
    if case["kind"] == "experts":
        fmt = FP4 if case["act"] == "a4" else FP8
        xd = _exact_rounded(s["x"].double(), fmt)
        o = torch.empty(len(tok), d, dtype=torch.float64, device=DEV)
        for e, r in spans:
            ab = xd[tok[r]] @ _exact_matrix(s["W13"][e], s["W13s"][e]).t()
            ab = ab.view(-1, f // 16, 2, 16)
            a, b = ab[:, :, 0].reshape(-1, f), ab[:, :, 1].reshape(-1, f)
            o[r] = _exact_rounded(a * torch.sigmoid(a) * b, fmt) @ _exact_matrix(s["W2"][e], s["W2s"][e]).t()
        return o
    P = len(tok)
    got = {n: torch.zeros(P, d, dtype=torch.float64, device=DEV) for n in ("o", "dXp")}
    got |= {n: torch.zeros(s[n[1:]].shape, dtype=torch.float64, device=DEV) for n in ("dW1", "dW3", "dW2")}
    got["dprob"] = torch.zeros(P, dtype=torch.float64, device=DEV)
    for e, r in spans:
        x, dO, p = s["x"].double()[tok[r]], s["dO"][r].double(), s["row_prob"][r].double()[:, None]
        W1, W3, W2 = (s[n][e].double() for n in ("W1", "W3", "W2"))
        if case["kind"] == "train":
            a, b = x @ W1, x @ W3
            got["o"][r] = (p * a * torch.sigmoid(a) * b) @ W2
            a, b = _exact_rounded(a, FP8), _exact_rounded(b, FP8)
        else:
            sc = torch.repeat_interleave(_exact_pow2(s["abs"][r].long() - 127), 32, dim=1)
            ab = s["abq"][r].view(torch.float8_e4m3fn).double() * sc
            a, b = ab[:, :f], ab[:, f:]
        sg = torch.sigmoid(a)
        h, dh = a * sg * b, dO @ W2.t()
        got["dprob"][r] = (h * dh).sum(1)
        da, db = p * dh * b * (sg + a * sg * (1 - sg)), p * dh * a * sg
        got["dXp"][r] = da @ W1.t() + db @ W3.t()
        got["dW1"][e], got["dW3"][e], got["dW2"][e] = x.t() @ da, x.t() @ db, (p * h).t() @ dO
    got.pop("dprob" if case["kind"] == "train" else "o")
    return got
