"""Cases and plain forms of the microscaled 4-bit (mx4) operators.

An mx4 matrix holds every row as 4-bit e2m1 codes (magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
and a sign, the even column in the low half of a byte) with one power-of-two scale for
each 32 columns, stored as its exponent + 127 in one byte (255: not a number).  Three
operators are measured:

  quantize  a batch of matrices to mx4 and back;
  ffn       the expert FFN of a routed batch, both operands mx4: the kept rows of x are
            quantised, multiplied with the experts' W1 and W3, silu(g) * u is quantised
            again and multiplied with W2;
  layer     the whole layer (router, dispatch, experts, combine, gate statistics) on mx4
            expert weights: for at most 16 tokens with bf16 activations ("bf16"), for any
            number with quantised rows ("mx4").

Sizes are those of this repository's workloads (d = 4096, 8 experts of 1376 neurons,
16 of 688) and smaller or odd ones around them.
"""
import torch

own = False  # set from outside: True runs the framework's kernels, False the plain forms

BLOCK = 32  # columns that share a scale

# outputs and intermediates of the whole layer, held by the caller
_BUFFERS = ("y", "loss", "counts", "importance", "f", "P", "topk_idx", "topk_w", "probs_sum", "row_token",
            "slot_row", "kept", "offsets", "x_q", "x_s", "h", "h_q", "h_s", "out")


# ------------------------------------------------------------------------- the cases
def _q(name, G, rows, K, dtype):
    return {"name": name, "op": "quantize", "G": G, "rows": rows, "K": K, "dtype": dtype}


def _f(name, T, E, k, m, d, cf=-1.0):
    return {"name": name, "op": "ffn", "T": T, "E": E, "k": k, "m": m, "d": d, "cf": cf}


def _l(name, T, E, k, m, d, act, noisy=False, router="mixtral", rescale=True):
    return {"name": name, "op": "layer", "T": T, "E": E, "k": k, "m": m, "d": d, "act": act,
            "noisy": noisy, "router": router, "rescale": rescale}


def listed():
    return [
        # a few f32 rows of an odd width, as a test or a calibration run has them
        _q("quantize_f32_rows", 1, 37, 200, "f32"),
        # the down projections and the up projections of a whole layer, once after loading
        _q("quantize_w2", 8, 4096, 1376, "bf16"),
        _q("quantize_w13", 8, 2752, 4096, "bf16"),
        # one token through the row path; a ragged batch of a server; 16 small experts with
        # a capacity that drops rows; a training-sized prompt batch
        _f("ffn_t1", 1, 8, 2, 1376, 4096),
        _f("ffn_t203", 203, 8, 2, 1376, 4096),
        _f("ffn_t4096_16x688_cf4", 4096, 16, 4, 688, 4096, 4.0),
        _f("ffn_t16384", 16384, 8, 2, 1376, 4096),
        # decode steps: one token, an odd few with a noisy ST router on a small layer, eight
        # and sixteen tokens
        _l("layer_t1", 1, 8, 2, 1376, 4096, "bf16"),
        _l("layer_t5_small_st", 5, 6, 3, 172, 512, "bf16", True, "st"),
        _l("layer_t8", 8, 8, 2, 1376, 4096, "bf16"),
        _l("layer_t16_16x688", 16, 16, 4, 688, 4096, "bf16"),
        # a prompt through the whole layer with quantised rows
        _l("layer_t2048_rows", 2048, 8, 2, 1376, 4096, "mx4", True),
    ]


def _log(rng, lo, hi, step=1):
    v = lo * (hi / lo) ** rng.random()
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["quantize", "ffn", "layer", "layer"])
    if op == "quantize":
        while True:
            G, rows, K = _log(rng, 1, 8), _log(rng, 1, 8192), _log(rng, 8, 8192, 8)
            if G * rows * K <= 8 * 2752 * 4096:
                return {"op": op, "G": G, "rows": rows, "K": K, "dtype": rng.choice(["f32", "bf16"])}
    E = rng.choice([1, 4, 6, 8, 16])
    k = rng.randint(1, min(E, 4))
    m, d = _log(rng, 64, 1376), _log(rng, 64, 4096, 32)
    if op == "ffn":
        T = _log(rng, 1, 16384 if E * m <= 11008 else 4096)
        T = max(1, min(T, 32768 // k))
        return {"op": op, "T": T, "E": E, "k": k, "m": m, "d": d,
                "cf": rng.choice([-1.0, -1.0, 0.75 * k, 1.5 * k])}
    few = rng.random() < 0.75
    T = rng.randint(1, 16) if few else _log(rng, 1, 4096)
    return {"op": op, "T": T, "E": E, "k": k, "m": m, "d": d, "act": "bf16" if few else "mx4",
            "noisy": rng.random() < 0.5, "router": rng.choice(["mixtral", "st"]),
            "rescale": rng.random() < 0.5}


def _up(v, n):
    return (v + n - 1) // n * n


def _code_bytes(G, rows, K):
    return G * rows * (_up(K, BLOCK) // 2)


def _scale_bytes(G, rows, K):
    return G * rows * (_up(K, BLOCK) // BLOCK)


def work(case):
    """Bytes: inputs and outputs once (scales without their padding); operations: the products."""
    if case["op"] == "quantize":
        n, es = case["G"] * case["rows"] * case["K"], 4 if case["dtype"] == "f32" else 2
        mx4 = _code_bytes(case["G"], case["rows"], case["K"]) + _scale_bytes(case["G"], case["rows"], case["K"])
        return {"bytes": 2 * n * es + 2 * mx4, "flops": 0}
    T, E, k, m, d = (case[n] for n in ("T", "E", "k", "m", "d"))
    rows = T * k
    if case.get("cf", -1.0) >= 0:
        rows = min(rows, E * -int(-T * case["cf"] // E))
    hit = E * (1.0 - (1.0 - k / E) ** T)  # experts that a batch of T tokens reaches, on average
    weights = 3 * m * d * (0.5 + 1.0 / BLOCK)
    if case["op"] == "ffn":
        return {"bytes": hit * weights + 2 * T * d + 2 * rows * d, "flops": 6.0 * rows * m * d}
    router = (2 if case["noisy"] else 1) * E * d * 2
    return {"bytes": hit * weights + 4 * T * d + router,
            "flops": 6.0 * rows * m * d + router * T}


# ------------------------------------------------------------------- inputs and layouts
def _pack(v):
    """4-bit codes [..., K] (uint8) -> bytes [..., K / 2], the even column in the low half."""
    return v[..., 0::2] | (v[..., 1::2] << 4)


def _tiles(s):
    """Scales [G][rows][blocks] -> tiles of 128 rows x 4 blocks, 512 bytes each:
    [G][rows / 128][blocks / 4][row % 32][row / 32 % 4][block % 4], padded with zeros."""
    G, rows, nb = s.shape
    p = torch.zeros(G, _up(rows, 128), _up(nb, 4), dtype=torch.uint8, device=s.device)
    p[:, :rows, :nb] = s
    p = p.view(G, p.shape[1] // 128, 4, 32, p.shape[2] // 4, 4)
    return p.permute(0, 1, 4, 3, 2, 5).contiguous()


def _untiles(t, rows, nb):
    G, tr, tk = t.shape[:3]
    return t.permute(0, 1, 4, 3, 2, 5).reshape(G, tr * 128, tk * 4)[:, :rows, :nb]


def _make_codes(w):
    """Gaussian weights [rows][K] as mx4 codes and scales, as a user's weights come."""
    rows, K = w.shape
    w = torch.nn.functional.pad(w.float(), (0, _up(K, BLOCK) - K)).view(rows, -1, BLOCK)
    e = (torch.frexp(w.abs().amax(-1))[1] - 3).clamp(-127, 125)
    a = w.abs() * torch.exp2(-e.float()).unsqueeze(-1)
    code = torch.bucketize(a, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device))
    code = (code + 8 * (w < 0)).to(torch.uint8).view(rows, -1)
    return _pack(code), (e + 127).to(torch.uint8)


def _weights(g, E, m, d):
    """E experts: W1 and W3 rows in groups of 16 and 16 (m16 = m rounded up to 16), W2
    [d][m8]; zero neurons past m."""
    m16, m8 = _up(m, 16), _up(m, 8)
    q13, s13, q2, s2 = [], [], [], []
    for _ in range(E):
        w = torch.zeros(2, m16, d, device="cuda")
        w[:, :m] = torch.randn(2, m, d, generator=g, device="cuda") * 0.02
        c, s = _make_codes(w.view(2, m16 // 16, 16, d).transpose(0, 1).reshape(2 * m16, d))
        q13.append(c)
        s13.append(s)
        w = torch.zeros(d, m8, device="cuda")
        w[:, :m] = torch.randn(d, m, generator=g, device="cuda") * 0.02
        c, s = _make_codes(w)
        q2.append(c)
        s2.append(s)
    return {"W13_q": torch.stack(q13), "W13_s": _tiles(torch.stack(s13)),
            "W2_q": torch.stack(q2), "W2_s": _tiles(torch.stack(s2))}


def _row_scales(T, k, E, K):
    return torch.zeros((T * k // 128 + E + 1) * (_up(K, 128) // 128) * 512, dtype=torch.uint8, device="cuda")


def _rows(T, k, K):
    return torch.zeros(T * k, _up(K, BLOCK) // 2, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "quantize":
        G, rows, K = case["G"], case["rows"], case["K"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        src = torch.empty(G, rows, K, dtype=dt, device="cuda")
        src.normal_(0.0, 0.02, generator=g)
        # rows of very different sizes, a row of zeros among them
        size = torch.randint(-6, 7, (G, rows, 1), generator=g, device="cuda").float()
        src.mul_(torch.exp2(size).to(dt))
        src[:, rows // 2] = 0
        tr, tk = _up(rows, 128) // 128, _up(K, 128) // 128
        return {"case": case, "src": src,
                "codes": torch.zeros(G, rows, _up(K, BLOCK) // 2, dtype=torch.uint8, device="cuda"),
                "scales": torch.zeros(G, tr, tk, 32, 4, 4, dtype=torch.uint8, device="cuda"),
                "back": torch.empty_like(src)}
    T, E, k, m, d = (case[n] for n in ("T", "E", "k", "m", "d"))
    s = {"case": case, **_weights(g, E, m, d)}
    s["x"] = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    s["x_q"], s["x_s"] = _rows(T, k, d), _row_scales(T, k, E, d)
    s["h_q"], s["h_s"] = _rows(T, k, m), _row_scales(T, k, E, m)
    s["out"] = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")  # rows past the kept ones stay
    i32 = {"dtype": torch.int32, "device": "cuda"}
    f32 = {"dtype": torch.float32, "device": "cuda"}
    if case["op"] == "ffn":
        # a routed batch and its dispatch tables: stable by token, rows past the capacity dropped
        idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].contiguous()
        cap = T * k if case["cf"] < 0 else -int(-T * case["cf"] // E)
        flat = idx.reshape(-1)
        order = flat.argsort(stable=True)
        counts = torch.bincount(flat, minlength=E)
        first = counts.cumsum(0) - counts
        rank = torch.empty_like(flat)
        rank[order] = torch.arange(T * k, device="cuda") - first[flat[order]]
        kept = counts.clamp(max=cap)
        offsets = torch.cat([kept.new_zeros(1), kept.cumsum(0)])
        slot = torch.where(rank < cap, offsets[flat] + rank, -1)
        s["topk_idx"], s["slot_row"] = idx.to(torch.int32), slot.view(T, k).to(torch.int32)
        s["offsets"], s["most"] = offsets.to(torch.int32), int(kept.max())
    else:
        s["Wg"] = (torch.randn(d, E, generator=g, device="cuda") * 0.02).bfloat16()
        s["Wnoise"] = (torch.randn(d, E, generator=g, device="cuda") * 0.02).bfloat16() if case["noisy"] else None
        s["noise"] = torch.randn(T, E, generator=g, device="cuda") if case["noisy"] else None
        s["h"] = torch.zeros(T * k, _up(m, 8), dtype=torch.bfloat16, device="cuda")
        s["y"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        for n, shape, kind in (("loss", (1,), f32), ("counts", (E,), i32), ("importance", (E,), f32),
                               ("f", (E,), f32), ("P", (E,), f32), ("topk_idx", (T, k), i32),
                               ("topk_w", (T, k), f32), ("probs_sum", (E,), f32), ("row_token", (T * k,), i32),
                               ("slot_row", (T, k), i32), ("kept", (E,), i32), ("offsets", (E + 1,), i32)):
            s[n] = torch.empty(shape, **kind)
    # the scratch that a program keeps between calls, zeroed once
    s["ws"] = torch.zeros(4 * 128 * d + 64 * _up(T, 64) * E + 65536 * 8, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------- plain forms
def _plain_codes(x):
    """x [..., K] (f32, K a multiple of 32) -> (signed e2m1 values, exponents), exact."""
    v = x.view(*x.shape[:-1], -1, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    e = ((amax.view(torch.int32) >> 23) - 129).clamp(min=-127)  # floor(log2(amax)) - 2
    a = v.abs() * torch.exp2(-e.float())
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)  # ties to even, as the codes have them
    return torch.copysign(q, v), e


def _plain_mx4(x):
    """The mx4 values of x [..., K] in f32."""
    K = x.shape[-1]
    q, e = _plain_codes(torch.nn.functional.pad(x.float(), (0, _up(K, BLOCK) - K)).contiguous())
    return (q * torch.exp2(e.float())).view(*x.shape[:-1], -1)[..., :K]


_TABLE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _plain_matrix(codes, scales, rows, dtype=torch.float32):
    """f32 values [G][rows][K32] of an mx4 matrix."""
    pairs = torch.stack([codes & 15, codes >> 4], -1).view(*codes.shape[:-1], -1)
    v = torch.tensor(_TABLE, dtype=dtype, device=codes.device)[pairs.int()]
    nb = v.shape[-1] // BLOCK
    e = _untiles(scales, rows, nb).to(dtype) - 127
    return (v.view(*v.shape[:-1], nb, BLOCK) * torch.exp2(e).unsqueeze(-1)).view(v.shape)


def _plain_w13(s, E, m, d, dtype=torch.float32):
    w = _plain_matrix(s["W13_q"], s["W13_s"], 2 * _up(m, 16), dtype).view(E, -1, 2, 16, d)
    return w[:, :, 0].reshape(E, -1, d)[:, :m], w[:, :, 1].reshape(E, -1, d)[:, :m]


def _plain_w2(s, E, m, d, dtype=torch.float32):
    return _plain_matrix(s["W2_q"], s["W2_s"], d, dtype)[:, :, :m]


def _silu_mul(g, u):
    return g / (1 + torch.exp(-g)) * u


def _plain_experts(s, rows, E, m, d, quantised):
    """rows [E][n][d] (f32) through every expert: [E][n][d] f32."""
    w1, w3 = _plain_w13(s, E, m, d)
    h = _silu_mul(rows @ w1.transpose(1, 2), rows @ w3.transpose(1, 2))
    del w1, w3
    h = _plain_mx4(h) if quantised else h
    return h @ _plain_w2(s, E, m, d).transpose(1, 2)


def _plain_routed(s, x, idx, slot, offsets, most, E, m, d):
    """The kept rows of x (f32) through their experts, rows mx4: out [T k + 1][d] f32 in row
    order, zeros past the kept rows (the last row takes what is dropped)."""
    T, k = idx.shape
    flat, at = idx.reshape(-1).long(), slot.reshape(-1).long()
    kept = at >= 0
    place = torch.where(kept, flat * most + at - offsets[flat].long(), E * most)
    grid = torch.zeros(E * most + 1, d, device=x.device)
    grid[place] = _plain_mx4(x).repeat_interleave(k, 0)
    y = _plain_experts(s, grid[:-1].view(E, most, d), E, m, d, True).reshape(E * most, d)
    out = torch.zeros(T * k + 1, d, device=x.device)
    out[torch.where(kept, at, T * k)] = y[place.clamp(max=E * most - 1)]
    return out


def _plain_route(s, case):
    """Logits in 64 bits (the choice of experts lies next to a border), gates rounded at the end."""
    x = s["x"].double()
    H = x @ s["Wg"].double()
    if case["noisy"]:
        H = H + s["noise"].double() * torch.log1p(torch.exp(x @ s["Wnoise"].double()))
    top, idx = torch.sort(H, dim=1, descending=True, stable=True)
    k, E, T = case["k"], case["E"], case["T"]
    idx = idx[:, :k]
    p = torch.exp(H - top[:, :1])
    p = p / p.sum(1, keepdim=True)
    G = p.gather(1, idx)
    if case["router"] == "mixtral":
        G = torch.exp(top[:, :k] - top[:, :1])
        G = G / G.sum(1, keepdim=True)
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    importance = torch.zeros(E, dtype=torch.float64, device=x.device).index_add_(0, idx.reshape(-1), G.reshape(-1))
    P = p.mean(0)
    loss = 0.01 * (counts.double() / (T * k) * P).sum().view(1)
    return idx, G, counts, importance, P, loss


def _plain_run(s):
    case = s["case"]
    if case["op"] == "quantize":
        return {"values": _plain_mx4(s["src"]).to(s["src"].dtype)}
    T, E, k, m, d = (case[n] for n in ("T", "E", "k", "m", "d"))
    x = s["x"].float()
    if case["op"] == "ffn":
        out = _plain_routed(s, x, s["topk_idx"], s["slot_row"], s["offsets"], s["most"], E, m, d)
        return {"out": out[:-1].bfloat16()}
    idx, G, counts, importance, P, loss = _plain_route(s, case)
    rows = _plain_mx4(x) if case["act"] == "mx4" else x
    # every expert on every token, then the chosen ones of each
    y = _plain_experts(s, rows.expand(E, T, d), E, m, d, case["act"] == "mx4")
    y = y[idx, torch.arange(T, device=x.device).view(T, 1)]
    y = (G.float().unsqueeze(-1) * y).sum(1) * (E / k if case["rescale"] else 1.0)
    return {"y": y.bfloat16(), "topk_idx": idx.to(torch.int32), "topk_w": G.float(),
            "counts": counts.to(torch.int32), "importance": importance.float(), "P": P.float(),
            "loss": loss.float()}


# ---------------------------------------------------------------- the framework's calls
def _handles(s, moe):
    """What a program makes once and keeps: the layer's description, the experts, buffers and scratch."""
    case = s["case"]
    p = moe.params(case["T"], case["d"], case["E"], case["k"], case["m"],
                   router_type=moe.ST if case.get("router") == "st" else moe.MIXTRAL,
                   rescale=case.get("rescale", False), balance_lambda=0.01)
    W = moe.Mx4Experts(s["W13_q"], s["W13_s"], s["W2_q"], s["W2_s"])
    bufs = moe.Mx4Buffers(p, **{n: s[n] for n in _BUFFERS}) if case["op"] == "layer" else None
    return p, W, moe.Workspace(p, buf=s["ws"]), bufs


def _own_run(s):
    import top_routing_grouped_noisy_b200 as moe
    case = s["case"]
    if case["op"] == "quantize":
        moe.moe_mx4_quantize(s["src"], out=(s["codes"], s["scales"]))
        moe.moe_mx4_dequantize(s["codes"], s["scales"], case["K"], out=s["back"])
        return {"values": s["back"]}
    if "handles" not in s:
        s["handles"] = _handles(s, moe)
    p, W, ws, bufs = s["handles"]
    if case["op"] == "ffn":
        moe.moe_mx4_dispatch(p, s["x"], s["topk_idx"], s["slot_row"], s["offsets"], s["x_q"], s["x_s"])
        moe.moe_expert_ffn_mx4(p, s["x_q"], s["x_s"], s["offsets"], W, s["h_q"], s["h_s"], s["out"], ws)
        return {"out": s["out"]}
    moe.moe_forward_mx4(p, s["x"], s["Wg"], W, ws, bufs, Wnoise=s["Wnoise"], noise=s["noise"],
                        act=moe.MX4_ACT_BF16 if case["act"] == "bf16" else moe.MX4_ACT_MX4)
    return {n: s[n] for n in ("y", "topk_idx", "topk_w", "counts", "importance", "P", "loss")}


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ------------------------------------------------------------------------- in 64 bits
def _exact_mx4(x):
    """mx4 values of x [rows][K] in 64 bits, by comparison with the midpoints between codes:
    a tie goes to the code of even index."""
    K = x.shape[1]
    v = torch.zeros(x.shape[0], _up(K, BLOCK), dtype=torch.float64, device=x.device)
    v[:, :K] = x
    v = v.view(x.shape[0], -1, BLOCK)
    top = v.abs().max(2, keepdim=True)[0]
    e = torch.where(top > 0, torch.frexp(top)[1] - 1, -125).clamp(min=-125) - 2
    unit = torch.exp2(e.double())
    code = torch.zeros(v.shape, dtype=torch.int8, device=x.device)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += v.abs() > mid * unit if i % 2 == 0 else v.abs() >= mid * unit
    value = torch.tensor(_TABLE[:8], dtype=torch.float64, device=x.device)[code.int()] * unit
    return torch.where(v < 0, -value, value).view(x.shape[0], -1)[:, :K]


def _exact_matrix(codes, scales, g, rows):
    """Matrix g of an mx4 batch in 64 bits, read from its bytes by the layout's definition."""
    c = codes[g]
    K = 2 * c.shape[1]
    col = torch.arange(K, device=c.device)
    nib = torch.where(col % 2 == 0, c[:, col // 2] & 15, c[:, col // 2] >> 4).int()
    r = torch.arange(rows, device=c.device).view(-1, 1)
    b = (col // BLOCK).view(1, -1)
    tk = scales.shape[2]
    at = ((r // 128) * tk + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    s = scales[g].reshape(-1)[at].double()
    return torch.tensor(_TABLE, dtype=torch.float64, device=c.device)[nib] * torch.exp2(s - 127)


def _exact_expert(s, e, rows, m, d, quantised):
    m16 = _up(m, 16)
    w = _exact_matrix(s["W13_q"], s["W13_s"], e, 2 * m16)
    n = torch.arange(m, device=w.device)
    gate = n // 16 * 32 + n % 16
    g, u = rows @ w[gate].T, rows @ w[gate + 16].T
    h = g * torch.sigmoid(g) * u
    h = _exact_mx4(h) if quantised else h
    return h @ _exact_matrix(s["W2_q"], s["W2_s"], e, d)[:, :m].T


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        K = case["K"]
        v = [_exact_mx4(a.double()) for a in s["src"]]
        return {"values": torch.stack(v).view(case["G"], case["rows"], K)}
    T, E, k, m, d = (case[n] for n in ("T", "E", "k", "m", "d"))
    x = s["x"].double()
    if case["op"] == "ffn":
        x = _exact_mx4(x)
        out = torch.zeros(T * k, d, dtype=torch.float64, device=x.device)
        for e in range(E):
            t, j = torch.nonzero((s["topk_idx"] == e) & (s["slot_row"] >= 0), as_tuple=True)
            if len(t):
                out[s["slot_row"][t, j].long()] = _exact_expert(s, e, x[t], m, d, True)
        return {"out": out}
    H = torch.einsum("td,de->te", x, s["Wg"].double())
    if case["noisy"]:
        H = H + s["noise"].double() * torch.nn.functional.softplus(
            torch.einsum("td,de->te", x, s["Wnoise"].double()))
    p = torch.softmax(H, 1)
    left, idx = H.clone(), []
    for _ in range(k):  # the largest that is left; of equals the first
        best = torch.argmax(left, 1)
        idx.append(best)
        left[torch.arange(T, device=x.device), best] = -float("inf")
    idx = torch.stack(idx, 1)
    picked = H.gather(1, idx)
    G = torch.softmax(picked, 1) if case["router"] == "mixtral" else p.gather(1, idx)
    y = torch.zeros(T, d, dtype=torch.float64, device=x.device)
    importance = torch.zeros(E, dtype=torch.float64, device=x.device)
    rows = _exact_mx4(x) if case["act"] == "mx4" else x
    share = torch.zeros(E, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        share[e] = len(t) / (T * k)
        if len(t):
            importance[e] = G[t, j].sum()
            y[t] += G[t, j].unsqueeze(1) * _exact_expert(s, e, rows[t], m, d, case["act"] == "mx4")
    y = y * (E / k if case["rescale"] else 1.0)
    P = p.sum(0) / T
    return {"y": y, "topk_idx": None, "topk_w": G, "counts": None, "importance": importance, "P": P,
            "loss": (0.01 * share @ P).view(1)}
