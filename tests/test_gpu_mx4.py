"""The mx4 kernels against the plain format in 64 bits: quantisation and the row dispatch
bit for bit."""
import numpy as np
import pytest
import torch

import mx4_plain as mp
import top_routing_grouped_noisy_b200 as moe

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _matrix(G, rows, K, dtype, seed, spread=20):
    """Values over many octaves, zero blocks, ties and saturating values among them."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(G, rows, K, generator=g) * torch.exp2(
        torch.randint(-spread, spread + 1, (G, rows, (K + 31) // 32), generator=g).float()
    ).repeat_interleave(32, -1)[..., :K]
    pick = torch.rand(v.shape, generator=g)
    grid = torch.randint(-16, 17, v.shape, generator=g) * 0.25  # ties between codes
    v = torch.where(pick < 0.2, grid, v)
    v[:, rows // 2, : 32] = 0
    return v.to(DT[dtype])


def _check_batch(src, codes, scales):
    G, rows, K = src.shape
    nb = (K + 31) // 32
    tr, tk = (rows + 127) // 128, (K + 127) // 128
    got = mp.unpack_codes(codes)
    t = scales.reshape(G, tr, tk, 512)
    for g in range(G):
        c, b = mp.quantize(mp.f64(src[g]))
        np.testing.assert_array_equal(got[g], c)
        # every byte of the tiles: zeros past the rows and the blocks
        full = np.zeros((tr * 128, tk * 4), np.uint8)
        full[:rows, :nb] = b
        np.testing.assert_array_equal(mp.scale_bytes(t[g], tr * 128, tk * 4), full)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,rows,K", [(1, 1, 8), (1, 1, 32), (2, 3, 40), (1, 37, 200),
                                      (3, 128, 128), (2, 129, 160), (1, 257, 1376), (1, 5, 8192)])
def test_quantize_exact(G, rows, K, dtype):
    src = _matrix(G, rows, K, dtype, 7 * rows + K).cuda()
    codes = torch.full((G, rows, (K + 31) // 32 * 16), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((G, (rows + 127) // 128, (K + 127) // 128, 32, 4, 4), 0xAA,
                        dtype=torch.uint8, device="cuda")
    moe.moe_mx4_quantize(src, out=(codes, scales))
    _check_batch(src, codes, scales)
    for out_dtype in DT:
        back = moe.moe_mx4_dequantize(codes, scales, K, dtype=DT[out_dtype])
        np.testing.assert_array_equal(mp.f64(back), mp.matrix_values(codes, scales)[..., :K])


def test_quantize_edges():
    """Infinities, NaN, the largest and smallest values of the type."""
    src = torch.zeros(1, 8, 64)
    src[0, 0, 3] = float("inf")
    src[0, 1, 40] = float("nan")
    src[0, 2, :4] = torch.tensor([3.0e38, -3.4e38, 1.0, 2.0e37])
    src[0, 3, :3] = torch.tensor([1e-38, 1e-40, 3e-39])  # subnormal in f32
    src[0, 4, 33] = 1e-45
    src[0, 5, :2] = torch.tensor([2.0 ** -125, 2.0 ** -127])
    src[0, 6, :2] = torch.tensor([-0.0, 0.0])
    src = src.cuda()
    codes, scales = moe.moe_mx4_quantize(src)
    _check_batch(src, codes, scales)
    for dt in DT.values():
        back = mp.f64(moe.moe_mx4_dequantize(codes, scales, 64, dtype=dt))
        assert np.isnan(back[0, 0, :32]).all() and np.isnan(back[0, 1, 32:]).all()
        ref = mp.matrix_values(codes, scales)
        np.testing.assert_array_equal(back, ref)
    # a second pass over the values changes nothing
    again = moe.moe_mx4_quantize(moe.moe_mx4_dequantize(codes, scales, 64))
    ok = ~np.isnan(ref)
    np.testing.assert_array_equal(mp.matrix_values(*again)[ok], ref[ok])


def test_quantize_spaced_rows_and_streams():
    """Rows spaced ld apart, columns between them untouched; on another stream."""
    wide = _matrix(1, 2 * 50, 96, "bf16", 3).cuda().view(2, 50, 96)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        codes, scales = moe.moe_mx4_quantize(wide[..., :72])
        out = torch.full((2, 50, 96), 7.0, device="cuda", dtype=torch.bfloat16)
        moe.moe_mx4_dequantize(codes, scales, 72, out=out[..., :72])
    s.synchronize()
    _check_batch(wide[..., :72].contiguous(), codes, scales)
    np.testing.assert_array_equal(mp.f64(out[..., :72]), mp.matrix_values(codes, scales)[..., :72])
    assert (out[..., 72:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,cap", [(1, 32, 1, 1, -1), (7, 96, 4, 2, -1), (300, 160, 8, 2, -1),
                                         (300, 160, 8, 2, 20), (257, 64, 16, 4, 0), (130, 4096, 3, 3, 97)])
def test_dispatch_rows(T, d, E, k, cap, dtype):
    """The kept rows hold their token's mx4 row; everything else keeps what it held."""
    x = _matrix(1, T, d, dtype, T + d)[0].cuda()
    g = torch.Generator().manual_seed(T)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32).contiguous()
    idx[T // 2, 0] = E + 3  # an index outside is dropped
    idx = idx.cuda()
    p = moe.params(T, d, E, k, 32, dtype=DT[dtype], capacity=cap)
    ws = moe.Workspace(p)
    i32 = dict(dtype=torch.int32, device="cuda")
    row_token, slot = torch.empty(T * k, **i32), torch.empty(T, k, **i32)
    counts, kept, off = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
    moe.moe_dispatch_rows(p, idx, ws, row_token, slot, counts, kept, off)
    x_q = torch.full((moe.moe_mx4_rows_bytes(p, d),), 0xAA, dtype=torch.uint8, device="cuda")
    x_s = torch.full((moe.moe_mx4_row_scales_bytes(p, d),), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_mx4_dispatch(p, x, idx, slot, off, x_q, x_s)
    off, rt = off.cpu().numpy(), row_token.cpu().numpy()
    R = int(off[-1])
    c, b = mp.quantize(mp.f64(x))
    ref = mp.values(c, b)
    np.testing.assert_array_equal(mp.rows_values(x_q, x_s, d, off)[:, :d], ref[rt[:R]])
    assert (x_q.view(T * k, -1)[R:] == 0xAA).all()
    # scale bytes: the rows' words and no others
    tk = (d + 127) // 128
    t = x_s.view(-1, tk, 512).cpu().numpy().copy()
    for e in range(E):
        n = int(off[e + 1] - off[e])
        for r in range(n):
            at = (r % 32) * 16 + r % 128 // 32 * 4
            w = t[off[e] // 128 + e + r // 128, :, at:at + 4]
            full = np.zeros(tk * 4, np.uint8)
            full[: d // 32] = b[rt[off[e] + r]]
            np.testing.assert_array_equal(w.reshape(-1), full)
            w[:] = 0xAA
    assert (t == 0xAA).all()


# --------------------------------------------------------------------------- experts

def _experts(E, m, d, seed, spread=3):
    """mx4 experts with scales over several octaves; values exactly as stored (f64)."""
    g = torch.Generator().manual_seed(seed)
    m16, m8 = mp.up(m, 16), mp.up(m, 8)

    def draw(rows, K):
        v = torch.randn(E, rows, K, generator=g) / K ** 0.5
        return v * torch.exp2(torch.randint(-spread, spread + 1, (E, rows, 1), generator=g).float())

    w13 = torch.zeros(E, m16 // 16, 2, 16, d)
    w1, w3 = draw(m16, d), draw(m16, d)
    w1[:, m:], w3[:, m:] = 0, 0
    w13[:, :, 0], w13[:, :, 1] = w1.view(E, -1, 16, d), w3.view(E, -1, 16, d)
    w2 = torch.zeros(E, d, m8)
    w2[:, :, :m] = draw(d, m)
    W = moe.Mx4Experts.quantize(w13.cuda(), w2.cuda(), E, m, d)
    v13 = mp.matrix_values(W.W13_q, W.W13_s).reshape(E, m16 // 16, 2, 16, d)
    v2 = mp.matrix_values(W.W2_q, W.W2_s)[:, :, :m]
    return W, v13[:, :, 0].reshape(E, m16, d)[:, :m], v13[:, :, 1].reshape(E, m16, d)[:, :m], v2


class _Routed:
    """A routed batch with its mx4 rows; idx [T][k] on the host."""

    def __init__(self, idx, x, E, m, cap=-1):
        T, k = idx.shape
        d = x.shape[1]
        self.p = moe.params(T, d, E, k, m, capacity=cap)
        self.ws = moe.Workspace(self.p)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.x, self.idx = x.cuda(), idx.to(torch.int32).cuda().contiguous()
        self.row_token, self.slot = torch.empty(T * k, **i32), torch.empty(T, k, **i32)
        counts, kept, off = torch.empty(E, **i32), torch.empty(E, **i32), torch.empty(E + 1, **i32)
        moe.moe_dispatch_rows(self.p, self.idx, self.ws, self.row_token, self.slot, counts, kept, off)
        fill = lambda n: torch.full((n,), 0xAA, dtype=torch.uint8, device="cuda")
        self.x_q, self.x_s = (fill(moe.moe_mx4_rows_bytes(self.p, d)),
                              fill(moe.moe_mx4_row_scales_bytes(self.p, d)))
        # scales past the rows read as NaN (255): they may not reach a kept row
        self.x_s.fill_(255)
        moe.moe_mx4_dispatch(self.p, self.x, self.idx, self.slot, off, self.x_q, self.x_s)
        self.h_q, self.h_s = (fill(moe.moe_mx4_rows_bytes(self.p, m)),
                              fill(moe.moe_mx4_row_scales_bytes(self.p, m)))
        self.h_s.fill_(255)
        self.out = torch.full((T * k, d), 7.0, dtype=torch.bfloat16, device="cuda")
        self.offsets, self.off = off, off.cpu().numpy()
        self.R = int(self.off[-1])

    def rows(self):
        return mp.rows_values(self.x_q, self.x_s, self.p.d, self.off)


def _acc_bound(K):
    """Bound of an f32 accumulation of K products relative to the sum of their
    magnitudes: at most K/64 + 64 additions follow one another, each off by 2^-23 (a
    truncating adder) of a partial sum no larger than that sum."""
    return (K / 64 + 64) * 2.0 ** -23


def _quantize_with(v, s):
    """v [..][32] on the grid of exponent s [..]: nearest, ties to even, saturating."""
    step = np.exp2(s.astype(np.float64))[..., None]
    a = np.abs(v) / step
    st = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.sign(v) * np.minimum(np.rint(a / st) * st, 6.0) * step


def _check_up(rt, w1, w3, m):
    """Every h code is the rounding of a value within the f32 accumulation bound of the
    64-bit h, every scale that of a maximum within it, and few differ from the 64-bit
    quantisation itself."""
    x, k32 = rt.rows(), mp.up(m, 32)
    d = x.shape[1]
    got = mp.rows_values(rt.h_q, rt.h_s, m, rt.off)
    differ = total = 0
    tk = mp.up(m, 128) // 128
    tiles = rt.h_s.view(-1, tk, 512)
    for e in range(len(w1)):
        a, b = int(rt.off[e]), int(rt.off[e + 1])
        if a == b:
            continue
        xs = x[a:b]
        g, u = xs @ w1[e].T, xs @ w3[e].T
        sg, su = np.abs(xs) @ np.abs(w1[e]).T, np.abs(xs) @ np.abs(w3[e]).T
        sig = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
        h = g * sig * u
        # |silu'| <= 1.1; the exponential, quotient and products add a few ulps
        err = _acc_bound(d) * (1.1 * sg * np.abs(u) + np.abs(g * sig) * su) * 1.01 \
            + (8 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(h) + 1e-37
        pad = lambda z: np.pad(z, ((0, 0), (0, k32 - m))).reshape(b - a, -1, 32)
        h3, e3, v3 = pad(h), pad(err), got[a:b].reshape(b - a, -1, 32)
        bytes_ = mp.scale_bytes(tiles, b - a, k32 // 32, a // 128 + e).astype(int)
        s = bytes_ - 127
        for sign in (-1, 1):  # the scale is that of a maximum inside the bound
            top = np.maximum(np.abs(h3) + sign * e3, 0).max(-1)
            lim = np.where(top > 0, np.maximum(np.floor(np.log2(np.maximum(top, 1e-300))) - 2, -127), -127)
            assert (sign * (lim - s) >= 0).all()
        lo, hi = _quantize_with(h3 - e3, s), _quantize_with(h3 + e3, s)
        assert (v3 >= lo).all() and (v3 <= hi).all()
        # bytes of the scale word past the last block are zero
        rest = mp.scale_bytes(tiles, b - a, tk * 4, a // 128 + e)[:, k32 // 32:]
        assert (rest == 0).all()
        c, sb = mp.quantize(h)
        differ += (mp.values(c, sb) != got[a:b]).sum()
        total += h.size
    assert differ <= 0.01 * total + 2, (differ, total)


def _check_down(rt, v2, m):
    h = mp.rows_values(rt.h_q, rt.h_s, m, rt.off)[:, :m]
    got = mp.f64(rt.out)
    for e in range(len(v2)):
        a, b = int(rt.off[e]), int(rt.off[e + 1])
        ref = h[a:b] @ v2[e].T
        tol = 2.0 ** -8 * np.abs(ref) + _acc_bound(m) * (np.abs(h[a:b]) @ np.abs(v2[e]).T) + 1e-37
        assert (np.abs(got[a:b] - ref) <= tol).all()
    assert (got[rt.R:] == 7.0).all() and (rt.h_q.view(len(got), -1)[rt.R:] == 0xAA).all()


EXPERT_CASES = [  # T, E, k, m, d, capacity
    (1, 1, 1, 16, 32, -1), (1, 4, 2, 64, 64, -1), (3, 2, 1, 24, 96, -1), (5, 3, 3, 100, 160, -1),
    (64, 4, 2, 172, 512, -1), (129, 1, 1, 96, 256, -1), (200, 8, 2, 344, 288, -1),
    (300, 5, 2, 130, 224, 50), (700, 3, 2, 200, 1024, -1), (40, 64, 8, 48, 128, -1),
    (256, 2, 1, 1376, 320, -1),
    # thousands of rows: wider tiles, one or several of them, ragged ends
    (4096, 1, 1, 64, 96, -1), (2100, 3, 2, 200, 320, -1), (1500, 8, 3, 136, 544, 450),
    (2300, 5, 2, 400, 288, -1), (1100, 16, 4, 260, 64, 290),
    # the second product's K in one to six blocks of 256, and in more
    (2048, 4, 2, 768, 576, -1), (2100, 2, 2, 1504, 320, -1), (2060, 3, 2, 1568, 160, -1),
]


@pytest.mark.parametrize("T,E,k,m,d,cap", EXPERT_CASES)
def test_expert_ffn(T, E, k, m, d, cap):
    g = torch.Generator().manual_seed(T * 31 + m)
    x = (torch.randn(T, d, generator=g) * torch.exp2(
        torch.randint(-4, 5, (T, 1), generator=g).float())).bfloat16()
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    W, w1, w3, w2 = _experts(E, m, d, T + d)
    rt = _Routed(idx, x, E, m, cap)
    moe.moe_expert_up_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q, rt.h_s, rt.ws)
    _check_up(rt, w1, w3, m)
    moe.moe_expert_down_mx4(rt.p, rt.h_q, rt.h_s, rt.offsets, W, rt.out, rt.ws)
    _check_down(rt, w2, m)
    out = rt.out.clone()
    rt.out.fill_(7.0)
    moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q, rt.h_s, rt.out, rt.ws)
    assert torch.equal(rt.out, out)
    assert moe.moe_get_device_status(rt.ws) == 0


MORE_CASES = [
    # rows enough for the CTA-pair kernels, most of them dropped so that the tiles are ragged:
    # K of the first product in 1, 2, 4 and more blocks of 256, of the second (A resident) in
    # 2 to 6, and in more (A streamed)
    (16000, 5, 4, 500, 96, 333), (16000, 2, 2, 500, 320, 1000), (12000, 3, 3, 360, 800, 300),
    (6000, 2, 2, 700, 800, 511), (6000, 2, 2, 1000, 800, 700), (4100, 2, 2, 1270, 800, 257),
    (2300, 2, 2, 1500, 1600, 900), (4100, 2, 2, 1600, 800, 600), (1700, 2, 2, 1000, 2336, -1),
    # experts in more than one row of 32, and more than 8
    (12000, 40, 4, 700, 1056, 70), (9000, 12, 2, 1000, 1600, 300),
    # nothing kept
    (9000, 12, 2, 1000, 1600, 0), (64, 4, 2, 64, 96, 0),
    # one neuron
    (5, 2, 1, 1, 32, -1),
]


@pytest.mark.parametrize("T,E,k,m,d,cap", MORE_CASES)
def test_expert_ffn_more(T, E, k, m, d, cap):
    test_expert_ffn(T, E, k, m, d, cap)


@pytest.mark.parametrize("T,m,d", [(40, 64, 128), (8000, 700, 1056)])
def test_expert_offsets_out_of_range(T, m, d):
    """Offsets that no dispatch writes are reported; nothing outside the buffers is touched."""
    g = torch.Generator().manual_seed(T)
    E, k = 4, 2
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    W = _experts(E, m, d, T)[0]
    rt = _Routed(idx, torch.randn(T, d, generator=g).bfloat16(), E, m)
    n, guard = T * k * d, 1 << 16
    big = torch.full((n + 2 * guard,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[guard:guard + n].view(T * k, d)
    for bad in ([0, T * k // 2, 5, 9, T * k], [-300, 3, 4, T, 2 ** 31 - 1], [T * k + 999] * 5):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda: moe.moe_expert_up_mx4(rt.p, rt.x_q, rt.x_s, off, W, rt.h_q, rt.h_s, rt.ws),
                     lambda: moe.moe_expert_down_mx4(rt.p, rt.h_q, rt.h_s, off, W, out, rt.ws)):
            call()
            assert moe.moe_get_device_status(rt.ws) == moe.MOE_ERR_DEVICE_BADINDEX
        assert (big[:guard] == 7).all() and (big[guard + n:] == 7).all()
    # falling offsets count as the largest before them: rows T*k/2.. of expert 3 alone
    rt.h_q.fill_(0xAA)
    rt.out.fill_(7.0)
    off = torch.tensor([0, 0, 0, T * k // 2, T * k // 4], dtype=torch.int32, device="cuda")
    moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, off, W, rt.h_q, rt.h_s, rt.out, rt.ws)
    assert moe.moe_get_device_status(rt.ws) == moe.MOE_ERR_DEVICE_BADINDEX
    assert (rt.out[T * k // 2:] == 7).all() and (rt.h_q.view(T * k, -1)[T * k // 2:] == 0xAA).all()
    moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q, rt.h_s, rt.out, rt.ws)
    assert moe.moe_get_device_status(rt.ws) == 0


def test_dispatch_slots_out_of_range():
    """Slots and offsets outside the buffers are skipped."""
    T, E, k, d = 33, 4, 2, 96
    p = moe.params(T, d, E, k, 32)
    nq, ns, pad = moe.moe_mx4_rows_bytes(p, d), moe.moe_mx4_row_scales_bytes(p, d), 1 << 16
    q = torch.full((nq + 2 * pad,), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((ns + 2 * pad,), 0xAA, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.ones(T, d, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(T, k, **i32)
    slot = torch.tensor([T * k, T * k + 5, 2 ** 31 - 1, -7, 3], **i32).repeat(14)[: T * k].view(T, k)
    for off in ([4] * 5, [-9] * 5):  # row 3 lies before its expert's offset, or that below 0
        moe.moe_mx4_dispatch(p, x, idx, slot.contiguous(), torch.tensor(off, **i32),
                             q[pad:pad + nq], s[pad:pad + ns])
        assert (q == 0xAA).all() and (s == 0xAA).all()


@pytest.mark.parametrize("T,m,d", [(7, 96, 256), (300, 172, 512), (6000, 500, 800)])
def test_weights_rewritten_right_before(T, m, d):
    """Weights quantised on the same stream right before the products, eager and replayed: the
    second product's early loads read the new ones."""
    g = torch.Generator().manual_seed(T)
    E, k = 4, 2
    m16, m8 = mp.up(m, 16), mp.up(m, 8)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    rt = _Routed(idx, torch.randn(T, d, generator=g).bfloat16(), E, m)
    ffn = lambda W, out: moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q,
                                                rt.h_s, out, rt.ws)
    src, refs = [], []
    for seed in range(3):
        gg = torch.Generator(device="cuda").manual_seed(seed)
        w13 = torch.randn(E, 2 * m16, d, generator=gg, device="cuda").bfloat16()
        w2 = torch.randn(E, d, m8, generator=gg, device="cuda").bfloat16()
        W = moe.Mx4Experts.quantize(w13, w2, E, m, d)
        torch.cuda.synchronize()
        out = torch.empty_like(rt.out)
        ffn(W, out)
        torch.cuda.synchronize()
        src.append((w13, w2))
        refs.append(out)
    w13, w2 = (t.clone() for t in src[0])
    W = moe.Mx4Experts.quantize(w13, w2, E, m, d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        def step():
            moe.moe_mx4_quantize(w13, out=(W.W13_q, W.W13_s))
            moe.moe_mx4_quantize(w2, out=(W.W2_q, W.W2_s))
            ffn(W, rt.out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
        for run in (step, graph.replay):
            for _ in range(4):
                for (a, b), ref in zip(src, refs):
                    w13.copy_(a)
                    w2.copy_(b)
                    run()
                    assert torch.equal(rt.out[: rt.R], ref[: rt.R])
    st.synchronize()
    assert moe.moe_get_device_status(rt.ws) == 0


@pytest.mark.parametrize("T,m,d", [(40, 96, 256), (8000, 700, 1056)])
def test_expert_ffn_nan_token(T, m, d):
    """A NaN or an infinity in a token's row stays with that token."""
    g = torch.Generator().manual_seed(T)
    E, k = 4, 2
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    W = _experts(E, m, d, T)[0]
    x = torch.randn(T, d, generator=g).bfloat16()
    outs = []
    for bad in (False, True):
        if bad:
            x[7, 5], x[T - 1, d - 1] = float("nan"), float("-inf")
        rt = _Routed(idx, x, E, m)
        moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q, rt.h_s, rt.out, rt.ws)
        outs.append(rt.out.clone())
    hit = (rt.row_token == 7) | (rt.row_token == T - 1)
    assert torch.isnan(outs[1][hit]).all() and int(hit.sum()) == 2 * k
    assert torch.equal(outs[0][~hit], outs[1][~hit])


def test_two_streams_at_once():
    """Calls on two streams with a workspace each, in flight together."""
    layers = [_Layer(T=16, E=8, k=2, m=344, d=1024, seed=s) for s in range(2)]
    acts = (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4)
    refs = [[L.run(a).y.clone() for a in acts] for L in layers]
    bufs = [[[moe.Mx4Buffers(L.p, act=a) for _ in range(6)] for a in acts] for L in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for i in range(6):
        for n, (L, st) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(st):
                for a, b in zip(acts, bufs[n]):
                    L.run(a, b[i])
    torch.cuda.synchronize()
    for n, L in enumerate(layers):
        for ref, b in zip(refs[n], bufs[n]):
            assert all(torch.equal(c.y, ref) for c in b)
        assert moe.moe_get_device_status(L.ws) == 0


LIMIT_NS = 2_000_000_000


def _cold():
    """Nothing in L2, so that the first waits are long."""
    torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,E,m,d", [(40, 2, 96, 512), (2000, 64, 688, 4096), (16000, 8, 1376, 4096)])
def test_expert_wait_limit(T, E, m, d):
    """With a wait limit of 0 the products give up at a wait that is not over at its second
    look (the larger batches have such waits), report it and return: either that or the
    output is whole.  The next are right."""
    g = torch.Generator(device="cuda").manual_seed(T)
    k = 2
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].cpu()
    W = moe.Mx4Experts.quantize(
        torch.randn(E, 2 * mp.up(m, 16), d, generator=g, device="cuda").bfloat16(),
        torch.randn(E, d, mp.up(m, 8), generator=g, device="cuda").bfloat16(), E, m, d)
    rt = _Routed(idx, torch.randn(T, d, generator=g, device="cuda").bfloat16(), E, m)
    ffn = lambda: moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, W, rt.h_q, rt.h_s,
                                         rt.out, rt.ws)
    ffn()
    ref = rt.out.clone()
    assert moe.moe_get_device_status(rt.ws) == 0
    _cold()
    moe.moe_set_wait_limit_ns(0)
    try:
        ffn()
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(LIMIT_NS)
    status = moe.moe_get_device_status(rt.ws)
    assert status == moe.MOE_ERR_DEVICE_TIMEOUT or (status == 0 and torch.equal(rt.out, ref))
    ffn()
    assert torch.equal(rt.out, ref) and moe.moe_get_device_status(rt.ws) == 0


# --------------------------------------------------------------------------- the layer
import types  # noqa: E402

import harness as H  # noqa: E402


class _Layer:
    def __init__(self, T, E, k, m, d, noisy=False, router=moe.MIXTRAL, cap=-1, rescale=True,
                 bias=False, seed=0):
        g = torch.Generator().manual_seed(1000 + seed + 17 * T + d)
        self.w = types.SimpleNamespace(T=T, E=E, k=k, m=m, d=d, router=router, lam=0.01)
        r = lambda *s: torch.randn(*s, generator=g)
        self.inp = {"x": r(T, d).bfloat16(), "Wg": (r(d, E) * 0.05).bfloat16(),
                    "Wnoise": (r(d, E) * 0.05).bfloat16() if noisy else None,
                    "eps": r(T, E) if noisy else None, "bias": r(E) if bias else None}
        self.W, self.w1, self.w3, self.w2 = _experts(E, m, d, seed + T + d)
        self.p = moe.params(T, d, E, k, m, router_type=router, capacity=cap, rescale=rescale,
                            balance_lambda=0.01)
        self.ws = moe.Workspace(self.p)
        self.dev = {n: None if v is None else v.cuda() for n, v in self.inp.items()}
        self.scale = E / k if rescale else 1.0

    def run(self, act, bufs=None, **kw):
        bufs = moe.Mx4Buffers(self.p, act=act) if bufs is None else bufs
        v = self.dev
        moe.moe_forward_mx4(self.p, v["x"], v["Wg"], self.W, self.ws, bufs, act=act,
                            Wnoise=v["Wnoise"], noise=v["eps"], bias=v["bias"], **kw)
        return bufs

    def check_tables(self, b):
        """Routing against the oracle, the tables against a stable sort of the indices."""
        r, _ = H.check_routing(self.w, self.inp, b, 5e-5)
        import oracle
        d = oracle.dispatch(b.topk_idx.cpu().numpy(), self.w.E, self.p.capacity)
        for n in ("counts", "kept", "offsets", "slot_row"):
            np.testing.assert_array_equal(getattr(b, n).cpu().numpy(), d[n])
        np.testing.assert_array_equal(b.row_token.cpu().numpy()[: d["R"]], d["row_token"])
        T, k = self.w.T, self.w.k
        np.testing.assert_allclose(b.f.cpu().numpy(), d["counts"] / (T * k), rtol=1e-6)
        np.testing.assert_allclose(b.P.cpu().numpy(), b.probs_sum.cpu().numpy() / T, rtol=1e-6)
        H.check_loss(self.w, b, r)
        return d

    def combine(self, out, b, d):
        """y from expert rows `out` and the kernel's own gate weights, and sum |.|."""
        G, slot = mp.f64(b.topk_w), d["slot_row"]
        rows = np.where((slot >= 0)[..., None], out[np.maximum(slot, 0)], 0.0) if len(out) else \
            np.zeros((*slot.shape, self.w.d))
        terms = self.scale * G[..., None] * rows
        return terms.sum(1), np.abs(terms).sum(1)


def _check_few(L, b):
    d = L.check_tables(b)
    w, off, R = L.w, d["offsets"], d["R"]
    x = mp.f64(L.inp["x"])
    h = mp.f64(b.h)[:R, : w.m]
    out, mag = np.zeros((R, w.d)), np.zeros((R, w.d))
    for e in range(w.E):
        rows = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        xs = x[d["row_token"][rows]]
        g, u = xs @ L.w1[e].T, xs @ L.w3[e].T
        # activations scaled into f16: off by at most 2^-38 of the row's maximum each
        tiny = 2.0 ** -38 * np.abs(xs).max(1, keepdims=True)
        eg = _acc_bound(w.d) * (np.abs(xs) @ np.abs(L.w1[e]).T) + tiny * np.abs(L.w1[e]).sum(1)
        eu = _acc_bound(w.d) * (np.abs(xs) @ np.abs(L.w3[e]).T) + tiny * np.abs(L.w3[e]).sum(1)
        s = g / (1 + np.exp(-g))
        ref = s * u
        tol = 1.1 * eg * np.abs(u) + np.abs(s) * eu + eg * eu + \
            (2.0 ** -8 + (8 + 1.2 * np.abs(g)) * 2.0 ** -23) * np.abs(ref) + 1e-37
        assert (np.abs(h[rows] - ref) <= tol * 1.02).all()
        hs = h[rows]
        out[rows] = hs @ L.w2[e].T
        tiny = 2.0 ** -38 * np.abs(hs).max(1, keepdims=True)
        mag[rows] = _acc_bound(w.m) * (np.abs(hs) @ np.abs(L.w2[e]).T) + tiny * np.abs(L.w2[e]).sum(1)
    y, top = L.combine(out, b, d)
    err, _ = L.combine(mag, b, d)
    tol = 2.0 ** -8 * np.abs(y) + np.abs(err) + (w.k + 2) * 2.0 ** -24 * top + 1e-37
    assert (np.abs(mp.f64(b.y) - y) <= tol * 1.02).all()
    assert moe.moe_get_device_status(L.ws) == 0


FEW_CASES = [
    dict(T=1, E=1, k=1, m=16, d=32), dict(T=1, E=8, k=2, m=64, d=256),
    dict(T=3, E=6, k=3, m=172, d=512, noisy=True, router=moe.ST),
    dict(T=8, E=8, k=2, m=344, d=1024, cap=1), dict(T=9, E=16, k=4, m=100, d=320, noisy=True, bias=True),
    dict(T=16, E=32, k=8, m=48, d=160, rescale=False), dict(T=16, E=4, k=2, m=40, d=96, cap=0),
    dict(T=5, E=5, k=1, m=1000, d=64), dict(T=13, E=3, k=3, m=72, d=8192),
    dict(T=16, E=2, k=2, m=5000, d=64), dict(T=7, E=12, k=5, m=24, d=4096, noisy=True),
    dict(T=2, E=24, k=8, m=130, d=736, router=moe.ST), dict(T=2, E=2, k=1, m=1, d=32),
]


@pytest.mark.parametrize("case", FEW_CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_layer_few(case):
    L = _Layer(**case)
    b = moe.Mx4Buffers(L.p, act=moe.MX4_ACT_BF16)
    for t in (b.y, b.h):
        t.fill_(float("nan"))
    L.run(moe.MX4_ACT_BF16, b)
    _check_few(L, b)
    y = b.y.clone()
    L.run(moe.MX4_ACT_BF16, b)  # the same bits again
    assert torch.equal(b.y.view(torch.int16), y.view(torch.int16))


def test_layer_few_nan_token():
    """A token whose logits are not finite is dropped (y = 0, status set); the others are
    what they are without it."""
    L = _Layer(T=4, E=4, k=2, m=64, d=128)
    good = L.run(moe.MX4_ACT_BF16).y.clone()
    L.dev["x"][2, 5] = float("inf")
    L.dev["x"][2, 6] = float("nan")
    b = L.run(moe.MX4_ACT_BF16)
    assert moe.moe_get_device_status(L.ws) == moe.MOE_ERR_DEVICE_BADINDEX
    assert (b.topk_idx[2] == -1).all() and (b.y[2] == 0).all()
    for t in (0, 1, 3):
        assert torch.equal(b.y[t], good[t])


def test_layer_few_nan_weights():
    """A NaN scale reaches exactly the outputs whose weights it belongs to."""
    L = _Layer(T=3, E=2, k=2, m=32, d=128)
    L.W.W2_s.view(2, -1)[1, 5 * 16] = 255  # expert 1, W2 row 5, block 0
    b = L.run(moe.MX4_ACT_BF16)
    nan = torch.isnan(b.y)
    assert nan[:, 5].all() and nan.sum() == 3


@pytest.mark.parametrize("T,E,k,m,d,cap", [(1, 8, 2, 64, 256, -1), (40, 6, 3, 172, 512, 9),
                                           (300, 8, 2, 96, 160, -1), (33, 64, 8, 48, 128, -1)])
def test_layer_rows(T, E, k, m, d, cap):
    """MX4_ACT_MX4 is its steps: route, tables, mx4 dispatch, experts, combine."""
    L = _Layer(T=T, E=E, k=k, m=m, d=d, cap=cap, noisy=T % 2 == 0)
    b = L.run(moe.MX4_ACT_MX4)
    tab = L.check_tables(b)
    rt = _Routed(b.topk_idx.cpu(), L.inp["x"], E, m, cap)
    moe.moe_expert_ffn_mx4(rt.p, rt.x_q, rt.x_s, rt.offsets, L.W, rt.h_q, rt.h_s, rt.out, rt.ws)
    R = tab["R"]
    assert torch.equal(b.out[:R], rt.out[:R])
    _check_up(rt, L.w1, L.w3, m)
    _check_down(rt, L.w2, m)
    y, top = L.combine(mp.f64(b.out)[:R], b, tab)
    assert (np.abs(mp.f64(b.y) - y) <= 2.0 ** -8 * np.abs(y) + (k + 2) * 2.0 ** -24 * top + 1e-37).all()


@pytest.mark.parametrize("act", [moe.MX4_ACT_BF16, moe.MX4_ACT_MX4])
def test_layer_empty_batch(act):
    L = _Layer(T=1, E=4, k=2, m=32, d=64)
    p = moe.params(0, 64, 4, 2, 32, balance_lambda=0.01)
    b = moe.Mx4Buffers(p, act=None)
    moe.moe_forward_mx4(p, L.dev["x"][:0], L.dev["Wg"], L.W, L.ws, b, act=act)
    assert b.counts.tolist() == [0] * 4 and b.offsets.tolist() == [0] * 5 and b.loss.item() == 0


@pytest.mark.parametrize("act", [moe.MX4_ACT_BF16, moe.MX4_ACT_MX4])
def test_layer_graphs_and_streams(act):
    """Two captured graphs and eager calls that share the workspace, one after the other."""
    A, B = _Layer(T=5, E=8, k=2, m=96, d=256), _Layer(T=11, E=8, k=2, m=96, d=256)
    B.ws = A.ws = moe.Workspace(B.p)
    refs = [L.run(act).y.clone() for L in (A, B)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs, bufs = [], []
    with torch.cuda.stream(s):
        for L in (A, B):
            b = moe.Mx4Buffers(L.p, act=act)
            L.run(act, b)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                L.run(act, b)
            graphs.append(g)
            bufs.append(b)
        for _ in range(3):
            for g, b, L, ref in zip(graphs, bufs, (A, B), refs):
                b.y.fill_(float("nan"))
                g.replay()
                assert torch.equal(b.y, ref)
                assert torch.equal(L.run(act).y, ref)
    s.synchronize()
    assert moe.moe_get_device_status(A.ws) == 0


def test_layer_few_wait_limit():
    """The same for the grid barrier of the few-token layer."""
    L = _Layer(T=8, E=8, k=2, m=344, d=1024)
    ref = L.run(moe.MX4_ACT_BF16).y.clone()
    _cold()
    moe.moe_set_wait_limit_ns(0)
    try:
        y = L.run(moe.MX4_ACT_BF16).y
        torch.cuda.synchronize()
    finally:
        moe.moe_set_wait_limit_ns(LIMIT_NS)
    status = moe.moe_get_device_status(L.ws)
    assert status == moe.MOE_ERR_DEVICE_TIMEOUT or (status == 0 and torch.equal(y, ref))
    for _ in range(3):
        assert torch.equal(L.run(moe.MX4_ACT_BF16).y, ref)
    assert moe.moe_get_device_status(L.ws) == 0


@pytest.mark.parametrize("mode", [moe.DISJOINT, moe.STACKED])
def test_partition_quantize_and_serve(mode):
    """As a server uses them: expert weights from a dense FFN (or stacked experts), quantised
    once; a prompt through quantised rows, then decode steps with bf16 activations on the same
    workspace, each compared with moe_forward on the dequantised weights."""
    E, k, m, d, T = 8, 2, 96, 256, 200
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.06).bfloat16()
    if mode == moe.DISJOINT:
        W1, W3, W2 = r(E * m, d), r(E * m, d), r(d, E * m)
    else:
        W1, W3, W2 = r(E, m, d), r(E, m, d), r(E, d, m)
    p = moe.params(T, d, E, k, m, balance_lambda=0.01)
    ws = moe.Workspace(p)
    perm = torch.randperm(E * m, generator=g, device="cuda").int() if mode == moe.DISJOINT else None
    W13_e, W2_e = moe.moe_partition_experts(W1, W3, W2, E, mode=mode, perm=perm, ws=ws)
    W = moe.Mx4Experts.quantize(W13_e, W2_e, E, m, d)
    m16, m8 = mp.up(m, 16), mp.up(m, 8)
    D13 = moe.moe_mx4_dequantize(W.W13_q, W.W13_s, d).reshape(-1)
    D2 = moe.moe_mx4_dequantize(W.W2_q, W.W2_s, m8).reshape(-1)
    x, Wg = r(T, d) * 20, r(d, E)

    # the prompt: the layer is its public steps, one by one
    b = moe.Mx4Buffers(p, act=moe.MX4_ACT_MX4)
    moe.moe_forward_mx4(p, x, Wg, W, ws, b, act=moe.MX4_ACT_MX4)
    s = moe.Mx4Buffers(p, act=moe.MX4_ACT_MX4)
    moe.moe_route(p, x, Wg, None, None, None, ws, s.topk_idx, s.topk_w, s.probs_sum, s.importance)
    moe.moe_dispatch_rows(p, s.topk_idx, ws, s.row_token, s.slot_row, s.counts, s.kept, s.offsets)
    moe.moe_mx4_dispatch(p, x, s.topk_idx, s.slot_row, s.offsets, s.x_q, s.x_s)
    moe.moe_expert_up_mx4(p, s.x_q, s.x_s, s.offsets, W, s.h_q, s.h_s, ws)
    moe.moe_expert_down_mx4(p, s.h_q, s.h_s, s.offsets, W, s.out, ws)
    moe.moe_combine(p, s.out, s.slot_row, s.topk_w, s.y)
    assert torch.equal(b.y, s.y) and torch.equal(b.topk_idx, s.topk_idx)

    # decode steps of every small size: against the same weights in bf16
    v13 = mp.f64(D13).reshape(E, m16 // 16, 2, 16, d)
    v1, v3 = (v13[:, :, i].reshape(E, m16, d)[:, :m] for i in (0, 1))
    v2 = mp.f64(D2).reshape(E, d, m8)[:, :, :m]
    at = 0
    for n in (1, 2, 5, 8, 9, 16):
        q = moe.params(n, d, E, k, m, balance_lambda=0.01)
        xs = x[at:at + n].contiguous()
        at += n
        f = moe.Mx4Buffers(q, act=moe.MX4_ACT_BF16)
        moe.moe_forward_mx4(q, xs, Wg, W, ws, f)
        o = moe.ForwardBuffers(q)
        moe.moe_forward(q, xs, Wg, D13, D2, ws, o)
        assert torch.equal(f.topk_idx, o.topk_idx) and torch.equal(f.slot_row, o.slot_row)
        # both round h to bf16 (2^-8 each), moe_forward the expert outputs as well, and y twice
        X, G, I = mp.f64(xs), mp.f64(f.topk_w), f.topk_idx.cpu().numpy()
        y, tol = np.zeros((n, d)), np.zeros((n, d))
        for t in range(n):
            for j in range(k):
                e = I[t, j]
                gate, up = v1[e] @ X[t], v3[e] @ X[t]
                h = gate / (1 + np.exp(-gate)) * up
                acc = _acc_bound(d) * ((np.abs(v1[e]) @ np.abs(X[t])) * 1.1 * np.abs(up)
                                       + (np.abs(v3[e]) @ np.abs(X[t])) * np.abs(h / up))
                dh = 2 * (2.0 ** -8 + 2.0 ** -20) * np.abs(h) + 2.1 * acc
                o_ = v2[e] @ h
                y[t] += G[t, j] * o_
                tol[t] += G[t, j] * (np.abs(v2[e]) @ (dh + 2 * _acc_bound(m) * np.abs(h))
                                     + 2.0 ** -8 * np.abs(o_) * 1.1 + 2.0 ** -20 * np.abs(o_))
        y, tol = y * (E / k if q.rescale else 1), tol * (E / k if q.rescale else 1)
        tol += 2 * 2.0 ** -8 * (np.abs(y) + tol)
        assert (np.abs(mp.f64(f.y) - mp.f64(o.y)) <= tol).all()
        assert (np.abs(mp.f64(f.y) - y) <= tol).all()
    assert moe.moe_get_device_status(ws) == 0
