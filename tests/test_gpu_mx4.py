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
