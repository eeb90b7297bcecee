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
