"""The microscaled 4-bit format in plain numpy and torch (64 bits), for the mx4 tests:
written from the format's definition, without the library."""
import numpy as np
import torch

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def up(v, n):
    return (v + n - 1) // n * n


def quantize(v):
    """v [rows][K] f64 -> (codes [rows][K32] 0..15, scale bytes [rows][K32 / 32]).  The
    scale exponent is floor(log2(max)) - 2, at least -127; the nearest code is found by
    comparing distances, a tie taking the even code."""
    rows, K = v.shape
    k32 = up(K, 32)
    x = np.zeros((rows, k32))
    x[:, :K] = v
    x = x.reshape(rows, -1, 32)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    top = np.abs(x).max(-1)
    e = np.frexp(np.where(top > 0, top, 1.0))[1] - 1  # floor(log2), exact
    s = np.where(top > 0, np.maximum(e - 2, -127), -127)
    a = np.abs(x) / np.exp2(s.astype(np.float64))[..., None]
    dist = np.abs(a[..., None] - CODES)
    near = dist.argmin(-1)  # the lower of two equally near codes
    tie = (near < 7) & (dist[..., :7] == dist[..., 1:]).any(-1)
    nxt = np.take_along_axis(dist, np.minimum(near + 1, 7)[..., None], -1)[..., 0]
    tie &= nxt == np.take_along_axis(dist, near[..., None], -1)[..., 0]
    near = near + (tie & (near % 2 == 1))
    near = np.where(a >= 6, 7, near)
    code = near + 8 * np.signbit(x)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255, s + 127)
    return code.reshape(rows, k32).astype(np.uint8), byte.astype(np.uint8)


def values(codes, bytes_):
    """f64 values of codes [rows][K32] and scale bytes [rows][K32 / 32]."""
    v = np.where(codes & 8, -1.0, 1.0) * CODES[codes & 7]
    s = np.where(bytes_ == 255, np.nan, np.exp2(bytes_.astype(np.float64) - 127))
    return (v.reshape(*s.shape, 32) * s[..., None]).reshape(v.shape)


def unpack_codes(q):
    """Library codes [..., K32 / 2] uint8 -> one code per element."""
    q = q.cpu().numpy()
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)


def scale_bytes(tiles, rows, nb, tile0=0):
    """Scale bytes [rows][nb] of the matrix that starts at tile row tile0; tiles
    [tile rows][tiles of a row][512] uint8 (flat 512-byte tiles)."""
    t = tiles.cpu().numpy()
    r, b = np.arange(rows)[:, None], np.arange(nb)[None, :]
    return t[tile0 + r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def matrix_values(codes, scales):
    """Library batch (codes [G][rows][K32/2], scales) -> f64 values [G][rows][K32]."""
    G, rows, half = codes.shape
    c = unpack_codes(codes)
    tr, tk = up(rows, 128) // 128, up(2 * half, 128) // 128
    t = scales.reshape(G, tr, tk, 512)
    return np.stack([values(c[g], scale_bytes(t[g], rows, 2 * half // 32)) for g in range(G)])


def rows_values(x_q, x_s, K, offsets):
    """Expert rows (x_q [T*k][K32/2], x_s flat bytes) -> f64 values [R][K32]."""
    k32, tk = up(K, 32), up(K, 128) // 128
    c = unpack_codes(x_q.reshape(-1, k32 // 2))
    t = x_s.reshape(-1, tk, 512)
    out = []
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        out.append(values(c[a:b], scale_bytes(t, b - a, k32 // 32, a // 128 + e)))
    return np.concatenate(out) if out else np.zeros((0, k32))


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()
