"""The mx4 calls without a GPU: sizes, refusals before anything reaches the device, the
plain format against hand-worked blocks, and the tile placement of ragged expert rows."""
import ctypes as C

import numpy as np
import pytest

import mx4_plain as mp
import top_routing_grouped_noisy_b200 as moe


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def _fake(i=0, off=0):
    return C.c_void_p(0x100000 + 4096 * i + off)


def test_sizes():
    assert moe.moe_mx4_codes_bytes(8, 2752, 4096) == 8 * 2752 * 2048
    assert moe.moe_mx4_codes_bytes(1, 3, 40) == 3 * 32
    assert moe.moe_mx4_scales_bytes(8, 2752, 4096) == 8 * 22 * 32 * 512
    assert moe.moe_mx4_scales_bytes(1, 129, 136) == 2 * 2 * 512
    for bad in ((0, 1, 32), (1, 0, 32), (1, 1, 0), (1, 1, 12)):
        assert moe.moe_mx4_codes_bytes(*bad) == 0 and moe.moe_mx4_scales_bytes(*bad) == 0
    p = moe.params(100, 64, 8, 2, 40)
    assert moe.moe_mx4_rows_bytes(p, 64) == 200 * 32
    assert moe.moe_mx4_rows_bytes(p, 40) == 200 * 32
    assert moe.moe_mx4_row_scales_bytes(p, 64) == (200 // 128 + 9) * 512
    assert moe.moe_mx4_rows_bytes(moe.params(0, 64, 8, 2, 40), 64) == 32
    assert moe.moe_mx4_rows_bytes(moe.params(4, 60, 8, 2, 40), 64) == 0


def test_quantize_refusals(L):
    f = [_fake(i) for i in range(3)]

    def q(src=f[0], dtype=moe.MOE_BF16, G=2, rows=3, K=64, ld=64, codes=f[1], scales=f[2]):
        return L.moe_mx4_quantize(src, dtype, G, rows, K, ld, codes, scales, None)

    def dq(codes=f[0], scales=f[1], dtype=moe.MOE_F32, G=2, rows=3, K=64, ld=64, dst=f[2]):
        return L.moe_mx4_dequantize(codes, scales, dtype, G, rows, K, ld, dst, None)

    for call in (q, dq):
        assert call(dtype=5) == moe.MOE_ERR_DTYPE
        assert call(G=0) == moe.MOE_ERR_INVALID_ARG
        assert call(rows=0) == moe.MOE_ERR_INVALID_ARG
        assert call(K=0) == moe.MOE_ERR_SHAPE
        assert call(K=60, ld=64) == moe.MOE_ERR_SHAPE
        assert call(ld=56) == moe.MOE_ERR_SHAPE
        assert call(ld=68) == moe.MOE_ERR_SHAPE
        assert call(codes=None) == moe.MOE_ERR_INVALID_ARG
        assert call(scales=_fake(1, 8)) == moe.MOE_ERR_ALIGN
    assert q(src=None) == moe.MOE_ERR_INVALID_ARG
    assert b"'src'" in L.moe_last_error_string()
    assert dq(dst=_fake(2, 4)) == moe.MOE_ERR_ALIGN


def test_dispatch_refusals(L):
    p = moe.params(16, 64, 8, 2, 16)
    f = [_fake(i) for i in range(6)]
    assert L.moe_mx4_dispatch(None, *f, None) == moe.MOE_ERR_INVALID_ARG
    assert L.moe_mx4_dispatch(C.byref(moe.params(16, 40, 8, 2, 16)), *f, None) == moe.MOE_ERR_SHAPE
    for i in range(6):
        a = list(f)
        a[i] = None
        assert L.moe_mx4_dispatch(C.byref(p), *a, None) == moe.MOE_ERR_INVALID_ARG
        a[i] = _fake(i, 8)
        assert L.moe_mx4_dispatch(C.byref(p), *a, None) == moe.MOE_ERR_ALIGN
    # an empty batch has nothing to do: token-sized buffers may be NULL
    p = moe.params(0, 64, 8, 2, 16)
    assert L.moe_mx4_dispatch(C.byref(p), None, None, None, f[3], None, None, None) == moe.MOE_OK


def test_python_refusals():
    import torch
    with pytest.raises(ValueError):
        moe.moe_mx4_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        moe.moe_mx4_quantize(torch.zeros(64))


def test_plain_format_by_hand():
    v = np.zeros((4, 32))
    v[0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]  # max 6: s = 0; every tie
    v[1, :4] = [7.9, -7.9, -0.2, 8e-3]                    # max 7.9: s = 0, saturates
    v[2, 0] = 2.0 ** -126
    v[3, 1] = np.inf
    c, b = mp.quantize(v)
    assert b[:, 0].tolist() == [127, 127, 0, 255]
    assert mp.CODES[c[0, :8]].tolist() == [6, 4, 4, 2, 2, 1, 1, 0]
    assert c[1, :4].tolist() == [7, 15, 8, 0]
    assert mp.values(c, b)[2, 0] == 2.0 ** -126  # 2 * 2^-127
    assert np.isnan(mp.values(c, b)[3]).all()


@pytest.mark.parametrize("seed", range(4))
def test_expert_tiles_do_not_overlap(seed):
    """The tile rows of ragged experts: offsets[e]/128 + e onwards, in order, inside
    T*k/128 + E + 1."""
    rng = np.random.default_rng(seed)
    E = int(rng.integers(1, 65))
    n = rng.integers(0, 300, E) * (rng.random(E) < 0.7)
    off = np.concatenate([[0], n.cumsum()])
    end = 0
    for e in range(E):
        first = off[e] // 128 + e
        assert first >= end
        end = first + -(-int(n[e]) // 128)
    assert end <= off[-1] // 128 + E + 1


def test_expert_refusals(L):
    p = moe.params(16, 64, 8, 2, 16)
    n = moe.moe_workspace_size(p)
    ws = _fake(20)
    calls = {
        "up": (L.moe_expert_up_mx4, 7, {0: "x_q", 3: "W13_q", 6: "h_s"}),
        "down": (L.moe_expert_down_mx4, 6, {1: "h_s", 4: "W2_s", 5: "out"}),
        "ffn": (L.moe_expert_ffn_mx4, 10, {2: "offsets", 6: "W2_s", 9: "out"}),
    }
    for fn, count, names in calls.values():
        f = [_fake(i) for i in range(count)]
        assert fn(None, *f, ws, n, None) == moe.MOE_ERR_INVALID_ARG
        assert fn(C.byref(moe.params(16, 72, 8, 2, 16)), *f, ws, n, None) == moe.MOE_ERR_SHAPE
        f32 = moe.params(16, 64, 8, 2, 16, dtype=moe.MOE_F32)
        assert fn(C.byref(f32), *f, ws, 1 << 24, None) == moe.MOE_ERR_DTYPE
        assert fn(C.byref(p), *f, None, n, None) == moe.MOE_ERR_INVALID_ARG
        assert fn(C.byref(p), *f, ws, n - 1, None) == moe.MOE_ERR_WORKSPACE
        for i in range(count):
            a = list(f)
            a[i] = None
            assert fn(C.byref(p), *a, ws, n, None) == moe.MOE_ERR_INVALID_ARG
            if i in names:
                assert ("'%s'" % names[i]).encode() in L.moe_last_error_string()
            a[i] = _fake(i, 8)
            assert fn(C.byref(p), *a, ws, n, None) == moe.MOE_ERR_ALIGN


def test_forward_refusals(L):
    p = moe.params(16, 64, 8, 2, 16)
    n = moe.moe_workspace_size(p)
    ws = _fake(40)

    def call(p=p, act=moe.MX4_ACT_BF16, n=n, drop=(), skew=(), noise=False):
        b = moe._Mx4Buffers()
        for i, f in enumerate(moe._MX4_FIELDS):
            if f in ("Wnoise", "noise") and not noise:
                continue
            if f not in drop:
                setattr(b, f, 0x100000 + 4096 * i + (8 if f in skew else 0))
        return L.moe_forward_mx4(C.byref(p), C.byref(b), act, ws, n, None)

    assert L.moe_forward_mx4(C.byref(p), None, 0, ws, n, None) == moe.MOE_ERR_INVALID_ARG
    assert call(act=2) == moe.MOE_ERR_INVALID_ARG
    assert call(n=n - 1) == moe.MOE_ERR_WORKSPACE
    big = 1 << 26
    assert call(moe.params(16, 64, 8, 2, 16, dtype=moe.MOE_F32), n=big) == moe.MOE_ERR_DTYPE
    assert call(moe.params(16, 72, 8, 2, 16), n=big) == moe.MOE_ERR_SHAPE
    assert call(moe.params(17, 64, 8, 2, 16), n=big) == moe.MOE_ERR_UNSUPPORTED
    assert b"16 tokens" in L.moe_last_error_string()
    assert call(moe.params(4, 64, 33, 2, 16), n=big) == moe.MOE_ERR_UNSUPPORTED
    assert call(moe.params(4, 64, 17, 2, 16), n=big, noise=True) == moe.MOE_ERR_UNSUPPORTED
    assert call(noise=True, drop=("noise",)) == moe.MOE_ERR_INVALID_ARG
    for f in moe._MX4_FIELDS:
        if f in ("Wnoise", "noise", "bias", "router_packed", "x_q", "x_s", "h_q", "h_s", "out"):
            continue
        assert call(drop=(f,)) == moe.MOE_ERR_INVALID_ARG, f
        assert call(skew=(f,)) == moe.MOE_ERR_ALIGN, f
    for f in ("x_q", "x_s", "h_q", "h_s", "out"):
        assert call(act=moe.MX4_ACT_MX4, drop=(f,)) == moe.MOE_ERR_INVALID_ARG, f
        assert call(act=moe.MX4_ACT_MX4, skew=(f,)) == moe.MOE_ERR_ALIGN, f


def test_buffers_given_by_name():
    import torch
    p = moe.params(4, 64, 8, 2, 16)
    y = torch.zeros(4, 64, dtype=torch.bfloat16)
    b = moe.Mx4Buffers(p, device="cpu", y=y)
    assert b.y is y and b.out.shape == (8, 64) and b.h.shape == (8, 16)
    assert moe.Mx4Buffers(p, act=moe.MX4_ACT_BF16, device="cpu").x_q is None
    assert moe.Mx4Buffers(p, act=moe.MX4_ACT_MX4, device="cpu").h is None
    with pytest.raises(TypeError):
        moe.Mx4Buffers(p, device="cpu", nothing=y)
    with pytest.raises(ValueError):
        moe.Mx4Buffers(p, device="cpu", y=y[:3])
    with pytest.raises(ValueError):
        moe.Mx4Buffers(p, device="cpu", y=y.float())


def test_workspace_given():
    import torch
    p = moe.params(4, 64, 8, 2, 16)
    n = moe.moe_workspace_size(p)
    for buf in (torch.zeros(n - 1, dtype=torch.uint8), torch.zeros(n, dtype=torch.float32)):
        with pytest.raises(moe.MoeError):
            moe.Workspace(p, buf=buf)
