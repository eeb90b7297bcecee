"""What the mx4 handles and calls hand to the library, without a GPU: CPU tensors that say they
are on the device, and a library that writes down what it is given."""
import copy
import ctypes as C
import io
import pickle

import pytest
import torch

import top_routing_grouped_noisy_b200 as moe

E, K, M, D, T = 4, 2, 40, 96, 5
U8, BF16, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
WEIGHTS = ("W13_q", "W13_s", "W2_q", "W2_s")


class OnDevice(torch.Tensor):
    """A CPU tensor that passes for one on the current device."""
    index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index

    def __deepcopy__(self, memo):
        memo[id(self)] = t = self.clone()
        return t


def dev(*shape, dtype=U8, **kw):
    return torch.zeros(*shape, dtype=dtype, **kw).as_subclass(OnDevice)


class _Workspace:
    def __init__(self, p):
        self.buf = dev(moe.moe_workspace_size(p))
        self.nbytes = self.buf.numel()

    @property
    def ptr(self):
        return self.buf.data_ptr()


class _Recorder:
    """The library: host-only calls pass through, the others are written down."""

    def __init__(self, real):
        self._real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name.endswith("_elems") or name in (
                "moe_h_ld", "moe_workspace_size", "moe_last_error_string"):
            return getattr(self._real, name)

        def call(*a):
            self.calls.append((name, a))
            if name == "moe_forward_mx4":
                self.struct = {n: getattr(a[1]._obj, n) for n in moe._MX4_FIELDS}
            return moe.MOE_OK
        return call


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(moe.lib())
    monkeypatch.setattr(moe, "lib", lambda: r)
    monkeypatch.setattr(moe, "_stream", lambda stream=None: 7)
    monkeypatch.setattr(moe, "_current_device", lambda: 0, raising=False)
    return r


def params(T=T, m=M, d=D, E=E, k=K, **kw):
    return moe.params(T, d, E, k, m, **kw)


def experts(m=M, d=D, E=E):
    m16, m8 = (m + 15) // 16 * 16, (m + 7) // 8 * 8
    return moe.Mx4Experts(dev(moe.moe_mx4_codes_bytes(E, 2 * m16, d)),
                          dev(moe.moe_mx4_scales_bytes(E, 2 * m16, d)),
                          dev(moe.moe_mx4_codes_bytes(E, d, m8)),
                          dev(moe.moe_mx4_scales_bytes(E, d, m8)))


def buffers(p, act=None):
    b = moe.Mx4Buffers(p, act=act, device="cpu")
    for n in moe._MX4_FIELDS[10:]:
        t = getattr(b, n)
        if t is not None:
            setattr(b, n, t.as_subclass(OnDevice))
    return b


class Layer:
    def __init__(self, p=None, act=None):
        self.p = p if p is not None else params()
        self.W, self.b, self.ws = experts(), buffers(self.p, act), _Workspace(self.p)
        self.x, self.Wg = dev(self.p.T, D, dtype=BF16), dev(D, E, dtype=BF16)

    def run(self, act=moe.MX4_ACT_BF16, **kw):
        a = dict(x=self.x, Wg=self.Wg, W=self.W, ws=self.ws, bufs=self.b)
        a.update(kw)
        return moe.moe_forward_mx4(self.p, act=act, **a)


def test_layer_gets_every_pointer(rec):
    L = Layer()
    for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
        L.run(act)
        s = rec.struct
        for n in WEIGHTS:
            assert s[n] == getattr(L.W, n).data_ptr()
        used = [n for n in moe._MX4_FIELDS[10:]
                if n not in (("x_q", "x_s", "h_q", "h_s", "out") if act == 0 else ("h",))]
        for n in used:
            assert s[n] == getattr(L.b, n).data_ptr(), n
        assert s["x"] == L.x.data_ptr() and s["Wg"] == L.Wg.data_ptr()
        assert s["Wnoise"] is None and s["router_packed"] is None


def _swap_data(t):
    t.data = t.data.clone()


def _swap_set(t):
    t.set_(t.clone())


def _swap_storage(t):
    n = t.untyped_storage().nbytes()
    keep = torch.zeros(n + 64, dtype=U8)  # so that the next allocation lies elsewhere
    t.untyped_storage().resize_(0)
    t.untyped_storage().resize_(n + (1 << 16))
    return keep


@pytest.mark.parametrize("swap", [_swap_data, _swap_set, _swap_storage])
def test_storage_replaced_in_place(rec, swap):
    """A tensor of a handle whose storage is another one since: the calls take the new one."""
    L = Layer()
    L.run()
    for owner, n in [(L.W, n) for n in WEIGHTS] + [(L.b, n) for n in ("y", "h", "topk_idx")]:
        t = getattr(owner, n)
        old = t.data_ptr()
        keep = swap(t)
        if t.data_ptr() == old and swap is _swap_storage:
            continue  # the allocator gave the same place again
        assert t.data_ptr() != old
        L.run()
        assert rec.struct[n] == t.data_ptr(), n
        del keep
    moe.moe_expert_up_mx4(L.p, L.b.x_q, L.b.x_s, L.b.offsets, L.W, L.b.h_q, L.b.h_s, L.ws)
    assert rec.calls[-1][1][4:6] == (L.W.W13_q.data_ptr(), L.W.W13_s.data_ptr())
    moe.moe_expert_down_mx4(L.p, L.b.h_q, L.b.h_s, L.b.offsets, L.W, L.b.out, L.ws)
    assert rec.calls[-1][1][4:6] == (L.W.W2_q.data_ptr(), L.W.W2_s.data_ptr())


def _by_pickle(h):
    return pickle.loads(pickle.dumps(h))


def _by_save(h):
    f = io.BytesIO()
    torch.save(h, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, _by_pickle, _by_save])
def test_handles_copied(rec, how):
    """A copy is a handle of its own: a tensor set on it is not the original's."""
    L = Layer()
    W, b = how(L.W), how(L.b)
    L.run(W=W, bufs=b)
    for owner, names in ((W, WEIGHTS), (b, ("y", "h", "offsets"))):
        for n in names:
            assert rec.struct[n] == getattr(owner, n).data_ptr(), n
    shared = how is copy.copy
    assert (W.W2_q.data_ptr() == L.W.W2_q.data_ptr()) is shared
    assert (b.y.data_ptr() == L.b.y.data_ptr()) is shared
    W.W2_q, b.y = L.W.W2_q.clone(), L.b.y.clone()
    L.run()
    assert rec.struct["W2_q"] == L.W.W2_q.data_ptr() != W.W2_q.data_ptr()
    assert rec.struct["y"] == L.b.y.data_ptr() != b.y.data_ptr()
    L.run(W=W, bufs=b)
    assert rec.struct["W2_q"] == W.W2_q.data_ptr() and rec.struct["y"] == b.y.data_ptr()


def test_attribute_taken_away(rec):
    L = Layer()
    L.run()
    n = len(rec.calls)
    del L.b.h, L.W.W2_s
    for kw in ({}, {"W": experts()}):
        with pytest.raises(AttributeError):
            L.run(**kw)
    L.b.h = None  # the library says which it misses
    L.run(W=experts())
    assert rec.struct["h"] is None and len(rec.calls) == n + 1


def test_cpu_tensors_refused(rec):
    L = Layer()
    n = len(rec.calls)
    for owner, name in ((L.W, "W13_q"), (L.b, "y"), (L.b, "topk_w")):
        good = getattr(owner, name)
        setattr(owner, name, torch.zeros(good.shape, dtype=good.dtype))
        with pytest.raises(ValueError, match="CUDA"):
            L.run()
        setattr(owner, name, good)
    L.run()
    assert len(rec.calls) == n + 1
