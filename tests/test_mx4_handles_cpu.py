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


def _calls(L, noisy=False):
    """name, the call, and its tensors by argument: a changed copy of them may be given to it."""
    p, b, W, i32 = L.p, L.b, L.W, dict(dtype=I32)
    rows = p.T * p.k
    t = {n: getattr(b, n) for n in ("topk_idx", "slot_row", "offsets", "x_q", "x_s", "h_q", "h_s",
                                    "out")}
    w13 = {n: getattr(W, n) for n in WEIGHTS[:2]}
    w2 = {n: getattr(W, n) for n in WEIGHTS[2:]}
    of = lambda a: moe.Mx4Experts(*(a.pop(n, None) for n in WEIGHTS))
    pick = lambda *ns: {n: t[n] for n in ns}

    def experts_call(fn):
        def call(a):
            W = of(a)
            return fn(p, W=W, ws=L.ws, **a)
        return call

    yield "dispatch", lambda a: moe.moe_mx4_dispatch(p, **a), \
        {"x": L.x, **pick("topk_idx", "slot_row", "offsets", "x_q", "x_s")}
    yield "up", experts_call(moe.moe_expert_up_mx4), \
        {**pick("x_q", "x_s", "offsets", "h_q", "h_s"), **w13}
    yield "down", experts_call(moe.moe_expert_down_mx4), \
        {**pick("h_q", "h_s", "offsets", "out"), **w2}
    yield "ffn", experts_call(moe.moe_expert_ffn_mx4), \
        {**pick("x_q", "x_s", "offsets", "h_q", "h_s", "out"), **w13, **w2}
    more = {"x": L.x, "Wg": L.Wg, "Wnoise": dev(D, E, dtype=BF16), "noise": dev(T, E, dtype=F32),
            "bias": dev(E, dtype=F32),
            "router_packed": dev(moe.moe_router_packed_bytes(p, True))}
    for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
        names = moe._MX4_OUTPUTS + (["h"] if act == moe.MX4_ACT_BF16 else moe._MX4_ROWS)

        def forward(a, act=act, names=names):
            W, bufs = of(a), copy.copy(b)
            for n in names:
                setattr(bufs, n, a.pop(n))
            return moe.moe_forward_mx4(p, W=W, ws=L.ws, bufs=bufs, act=act, **a)

        yield "forward%d" % act, forward, \
            {**more, **{n: getattr(b, n) for n in names}, **w13, **w2}


def _shorter(t):
    return t.reshape(-1)[:-1]


def _longer(t):
    return torch.cat([t.reshape(-1), t.reshape(-1)[:1]]).as_subclass(OnDevice)


def _other_type(t):
    return t.to(torch.int16 if t.dtype == BF16 else (F32 if t.dtype == I32 else
                                                     (I32 if t.dtype == F32 else torch.int8)))


def _spaced(t):
    return torch.stack([t.reshape(-1), t.reshape(-1)], 1).as_subclass(OnDevice)[:, 0]


def _elsewhere(t):
    t = t.clone()
    t.index = 1
    return t


def _on_host(t):
    return t.as_subclass(torch.Tensor)


def _emptied(t):
    """A view into a storage that was taken away: data_ptr() is a bare offset."""
    flat = torch.zeros(t.nbytes + 256, dtype=U8).as_subclass(OnDevice)
    v = flat[256:].view(t.dtype)
    flat.untyped_storage().resize_(0)
    return v


REFUSED = {"shorter": _shorter, "type": _other_type, "spaced": _spaced, "device": _elsewhere,
           "host": _on_host}


@pytest.mark.parametrize("how", REFUSED)
def test_tensors_refused(rec, how):
    """Too few elements, another type, spaced out, on another device or the host: ValueError
    before anything is launched, whichever argument it is."""
    L = Layer()
    for call_name, call, args in _calls(L):
        call(dict(args))
        n = len(rec.calls)
        for name, t in args.items():
            if how == "spaced" and t.numel() == 1:
                continue  # one element is contiguous
            if how == "type" and name == "router_packed":
                continue  # moe_router_pack fills a buffer of any type
            bad = REFUSED[how](t)
            with pytest.raises(ValueError):
                call({**args, name: bad})
                pytest.fail("%s took %s (%s)" % (call_name, name, how))
            assert len(rec.calls) == n, (call_name, name)


def test_weights_of_another_layer_refused(rec):
    """Weights have to have the layer's sizes: more bytes are another layout.  Their storage has
    to be there."""
    L = Layer()
    for call_name, call, args in _calls(L):
        n = len(rec.calls)
        for name in set(args) & {*WEIGHTS, "Wg", "Wnoise", "bias"}:
            for bad in (_longer, _emptied):
                with pytest.raises(ValueError):
                    call({**args, name: bad(args[name])})
                    pytest.fail("%s took %s (%s)" % (call_name, name, bad))
        assert len(rec.calls) == n
    for W in (experts(m=M - 8), experts(m=2 * M), experts(d=D + 32), experts(E=E + 1)):
        for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
            with pytest.raises(ValueError, match="W"):
                L.run(act, W=W)
    assert len(rec.calls) == n


def test_not_a_tensor(rec):
    L = Layer()
    for _, call, args in _calls(L):
        for name in args:
            for bad in (3, "x", [1.0]):
                with pytest.raises(TypeError):
                    call({**args, name: bad})


def test_buffers_of_another_batch_refused(rec):
    """Buffers made for T tokens serve T or fewer."""
    small, big = Layer(params(T=4)), Layer(params(T=16))
    n = len(rec.calls)
    for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
        with pytest.raises(ValueError, match="y: needs at least"):
            big.run(act, bufs=small.b)
        with pytest.raises(ValueError):
            big.run(act, bufs=buffers(params(T=16, d=64)))
        with pytest.raises(ValueError):
            big.run(act, bufs=buffers(params(T=16, E=2)))
    with pytest.raises(ValueError, match="h: needs at least"):
        big.run(bufs=buffers(params(T=16, m=8)))
    with pytest.raises(ValueError, match="h_q: needs at least"):
        big.run(moe.MX4_ACT_MX4, bufs=buffers(params(T=16, m=8)))
    assert len(rec.calls) == n
    for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
        small.run(act, bufs=big.b)
    assert len(rec.calls) == n + 2


@pytest.mark.parametrize("act", [moe.MX4_ACT_BF16, moe.MX4_ACT_MX4])
def test_empty_batch_and_none(rec, act):
    """T = 0 needs no rows; what is None the library judges."""
    L = Layer(params(T=0))
    L.run(act)
    for n in ("x_q", "x_s", "h_q", "h_s", "out", "y", "topk_idx"):
        setattr(L.b, n, None)
    L.run(act)
    assert rec.struct["x_q"] is None and rec.struct["y"] is None and len(rec.calls) == 2


def test_sizes_that_the_library_refuses(monkeypatch):
    """Sizes outside the contract are the library's to refuse, before it looks at a tensor."""
    monkeypatch.setattr(moe, "_stream", lambda stream=None: None)
    x = dev(4, D, dtype=BF16)
    for p in (params(T=-1), params(E=65), params(m=0), params(k=9)):
        with pytest.raises(moe.MoeError):
            moe.moe_mx4_dispatch(p, x, x, x, x, x, x)
        with pytest.raises(moe.MoeError):
            moe.moe_expert_down_mx4(p, x, x, x, experts(), x, _Workspace(params()))


def test_quantize_other_device(rec):
    src, codes = dev(2, 3, 64, dtype=F32), dev(2, 3, 32)
    scales = dev(2, 1, 1, 32, 4, 4)
    moe.moe_mx4_quantize(src, out=(codes, scales))
    moe.moe_mx4_dequantize(codes, scales, 64, out=src)
    n = len(rec.calls)
    for i in range(3):
        a = [src, codes, scales]
        a[i] = _elsewhere(a[i])
        with pytest.raises(ValueError, match="device 1"):
            moe.moe_mx4_quantize(a[0], out=(a[1], a[2]))
        with pytest.raises(ValueError, match="device 1"):
            moe.moe_mx4_dequantize(a[1], a[2], 64, out=a[0])
    assert len(rec.calls) == n


def test_router_packed_of_any_type(rec):
    """moe_router_pack fills the buffer it is given, whatever its type; so is it taken."""
    L = Layer()
    n = moe.moe_router_packed_bytes(L.p, False)
    for dtype in (U8, BF16, F32):
        t = dev(n // dtype.itemsize, dtype=dtype)
        L.run(moe.MX4_ACT_MX4, router_packed=t)
        assert rec.struct["router_packed"] == t.data_ptr()
        with pytest.raises(ValueError):
            L.run(moe.MX4_ACT_MX4, router_packed=t[1:].clone())


def test_f32_layers_are_the_librarys_to_refuse(monkeypatch):
    """With the tensors of a bf16 layer the error is that of the library, not one of sizes."""
    monkeypatch.setattr(moe, "_stream", lambda stream=None: None)
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    L = Layer()
    p32 = params(dtype=moe.MOE_F32)
    L.ws = _Workspace(p32)
    L.p = p32
    for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
        with pytest.raises(moe.MoeError, match="bf16"):
            L.run(act)
    x = dev(T, D, dtype=F32)  # the dispatch takes them
    L.p = params(T=0, dtype=moe.MOE_F32)
    moe.moe_mx4_dispatch(L.p, x[:0], L.b.topk_idx, L.b.slot_row, L.b.offsets, L.b.x_q, L.b.x_s)
    with pytest.raises(ValueError, match="x: needs"):
        moe.moe_mx4_dispatch(p32, L.x, L.b.topk_idx, L.b.slot_row, L.b.offsets, L.b.x_q, L.b.x_s)


def test_workspace_replaced(monkeypatch):
    """The workspace's size is that of its buffer at the call: with a smaller buffer in its place
    the call is refused."""
    class Init:  # the library but for moe_workspace_init, which needs a device
        def __getattr__(self, name):
            return getattr(real, name) if name != "moe_workspace_init" else lambda *a: moe.MOE_OK

    real, init = moe.lib(), Init()
    monkeypatch.setattr(moe, "lib", lambda: init)
    monkeypatch.setattr(moe, "_stream", lambda stream=None: None)
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    L = Layer()
    n = moe.moe_workspace_size(L.p)
    for buf in (None, dev(n + 512)):
        ws = moe.Workspace(L.p, buf=buf if buf is not None else dev(n))
        assert ws.nbytes == ws.buf.numel()
        ws.buf = dev(n - 256)
        assert ws.nbytes == n - 256
        for act in (moe.MX4_ACT_BF16, moe.MX4_ACT_MX4):
            with pytest.raises(moe.MoeError, match="workspace"):
                L.run(act, ws=ws)
        ws.buf = dev(n)
        ws.buf.data = torch.zeros(n // 2, dtype=U8)
        with pytest.raises(moe.MoeError, match="workspace"):
            L.run(ws=ws)
