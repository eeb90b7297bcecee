"""Python binding of libmoe.so, the B200 (sm_100a) sparse Mixture-of-Experts SwiGLU
FFN layer: the forward pass (noisy Top-K routing, capacity dispatch, grouped expert
GEMMs on tcgen05 tensor cores, gate-weighted combine, gate statistics), its backward
(moe_backward and its steps), the residual layer with shared neurons, the expert
construction (moe_partition_*), the clustering partition (moe_cluster_partition) and
the non-collective steps of the expert-parallel layer (moe_ep_*; the layer itself is
``expert_parallel.ExpertParallelMoE``).

The functions mirror the C ABI in ``include/moe.h`` one to one and only marshal
arguments: torch tensors are passed as device pointers together with torch's
current CUDA stream; every step of the layer runs in the library's kernels.
PyTorch provides device memory and streams only.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
import ctypes as C
import functools
import operator
import os

import torch

__all__ = [
    "MoeError", "Params", "lib", "params", "moe_capacity", "moe_version", "moe_launch_count",
    "moe_partition_experts", "moe_workspace_size", "Workspace", "moe_route", "moe_route_packed",
    "moe_router_pack", "moe_router_packed_bytes", "moe_dispatch", "moe_dispatch_routed", "moe_dispatch_noalloc", "moe_dispatch_rows", "moe_expert_up_gather",
    "moe_expert_up", "moe_expert_down", "moe_expert_ffn", "moe_combine", "moe_gate_stats",
    "moe_forward", "ForwardBuffers", "moe_get_device_status", "moe_set_wait_limit_ns",
    "moe_set_gemm_band_rows",
    "packed_w13_elems", "packed_w2_elems", "h_ld", "Pipeline", "moe_partition_residual",
    "moe_combine_residual", "moe_forward_residual", "moe_cluster_workspace_size",
    "moe_cluster_partition", "moe_cluster_distances", "moe_backward_workspace_size",
    "moe_combine_backward", "moe_expert_down_backward", "moe_expert_up_backward",
    "moe_route_backward", "moe_backward", "BackwardBuffers",
    "moe_backward_residual_workspace_size", "moe_backward_residual", "EpPlan", "moe_ep_plan",
    "moe_ep_mask_slots", "moe_ep_gate_stats", "EP_CAPACITY_GLOBAL", "EP_CAPACITY_LOCAL",
    "moe_mx4_codes_bytes", "moe_mx4_scales_bytes", "moe_mx4_rows_bytes",
    "moe_mx4_row_scales_bytes", "moe_mx4_quantize", "moe_mx4_dequantize", "moe_mx4_dispatch",
    "moe_expert_up_mx4", "moe_expert_down_mx4", "moe_expert_ffn_mx4", "Mx4Experts",
    "moe_forward_mx4", "Mx4Buffers", "MX4_ACT_BF16", "MX4_ACT_MX4", "MX4_FEW_TOKENS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_SHAPE = -2
MOE_ERR_ALIGN = -3
MOE_ERR_DTYPE = -4
MOE_ERR_CUDA = -5
MOE_ERR_DEVICE_TIMEOUT = -6
MOE_ERR_DEVICE_BADINDEX = -7
MOE_ERR_WORKSPACE = -8
MOE_ERR_UNSUPPORTED = -9

MOE_F32 = 0
MOE_BF16 = 1
MIXTRAL = 0
ST = 1
DISJOINT = 0
COPY = 1
STACKED = 2
EP_CAPACITY_GLOBAL = 0
EP_CAPACITY_LOCAL = 1
MX4_ACT_BF16 = 0
MX4_ACT_MX4 = 1
MX4_FEW_TOKENS = 16


class MoeError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("libmoe error %d: %s" % (code, msg))
        self.code = code


class Params(C.Structure):
    _fields_ = [("T", C.c_int32), ("d", C.c_int32), ("E", C.c_int32), ("k", C.c_int32),
                ("m", C.c_int32), ("dtype", C.c_int32), ("router_type", C.c_int32),
                ("capacity", C.c_int32), ("rescale", C.c_int32), ("balance_lambda", C.c_float)]


_BUF_FIELDS = ["x", "Wg", "Wnoise", "noise", "bias", "W13_e", "W2_e", "y", "loss", "counts",
               "importance", "f", "P", "topk_idx", "topk_w", "probs_sum", "x_perm", "row_token",
               "slot_row", "kept", "offsets", "h", "out", "router_packed"]


class _Buffers(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in _BUF_FIELDS]


_MX4_FIELDS = ["x", "Wg", "Wnoise", "noise", "bias", "W13_q", "W13_s", "W2_q", "W2_s",
               "router_packed", "y", "loss", "counts", "importance", "f", "P", "topk_idx", "topk_w",
               "probs_sum", "row_token", "slot_row", "kept", "offsets", "h", "x_q", "x_s", "h_q",
               "h_s", "out"]
# the caller's outputs and tables; h of bf16 activations lies between them and these of mx4 ones
_MX4_OUTPUTS, _MX4_ROWS = _MX4_FIELDS[10:-6], _MX4_FIELDS[-5:]
_mx4_few_tensors = operator.attrgetter(*_MX4_OUTPUTS, "h")
_mx4_row_tensors = operator.attrgetter(*_MX4_OUTPUTS, *_MX4_ROWS)


class _Mx4Buffers(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in _MX4_FIELDS]


_BWD_FIELDS = ["dy", "dx", "dWg", "dWnoise", "dbias", "dW13_e", "dW2_e", "d_out", "dG", "dh",
               "dx_perm"]


class _BwdBuffers(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in _BWD_FIELDS]


_lib = None


def lib():
    """The loaded libmoe.so (raises ImportError when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libmoe.so not found at %s; build it with "
                              "`python -m top_routing_grouped_noisy_b200.build`" % LIB_PATH)
        L = C.CDLL(LIB_PATH)
        v, i32, i64, sz, f64 = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_double
        P = C.POINTER(Params)
        sig = {
            "moe_version": (C.c_char_p, []),
            "moe_last_error_string": (C.c_char_p, []),
            "moe_launch_count": (C.c_uint64, []),
            "moe_set_wait_limit_ns": (None, [C.c_uint64]),
            "moe_set_gemm_band_rows": (None, [C.c_int32]),
            "moe_capacity": (i32, [i32, i32, f64]),
            "moe_packed_w13_elems": (i64, [i32, i32, i32]),
            "moe_packed_w2_elems": (i64, [i32, i32, i32]),
            "moe_h_ld": (i32, [i32]),
            "moe_partition_experts": (C.c_int, [v, v, v, i32, i32, i32, i32, v, i32, v, v, v, v]),
            "moe_workspace_size": (sz, [P]),
            "moe_workspace_init": (C.c_int, [v, sz, v]),
            "moe_route": (C.c_int, [P, v, v, v, v, v, v, v, v, v, v, sz, v]),
            "moe_route_packed": (C.c_int, [P, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            "moe_router_pack": (C.c_int, [P, v, v, v, v]),
            "moe_router_packed_bytes": (sz, [P, i32]),
            "moe_dispatch": (C.c_int, [P, v, v, v, v, v, v, v, v, v, sz, v]),
            "moe_dispatch_routed": (C.c_int, [P, v, v, v, v, v, v, v, v, v, sz, v]),
            "moe_dispatch_noalloc": (C.c_int, [P, v, v, v, v, v, v, v, v, v, v]),
            "moe_dispatch_rows": (C.c_int, [P, v, v, v, v, v, v, v, sz, v]),
            "moe_expert_up_gather": (C.c_int, [P, v, v, v, v, v, v, sz, v]),
            "moe_expert_up": (C.c_int, [P, v, v, v, v, v, sz, v]),
            "moe_expert_down": (C.c_int, [P, v, v, v, v, v, sz, v]),
            "moe_expert_ffn": (C.c_int, [P, v, v, v, v, v, v, v, sz, v]),
            "moe_combine": (C.c_int, [P, v, v, v, v, v]),
            "moe_gate_stats": (C.c_int, [P, v, v, v, v, v, v]),
            "moe_forward": (C.c_int, [P, C.POINTER(_Buffers), v, sz, v]),
            "moe_get_device_status": (C.c_int, [v, C.POINTER(i32), i32, v]),
            "moe_partition_residual": (C.c_int, [v, v, v, i32, i32, i32, v, i32, v, i32, v, v,
                                                 v, v, v, v]),
            "moe_combine_residual": (C.c_int, [P, v, v, v, v, v, v]),
            "moe_forward_residual": (C.c_int, [P, C.POINTER(_Buffers), v, v, i32, v, v, v, sz,
                                               v]),
            "moe_cluster_workspace_size": (sz, [i32, i32, i32]),
            "moe_cluster_partition": (C.c_int, [v, i32, i32, i32, i32, i32, v, v, v, v, v, sz,
                                                v]),
            "moe_cluster_distances": (C.c_int, [v, i32, i32, i32, i32, v, v, v]),
            "moe_backward_workspace_size": (sz, [P]),
            "moe_combine_backward": (C.c_int, [P, v, v, v, v, v, v, v]),
            "moe_expert_down_backward": (C.c_int, [P, v, v, v, v, v, v, v, sz, v]),
            "moe_expert_up_backward": (C.c_int, [P, v, v, v, v, v, v, v, sz, v]),
            "moe_route_backward": (C.c_int, [P, v, v, v, v, v, v, v, v, v, C.c_float, v, v, v,
                                             v, v, v, v, sz, v]),
            "moe_backward": (C.c_int, [P, C.POINTER(_Buffers), C.POINTER(_BwdBuffers),
                                       C.c_float, v, sz, v]),
            "moe_backward_residual_workspace_size": (sz, [P, i32]),
            "moe_backward_residual": (C.c_int, [P, C.POINTER(_Buffers), C.POINTER(_BwdBuffers), v,
                                                v, i32, v, v, v, v, v, C.c_float, v, sz, v]),
            "moe_ep_plan": (C.c_int, [v, i32, i32, i32, i32, i32, v, v, v, v, v, v]),
            "moe_ep_mask_slots": (C.c_int, [P, v, v, v, v, v]),
            "moe_ep_gate_stats": (C.c_int, [P, v, i32, v, v, v, v, v, v]),
            "moe_mx4_codes_bytes": (sz, [i32, i32, i32]),
            "moe_mx4_scales_bytes": (sz, [i32, i32, i32]),
            "moe_mx4_rows_bytes": (sz, [P, i32]),
            "moe_mx4_row_scales_bytes": (sz, [P, i32]),
            "moe_mx4_quantize": (C.c_int, [v, i32, i32, i32, i32, i64, v, v, v]),
            "moe_mx4_dequantize": (C.c_int, [v, v, i32, i32, i32, i32, i64, v, v]),
            "moe_mx4_dispatch": (C.c_int, [P, v, v, v, v, v, v, v]),
            "moe_expert_up_mx4": (C.c_int, [P, v, v, v, v, v, v, v, v, sz, v]),
            "moe_expert_down_mx4": (C.c_int, [P, v, v, v, v, v, v, v, sz, v]),
            "moe_expert_ffn_mx4": (C.c_int, [P, v, v, v, v, v, v, v, v, v, v, v, sz, v]),
            "moe_forward_mx4": (C.c_int, [P, C.POINTER(_Mx4Buffers), i32, v, sz, v]),
            "moe_pipeline_create": (C.c_int, [P, v, v, v, v, v, i32, C.POINTER(v)]),
            "moe_pipeline_submit": (C.c_int, [v, v, v, v, v, C.POINTER(i64)]),
            "moe_pipeline_wait": (C.c_int, [v, i64]),
            "moe_pipeline_destroy": (C.c_int, [v]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc):
    if rc != MOE_OK:
        raise MoeError(rc, lib().moe_last_error_string().decode())


def _p(t):
    if t is None:
        return None
    if type(t) is torch.Tensor and t.is_cuda and t.is_contiguous():
        return t.data_ptr() or None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor, got %r" % type(t))
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors (got a %s tensor)" % t.device)
    if not t.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors")
    return t.data_ptr() or None


# the current stream's handle without building a torch.cuda.Stream (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)
_started = False


def _stream(stream=None):
    global _started
    if stream is not None:
        return stream.cuda_stream
    if not _started:
        s = torch.cuda.current_stream().cuda_stream  # starts CUDA
        _started = _raw_stream is not None and _device is not None
        return s
    return _raw_stream(_device())


def _current_device():
    """Index of the current device; -2 before CUDA has started, when no tensor lies on one."""
    if _started:
        return _device()
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _dtype_code(dt):
    if dt == torch.bfloat16:
        return MOE_BF16
    if dt == torch.float32:
        return MOE_F32
    raise TypeError("libmoe computes in bf16 or f32, not %s" % dt)


def moe_version() -> str:
    return lib().moe_version().decode()


def moe_launch_count() -> int:
    return int(lib().moe_launch_count())


def moe_set_wait_limit_ns(ns: int) -> None:
    lib().moe_set_wait_limit_ns(int(ns))


def moe_set_gemm_band_rows(rows: int) -> None:
    """Tuning knob of the 2-SM expert GEMMs' tile order (results do not change)."""
    lib().moe_set_gemm_band_rows(int(rows))


def moe_capacity(T: int, E: int, cf: float) -> int:
    return int(lib().moe_capacity(T, E, float(cf)))


def packed_w13_elems(E, m, d):
    return int(lib().moe_packed_w13_elems(E, m, d))


def packed_w2_elems(E, m, d):
    return int(lib().moe_packed_w2_elems(E, m, d))


def h_ld(m):
    return int(lib().moe_h_ld(m))


def params(T, d, E, k, m, dtype=torch.bfloat16, router_type=MIXTRAL, capacity=-1,
           rescale=False, balance_lambda=0.0) -> Params:
    return Params(T, d, E, k, m, _dtype_code(dtype) if isinstance(dtype, torch.dtype) else dtype,
                  router_type, capacity, 1 if rescale else 0, balance_lambda)


def moe_workspace_size(p: Params) -> int:
    return int(lib().moe_workspace_size(C.byref(p)))


class Workspace:
    """Caller-owned scratch for the library (a zeroed torch uint8 buffer): a new one, or
    ``buf``, a CUDA uint8 tensor of at least moe_workspace_size(p) bytes, which is zeroed."""

    def __init__(self, p: Params, device=None, nbytes=None, buf=None):
        n = nbytes if nbytes is not None else moe_workspace_size(p)
        if n <= 0:
            raise MoeError(MOE_ERR_INVALID_ARG, "invalid parameters for the workspace")
        if buf is not None:
            if buf.dtype != torch.uint8 or buf.numel() < n:
                raise MoeError(MOE_ERR_WORKSPACE, "the workspace needs %d uint8 elements" % n)
        self.buf = buf if buf is not None else torch.empty(n, dtype=torch.uint8,
                                                           device=device or "cuda")
        _check(lib().moe_workspace_init(_p(self.buf), self.nbytes, _stream()))

    @property
    def ptr(self):
        return self.buf.data_ptr()

    @property
    def nbytes(self):
        return self.buf.nbytes


def moe_get_device_status(ws: Workspace, clear=True, stream=None) -> int:
    st = C.c_int32(0)
    _check(lib().moe_get_device_status(ws.ptr, C.byref(st), 1 if clear else 0, _stream(stream)))
    return st.value


def moe_partition_experts(W1, W3, W2, E, mode=DISJOINT, perm=None, ws=None, out=None,
                          stream=None):
    """a0: packed expert weights (W13_e, W2_e) from a dense FFN (or stacked experts)."""
    dt = _dtype_code(W1.dtype)
    if mode == STACKED:
        d_ff, d = W1.shape[1], W1.shape[2]
    else:
        d_ff, d = W1.shape
    m = d_ff // E if mode == DISJOINT else d_ff
    if out is None:
        W13_e = torch.empty(packed_w13_elems(E, m, d), dtype=W1.dtype, device=W1.device)
        W2_e = torch.empty(packed_w2_elems(E, m, d), dtype=W1.dtype, device=W1.device)
    else:
        W13_e, W2_e = out
    _check(lib().moe_partition_experts(_p(W1), _p(W3), _p(W2), d, d_ff, E, mode, _p(perm), dt,
                                       _p(W13_e), _p(W2_e), ws.ptr if ws is not None else None,
                                       _stream(stream)))
    return W13_e, W2_e


def moe_route(p, x, Wg, Wnoise, noise, bias, ws, topk_idx, topk_w, probs_sum, importance,
              stream=None):
    _check(lib().moe_route(C.byref(p), _p(x), _p(Wg), _p(Wnoise), _p(noise), _p(bias),
                           _p(topk_idx), _p(topk_w), _p(probs_sum), _p(importance), ws.ptr,
                           ws.nbytes, _stream(stream)))


def moe_router_packed_bytes(p, noisy) -> int:
    return int(lib().moe_router_packed_bytes(C.byref(p), 1 if noisy else 0))


def moe_router_pack(p, Wg, Wnoise=None, out=None, stream=None):
    """The router weights packed once for the tensor-core router (include/moe.h);
    returns the packed device buffer (uint8)."""
    n = moe_router_packed_bytes(p, Wnoise is not None)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=Wg.device)
    _check(lib().moe_router_pack(C.byref(p), _p(Wg), _p(Wnoise), _p(out), _stream(stream)))
    return out


def moe_route_packed(p, x, Wg, Wnoise, Wt, noise, bias, ws, topk_idx, topk_w, probs_sum,
                     importance, stream=None):
    _check(lib().moe_route_packed(C.byref(p), _p(x), _p(Wg), _p(Wnoise), _p(Wt), _p(noise),
                                  _p(bias), _p(topk_idx), _p(topk_w), _p(probs_sum),
                                  _p(importance), ws.ptr, ws.nbytes, _stream(stream)))


def moe_dispatch(p, x, topk_idx, ws, x_perm, row_token, slot_row, counts, kept, offsets,
                 stream=None):
    _check(lib().moe_dispatch(C.byref(p), _p(x), _p(topk_idx), _p(x_perm), _p(row_token),
                              _p(slot_row), _p(counts), _p(kept), _p(offsets), ws.ptr,
                              ws.nbytes, _stream(stream)))


def moe_dispatch_routed(p, x, topk_idx, ws, x_perm, row_token, slot_row, counts, kept, offsets,
                        stream=None):
    """a2 right after moe_route on the same workspace: reuses the chunk counts the
    router left there (topk_idx must be that call's output, unchanged)."""
    _check(lib().moe_dispatch_routed(C.byref(p), _p(x), _p(topk_idx), _p(x_perm),
                                     _p(row_token), _p(slot_row), _p(counts), _p(kept),
                                     _p(offsets), ws.ptr, ws.nbytes, _stream(stream)))


def moe_dispatch_rows(p, topk_idx, ws, row_token, slot_row, counts, kept, offsets, stream=None):
    """a2 tables only (no permuted copy of x)."""
    _check(lib().moe_dispatch_rows(C.byref(p), _p(topk_idx), _p(row_token), _p(slot_row),
                                   _p(counts), _p(kept), _p(offsets), ws.ptr, ws.nbytes,
                                   _stream(stream)))


def moe_expert_up_gather(p, x, row_token, offsets, W13_e, h, ws, stream=None):
    """a3 gathering rows of x through row_token (bf16)."""
    _check(lib().moe_expert_up_gather(C.byref(p), _p(x), _p(row_token), _p(offsets), _p(W13_e),
                                      _p(h), ws.ptr, ws.nbytes, _stream(stream)))


def moe_dispatch_noalloc(p, x, topk_idx, x_perm, row_token, slot_row, counts, kept, offsets,
                         status, stream=None):
    """a2 without a workspace (fixed scratch inside the library; see include/moe.h).
    ``status`` is a device int32 tensor the caller zeroes; it is required for T > 0,
    being the only place a bad expert index is reported."""
    _check(lib().moe_dispatch_noalloc(C.byref(p), _p(x), _p(topk_idx), _p(x_perm),
                                      _p(row_token), _p(slot_row), _p(counts), _p(kept),
                                      _p(offsets), _p(status), _stream(stream)))


def moe_expert_up(p, x_perm, offsets, W13_e, h, ws, stream=None):
    _check(lib().moe_expert_up(C.byref(p), _p(x_perm), _p(offsets), _p(W13_e), _p(h), ws.ptr,
                               ws.nbytes, _stream(stream)))


def moe_expert_down(p, h, offsets, W2_e, out, ws, stream=None):
    _check(lib().moe_expert_down(C.byref(p), _p(h), _p(offsets), _p(W2_e), _p(out), ws.ptr,
                                 ws.nbytes, _stream(stream)))


def moe_expert_ffn(p, x_perm, offsets, W13_e, W2_e, h, out, ws, stream=None):
    _check(lib().moe_expert_ffn(C.byref(p), _p(x_perm), _p(offsets), _p(W13_e), _p(W2_e), _p(h),
                                _p(out), ws.ptr, ws.nbytes, _stream(stream)))


def moe_combine(p, out, slot_row, topk_w, y, stream=None):
    _check(lib().moe_combine(C.byref(p), _p(out), _p(slot_row), _p(topk_w), _p(y),
                             _stream(stream)))


def moe_gate_stats(p, counts, probs_sum, f, P, loss, stream=None):
    _check(lib().moe_gate_stats(C.byref(p), _p(counts), _p(probs_sum), _p(f), _p(P), _p(loss),
                                _stream(stream)))


class EpPlan:
    """Exchange plan of one rank of the expert-parallel layer (host int32 tensors):
    keep_all [N][E], send_row/send_cnt [E] (indexed by expert), recv_row/recv_cnt [E]
    (entry p*(E/N)+l: rank p's run for local expert l), in_offsets [E/N+1]."""

    def __init__(self, N, E, rank, keep_all, send_row, send_cnt, recv_row, recv_cnt, in_offsets):
        self.N, self.E, self.rank = N, E, rank
        self.E_local = E // N
        self.keep_all, self.send_row, self.send_cnt = keep_all, send_row, send_cnt
        self.recv_row, self.recv_cnt, self.in_offsets = recv_row, recv_cnt, in_offsets

    @property
    def rows_in(self) -> int:
        return int(self.in_offsets[-1])

    def send_runs(self):
        """(peer, first row, rows, expert) of the run this rank sends for each expert."""
        El = self.E_local
        return [(e // El, int(self.send_row[e]), int(self.send_cnt[e]), e)
                for e in range(self.E)]

    def recv_runs(self):
        """(peer, first row, rows, expert) of every run this rank receives, grouped by
        peer and in expert order inside a peer (the order the peer sends them in)."""
        El = self.E_local
        return [(i // El, int(self.recv_row[i]), int(self.recv_cnt[i]), self.rank * El + i % El)
                for i in range(self.E)]


def _host_i32(t, name):
    if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.int32 or \
            not t.is_contiguous():
        raise ValueError("%s must be a contiguous host int32 tensor" % name)
    return t.data_ptr()


def moe_ep_plan(counts_all, rank, capacity=-1, scope=EP_CAPACITY_GLOBAL) -> EpPlan:
    """counts_all: host int32 [N][E] (every rank's routed counts).  Runs on the host."""
    c = torch.as_tensor(counts_all, dtype=torch.int32).contiguous()
    if c.dim() != 2:
        raise ValueError("counts_all must be [N][E]")
    N, E = c.shape
    El = E // N if N > 0 and E >= N else 0
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)
    keep, srow, scnt, rrow, rcnt, ioff = z(N, E), z(E), z(E), z(E), z(E), z(El + 1)
    _check(lib().moe_ep_plan(_host_i32(c, "counts_all"), N, E, int(rank), int(capacity),
                             int(scope), keep.data_ptr(), srow.data_ptr(), scnt.data_ptr(),
                             rrow.data_ptr(), rcnt.data_ptr(), ioff.data_ptr()))
    return EpPlan(N, E, int(rank), keep, srow, scnt, rrow, rcnt, ioff)


def moe_ep_mask_slots(p, topk_idx, offsets, keep, slot_row, stream=None):
    """keep: host int32 [E] (this rank's row of EpPlan.keep_all)."""
    keep = torch.as_tensor(keep, dtype=torch.int32).contiguous()
    if keep.numel() < p.E:
        raise ValueError("keep needs E entries")
    _check(lib().moe_ep_mask_slots(C.byref(p), _p(topk_idx), _p(offsets),
                                   _host_i32(keep, "keep"), _p(slot_row), _stream(stream)))


def moe_ep_gate_stats(p, counts_all, N, probs_sum, counts, f, P, loss, stream=None):
    _check(lib().moe_ep_gate_stats(C.byref(p), _p(counts_all), int(N), _p(probs_sum),
                                   _p(counts), _p(f), _p(P), _p(loss), _stream(stream)))


class ForwardBuffers:
    """Every intermediate and output tensor of one layer forward, allocated with torch."""

    def __init__(self, p: Params, device="cuda"):
        dt = torch.bfloat16 if p.dtype == MOE_BF16 else torch.float32
        T, d, E, k = p.T, p.d, p.E, p.k
        rows = max(T * k, 1)
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.y = torch.empty(max(T, 1), d, dtype=dt, device=device)[:T]
        self.loss = torch.empty(1, **f32)
        self.counts = torch.empty(E, **i32)
        self.importance = torch.empty(E, **f32)
        self.f = torch.empty(E, **f32)
        self.P = torch.empty(E, **f32)
        self.topk_idx = torch.empty(max(T, 1), k, **i32)[:T]
        self.topk_w = torch.empty(max(T, 1), k, **f32)[:T]
        self.probs_sum = torch.empty(E, **f32)
        self.x_perm = torch.empty(rows, d, dtype=dt, device=device)
        self.row_token = torch.empty(rows, **i32)
        self.slot_row = torch.empty(max(T, 1), k, **i32)[:T]
        self.kept = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.h = torch.empty(rows, h_ld(p.m), dtype=dt, device=device)
        self.out = torch.empty(rows, d, dtype=dt, device=device)
        self.router_packed = None  # optional: moe_router_pack output for moe_forward


def moe_forward(p, x, Wg, W13_e, W2_e, ws, bufs: ForwardBuffers, Wnoise=None, noise=None,
                bias=None, stream=None, router_packed=None):
    b = _Buffers()
    vals = dict(x=x, Wg=Wg, Wnoise=Wnoise, noise=noise, bias=bias, W13_e=W13_e, W2_e=W2_e)
    if router_packed is not None:  # else bufs.router_packed (None: packed per call)
        vals["router_packed"] = router_packed
    for n in _BUF_FIELDS:
        t = vals[n] if n in vals else getattr(bufs, n)
        setattr(b, n, _p(t))
    _check(lib().moe_forward(C.byref(p), C.byref(b), ws.ptr, ws.nbytes, _stream(stream)))
    return bufs


def moe_partition_residual(W1, W3, W2, E, shared_idx, perm_rest, ws=None, stream=None):
    """a0 of the residual MoE: E disjoint experts over perm_rest and the shared block
    over shared_idx; returns (W13_e, W2_e, W13_s, W2_s) (include/moe.h)."""
    dt = _dtype_code(W1.dtype)
    d_ff, d = W1.shape
    m_s = shared_idx.numel()
    m = (d_ff - m_s) // E
    mk = lambda n: torch.empty(n, dtype=W1.dtype, device=W1.device)
    W13_e, W2_e = mk(packed_w13_elems(E, m, d)), mk(packed_w2_elems(E, m, d))
    W13_s, W2_s = mk(packed_w13_elems(1, m_s, d)), mk(packed_w2_elems(1, m_s, d))
    _check(lib().moe_partition_residual(_p(W1), _p(W3), _p(W2), d, d_ff, E, _p(shared_idx), m_s,
                                        _p(perm_rest), dt, _p(W13_e), _p(W2_e), _p(W13_s),
                                        _p(W2_s), ws.ptr if ws is not None else None,
                                        _stream(stream)))
    return W13_e, W2_e, W13_s, W2_s


def moe_combine_residual(p, out, slot_row, topk_w, resid, y, stream=None):
    _check(lib().moe_combine_residual(C.byref(p), _p(out), _p(slot_row), _p(topk_w), _p(resid),
                                      _p(y), _stream(stream)))


def moe_forward_residual(p, x, Wg, W13_e, W2_e, W13_s, W2_s, m_s, ws, bufs: ForwardBuffers, h_s,
                         out_s, Wnoise=None, noise=None, bias=None, stream=None):
    """The residual MoE layer: routed experts plus the shared block (include/moe.h)."""
    b = _Buffers()
    vals = dict(x=x, Wg=Wg, Wnoise=Wnoise, noise=noise, bias=bias, W13_e=W13_e, W2_e=W2_e)
    for n in _BUF_FIELDS:
        t = vals[n] if n in vals else getattr(bufs, n)
        setattr(b, n, _p(t))
    _check(lib().moe_forward_residual(C.byref(p), C.byref(b), _p(W13_s), _p(W2_s), int(m_s),
                                      _p(h_s), _p(out_s), ws.ptr, ws.nbytes, _stream(stream)))
    return bufs


def _host_ptr(t, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %r" % (name, type(t)))
    if t.is_cuda:
        raise ValueError("%s: the pipeline takes host tensors (pinned for overlap)" % name)
    if not t.is_contiguous():
        raise ValueError("%s: the pipeline takes contiguous tensors" % name)
    return t.data_ptr() or None


class Pipeline:
    """Host-buffer pipeline (include/moe_pipeline.h): batches in host memory go
    through the layer with up to ``depth`` of them in flight, copies overlapping
    the compute.  The weights are device tensors that must outlive the pipeline."""

    def __init__(self, p: Params, Wg, W13_e, W2_e, Wnoise=None, bias=None, depth=2):
        self._p = p
        self._keep = (Wg, W13_e, W2_e, Wnoise, bias)
        h = C.c_void_p(None)
        _check(lib().moe_pipeline_create(C.byref(p), _p(Wg), _p(Wnoise), _p(bias), _p(W13_e),
                                         _p(W2_e), int(depth), C.byref(h)))
        self._h = h
        self._held = {}

    def submit(self, x_host, y_host, loss_host, noise_host=None) -> int:
        """Enqueue one batch; returns its ticket.  The host tensors are held until
        wait() has returned for that ticket."""
        t = C.c_int64(-1)
        _check(lib().moe_pipeline_submit(self._h, _host_ptr(x_host, "x_host"),
                                         _host_ptr(noise_host, "noise_host"),
                                         _host_ptr(y_host, "y_host"),
                                         _host_ptr(loss_host, "loss_host"), C.byref(t)))
        self._held[t.value] = (x_host, noise_host, y_host, loss_host)
        return t.value

    def wait(self, ticket: int) -> None:
        _check(lib().moe_pipeline_wait(self._h, int(ticket)))
        for k in [k for k in self._held if k <= ticket]:
            del self._held[k]

    def close(self) -> None:
        if self._h is not None and self._h.value is not None:
            h, self._h = self._h, None
            self._held.clear()
            _check(lib().moe_pipeline_destroy(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_cluster_workspace_size(d, d_ff, E) -> int:
    return int(lib().moe_cluster_workspace_size(d, d_ff, E))


def moe_cluster_partition(F, E, n_iter, init_idx, ws=None, stream=None):
    """Balanced k-means partition of the rows of F [d_ff][d] into E clusters of
    d_ff/E neurons (include/moe.h).  Returns (assign, centers, perm, ws); ws is a
    Workspace-like object whose status word records a bad init index."""
    dt = _dtype_code(F.dtype)
    d_ff, d = F.shape
    dev = F.device
    if ws is None:
        n = moe_cluster_workspace_size(d, d_ff, E)
        if n <= 0:
            raise MoeError(MOE_ERR_SHAPE, "invalid shape for the clustering workspace")
        ws = Workspace(None, device=dev, nbytes=n)
    assign = torch.empty(d_ff, dtype=torch.int32, device=dev)
    perm = torch.empty(d_ff, dtype=torch.int32, device=dev)
    centers = torch.empty(E, d, dtype=torch.float64, device=dev)
    _check(lib().moe_cluster_partition(_p(F), d, d_ff, E, dt, n_iter, _p(init_idx), _p(assign),
                                       _p(centers), _p(perm), ws.ptr, ws.nbytes,
                                       _stream(stream)))
    return assign, centers, perm, ws


def moe_cluster_distances(F, centers, out=None, stream=None):
    """D [d_ff][E] f64: squared distances of the rows of F to the centers (f64)."""
    d_ff, d = F.shape
    E = centers.shape[0]
    D = out if out is not None else torch.empty(d_ff, E, dtype=torch.float64, device=F.device)
    _check(lib().moe_cluster_distances(_p(F), d, d_ff, E, _dtype_code(F.dtype), _p(centers),
                                       _p(D), _stream(stream)))
    return D


# --------------------------------------------------------------------------- backward

def moe_backward_workspace_size(p) -> int:
    return int(lib().moe_backward_workspace_size(C.byref(p)))


class BackwardBuffers:
    """Outputs and intermediates of moe_backward for layer p (include/moe.h)."""

    def __init__(self, p: Params, noisy: bool, biased: bool, device="cuda"):
        T, d, E, k = p.T, p.d, p.E, p.k
        dt = torch.bfloat16
        f32 = dict(dtype=torch.float32, device=device)
        rows = max(T * k, 1)
        self.dx = torch.empty(T, d, dtype=dt, device=device)
        self.dWg = torch.empty(d, E, **f32)
        self.dWnoise = torch.empty(d, E, **f32) if noisy else None
        self.dbias = torch.empty(E, **f32) if biased else None
        self.dW13_e = torch.empty(packed_w13_elems(E, p.m, d), dtype=dt, device=device)
        self.dW2_e = torch.empty(packed_w2_elems(E, p.m, d), dtype=dt, device=device)
        self.d_out = torch.empty(rows, d, dtype=dt, device=device)
        self.dG = torch.empty(T, k, **f32)
        self.dh = torch.empty(rows, h_ld(p.m), dtype=dt, device=device)
        self.dx_perm = torch.empty(rows, d, dtype=dt, device=device)


def moe_combine_backward(p, dy, out, slot_row, topk_w, d_out, dG, stream=None):
    _check(lib().moe_combine_backward(C.byref(p), _p(dy), _p(out), _p(slot_row), _p(topk_w),
                                      _p(d_out), _p(dG), _stream(stream)))


def moe_expert_down_backward(p, d_out, h, offsets, W2_e, dh, dW2_e, ws, stream=None):
    _check(lib().moe_expert_down_backward(C.byref(p), _p(d_out), _p(h), _p(offsets), _p(W2_e),
                                          _p(dh), _p(dW2_e), ws.ptr, ws.nbytes, _stream(stream)))


def moe_expert_up_backward(p, x_perm, dh, offsets, W13_e, dx_perm, dW13_e, ws, stream=None):
    _check(lib().moe_expert_up_backward(C.byref(p), _p(x_perm), _p(dh), _p(offsets), _p(W13_e),
                                        _p(dx_perm), _p(dW13_e), ws.ptr, ws.nbytes,
                                        _stream(stream)))


def moe_route_backward(p, x, Wg, topk_idx, topk_w, dG, counts, dx_perm, slot_row, dx, dWg, ws,
                       Wnoise=None, noise=None, bias=None, dWnoise=None, dbias=None, dLb=1.0,
                       stream=None):
    _check(lib().moe_route_backward(C.byref(p), _p(x), _p(Wg), _p(Wnoise), _p(noise), _p(bias),
                                    _p(topk_idx), _p(topk_w), _p(dG), _p(counts), float(dLb),
                                    _p(dx_perm), _p(slot_row), _p(dx), _p(dWg), _p(dWnoise),
                                    _p(dbias), ws.ptr, ws.nbytes, _stream(stream)))


def moe_backward(p, x, Wg, W13_e, W2_e, fwd: "ForwardBuffers", g: BackwardBuffers, dy, ws,
                 Wnoise=None, noise=None, bias=None, dLb=1.0, stream=None):
    """The whole backward of the batch whose forward filled `fwd` (include/moe.h)."""
    b = _Buffers()
    vals = dict(x=x, Wg=Wg, Wnoise=Wnoise, noise=noise, bias=bias, W13_e=W13_e, W2_e=W2_e)
    for n in _BUF_FIELDS:
        t = vals[n] if n in vals else getattr(fwd, n)
        setattr(b, n, _p(t))
    gb = _BwdBuffers()
    for n in _BWD_FIELDS:
        setattr(gb, n, _p(dy if n == "dy" else getattr(g, n)))
    _check(lib().moe_backward(C.byref(p), C.byref(b), C.byref(gb), float(dLb), ws.ptr, ws.nbytes,
                              _stream(stream)))
    return g


def moe_backward_residual_workspace_size(p, m_s) -> int:
    return int(lib().moe_backward_residual_workspace_size(C.byref(p), int(m_s)))


def moe_backward_residual(p, x, Wg, W13_e, W2_e, W13_s, W2_s, m_s, h_s, fwd: "ForwardBuffers",
                          g: BackwardBuffers, dy, dh_s, dx_s, dW13_s, dW2_s, ws, Wnoise=None,
                          noise=None, bias=None, dLb=1.0, stream=None):
    """Backward of the residual MoE layer (include/moe.h)."""
    b = _Buffers()
    vals = dict(x=x, Wg=Wg, Wnoise=Wnoise, noise=noise, bias=bias, W13_e=W13_e, W2_e=W2_e)
    for n in _BUF_FIELDS:
        t = vals[n] if n in vals else getattr(fwd, n)
        setattr(b, n, _p(t))
    gb = _BwdBuffers()
    for n in _BWD_FIELDS:
        setattr(gb, n, _p(dy if n == "dy" else getattr(g, n)))
    _check(lib().moe_backward_residual(C.byref(p), C.byref(b), C.byref(gb), _p(W13_s), _p(W2_s),
                                       int(m_s), _p(h_s), _p(dh_s), _p(dx_s), _p(dW13_s),
                                       _p(dW2_s), float(dLb), ws.ptr, ws.nbytes, _stream(stream)))
    return g


# --------------------------------------------------------------------------- mx4

def moe_mx4_codes_bytes(G, rows, K) -> int:
    return int(lib().moe_mx4_codes_bytes(G, rows, K))


def moe_mx4_scales_bytes(G, rows, K) -> int:
    return int(lib().moe_mx4_scales_bytes(G, rows, K))


def moe_mx4_rows_bytes(p, K) -> int:
    return int(lib().moe_mx4_rows_bytes(C.byref(p), K))


def moe_mx4_row_scales_bytes(p, K) -> int:
    return int(lib().moe_mx4_row_scales_bytes(C.byref(p), K))


class _Mx4Needs:
    """What the mx4 calls take for a layer: for each call a list of (name, type, least bytes) of
    its tensors, and for the weights the same with their exact bytes (more are another layout)."""

    def __init__(self, p):
        T, d, E, k, m = p.T, p.d, p.E, p.k, p.m
        if moe_mx4_rows_bytes(p, d) == 0:  # outside the contract: the library says how
            _check(lib().moe_mx4_dispatch(C.byref(p), *[None] * 7))
        u8, i32, f32 = torch.uint8, torch.int32, torch.float32
        dt, es = torch.bfloat16, 2  # the library refuses other layers, but for the dispatch
        m16, m8, rows = (m + 15) // 16 * 16, (m + 7) // 8 * 8, T * k
        some = min(T, 1)  # an empty batch needs no rows
        need = dict(
            x=(dt, T * d * es), Wg=(dt, d * E * es), Wnoise=(dt, d * E * es),
            noise=(f32, T * E * 4), bias=(f32, E * 4), y=(dt, T * d * es), loss=(f32, 4),
            counts=(i32, E * 4), importance=(f32, E * 4), f=(f32, E * 4), P=(f32, E * 4),
            topk_idx=(i32, rows * 4), topk_w=(f32, rows * 4), probs_sum=(f32, E * 4),
            row_token=(i32, rows * 4), slot_row=(i32, rows * 4), kept=(i32, E * 4),
            offsets=(i32, (E + 1) * 4), h=(dt, rows * m8 * es), out=(dt, rows * d * es),
            router_packed=(u8, moe_router_packed_bytes(p, False)))
        for n, K in (("x", d), ("h", m)):
            need[n + "_q"] = (u8, some * moe_mx4_rows_bytes(p, K))
            need[n + "_s"] = (u8, some * moe_mx4_row_scales_bytes(p, K))
        pick = lambda *names: [(n, *need[n]) for n in names]
        self.dispatch = pick("x") if p.dtype == MOE_BF16 else [("x", f32, T * d * 4)]
        self.dispatch += pick("topk_idx", "slot_row", "offsets", "x_q", "x_s")
        self.up = pick("x_q", "x_s", "offsets", "h_q", "h_s")
        self.down = pick("h_q", "h_s", "offsets", "out")
        self.ffn = pick("x_q", "x_s", "offsets", "h_q", "h_s", "out")
        inputs = pick("x", "noise", "router_packed")
        noisy = inputs[:-1] + [("router_packed", u8, moe_router_packed_bytes(p, True))]
        # by activations (bf16, mx4) and noise
        rest = (pick(*_MX4_OUTPUTS, "h"), pick(*_MX4_OUTPUTS, *_MX4_ROWS))
        self.forward = [[i + r for i in (inputs, noisy)] for r in rest]
        self.W13 = [("W13_q", u8, E * 2 * m16 * ((d + 31) // 32 * 16)),
                    ("W13_s", u8, moe_mx4_scales_bytes(E, 2 * m16, d))]
        self.W2 = [("W2_q", u8, moe_mx4_codes_bytes(E, d, m8)),
                   ("W2_s", u8, moe_mx4_scales_bytes(E, d, m8))]
        self.W = self.W13 + self.W2
        self.all_weights = pick("Wg", "Wnoise", "bias") + self.W


@functools.lru_cache(maxsize=256)
def _mx4_needs_of(params_bytes):
    return _Mx4Needs(Params.from_buffer_copy(params_bytes))


def _mx4_needs(p):
    return _mx4_needs_of(bytes(p))


def _mx4_refuse(t, name, dtype, need, exact):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %r" % (name, type(t)))
    if not t.is_cuda:
        raise ValueError("%s: libmoe takes CUDA tensors (got a %s tensor)" % (name, t.device))
    if t.get_device() != _current_device():
        raise ValueError("%s: on device %d, the current one is %d"
                         % (name, t.get_device(), _current_device()))
    if not t.is_contiguous():
        raise ValueError("%s: libmoe takes contiguous tensors" % name)
    raise ValueError("%s: needs %s%d bytes of %s, got %d of %s%s" % (
        name, "" if exact else "at least ", need, dtype, t.nbytes, t.dtype,
        ", its storage taken away" if t.untyped_storage().nbytes() < t.nbytes else ""))


def _mx4_ptrs(needs, *tensors):
    """The device pointers of a call's tensors, each compared with what the layer needs: type,
    bytes, contiguous, on the current device.  None stays NULL, for the library to judge."""
    dev = _current_device()
    for t, (name, dtype, least) in zip(tensors, needs):
        try:
            if (t.dtype is dtype and t.nbytes >= least and t.get_device() == dev
                    and t.is_contiguous()):
                continue
        except AttributeError:
            if t is None:
                continue
        _mx4_refuse(t, name, dtype, least, False)
    return [None if t is None else t.data_ptr() or None for t in tensors]


def _mx4_weights(needs, *tensors):
    """The same for weights: exactly the layer's bytes.  Programs take the storage of weights
    away, to offload or to gather them: data_ptr() is 0 then (NULL), or where the tensor lies
    inside its storage a bare offset, which is refused here."""
    dev = _current_device()
    for t, (name, dtype, n) in zip(tensors, needs):
        try:
            if (t.dtype is dtype and t.nbytes == n and t.get_device() == dev
                    and t.is_contiguous()
                    and (t.storage_offset() == 0 or t.untyped_storage().nbytes()
                         >= t.storage_offset() * t.element_size() + n)):
                continue
        except AttributeError:
            if t is None:
                continue
        _mx4_refuse(t, name, dtype, n, True)
    return [None if t is None else t.data_ptr() or None for t in tensors]


def _mx4_rows(t):
    """(pointer, G, rows, K, ld) of a matrix or batch of matrices whose columns are
    contiguous and whose rows are evenly spaced through the batch."""
    if t.dim() not in (2, 3):
        raise ValueError("expected [rows][K] or [G][rows][K], got %d dimensions" % t.dim())
    b = t if t.dim() == 3 else t.unsqueeze(0)
    G, rows, K = b.shape
    ld = b.stride(1) if rows > 1 else (b.stride(0) if G > 1 else K)
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors (got a %s tensor)" % t.device)
    if t.get_device() != _current_device():
        raise ValueError("the matrix is on device %d, the current one is %d"
                         % (t.get_device(), _current_device()))
    if b.stride(2) != 1 or (G > 1 and b.stride(0) != rows * ld):
        raise ValueError("the rows of the matrices must be contiguous and evenly spaced")
    return t.data_ptr() or None, G, rows, K, ld


def _mx4_pair(codes, scales, G, rows, K):
    """Pointers of a batch's codes and scales, of the right sizes."""
    out, dev = [], _current_device()
    for name, t, n in (("codes", codes, G * rows * ((K + 31) // 32 * 16)),
                       ("scales", scales, G * ((rows + 127) // 128) * ((K + 127) // 128) * 512)):
        if t.dtype != torch.uint8 or t.numel() != n:
            raise ValueError("%s must hold %d uint8 elements" % (name, n))
        ptr = _p(t)
        if t.get_device() != dev:
            _mx4_refuse(t, name, torch.uint8, n, True)
        out.append(ptr)
    return out


def moe_mx4_quantize(src, out=None, stream=None):
    """src [rows][K] or [G][rows][K] (bf16 or f32; rows may be spaced) in mx4: (codes
    [G][rows][K32/2], scales [G][rows/128][K/128][32][4][4]) uint8 (include/moe.h)."""
    ptr, G, rows, K, ld = _mx4_rows(src)
    if out is None:
        u8 = dict(dtype=torch.uint8, device=src.device)
        out = (torch.empty(G, rows, (K + 31) // 32 * 16, **u8),
               torch.empty(G, (rows + 127) // 128, (K + 127) // 128, 32, 4, 4, **u8))
    codes, scales = _mx4_pair(out[0], out[1], G, rows, K)
    _check(lib().moe_mx4_quantize(ptr, _dtype_code(src.dtype), G, rows, K, ld, codes, scales,
                                  _stream(stream)))
    return out


def moe_mx4_dequantize(codes, scales, K, dtype=torch.bfloat16, out=None, stream=None):
    """The values [G][rows][K] of an mx4 batch (codes [G][rows][K32/2] as moe_mx4_quantize
    gives them); with ``out`` its dtype and row spacing count."""
    G, rows = codes.shape[0], codes.shape[1]
    if out is None:
        out = torch.empty(G, rows, K, dtype=dtype, device=codes.device)
    ptr, Go, ro, Ko, ld = _mx4_rows(out)
    if (Go, ro, Ko) != (G, rows, K):
        raise ValueError("out must be [%d][%d][%d]" % (G, rows, K))
    cp, sp = _mx4_pair(codes, scales, G, rows, K)
    _check(lib().moe_mx4_dequantize(cp, sp, _dtype_code(out.dtype), G, rows, K, ld, ptr,
                                    _stream(stream)))
    return out


class Mx4Experts:
    """The packed expert weights of a layer in mx4: W13_q / W13_s of W13_e [E][2*m16][d] and
    W2_q / W2_s of W2_e [E][d][m8].  A call reads where its tensors lie at that moment, so they
    may be set anew or get another storage between calls, and refuses (ValueError) any that are
    not of the layer's sizes, uint8, contiguous and on the current device."""

    def __init__(self, W13_q, W13_s, W2_q, W2_s):
        self.W13_q, self.W13_s, self.W2_q, self.W2_s = W13_q, W13_s, W2_q, W2_s

    @classmethod
    def quantize(cls, W13_e, W2_e, E, m, d, stream=None):
        """From the packed weights of moe_partition_experts (bf16 or f32)."""
        m16, m8 = (m + 15) // 16 * 16, (m + 7) // 8 * 8
        return cls(*moe_mx4_quantize(W13_e.view(E, 2 * m16, d), stream=stream),
                   *moe_mx4_quantize(W2_e.view(E, d, m8), stream=stream))


def moe_mx4_dispatch(p, x, topk_idx, slot_row, offsets, x_q, x_s, stream=None):
    """a2's row copy in mx4 (after moe_dispatch_rows)."""
    t = _mx4_ptrs(_mx4_needs(p).dispatch, x, topk_idx, slot_row, offsets, x_q, x_s)
    _check(lib().moe_mx4_dispatch(C.byref(p), *t, _stream(stream)))


def moe_expert_up_mx4(p, x_q, x_s, offsets, W: Mx4Experts, h_q, h_s, ws, stream=None):
    needs = _mx4_needs(p)
    t = _mx4_ptrs(needs.up, x_q, x_s, offsets, h_q, h_s)
    t[3:3] = _mx4_weights(needs.W13, W.W13_q, W.W13_s)
    _check(lib().moe_expert_up_mx4(C.byref(p), *t, ws.ptr, ws.nbytes, _stream(stream)))


def moe_expert_down_mx4(p, h_q, h_s, offsets, W: Mx4Experts, out, ws, stream=None):
    needs = _mx4_needs(p)
    t = _mx4_ptrs(needs.down, h_q, h_s, offsets, out)
    t[3:3] = _mx4_weights(needs.W2, W.W2_q, W.W2_s)
    _check(lib().moe_expert_down_mx4(C.byref(p), *t, ws.ptr, ws.nbytes, _stream(stream)))


def moe_expert_ffn_mx4(p, x_q, x_s, offsets, W: Mx4Experts, h_q, h_s, out, ws, stream=None):
    needs = _mx4_needs(p)
    t = _mx4_ptrs(needs.ffn, x_q, x_s, offsets, h_q, h_s, out)
    t[3:3] = _mx4_weights(needs.W, W.W13_q, W.W13_s, W.W2_q, W.W2_s)
    _check(lib().moe_expert_ffn_mx4(C.byref(p), *t, ws.ptr, ws.nbytes, _stream(stream)))


class Mx4Buffers:
    """Outputs and intermediates of moe_forward_mx4 for layer p, allocated with torch.
    ``act`` limits the intermediates to those of one form (None: both).  A tensor given by
    name (Mx4Buffers(p, y=mine)) is used instead of a new one.  A call for another layer than p
    refuses buffers that are too small for it."""

    def __init__(self, p: Params, act=None, device="cuda", **given):
        T, d, E, k, m = p.T, p.d, p.E, p.k, p.m
        rows = T * k
        i32, f32, b16, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
        shapes = dict(y=((T, d), b16), loss=((1,), f32), counts=((E,), i32),
                      importance=((E,), f32), f=((E,), f32), P=((E,), f32),
                      topk_idx=((T, k), i32), topk_w=((T, k), f32), probs_sum=((E,), f32),
                      row_token=((rows,), i32), slot_row=((T, k), i32), kept=((E,), i32),
                      offsets=((E + 1,), i32))
        if act != MX4_ACT_MX4:
            shapes["h"] = ((max(rows, 1), h_ld(m)), b16)
        if act != MX4_ACT_BF16:
            for n, K in (("x", d), ("h", m)):
                shapes[n + "_q"] = ((moe_mx4_rows_bytes(p, K),), u8)
                shapes[n + "_s"] = ((moe_mx4_row_scales_bytes(p, K),), u8)
            shapes["out"] = ((rows, d), b16)
        bad = set(given) - set(_MX4_FIELDS[10:])
        if bad:
            raise TypeError("not a buffer of moe_forward_mx4: %s" % ", ".join(sorted(bad)))
        for n in _MX4_FIELDS[10:]:
            t = given.get(n)
            if t is None and n in shapes:
                t = torch.empty(shapes[n][0], dtype=shapes[n][1], device=device)
            elif t is not None and n in shapes:
                need = 1
                for v in shapes[n][0]:
                    need *= v
                if t.dtype != shapes[n][1] or t.numel() < need:
                    raise ValueError("%s needs %d elements of %s" % (n, need, shapes[n][1]))
            setattr(self, n, t)


def moe_forward_mx4(p, x, Wg, W: Mx4Experts, ws, bufs: Mx4Buffers, act=MX4_ACT_BF16, Wnoise=None,
                    noise=None, bias=None, router_packed=None, stream=None):
    """The whole layer on mx4 expert weights (include/moe.h): at most 16 tokens with bf16
    activations (MX4_ACT_BF16), or any number with quantised rows (MX4_ACT_MX4)."""
    act = int(act)
    few = act == MX4_ACT_BF16 and p.T > 0
    if (isinstance(router_packed, torch.Tensor) and router_packed.dtype is not torch.uint8
            and router_packed.is_contiguous()):  # moe_router_pack fills a buffer of any type
        router_packed = router_packed.view(torch.uint8)
    needs = _mx4_needs(p)
    x, noise, router_packed, *t = _mx4_ptrs(
        needs.forward[0 if few else 1][0 if Wnoise is None else 1], x, noise, router_packed,
        *(_mx4_few_tensors if few else _mx4_row_tensors)(bufs))
    Wg, Wnoise, bias, *w = _mx4_weights(needs.all_weights, Wg, Wnoise, bias, W.W13_q, W.W13_s,
                                        W.W2_q, W.W2_s)
    if not few:
        t.insert(len(_MX4_OUTPUTS), None)  # h
    b = _Mx4Buffers(x, Wg, Wnoise, noise, bias, *w, router_packed, *t)
    _check(lib().moe_forward_mx4(C.byref(p), C.byref(b), act, ws.ptr, ws.nbytes,
                                 _stream(stream)))
    return bufs
