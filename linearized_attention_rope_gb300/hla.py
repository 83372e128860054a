"""ctypes binding of libhla (include/hla.h).

Argument marshalling only: tensors are passed as ``data_ptr()`` and the
stream as ``torch.cuda.current_stream().cuda_stream``.  Every step of the
layer runs in libhla's CUDA kernels; there is no Python or CPU fallback, and
calling into the library without a built ``libhla.so`` raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhla.so")

HLA_OK = 0
HLA_ERR_INVALID_ARG = 1
HLA_ERR_UNSUPPORTED = 2
HLA_ERR_STATE = 3
HLA_ERR_CUDA = 4
HLA_ERR_TIMEOUT = 5
HLA_ERR_WORKSPACE = 6

DTYPE_F32 = 0
DTYPE_BF16 = 1
DTYPE_E4M3 = 2  # caches only
ROPE_HALF = 0
ROPE_INTERLEAVED = 1
ROPE_SCALE_NONE = 0
ROPE_SCALE_LINEAR = 1
ROPE_SCALE_BANDS = 2
ROPE_SCALE_YARN = 3
FLAG_L2NORM_Q = 0x1
FLAG_SOFTMAX_OFF = 0x2
FLAG_LINEAR_OFF = 0x4
FLAG_GDN_RECURRENT = 0x8
FLAG_GLA = 0x10
FLAG_TEST_STALL = 0x20
FLAG_GDN_SCAN = 0x40

STATE_FIELDS = ("S", "k_ring", "v_ring", "pend_k", "pend_v", "pend_g", "pend_beta", "conv_q",
                "conv_k", "conv_v", "pos", "err", "scratch")


class HlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class CParams(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("n_sinks", ctypes.c_int), ("window", ctypes.c_int),
                ("conv_width", ctypes.c_int), ("rope_base", ctypes.c_float),
                ("dtype", ctypes.c_int), ("flags", ctypes.c_uint)]


class CState(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in STATE_FIELDS]


class CStateSizes(ctypes.Structure):
    _fields_ = [(name, ctypes.c_size_t) for name in STATE_FIELDS]


class CRopeParams(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int), ("scaling", ctypes.c_int),
                ("dtype", ctypes.c_int), ("original_len", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64)]


class CAttnParams(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("reserved", ctypes.c_int),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64)]


class CCacheParams(ctypes.Structure):
    _fields_ = [("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("cache_dtype", ctypes.c_int), ("page_size", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("reserved", ctypes.c_int)]


class CCache(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("k", "v", "k_exp", "v_exp", "page_table", "err")]


_vp = ctypes.c_void_p
_lib = None


def load():
    """Loads libhla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libhla.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(CParams)
        S = ctypes.POINTER(CState)
        lib.hla_status_string.argtypes = [ctypes.c_int]
        lib.hla_status_string.restype = ctypes.c_char_p
        lib.hla_state_bytes.argtypes = [P, ctypes.c_int, ctypes.POINTER(CStateSizes)]
        lib.hla_prefill_workspace_bytes.argtypes = [P, ctypes.c_int64, ctypes.c_int,
                                                    ctypes.POINTER(ctypes.c_size_t)]
        lib.hla_state_init.argtypes = [P, ctypes.c_int, S, _vp]
        lib.hla_prefill.argtypes = [P] + [_vp] * 10 + [ctypes.c_int, ctypes.c_int64, _vp, S, _vp,
                                                       ctypes.c_size_t, _vp]
        lib.hla_decode_step.argtypes = [P, ctypes.c_int] + [_vp] * 9 + [S, _vp, _vp]
        lib.hla_check_device_error.argtypes = [S, _vp, ctypes.POINTER(ctypes.c_int32)]
        lib.hla_check_workspace_error.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_int32)]
        lib.hla_prefill_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
        lib.hla_prefill_launch_count.argtypes = [P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        lib.hla_prefill_noalloc.argtypes = [P] + [_vp] * 10 + [ctypes.c_int, ctypes.c_int64, _vp, S, _vp]
        lib.hla_prefill_noalloc.restype = ctypes.c_int
        lib.hla_prefill_continue.argtypes = [P] + [_vp] * 10 + [ctypes.c_int, ctypes.c_int64, _vp, S, _vp,
                                                                ctypes.c_size_t, _vp]
        lib.hla_prefill_continue.restype = ctypes.c_int
        lib.hla_prefill_continue_workspace_bytes.argtypes = [P, ctypes.c_int64, ctypes.c_int,
                                                             ctypes.POINTER(ctypes.c_size_t)]
        lib.hla_prefill_continue_workspace_bytes.restype = ctypes.c_int
        lib.hla_prefill_diagnostics.argtypes = [P] + [_vp] * 10 + [ctypes.c_int, ctypes.c_int64, _vp, _vp, _vp,
                                                                   _vp, ctypes.c_size_t, _vp]
        lib.hla_prefill_diagnostics.restype = ctypes.c_int
        lib.hla_backward_workspace_bytes.argtypes = [P, ctypes.c_int64, ctypes.c_int,
                                                     ctypes.POINTER(ctypes.c_size_t)]
        lib.hla_backward_workspace_bytes.restype = ctypes.c_int
        lib.hla_backward.argtypes = [P] + [_vp] * 10 + [ctypes.c_int, ctypes.c_int64] + [_vp] * 10 + [
            _vp, ctypes.c_size_t, _vp]
        lib.hla_backward.restype = ctypes.c_int
        lib.hla_prefill_noalloc_check_error.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]
        lib.hla_prefill_noalloc_check_error.restype = ctypes.c_int
        RP, AP, CP = (ctypes.POINTER(t) for t in (CRopeParams, CAttnParams, CCacheParams))
        C, i64, size_p = ctypes.POINTER(CCache), ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
        for name, args in {
                "hla_rope_frequencies": [RP, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)],
                "hla_rope": [RP, _vp, _vp, _vp, i64, _vp, _vp, _vp],
                "hla_rope_backward": [RP, _vp, _vp, _vp, i64, _vp, _vp, _vp],
                "hla_attention_workspace_bytes": [AP, i64, i64, ctypes.c_int, ctypes.c_int, size_p],
                "hla_attention": [AP] + [_vp] * 5 + [ctypes.c_int, i64, i64, _vp, _vp, _vp, ctypes.c_size_t, _vp],
                "hla_attention_backward": [AP] + [_vp] * 8 + [ctypes.c_int, i64, i64] + [_vp] * 4 +
                                          [ctypes.c_size_t, _vp],
                "hla_cache_bytes": [CP, size_p, size_p],
                "hla_cache_write": [CP, C, _vp, _vp, _vp, _vp, ctypes.c_int, i64, _vp],
                "hla_cache_read": [CP, C, _vp, _vp, ctypes.c_int, i64, _vp, _vp, _vp],
                "hla_attention_decode_workspace_bytes": [AP, CP, size_p],
                "hla_attention_decode": [AP, CP, C, _vp, _vp, ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp],
                "hla_check_cache_error": [C, _vp, ctypes.POINTER(ctypes.c_int32)]}.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        for fn in ("hla_state_bytes", "hla_prefill_workspace_bytes", "hla_state_init", "hla_prefill",
                   "hla_decode_step", "hla_check_device_error", "hla_check_workspace_error",
                   "hla_prefill_stage_events", "hla_prefill_launch_count"):
            getattr(lib, fn).restype = ctypes.c_int
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().hla_status_string(status).decode()


def _check(rc: int, what: str):
    if rc != HLA_OK:
        raise HlaError(rc, what)


@dataclass
class Params:
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    n_sinks: int
    window: int
    dtype: int = DTYPE_BF16
    rope_base: float = 500000.0
    flags: int = FLAG_L2NORM_Q
    conv_width: int = 8

    def c(self) -> CParams:
        return CParams(self.n_q_heads, self.n_kv_heads, self.head_dim, self.n_sinks, self.window,
                       self.conv_width, self.rope_base, self.dtype, self.flags)

    @property
    def torch_dtype(self):
        return torch.float32 if self.dtype == DTYPE_F32 else torch.bfloat16


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def workspace_bytes(params: Params, total_tokens: int, n_seqs: int) -> int:
    n = ctypes.c_size_t()
    _check(load().hla_prefill_workspace_bytes(ctypes.byref(params.c()), total_tokens, n_seqs,
                                              ctypes.byref(n)), "hla_prefill_workspace_bytes")
    return n.value


def state_sizes(params: Params, n_seqs: int) -> dict:
    s = CStateSizes()
    _check(load().hla_state_bytes(ctypes.byref(params.c()), n_seqs, ctypes.byref(s)),
           "hla_state_bytes")
    return {name: getattr(s, name) for name in STATE_FIELDS}


class State:
    """Decode state of n_seqs sequences; the buffers are torch uint8 tensors."""

    def __init__(self, params: Params, n_seqs: int, device="cuda"):
        self.params, self.n_seqs = params, n_seqs
        self.buffers = {name: torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
                        for name, nbytes in state_sizes(params, n_seqs).items()}
        self.c = CState(*[b.data_ptr() for b in self.buffers.values()])

    def view(self, name: str):
        """Typed view of one buffer (S, pend_* and conv_* fp32; rings in the layer dtype;
        pos int64; err int32)."""
        b = self.buffers[name]
        dt = {"k_ring": self.params.torch_dtype, "v_ring": self.params.torch_dtype,
              "pos": torch.int64, "err": torch.int32}.get(name, torch.float32)
        n = state_sizes(self.params, self.n_seqs)[name] // torch.tensor([], dtype=dt).element_size()
        return b.view(dt)[:n]

    def init(self, stream=None):
        _check(load().hla_state_init(ctypes.byref(self.params.c()), self.n_seqs,
                                     ctypes.byref(self.c), _stream(stream)), "hla_state_init")
        return self

    def check_error(self, stream=None) -> int:
        """Synchronises, reads and clears the device error word; returns it (0 = fine)."""
        code = ctypes.c_int32()
        rc = load().hla_check_device_error(ctypes.byref(self.c), _stream(stream), ctypes.byref(code))
        if rc not in (HLA_OK, HLA_ERR_STATE, HLA_ERR_TIMEOUT):
            _check(rc, "device error word")
        return code.value


def alloc_workspace(params: Params, total_tokens: int, n_seqs: int, device="cuda"):
    return torch.empty(workspace_bytes(params, total_tokens, n_seqs), dtype=torch.uint8,
                       device=device)


def prefill(params: Params, q, k, v, g, beta, lam, wq, wk, wv, cu_seqlens, out, state=None,
            ws=None, stream=None):
    """hla_prefill on torch tensors (all on the GPU, contiguous)."""
    n_seqs = cu_seqlens.numel() - 1
    total = q.shape[0]
    if ws is None:
        ws = alloc_workspace(params, total, n_seqs, q.device)
    rc = load().hla_prefill(ctypes.byref(params.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                            _ptr(lam), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(cu_seqlens), n_seqs, total,
                            _ptr(out), None if state is None else ctypes.byref(state.c), _ptr(ws),
                            ws.numel(), _stream(stream))
    _check(rc, "hla_prefill")
    return ws


def continue_workspace_bytes(params: Params, total_tokens: int, n_seqs: int) -> int:
    n = ctypes.c_size_t()
    _check(load().hla_prefill_continue_workspace_bytes(ctypes.byref(params.c()), total_tokens, n_seqs,
                                                       ctypes.byref(n)), "hla_prefill_continue_workspace_bytes")
    return n.value


def prefill_continue(params: Params, q, k, v, g, beta, lam, wq, wk, wv, cu_seqlens, out, state: State, ws=None,
                     stream=None):
    """hla_prefill_continue: appends the tokens of every sequence to the context `state` holds."""
    n_seqs = cu_seqlens.numel() - 1
    total = q.shape[0]
    if ws is None:
        ws = torch.empty(continue_workspace_bytes(params, total, n_seqs), dtype=torch.uint8, device=q.device)
    rc = load().hla_prefill_continue(ctypes.byref(params.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                     _ptr(lam), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(cu_seqlens), n_seqs, total,
                                     _ptr(out), ctypes.byref(state.c), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "hla_prefill_continue")
    return ws


def prefill_diagnostics(params: Params, q, k, v, g, beta, lam, wq, wk, wv, cu_seqlens, out=None, ws=None,
                        stream=None):
    """hla_prefill_diagnostics: returns (branch_sq [n_seqs, Hq, 2], key_stats [total, Hkv, 2]), fp32
    tensors on the GPU (|o_sm|^2 and |lambda o_lin|^2 summed per sequence and head; key concentration
    and projection residual per position and kv head)."""
    n_seqs = cu_seqlens.numel() - 1
    total = q.shape[0]
    if ws is None:
        ws = alloc_workspace(params, total, n_seqs, q.device)
    if out is None:
        out = torch.empty_like(q)
    branch_sq = torch.empty((n_seqs, params.n_q_heads, 2), dtype=torch.float32, device=q.device)
    key_stats = torch.empty((total, params.n_kv_heads, 2), dtype=torch.float32, device=q.device)
    rc = load().hla_prefill_diagnostics(ctypes.byref(params.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                        _ptr(lam), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(cu_seqlens), n_seqs, total,
                                        _ptr(out), _ptr(branch_sq), _ptr(key_stats), _ptr(ws), ws.numel(),
                                        _stream(stream))
    _check(rc, "hla_prefill_diagnostics")
    return branch_sq, key_stats


def backward_workspace_bytes(params: Params, total_tokens: int, n_seqs: int) -> int:
    n = ctypes.c_size_t()
    _check(load().hla_backward_workspace_bytes(ctypes.byref(params.c()), total_tokens, n_seqs, ctypes.byref(n)),
           "hla_backward_workspace_bytes")
    return n.value


BACKWARD_GRADS = ("q", "k", "v", "g", "beta", "lam", "wq", "wk", "wv")


def backward(params: Params, q, k, v, g, beta, lam, wq, wk, wv, cu_seqlens, dout, grads=None, ws=None,
             stream=None):
    """hla_backward: the gradients of sum(dout * o) as a dict of fp32 GPU tensors named as in
    BACKWARD_GRADS, shaped like the inputs (q [total, Hq, d]; k, v [total, Hkv, d]; g, beta
    [total, Hq]; lam [Hq]; wq [Hq * d, 8]; wk, wv [Hkv * d, 8]).  `grads` (same dict) and `ws`
    (a uint8 tensor of backward_workspace_bytes) may be passed in to be reused."""
    n_seqs = cu_seqlens.numel() - 1
    total = q.shape[0]
    if ws is None:
        ws = torch.empty(backward_workspace_bytes(params, total, n_seqs), dtype=torch.uint8, device=q.device)
    if grads is None:
        src = dict(zip(BACKWARD_GRADS, (q, k, v, g, beta, lam, wq, wk, wv)))
        grads = {n: torch.empty(t.shape, dtype=torch.float32, device=q.device) for n, t in src.items()}
    rc = load().hla_backward(ctypes.byref(params.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(lam),
                             _ptr(wq), _ptr(wk), _ptr(wv), _ptr(cu_seqlens), n_seqs, total, _ptr(dout),
                             *[_ptr(grads[n]) for n in BACKWARD_GRADS], _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "hla_backward")
    return grads


def decode_step(params: Params, q, k, v, g, beta, lam, wq, wk, wv, state: State, out, stream=None):
    """hla_decode_step on torch tensors: q [N,Hq,d], k, v [N,Hkv,d], g, beta [N,Hq]."""
    rc = load().hla_decode_step(ctypes.byref(params.c()), state.n_seqs, _ptr(q), _ptr(k), _ptr(v),
                                _ptr(g), _ptr(beta), _ptr(lam), _ptr(wq), _ptr(wk), _ptr(wv),
                                ctypes.byref(state.c), _ptr(out), _stream(stream))
    _check(rc, "hla_decode_step")


def check_workspace_error(ws, stream=None) -> int:
    """Synchronises, reads and clears a prefill workspace's error word; returns it."""
    code = ctypes.c_int32()
    rc = load().hla_check_workspace_error(_ptr(ws), _stream(stream), ctypes.byref(code))
    if rc not in (HLA_OK, HLA_ERR_STATE, HLA_ERR_TIMEOUT):
        _check(rc, "workspace error word")
    return code.value


PREFILL_STAGES = ("features", "gdn", "softmax", "state_fill")
_stage_handles = None


def set_prefill_stage_events(events):
    """Makes hla_prefill record the given torch.cuda.Event objects (already
    recorded once, so their handles exist) at its stage boundaries on this
    thread; None switches the hook off."""
    global _stage_handles
    if events is None:
        _stage_handles = None
        _check(load().hla_prefill_stage_events(None, 0), "hla_prefill_stage_events")
        return
    _stage_handles = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(load().hla_prefill_stage_events(_stage_handles, len(events)), "hla_prefill_stage_events")


def prefill_launch_count(params: Params, with_state: bool = False) -> int:
    """hla_prefill_launch_count: kernels launched by one prefill call."""
    n = ctypes.c_int(0)
    _check(load().hla_prefill_launch_count(ctypes.byref(params.c()), int(with_state), ctypes.byref(n)),
           "hla_prefill_launch_count")
    return n.value


def prefill_noalloc(params: Params, q, k, v, g, beta, lam, wq, wk, wv, cu_seqlens, out, state=None,
                    stream=None):
    """hla_prefill_noalloc: the prefill with the library's own 64 MiB scratch, for
    callers that cannot allocate device memory; raises HlaError(HLA_ERR_WORKSPACE)
    for prefills that need more scratch than that."""
    rc = load().hla_prefill_noalloc(ctypes.byref(params.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                    _ptr(beta), _ptr(lam), _ptr(wq), _ptr(wk), _ptr(wv),
                                    _ptr(cu_seqlens), cu_seqlens.numel() - 1, q.shape[0], _ptr(out),
                                    None if state is None else ctypes.byref(state.c), _stream(stream))
    _check(rc, "hla_prefill_noalloc")


def prefill_noalloc_check_error(stream=None) -> int:
    """hla_prefill_noalloc_check_error: synchronises, reads and clears the error
    word of the library's own prefill buffer on the current device; returns it."""
    code = ctypes.c_int32()
    rc = load().hla_prefill_noalloc_check_error(_stream(stream), ctypes.byref(code))
    if rc not in (HLA_OK, HLA_ERR_STATE, HLA_ERR_TIMEOUT):
        _check(rc, "hla_prefill_noalloc_check_error")
    return code.value


# ---- full softmax layers: rotary positions, packed attention, paged cache, decode ----------------------
#
# These calls check their tensors (type, shape, device, strides) and raise HlaError with
# HLA_ERR_INVALID_ARG before anything is launched; they run on the tensors' device, on `stream` or that
# device's current stream.  Of tensors handed to a call on another `stream`, the memory is not given out again
# before that stream has passed the call.

_TORCH = {DTYPE_F32: torch.float32, DTYPE_BF16: torch.bfloat16, DTYPE_E4M3: torch.uint8}


def _refuse(what: str):
    raise HlaError(HLA_ERR_INVALID_ARG, what)


def _need(ok, what: str):
    if not ok:
        _refuse(what)


def _check_tensor(t, fn: str, name: str, dtype, shape, device, strided: bool = False) -> int:
    """The token stride of t in elements; t must have the type, shape and device given and be dense, or
    (strided) have dense rows at any token stride."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        _refuse(f"{fn}: {name}: expected a {dtype} tensor")
    if t.shape != shape:
        _refuse(f"{fn}: {name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        _refuse(f"{fn}: {name}: expected on {device}, got {t.device}")
    if t.is_contiguous() or t.numel() == 0:
        return shape[1] * shape[2] if len(shape) == 3 else 0
    if not (strided and len(shape) == 3 and t.stride(2) == 1 and (t.stride(1) == shape[2] or shape[1] == 1) and
            t.stride(0) >= shape[1] * shape[2]):
        _refuse(f"{fn}: {name}: expected dense {'rows' if strided else 'storage'}")
    return t.stride(0)


@functools.lru_cache(maxsize=256)
def _c(params, *strides):
    """A frozen parameter set's C form, by reference; made once per set and strides, never changed."""
    return ctypes.byref(params.c(*strides))


def _like(t, stride: int):
    """An uninitialised dense tensor of t's shape; stride: t's token stride, from _check_tensor."""
    if stride == t.shape[1] * t.shape[2]:
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _adr(t):
    """The address of a tensor as an int (0 for none), which ctypes takes as it is."""
    return None if t is None else t.data_ptr()


# A device's current stream as an int.  (Through torch.cuda.current_stream it takes 2 us, a tenth of a small call.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _here(device, stream):
    """The current stream of `device` as an int, or None if `stream` or `device` has to be made current first."""
    if device.type != "cuda":
        _refuse(f"expected CUDA tensors, got {device}")
    if stream is not None or device.index != torch.cuda.current_device():
        return None
    return _raw_stream(device.index)


def _on(device, stream, *tensors):
    """A context with `device` current, and `stream` too if one is given, so that buffers allocated in it belong
    to the stream that uses them; `tensors`, the call's own, stay theirs until that stream is done with them."""
    if stream is None:
        return torch.cuda.device(device)
    _need(stream.device == device, f"expected a stream of {device}, got one of {stream.device}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


@dataclass(frozen=True)
class RopeParams:
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    rot_dim: int = 0            # 0: the whole head
    layout: int = ROPE_HALF
    scaling: int = ROPE_SCALE_NONE
    dtype: int = DTYPE_BF16
    base: float = 500000.0
    factor: float = 1.0
    original_len: int = 8192
    low: float = 0.0            # band edges in turns; 0, 0: the scaling's own
    high: float = 0.0

    def c(self, q_stride: int = 0, k_stride: int = 0) -> CRopeParams:
        return CRopeParams(self.n_q_heads, self.n_kv_heads, self.head_dim, self.rot_dim or self.head_dim, self.layout,
                           self.scaling, self.dtype, self.original_len, self.base, self.factor, self.low, self.high,
                           q_stride, k_stride)


def rope_frequencies(params: RopeParams):
    """hla_rope_frequencies: (scaled angle per position of every pair, as a list; factor on rotated values)."""
    c = params.c()
    w, gain = (ctypes.c_double * max(1, c.rot_dim // 2))(), ctypes.c_double()
    _check(load().hla_rope_frequencies(ctypes.byref(c), w, ctypes.byref(gain)), "hla_rope_frequencies")
    return list(w), gain.value


def _rope(fn, params, q, k, positions, q_out, k_out, stream):
    dt = _TORCH.get(params.dtype)
    _need(dt is not None and dt != torch.uint8, f"{fn}: dtype")
    _need(isinstance(positions, torch.Tensor) and positions.dim() == 1, f"{fn}: positions must be a vector")
    n, dev, strides, outs = positions.numel(), positions.device, [0, 0], [q_out, k_out]
    _check_tensor(positions, fn, "positions", torch.int64, (n,), dev)
    for i, (x, o, heads, name) in enumerate(((q, q_out, params.n_q_heads, "q"), (k, k_out, params.n_kv_heads, "k"))):
        if x is None:
            _need(o is None, f"{fn}: {name}_out without {name}")
            continue
        shape = (n, heads, params.head_dim)
        strides[i] = _check_tensor(x, fn, name, dt, shape, dev, strided=True)
        if o is None:
            pass
        elif o.data_ptr() == x.data_ptr():
            _need(o.shape == x.shape and o.dtype == x.dtype and o.stride() == x.stride(), f"{fn}: {name}_out in place")
        else:
            _check_tensor(o, fn, name + "_out", dt, shape, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, q, k, positions, q_out, k_out):
            return _rope(fn, params, q, k, positions, q_out, k_out, None)
    for i, x in enumerate((q, k)):
        if x is not None and outs[i] is None:
            outs[i] = _like(x, strides[i])
    _check(getattr(load(), fn)(_c(params, *strides), _adr(q), _adr(k), positions.data_ptr(), n, _adr(outs[0]),
                               _adr(outs[1]), st), fn)
    return outs[0], outs[1]


def rope(params: RopeParams, q, k, positions, q_out=None, k_out=None, stream=None):
    """hla_rope: (q_out, k_out), q [T, Hq, d] and k [T, Hkv, d] (either may be None) rotated to positions
    [T] int64.  Rows may be slices of a wider tensor; q_out=q / k_out=k rotate in place."""
    return _rope("hla_rope", params, q, k, positions, q_out, k_out, stream)


def rope_backward(params: RopeParams, dq_out, dk_out, positions, dq=None, dk=None, stream=None):
    """hla_rope_backward: the gradients of rope's inputs from those of its outputs."""
    return _rope("hla_rope_backward", params, dq_out, dk_out, positions, dq, dk, stream)


@dataclass(frozen=True)
class AttnParams:
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    dtype: int = DTYPE_BF16
    scale: float = 0.0          # 0: 1 / sqrt(head_dim)

    def c(self, q_stride: int = 0, k_stride: int = 0, v_stride: int = 0) -> CAttnParams:
        return CAttnParams(self.n_q_heads, self.n_kv_heads, self.head_dim, self.dtype, self.scale, 0, q_stride,
                           k_stride, v_stride)


def _zeroed(n: int, device):
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the error word
    return ws


def attention_workspace_bytes(params: AttnParams, total_q: int, total_k: int, n_seqs: int,
                              backward: bool = False) -> int:
    """hla_attention_workspace_bytes: with which a call of these sizes takes the parts that suit it.  The workspace of the
    largest call serves every smaller one, in as many parts as it has room for."""
    n = ctypes.c_size_t()
    _check(load().hla_attention_workspace_bytes(_c(params), total_q, total_k, n_seqs, int(backward),
                                                ctypes.byref(n)), "hla_attention_workspace_bytes")
    return n.value


def alloc_attention_workspace(params: AttnParams, total_q: int, total_k: int, n_seqs: int, backward: bool = False,
                              device="cuda"):
    """A workspace for attention (and, backward=True, attention_backward) with its error word zeroed;
    check_workspace_error reads it."""
    n = attention_workspace_bytes(params, total_q, total_k, n_seqs)
    if backward:
        n = max(n, attention_workspace_bytes(params, total_q, total_k, n_seqs, True))
    return _zeroed(n, device)


def _check_packed(fn, params, q, k, v, cu_q, cu_k, ws):
    """Checks the inputs shared by attention and its gradient; returns (strides, total_q, total_k, n_seqs)."""
    dt = _TORCH.get(params.dtype)
    _need(dt is not None and dt != torch.uint8, f"{fn}: dtype")
    for x in (q, k, v):
        if not isinstance(x, torch.Tensor) or x.dim() != 3:
            _refuse(f"{fn}: q, k, v must be [T, H, d]")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.numel() < 2:
        _refuse(f"{fn}: cu_seqlens_q")
    dev, d, n, tq, tk = q.device, params.head_dim, cu_q.numel() - 1, q.shape[0], k.shape[0]
    strides = (_check_tensor(q, fn, "q", dt, (tq, params.n_q_heads, d), dev, strided=True),
               _check_tensor(k, fn, "k", dt, (tk, params.n_kv_heads, d), dev, strided=True),
               _check_tensor(v, fn, "v", dt, (tk, params.n_kv_heads, d), dev, strided=True))
    _check_tensor(cu_q, fn, "cu_seqlens_q", torch.int32, (n + 1,), dev)
    if cu_k is not None:
        _check_tensor(cu_k, fn, "cu_seqlens_k", torch.int32, (n + 1,), dev)
    _check_workspace(fn, ws, dev)
    return strides, tq, tk, n


def _check_workspace(fn, ws, dev):
    if ws is not None and not (isinstance(ws, torch.Tensor) and ws.dtype == torch.uint8 and ws.is_contiguous() and
                               ws.device == dev):
        _refuse(f"{fn}: ws must be a dense uint8 tensor on {dev}")


def attention(params: AttnParams, q, k, v, cu_seqlens_q, cu_seqlens_k=None, out=None, lse=None, ws=None, stream=None):
    """hla_attention: (out [Tq, Hq, d], lse [Tq, Hq] fp32) of causal attention over packed sequences.  q, k, v
    may be slices of one fused projection.  cu_seqlens_k: the key rows' offsets where they differ from the
    query rows' (chunks of prompts behind earlier keys).  Without `ws` one is allocated for the call, and what the device
    flags (a malformed table, a wait that ran out) cannot be read: where that may happen, pass a workspace and ask
    check_workspace_error."""
    strides, tq, tk, n = _check_packed("hla_attention", params, q, k, v, cu_seqlens_q, cu_seqlens_k, ws)
    dev, shape = q.device, (tq, params.n_q_heads, params.head_dim)
    if out is not None:
        _check_tensor(out, "hla_attention", "out", q.dtype, shape, dev)
    if lse is not None:
        _check_tensor(lse, "hla_attention", "lse", torch.float32, shape[:2], dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, ws):
            return attention(params, q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, ws)
    if out is None:
        out = _like(q, strides[0])
    if lse is None:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    if ws is None:
        ws = alloc_attention_workspace(params, tq, tk, n, device=dev)
    _check(load().hla_attention(_c(params, *strides), q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(),
                                _adr(cu_seqlens_k), n, tq, tk, out.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                                ws.numel(), st), "hla_attention")
    return out, lse


def attention_backward(params: AttnParams, q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k=None, grads=None,
                       ws=None, stream=None):
    """hla_attention_backward: {"q", "k", "v"} gradients of sum(dout * out), dense, in the layer's type, from
    attention's inputs and results.  `grads` (same dict) and `ws` may be passed in to be reused; without `ws`, what the
    device flags cannot be read (as for attention)."""
    fn = "hla_attention_backward"
    strides, tq, tk, n = _check_packed(fn, params, q, k, v, cu_seqlens_q, cu_seqlens_k, ws)
    dev = q.device
    for x, name in ((out, "out"), (dout, "dout")):
        _check_tensor(x, fn, name, q.dtype, tuple(q.shape), dev)
    _check_tensor(lse, fn, "lse", torch.float32, tuple(q.shape[:2]), dev)
    if grads is not None:
        for name, x in zip("qkv", (q, k, v)):
            _check_tensor(grads.get(name), fn, "grads." + name, x.dtype, tuple(x.shape), dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k, ws, *(grads or {}).values()):
            return attention_backward(params, q, k, v, out, lse, dout, cu_seqlens_q, cu_seqlens_k, grads, ws)
    if grads is None:
        grads = {name: _like(x, stride) for name, x, stride in zip("qkv", (q, k, v), strides)}
    if ws is None:
        ws = alloc_attention_workspace(params, tq, tk, n, backward=True, device=dev)
    _check(load().hla_attention_backward(_c(params, *strides), _adr(q), _adr(k), _adr(v), _adr(out), _adr(lse),
                                         _adr(dout), _adr(cu_seqlens_q), _adr(cu_seqlens_k), n, tq, tk,
                                         _adr(grads["q"]), _adr(grads["k"]), _adr(grads["v"]), _adr(ws), ws.numel(),
                                         st), fn)
    return grads


@dataclass(frozen=True)
class CacheParams:
    n_kv_heads: int
    head_dim: int
    page_size: int
    n_pages: int
    max_pages: int
    dtype: int = DTYPE_BF16         # of the rows written and read
    cache_dtype: int = DTYPE_E4M3   # E4M3, or dtype

    def c(self) -> CCacheParams:
        return CCacheParams(self.n_kv_heads, self.head_dim, self.dtype, self.cache_dtype, self.page_size, self.n_pages,
                            self.max_pages, 0)


class Cache:
    """A paged key / value cache: page_table int32 [n_seqs, max_pages] (kept, not copied: the caller updates it
    as sequences grow); k, v [n_pages, Hkv, page_size, d] and k_exp, v_exp uint8 [n_pages, Hkv, page_size] are
    allocated unless given."""

    def __init__(self, params: CacheParams, page_table, k=None, v=None, k_exp=None, v_exp=None):
        rows, exps = ctypes.c_size_t(), ctypes.c_size_t()
        _check(load().hla_cache_bytes(_c(params), ctypes.byref(rows), ctypes.byref(exps)),
               "hla_cache_bytes")
        _need(isinstance(page_table, torch.Tensor) and page_table.dim() == 2 and page_table.is_cuda,
              "Cache: page_table must be [n_seqs, max_pages] on the GPU")
        self.params, self.n_seqs, self.device = params, page_table.shape[0], page_table.device
        _check_tensor(page_table, "Cache", "page_table", torch.int32, (self.n_seqs, params.max_pages), self.device)
        self.page_table = page_table
        shape = (params.n_pages, params.n_kv_heads, params.page_size, params.head_dim)
        kind = _TORCH[params.cache_dtype]
        self.k, self.v = (self._buffer(t, n, kind, shape) for t, n in ((k, "k"), (v, "v")))
        if exps.value or params.cache_dtype == DTYPE_E4M3:
            self.k_exp, self.v_exp = (self._buffer(t, n, torch.uint8, shape[:3])
                                      for t, n in ((k_exp, "k_exp"), (v_exp, "v_exp")))
        else:
            _need(k_exp is None and v_exp is None, "Cache: exponents go with an E4M3 cache")
            self.k_exp = self.v_exp = None
        self.err = torch.zeros(4, dtype=torch.int32, device=self.device)
        self.tensors = (self.k, self.v, self.k_exp, self.v_exp, self.page_table, self.err)
        self._buffers = CCache(*[None if t is None else t.data_ptr() for t in self.tensors])
        self.c, self.cp = ctypes.byref(self._buffers), _c(params)

    def _buffer(self, t, name, dtype, shape):
        if t is None:
            return torch.zeros(shape, dtype=dtype, device=self.device)
        _check_tensor(t, "Cache", name, dtype, shape, self.device)
        return t

    def check_error(self, stream=None) -> int:
        """Synchronises, reads and clears the cache's error word; returns it (0 = fine)."""
        code = ctypes.c_int32()
        st = _here(self.device, stream)
        if st is None:
            with _on(self.device, stream):
                return self.check_error()
        rc = load().hla_check_cache_error(self.c, st, ctypes.byref(code))
        if rc not in (HLA_OK, HLA_ERR_STATE, HLA_ERR_TIMEOUT):
            _check(rc, "cache error word")
        return code.value


def _check_rows(fn, cache, cu_seqlens, start):
    dev = cache.device
    _check_tensor(cu_seqlens, fn, "cu_seqlens", torch.int32, (cache.n_seqs + 1,), dev)
    _check_tensor(start, fn, "start", torch.int64, (cache.n_seqs,), dev)


def cache_write(cache: Cache, k, v, cu_seqlens, start, stream=None):
    """hla_cache_write: packed rows k, v [T, Hkv, d] of cache.n_seqs sequences to positions start[n] + i."""
    fn, p = "hla_cache_write", cache.params
    _check_rows(fn, cache, cu_seqlens, start)
    _need(isinstance(k, torch.Tensor) and k.dim() == 3, f"{fn}: k must be [T, Hkv, d]")
    shape = (k.shape[0], p.n_kv_heads, p.head_dim)
    for t, name in ((k, "k"), (v, "v")):
        _check_tensor(t, fn, name, _TORCH[p.dtype], shape, cache.device)
    st = _here(cache.device, stream)
    if st is None:
        with _on(cache.device, stream, k, v, cu_seqlens, start, *cache.tensors):
            return cache_write(cache, k, v, cu_seqlens, start)
    _check(load().hla_cache_write(cache.cp, cache.c, _adr(k), _adr(v), _adr(cu_seqlens), _adr(start), cache.n_seqs,
                                  shape[0], st), fn)


def cache_read(cache: Cache, cu_seqlens, start, total_tokens: int, k=None, v=None, stream=None):
    """hla_cache_read: (k, v) [total_tokens, Hkv, d] in the layer's type, the rows at positions start[n] + i."""
    fn, p = "hla_cache_read", cache.params
    _check_rows(fn, cache, cu_seqlens, start)
    shape, dt = (total_tokens, p.n_kv_heads, p.head_dim), _TORCH[p.dtype]
    _need(total_tokens >= 0, f"{fn}: total_tokens")
    for t, name in ((k, "k"), (v, "v")):
        if t is not None:
            _check_tensor(t, fn, name, dt, shape, cache.device)
    st = _here(cache.device, stream)
    if st is None:
        with _on(cache.device, stream, k, v, cu_seqlens, start, *cache.tensors):
            return cache_read(cache, cu_seqlens, start, total_tokens, k, v)
    out = [torch.empty(shape, dtype=dt, device=cache.device) if t is None else t for t in (k, v)]
    _check(load().hla_cache_read(cache.cp, cache.c, _adr(cu_seqlens), _adr(start), cache.n_seqs, total_tokens,
                                 _adr(out[0]), _adr(out[1]), st), fn)
    return out[0], out[1]


def decode_workspace_bytes(params: AttnParams, cache_params: CacheParams) -> int:
    n = ctypes.c_size_t()
    _check(load().hla_attention_decode_workspace_bytes(_c(params), _c(cache_params),
                                                       ctypes.byref(n)), "hla_attention_decode_workspace_bytes")
    return n.value


def alloc_decode_workspace(params: AttnParams, cache: Cache):
    return torch.empty(decode_workspace_bytes(params, cache.params), dtype=torch.uint8, device=cache.device)


def attention_decode(params: AttnParams, cache: Cache, q, lens, out=None, ws=None, stream=None):
    """hla_attention_decode: out [N, Hq, d] of one query token per sequence, q [N, Hq, d] (rows may be slices of
    a wider tensor), over positions 0 .. lens[n] - 1 of the cache."""
    fn = "hla_attention_decode"
    _need(params.dtype == cache.params.dtype, f"{fn}: the layer's and the cache's row types differ")
    dt, dev, shape = _TORCH[params.dtype], cache.device, (cache.n_seqs, params.n_q_heads, params.head_dim)
    stride = _check_tensor(q, fn, "q", dt, shape, dev, strided=True)
    _check_tensor(lens, fn, "lens", torch.int64, (cache.n_seqs,), dev)
    if out is not None:
        _check_tensor(out, fn, "out", dt, shape, dev)
    _check_workspace(fn, ws, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, q, lens, out, ws, *cache.tensors):
            return attention_decode(params, cache, q, lens, out, ws)
    if out is None:
        out = _like(q, stride)
    if ws is None:
        ws = alloc_decode_workspace(params, cache)
    _check(load().hla_attention_decode(_c(params, stride), cache.cp, cache.c, _adr(q), _adr(lens), cache.n_seqs,
                                       _adr(out), _adr(ws), ws.numel(), st), fn)
    return out
