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
from typing import NamedTuple, Optional

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


class CNormParams(ctypes.Structure):
    _fields_ = [("n_cols", ctypes.c_int), ("n_heads", ctypes.c_int), ("dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("group", ctypes.c_int), ("eps", ctypes.c_float),
                ("offset", ctypes.c_float), ("reserved", ctypes.c_int), ("x_stride", ctypes.c_int64),
                ("residual_stride", ctypes.c_int64)]


class CRecurrenceParams(ctypes.Structure):
    _fields_ = [("n_channels", ctypes.c_int), ("gate_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("gate_dtype", ctypes.c_int), ("x_stride", ctypes.c_int64), ("g_stride", ctypes.c_int64)]


class CLinear4Params(ctypes.Structure):
    _fields_ = [("n_in", ctypes.c_int), ("n_out", ctypes.c_int), ("group", ctypes.c_int), ("dtype", ctypes.c_int),
                ("x_dtype", ctypes.c_int), ("x_group", ctypes.c_int), ("x_stride", ctypes.c_int64)]


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
        NP, GP, WP = (ctypes.POINTER(t) for t in (CNormParams, CRecurrenceParams, CLinear4Params))
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
                "hla_check_cache_error": [C, _vp, ctypes.POINTER(ctypes.c_int32)],
                "hla_rms_norm": [NP, _vp, _vp, _vp, i64, _vp, _vp, _vp, _vp],
                "hla_rms_norm_backward_workspace_bytes": [NP, size_p],
                "hla_rms_norm_backward": [NP, _vp, _vp, _vp, _vp, i64, _vp, _vp, _vp, ctypes.c_size_t, _vp],
                "hla_recurrence_workspace_bytes": [GP, i64, size_p],
                "hla_recurrence": [GP] + [_vp] * 4 + [ctypes.c_int, i64] + [_vp] * 4 + [ctypes.c_size_t, _vp],
                "hla_recurrence_backward": [GP] + [_vp] * 5 + [ctypes.c_int, i64] + [_vp] * 6 + [ctypes.c_size_t, _vp],
                "hla_recurrence_step": [GP, _vp, _vp, _vp, ctypes.c_int, _vp, _vp],
                "hla_linear4_workspace_bytes": [WP, i64, size_p],
                "hla_linear4": [WP] + [_vp] * 5 + [i64, _vp, _vp, ctypes.c_size_t, _vp],
                "hla_linear4_quantize": [WP] + [_vp] * 5}.items():
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


# ---- around the mixing: norms, the gated recurrence, products with 4-bit weights ------------------------


def _check_matrix(t, fn: str, name: str, dtype, shape, device) -> int:
    """The row stride of t in elements, as _check_tensor takes strided rows, for [rows, columns] as well."""
    if len(shape) == 3:
        return _check_tensor(t, fn, name, dtype, shape, device, strided=True)
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device and shape[0] > 1:
        rows, one = t.stride()
        if one == 1 and rows >= shape[1]:
            return rows
    _check_tensor(t, fn, name, dtype, shape, device)
    return shape[1]


def _sized(t, fn: str, name: str, *dims):
    """Refuses what is no tensor of one of the numbers of dimensions given."""
    if not isinstance(t, torch.Tensor) or t.dim() not in dims:
        _refuse(f"{fn}: {name}: expected a tensor of {dims} dimensions")


def _dense(t):
    """An uninitialised dense tensor of t's shape."""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _bytes(fn: str, params, *sizes) -> int:
    n = ctypes.c_size_t()
    _check(getattr(load(), fn)(_c(params), *sizes, ctypes.byref(n)), fn)
    return n.value


@dataclass(frozen=True)
class NormParams:
    n_cols: int
    n_heads: int = 1            # rows of n_cols per token: 1, or the heads of q or k
    dtype: int = DTYPE_BF16
    out_dtype: int = -1         # -1: dtype; DTYPE_E4M3: 8-bit floats with a power of two per group
    group: int = 0              # E4M3: 32, 128, or 0 (the whole row)
    eps: float = 1e-6
    offset: float = 0.0         # added to the weight

    def c(self, x_stride: int = 0, residual_stride: int = 0) -> CNormParams:
        return CNormParams(self.n_cols, self.n_heads, self.dtype, self.dtype if self.out_dtype < 0 else self.out_dtype,
                           self.group, self.eps, self.offset, 0, x_stride, residual_stride)


class Normed(NamedTuple):
    """out, exp (the exponents of 8-bit rows, else None), sum (x + residual; None without a residual)."""
    out: torch.Tensor
    exp: Optional[torch.Tensor]
    sum: Optional[torch.Tensor]


def _norm_rows(params: NormParams, fn: str, x, name: str):
    """Checks the rows x: [T, n_cols], or [T, n_heads, n_cols] for more heads than one."""
    dt = _TORCH.get(params.dtype)
    if dt is None or dt == torch.uint8:
        _refuse(f"{fn}: dtype")
    _sized(x, fn, name, 2 if params.n_heads == 1 else 3)
    shape = (x.shape[0], params.n_cols) if params.n_heads == 1 else (x.shape[0], params.n_heads, params.n_cols)
    return dt, shape, _check_matrix(x, fn, name, dt, shape, x.device)


def rms_norm(params: NormParams, x, weight=None, residual=None, out=None, exp=None, sum=None, stream=None) -> Normed:
    """hla_rms_norm: x (and residual) [T, n_cols], or [T, n_heads, n_cols], where tokens may be slices of a wider tensor;
    weight [n_cols].  The sum may be written over x or the residual (sum=residual), out over x, where those are
    dense."""
    fn, eight = "hla_rms_norm", params.out_dtype == DTYPE_E4M3
    dt, shape, xs = _norm_rows(params, fn, x, "x")
    dev, rs = x.device, 0
    if weight is not None:
        _check_tensor(weight, fn, "weight", dt, (params.n_cols,), dev)
    if residual is not None:
        rs = _check_matrix(residual, fn, "residual", dt, shape, dev)
        if sum is not None:
            _check_tensor(sum, fn, "sum", dt, shape, dev)
    else:
        _need(sum is None, f"{fn}: sum without residual")
    if out is not None:
        _check_tensor(out, fn, "out", torch.uint8 if eight else dt, shape, dev)
    groups = shape[:-1] + (params.n_cols // params.group if params.group else 1,) if eight else None
    if exp is not None:
        _need(eight, f"{fn}: exponents go with 8-bit rows")
        _check_tensor(exp, fn, "exp", torch.uint8, groups, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, x, weight, residual, out, exp, sum):
            return rms_norm(params, x, weight, residual, out, exp, sum)
    if residual is not None and sum is None:
        sum = _dense(x)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=dev) if eight else _dense(x)
    if eight and exp is None:
        exp = torch.empty(groups, dtype=torch.uint8, device=dev)
    _check(load().hla_rms_norm(_c(params, xs, rs), _adr(x), _adr(residual), _adr(weight), shape[0], _adr(out), _adr(exp),
                               _adr(sum), st), fn)
    return Normed(out, exp, sum)


def norm_workspace_bytes(params: NormParams) -> int:
    return _bytes("hla_rms_norm_backward_workspace_bytes", params)


def alloc_norm_workspace(params: NormParams, device="cuda"):
    """A workspace for rms_norm_backward."""
    return torch.empty(norm_workspace_bytes(params), dtype=torch.uint8, device=device)


def rms_norm_backward(params: NormParams, s, dout, weight=None, dsum=None, dx=None, dweight=None, ws=None, stream=None,
                      need_dweight: bool = True):
    """hla_rms_norm_backward: (dx, dweight) from s (rms_norm's sum, or its x without a residual), dout and, where the sum
    is used further, its gradient dsum.  dx is the gradient of x and of the residual; dweight [n_cols] fp32, None
    without a weight or with need_dweight False (the norm of a frozen backbone: no sums, no workspace).  dx may be dout
    or dsum."""
    fn = "hla_rms_norm_backward"
    dt, shape, xs = _norm_rows(params, fn, s, "s")
    dev = s.device
    for t, name in ((dout, "dout"), (dsum, "dsum"), (dx, "dx")):
        if t is not None or name == "dout":
            _check_tensor(t, fn, name, dt, shape, dev)
    if weight is not None:
        _check_tensor(weight, fn, "weight", dt, (params.n_cols,), dev)
    if dweight is not None:
        _need(weight is not None and need_dweight, f"{fn}: dweight without weight, or not wanted")
        _check_tensor(dweight, fn, "dweight", torch.float32, (params.n_cols,), dev)
    _check_workspace(fn, ws, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, s, dout, weight, dsum, dx, dweight, ws):
            return rms_norm_backward(params, s, dout, weight, dsum, dx, dweight, ws, None, need_dweight)
    if dx is None:
        dx = torch.empty_like(dout)
    if weight is not None and need_dweight:
        if dweight is None:
            dweight = torch.empty(params.n_cols, dtype=torch.float32, device=dev)
        if ws is None:
            ws = alloc_norm_workspace(params, dev)
    _check(load().hla_rms_norm_backward(_c(params, xs), _adr(s), _adr(weight), _adr(dout), _adr(dsum), shape[0], _adr(dx),
                                        _adr(dweight), _adr(ws), 0 if ws is None else ws.numel(), st), fn)
    return dx, dweight


@dataclass(frozen=True)
class RecurrenceParams:
    n_channels: int
    gate_dim: int = 1           # channels in a row that share a gate: 1, 64, 128
    dtype: int = DTYPE_BF16
    gate_dtype: int = DTYPE_F32

    def c(self, x_stride: int = 0, g_stride: int = 0) -> CRecurrenceParams:
        return CRecurrenceParams(self.n_channels, self.gate_dim, self.dtype, self.gate_dtype, x_stride, g_stride)


RECURRENCE_STATE_ROWS = 64


def recurrence_workspace_bytes(params: RecurrenceParams, total_tokens: int) -> int:
    return _bytes("hla_recurrence_workspace_bytes", params, total_tokens)


def alloc_recurrence_workspace(params: RecurrenceParams, total_tokens: int, device="cuda"):
    """A workspace for recurrence and recurrence_backward of up to total_tokens, its error word zeroed;
    check_workspace_error reads it."""
    return _zeroed(recurrence_workspace_bytes(params, total_tokens), device)


def alloc_recurrence_states(params: RecurrenceParams, total_tokens: int, device="cuda"):
    """The states that recurrence keeps for recurrence_backward."""
    return torch.empty((-(-total_tokens // RECURRENCE_STATE_ROWS), params.n_channels), dtype=torch.float32, device=device)


@functools.lru_cache(maxsize=256)
def _recurrence_types(params: RecurrenceParams, fn: str):
    """The types of x and g, and the gates of a row."""
    dt, gt = _TORCH.get(params.dtype), _TORCH.get(params.gate_dtype)
    _need(dt is not None and gt is not None and torch.uint8 not in (dt, gt), f"{fn}: dtype")
    _need(params.gate_dim > 0, f"{fn}: gate_dim")
    return dt, gt, params.n_channels // params.gate_dim


def _recurrence_rows(params: RecurrenceParams, fn: str, g, x):
    """Checks g [T, n_channels / gate_dim] and x [T, n_channels]; returns their types, T and strides."""
    dt, gt, gates = _recurrence_types(params, fn)
    _sized(x, fn, "x", 2)
    n, dev = x.shape[0], x.device
    return dt, gt, n, (_check_matrix(x, fn, "x", dt, (n, params.n_channels), dev),
                       _check_matrix(g, fn, "g", gt, (n, gates), dev))


def _check_states(params, fn, n, cu_seqlens, h0, states, dev, **rows):
    """Checks the table, the fp32 states per sequence (h0 and `rows`) and those per 64 rows; returns n_seqs."""
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        _refuse(f"{fn}: cu_seqlens")
    n_seqs = cu_seqlens.numel() - 1
    _check_tensor(cu_seqlens, fn, "cu_seqlens", torch.int32, (n_seqs + 1,), dev)
    for name, t in (("h0", h0), *rows.items()):
        if t is not None:
            _check_tensor(t, fn, name, torch.float32, (n_seqs, params.n_channels), dev)
    if states is not None:
        _check_tensor(states, fn, "states", torch.float32, (-(-n // RECURRENCE_STATE_ROWS), params.n_channels), dev)
    return n_seqs


def recurrence(params: RecurrenceParams, g, x, cu_seqlens, h0=None, out=None, h_last=None, states=None, ws=None,
               stream=None):
    """hla_recurrence: (out [T, n_channels], h_last [n_seqs, n_channels] fp32) of h = exp(g) h + x over packed sequences,
    from h0 (None: zeros).  g [T, n_channels / gate_dim] and x [T, n_channels] may be slices of a wider projection;
    h_last=h0 writes the states in place.  states (alloc_recurrence_states): kept for recurrence_backward.  Without `ws`
    one is allocated for the call, and what the device flags cannot be read."""
    fn = "hla_recurrence"
    dt, _, n, strides = _recurrence_rows(params, fn, g, x)
    dev = x.device
    n_seqs = _check_states(params, fn, n, cu_seqlens, h0, states, dev, h_last=h_last)
    if out is not None:
        _check_tensor(out, fn, "out", dt, tuple(x.shape), dev)
    _check_workspace(fn, ws, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, g, x, cu_seqlens, h0, out, h_last, states, ws):
            return recurrence(params, g, x, cu_seqlens, h0, out, h_last, states, ws)
    if out is None:
        out = _dense(x)
    if h_last is None:
        h_last = torch.empty((n_seqs, params.n_channels), dtype=torch.float32, device=dev)
    if ws is None:
        ws = alloc_recurrence_workspace(params, n, dev)
    _check(load().hla_recurrence(_c(params, *strides), _adr(g), _adr(x), _adr(h0), _adr(cu_seqlens), n_seqs, n, _adr(out),
                                 _adr(h_last), _adr(states), _adr(ws), ws.numel(), st), fn)
    return out, h_last


def recurrence_backward(params: RecurrenceParams, g, x, states, dout, cu_seqlens, h0=None, dh_last=None, grads=None,
                        ws=None, stream=None):
    """hla_recurrence_backward: {"g", "x"} gradients (and "h0", fp32, where h0 is given) of sum(dout * h) +
    sum(dh_last * h_last), from recurrence's inputs and the states it kept.  `grads` (same dict) and `ws` may be
    passed in to be reused."""
    fn = "hla_recurrence_backward"
    dt, gt, n, strides = _recurrence_rows(params, fn, g, x)
    dev, given = x.device, grads or {}
    _need(states is not None, f"{fn}: states")
    n_seqs = _check_states(params, fn, n, cu_seqlens, h0, states, dev, dh_last=dh_last, dh0=given.get("h0"))
    _check_tensor(dout, fn, "dout", dt, tuple(x.shape), dev)
    if grads is not None:
        _check_tensor(given.get("g"), fn, "grads.g", gt, tuple(g.shape), dev)
        _check_tensor(given.get("x"), fn, "grads.x", dt, tuple(x.shape), dev)
        _need((given.get("h0") is not None) == (h0 is not None), f"{fn}: grads.h0 goes with h0")
    _check_workspace(fn, ws, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, g, x, states, dout, cu_seqlens, h0, dh_last, ws, *given.values()):
            return recurrence_backward(params, g, x, states, dout, cu_seqlens, h0, dh_last, grads, ws)
    if grads is None:
        grads = {"g": _dense(g), "x": torch.empty_like(dout)}
        if h0 is not None:
            grads["h0"] = torch.empty_like(h0)
    if ws is None:
        ws = alloc_recurrence_workspace(params, n, dev)
    _check(load().hla_recurrence_backward(_c(params, *strides), _adr(g), _adr(x), _adr(h0), _adr(states),
                                          _adr(cu_seqlens), n_seqs, n, _adr(dout), _adr(dh_last), _adr(grads["g"]),
                                          _adr(grads["x"]), _adr(grads.get("h0")), _adr(ws), ws.numel(), st), fn)
    return grads


def recurrence_step(params: RecurrenceParams, g, x, h, out=None, stream=None):
    """hla_recurrence_step: one token per sequence; h [n_seqs, n_channels] fp32 becomes exp(g) h + x in place, and out
    is h in the layer's type."""
    fn = "hla_recurrence_step"
    dt, _, n, strides = _recurrence_rows(params, fn, g, x)
    dev = x.device
    _check_tensor(h, fn, "h", torch.float32, (n, params.n_channels), dev)
    if out is not None:
        _check_tensor(out, fn, "out", dt, tuple(x.shape), dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, g, x, h, out):
            return recurrence_step(params, g, x, h, out)
    if out is None:
        out = _dense(x)
    _check(load().hla_recurrence_step(_c(params, *strides), _adr(g), _adr(x), _adr(h), n, _adr(out), st), fn)
    return out


@dataclass(frozen=True)
class Linear4Params:
    n_in: int
    n_out: int
    group: int = 128            # inputs that share a scale: 32, 64, 128
    dtype: int = DTYPE_BF16     # of out, scales, offsets (and x)
    x_dtype: int = -1           # -1: dtype; DTYPE_E4M3: 8-bit rows with a power of two per x_group
    x_group: int = 0            # E4M3: 32, 128, or 0 (the whole row)

    def c(self, x_stride: int = 0) -> CLinear4Params:
        return CLinear4Params(self.n_in, self.n_out, self.group, self.dtype,
                              self.dtype if self.x_dtype < 0 else self.x_dtype, self.x_group, x_stride)


def linear4_workspace_bytes(params: Linear4Params, tokens: int) -> int:
    return _bytes("hla_linear4_workspace_bytes", params, tokens)


def alloc_linear4_workspace(params: Linear4Params, tokens: int, device="cuda"):
    """A workspace for linear4 of up to `tokens` rows."""
    return torch.empty(max(256, linear4_workspace_bytes(params, tokens)), dtype=torch.uint8, device=device)


def _linear4_weights(params: Linear4Params, fn: str, w, scales, offsets, dev):
    dt = _TORCH.get(params.dtype)
    if dt is None or dt == torch.uint8 or params.group <= 0:
        _refuse(f"{fn}: dtype or group")
    _check_tensor(w, fn, "w", torch.uint8, (params.n_out, params.n_in // 2), dev)
    shape = (params.n_out, params.n_in // params.group)
    _check_tensor(scales, fn, "scales", dt, shape, dev)
    if offsets is not None:
        _check_tensor(offsets, fn, "offsets", dt, shape, dev)
    return dt


def linear4(params: Linear4Params, x, w, scales, offsets=None, x_exp=None, out=None, ws=None, stream=None):
    """hla_linear4: out [T, n_out] = x W^T with W = scales (q - 8) + offsets; x [T, n_in] (tokens may be slices of a wider
    tensor; 8-bit rows: uint8, with x_exp [T, n_in / x_group]), w uint8 [n_out, n_in / 2]."""
    fn, eight = "hla_linear4", params.x_dtype == DTYPE_E4M3
    _sized(x, fn, "x", 2)
    dev, n = x.device, x.shape[0]
    dt = _linear4_weights(params, fn, w, scales, offsets, dev)
    stride = _check_matrix(x, fn, "x", torch.uint8 if eight else dt, (n, params.n_in), dev)
    if eight != (x_exp is not None):
        _refuse(f"{fn}: exponents go with 8-bit rows")
    if eight:
        _check_tensor(x_exp, fn, "x_exp", torch.uint8, (n, params.n_in // params.x_group if params.x_group else 1), dev)
    if out is not None:
        _check_tensor(out, fn, "out", dt, (n, params.n_out), dev)
    _check_workspace(fn, ws, dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, x, w, scales, offsets, x_exp, out, ws):
            return linear4(params, x, w, scales, offsets, x_exp, out, ws)
    if out is None:
        out = torch.empty((n, params.n_out), dtype=dt, device=dev)
    if ws is None and (dt != torch.bfloat16 or eight or stride % 8 or x.data_ptr() % 16):
        ws = alloc_linear4_workspace(params, n, dev)
    _check(load().hla_linear4(_c(params, stride), _adr(x), _adr(x_exp), _adr(w), _adr(scales), _adr(offsets), n, _adr(out),
                              _adr(ws), 0 if ws is None else ws.numel(), st), fn)
    return out


def linear4_quantize(params: Linear4Params, weight, with_offsets: bool = False, stream=None):
    """hla_linear4_quantize: (w, scales, offsets or None) of weight [n_out, n_in] in the layer's type."""
    fn = "hla_linear4_quantize"
    dt = _TORCH.get(params.dtype)
    _need(dt is not None and dt != torch.uint8 and params.group > 0, f"{fn}: dtype or group")
    _sized(weight, fn, "weight", 2)
    dev = weight.device
    _check_tensor(weight, fn, "weight", dt, (params.n_out, params.n_in), dev)
    st = _here(dev, stream)
    if st is None:
        with _on(dev, stream, weight):
            return linear4_quantize(params, weight, with_offsets)
    w = torch.empty((params.n_out, params.n_in // 2), dtype=torch.uint8, device=dev)
    scales, offsets = (torch.empty((params.n_out, params.n_in // params.group), dtype=dt, device=dev) if on else None
                       for on in (True, with_offsets))
    _check(load().hla_linear4_quantize(_c(params), _adr(weight), _adr(w), _adr(scales), _adr(offsets), st), fn)
    return w, scales, offsets
