"""Python binding of libgdn.so: argument marshalling for torch CUDA tensors.

Every step of the computation runs in the library's CUDA kernels; this module
only checks tensor placement/dtypes, allocates outputs and workspace with torch
when the caller does not pass them, and forwards pointers and the current CUDA
stream.  There is no CPU fallback: when ``libgdn.so`` is missing or cannot be
loaded, every call raises.

Names follow the C ABI in ``include/gdn.h`` and ``include/gdn_linattn.h``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# GDN_LIBRARY may name another build of the library (the bounds-checked one, for tests).
LIB_PATH = os.environ.get("GDN_LIBRARY") or os.path.join(_PKG, "libgdn.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA, GDN_ERR_TIMEOUT, \
    GDN_ERR_INTERNAL = range(7)
GDN_F32, GDN_BF16 = 0, 1
GDN_GATE_HEAD, GDN_GATE_CHANNEL = 0, 1
GDN_GATE_CONST = 2  # gdn_linattn_* only: one fixed decay per head

GDN_DEV_OK, GDN_DEV_TIMEOUT_PREP, GDN_DEV_TIMEOUT_SCAN, GDN_DEV_BOUNDS = 0, 1, 2, 16

EXPORTED = ("gdn_chunk_workspace_size", "gdn_chunk_fwd", "gdn_chunk_status", "gdn_chunk_fwd_static",
            "gdn_chunk_status_static", "gdn_decode_step", "gdn_decode_multi", "gdn_state_select", "gdn_prerule",
            "gdn_decode_step_prerule", "gdn_status_string", "gdn_last_error", "gdn_profile_enable",
            "gdn_profile_read")

# entry points of include/gdn_linattn.h
EXPORTED_LINATTN = ("gdn_linattn_workspace_size", "gdn_linattn_chunk_fwd", "gdn_linattn_decode_step",
                    "gdn_qk_norm_rope", "gdn_beam_workspace_size", "gdn_beam_select", "gdn_state_reorder")


class GdnDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("dk", ctypes.c_int64), ("dv", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("scale", ctypes.c_float), ("hk", ctypes.c_int32)]


class GdnQkRopeDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("hq", ctypes.c_int32), ("hk", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class GdnBeamDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("W", ctypes.c_int32), ("V", ctypes.c_int32), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("row_stride", ctypes.c_int64)]


class GdnKernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double)]


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH):
    """Load libgdn.so and declare its entry points.  Raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None and path == LIB_PATH:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m gated_delta_rule_64_b200.build`"
                               " (there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        dp = ctypes.POINTER(GdnDesc)
        lib.gdn_chunk_workspace_size.argtypes = [dp, i32, ctypes.POINTER(sz)]
        lib.gdn_chunk_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, vp, vp, sz, vp]
        lib.gdn_chunk_fwd_static.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, vp, vp]
        lib.gdn_chunk_status.argtypes = [vp, vp, ctypes.POINTER(i32)]
        lib.gdn_chunk_status_static.argtypes = [vp, ctypes.POINTER(i32)]
        lib.gdn_decode_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn_decode_multi.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp]
        lib.gdn_state_select.argtypes = [dp, vp, vp, vp, vp]
        lib.gdn_prerule.argtypes = [dp, vp, vp, vp, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn_decode_step_prerule.argtypes = [dp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp]
        lib.gdn_linattn_workspace_size.argtypes = [dp, i32, ctypes.POINTER(sz)]
        lib.gdn_linattn_chunk_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, vp, vp, sz, vp]
        lib.gdn_linattn_decode_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn_qk_norm_rope.argtypes = [ctypes.POINTER(GdnQkRopeDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp]
        bp = ctypes.POINTER(GdnBeamDesc)
        lib.gdn_beam_workspace_size.argtypes = [bp, ctypes.POINTER(sz)]
        lib.gdn_beam_select.argtypes = [bp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.gdn_state_reorder.argtypes = [vp, vp, i64, i32, sz, vp]
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_last_error.argtypes = []
        lib.gdn_last_error.restype = ctypes.c_char_p
        lib.gdn_profile_enable.argtypes = [ctypes.c_int]
        lib.gdn_profile_read.argtypes = [ctypes.POINTER(GdnKernelTime), i32, ctypes.POINTER(i32)]
        for name in ("gdn_chunk_workspace_size", "gdn_chunk_fwd", "gdn_chunk_status", "gdn_chunk_status_static",
                     "gdn_chunk_fwd_static", "gdn_decode_step",
                     "gdn_decode_multi", "gdn_state_select", "gdn_prerule", "gdn_decode_step_prerule",
                     "gdn_profile_enable", "gdn_profile_read") + EXPORTED_LINATTN:
            getattr(lib, name).restype = ctypes.c_int
        if path == LIB_PATH:
            _lib = lib
        return lib


def _check(lib, st: int):
    if st != GDN_OK:
        msg = lib.gdn_last_error().decode() or lib.gdn_status_string(st).decode()
        raise GdnError(st, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN_F32
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors (the library has no CPU path)")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def make_desc(B, T, H, dk, dv, dtype_code, per_channel, scale, hk=0) -> GdnDesc:
    """hk: query/key heads when fewer than the H value heads (0: H)."""
    return GdnDesc(B, T, H, dk, dv, dtype_code, GDN_GATE_CHANNEL if per_channel else GDN_GATE_HEAD,
                   float(scale), int(hk) if hk != H else 0)


def gdn_chunk_workspace_size(B, T, H, dk, dv, num_seqs, *, dtype=torch.bfloat16, per_channel=False,
                             hk=0) -> int:
    lib = load_library()
    d = make_desc(B, T, H, dk, dv, GDN_F32 if dtype == torch.float32 else GDN_BF16, per_channel, 1.0, hk)
    n = ctypes.c_size_t(0)
    _check(lib, lib.gdn_chunk_workspace_size(ctypes.byref(d), int(num_seqs), ctypes.byref(n)))
    return int(n.value)


def gdn_chunk_fwd(q, k, v, log_gate, beta, initial_state=None, cu_seqlens=None, *, scale=1.0,
                  snapshot_stride=0, out=None, final_state=True, snapshots=None, workspace=None,
                  stream=None):
    """Chunkwise prefill.  Shapes as in include/gdn.h:
    q, k (B,T,Hk,dk) with Hk dividing H (value head h reads query/key head h // (H // Hk)); v (B,T,H,dv); log_gate (B,T,H) or (B,T,H,dk); beta (B,T,H);
    initial_state (N,H,dv,dk) fp32 or None; cu_seqlens int32 (N+1) on the device or None.
    final_state: True to allocate, a tensor to fill (may be initial_state), or None.
    Returns (out, final_state, snapshots)."""
    lib = load_library()
    _need_cuda(q, k, v, log_gate, beta, initial_state, cu_seqlens)
    B, T, Hq, dk = q.shape
    H, dv = v.shape[-2], v.shape[-1]  # value heads; q and k may have fewer (Hq divides H)
    per_channel = log_gate.dim() == 4
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    dev = q.device
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    if final_state is True:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    if snapshot_stride and snapshots is None:
        n_snap = T // snapshot_stride
        snapshots = torch.empty((B, n_snap, H, dv, dk), dtype=torch.float32, device=dev)
    d = make_desc(B, T, H, dk, dv, _dtype_code(q), per_channel, scale, Hq)
    if workspace is None:
        ws_bytes = gdn_chunk_workspace_size(B, T, H, dk, dv, N, dtype=q.dtype, per_channel=per_channel, hk=Hq)
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    _need_cuda(out, final_state, snapshots, workspace)
    st = lib.gdn_chunk_fwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(beta),
                           _ptr(initial_state), _ptr(cu_seqlens), int(N), int(snapshot_stride), _ptr(out),
                           _ptr(final_state), _ptr(snapshots), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(lib, st)
    return out, final_state, snapshots


def gdn_chunk_status(workspace, stream=None):
    """Device status of the last gdn_chunk_fwd call that used `workspace` on `stream`
    (waits for the stream): (status, device_code); status GDN_OK, GDN_ERR_TIMEOUT
    or GDN_ERR_INTERNAL, device_code one of the GDN_DEV_* codes."""
    lib = load_library()
    _need_cuda(workspace)
    code = ctypes.c_int32(-1)
    st = lib.gdn_chunk_status(_ptr(workspace), _stream(stream), ctypes.byref(code))
    if st == GDN_ERR_CUDA or st == GDN_ERR_INVALID_ARG:
        _check(lib, st)
    return st, int(code.value)


def gdn_chunk_status_static(stream=None):
    """gdn_chunk_status for gdn_chunk_fwd_static (its built-in scratch on the current device)."""
    lib = load_library()
    code = ctypes.c_int32(-1)
    st = lib.gdn_chunk_status_static(_stream(stream), ctypes.byref(code))
    if st == GDN_ERR_CUDA or st == GDN_ERR_INVALID_ARG:
        _check(lib, st)
    return st, int(code.value)


def gdn_chunk_fwd_static(q, k, v, log_gate, beta, initial_state=None, cu_seqlens=None, *, scale=1.0,
                         snapshot_stride=0, out=None, final_state=True, snapshots=None, stream=None):
    """gdn_chunk_fwd for callers that cannot allocate device scratch: the library
    uses its built-in 64 MiB scratch array instead of a workspace (requests
    that need more are rejected).  This wrapper still allocates the outputs with
    torch when they are not passed; a caller that cannot allocate passes them."""
    lib = load_library()
    _need_cuda(q, k, v, log_gate, beta, initial_state, cu_seqlens)
    B, T, Hq, dk = q.shape
    H, dv = v.shape[-2], v.shape[-1]  # value heads; q and k may have fewer (Hq divides H)
    per_channel = log_gate.dim() == 4
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    dev = q.device
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    if final_state is True:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    elif final_state is False:
        final_state = None
    if snapshot_stride and snapshots is None:
        snapshots = torch.empty((B, T // snapshot_stride, H, dv, dk), dtype=torch.float32, device=dev)
    _need_cuda(out, final_state, snapshots)
    d = make_desc(B, T, H, dk, dv, _dtype_code(q), per_channel, scale, Hq)
    st = lib.gdn_chunk_fwd_static(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(beta),
                                  _ptr(initial_state), _ptr(cu_seqlens), int(N), int(snapshot_stride), _ptr(out),
                                  _ptr(final_state), _ptr(snapshots), _stream(stream))
    _check(lib, st)
    return out, final_state, snapshots


def gdn_decode_step(q, k, v, log_gate, beta, state, *, scale=1.0, out=None, stream=None):
    """One decode token per sequence; `state` (B,H,dv,dk) fp32 is updated in place.
    q, k (B,1,H,dk) or (B,H,dk); v (B,1,H,dv) or (B,H,dv); log_gate (B,[1,]H[,dk]); beta (B,[1,]H)."""
    lib = load_library()
    _need_cuda(q, k, v, log_gate, beta, state)
    B, H, dv, dk = state.shape
    per_channel = log_gate.dim() == q.dim()  # (.., H, dk) per channel, (.., H) per head
    if out is None:
        out = torch.empty((B, 1, H, dv), dtype=q.dtype, device=q.device)
    _need_cuda(out)
    d = make_desc(B, 1, H, dk, dv, _dtype_code(q), per_channel, scale, q.shape[-2])
    st = lib.gdn_decode_step(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(beta), _ptr(state),
                             _ptr(out), _stream(stream))
    _check(lib, st)
    return out


def gdn_decode_multi(q, k, v, log_gate, beta, state, *, n_tokens=None, commit=True, step_states=None, scale=1.0,
                     out=None, stream=None):
    """Up to T tokens per sequence in one pass over the state (speculative verify / multi-token decode).
    q, k (B,T,H,dk); v (B,T,H,dv); log_gate (B,T,H) or (B,T,H,dk); beta (B,T,H); state (B,H,dv,dk) fp32;
    n_tokens: int32 (B) on the device or None (all T); commit: write the state after n_tokens back;
    step_states: True to allocate, a (B,T,H,dv,dk) fp32 tensor, or None.  Returns (out, step_states)."""
    lib = load_library()
    _need_cuda(q, k, v, log_gate, beta, state)
    B, T, Hq, dk = q.shape
    H, dv = v.shape[-2], v.shape[-1]
    per_channel = log_gate.dim() == 4
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if step_states is True:
        step_states = torch.empty((B, T, H, dv, dk), dtype=torch.float32, device=q.device)
    _need_cuda(out)
    d = make_desc(B, T, H, dk, dv, _dtype_code(q), per_channel, scale, Hq)
    st = lib.gdn_decode_multi(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_gate), _ptr(beta),
                              _ptr(n_tokens), _ptr(state), 1 if commit else 0, _ptr(out), _ptr(step_states),
                              _stream(stream))
    _check(lib, st)
    return out, step_states


def gdn_prerule(x, a, b, conv_w, A_log, dt_bias, *, hk, dk, H, dv, cu_seqlens=None, conv_state_in=None,
                conv_state_out=None, stream=None):
    """Short convolution + SiLU, length-1 q/k and the gates from the raw projections.
    x (B,T,2*hk*dk+H*dv); a, b (B,T,H) in x's dtype; conv_w (C,K) fp32; A_log, dt_bias (H,) fp32;
    conv states (N,C,K-1) fp32 or None (conv_state_out may be conv_state_in).
    Returns (q (B,T,hk,dk), k, v (B,T,H,dv), log_gate (B,T,H), beta (B,T,H))."""
    lib = load_library()
    _need_cuda(x, a, b, conv_w, A_log, dt_bias, cu_seqlens, conv_state_in, conv_state_out)
    B, T, C = x.shape
    K = conv_w.shape[1]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    dev = x.device
    q = torch.empty((B, T, hk, dk), dtype=x.dtype, device=dev)
    k = torch.empty((B, T, hk, dk), dtype=x.dtype, device=dev)
    v = torch.empty((B, T, H, dv), dtype=x.dtype, device=dev)
    g = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    beta = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    d = make_desc(B, T, H, dk, dv, _dtype_code(x), False, 1.0, hk)
    st = lib.gdn_prerule(ctypes.byref(d), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), int(K), _ptr(A_log),
                         _ptr(dt_bias), _ptr(cu_seqlens), int(N), _ptr(conv_state_in), _ptr(conv_state_out),
                         _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _stream(stream))
    _check(lib, st)
    return q, k, v, g, beta


def gdn_decode_step_prerule(x, a, b, conv_w, A_log, dt_bias, conv_state, state, *, hk, dk, H, dv, scale=1.0,
                            out=None, stream=None):
    """One decode step from the raw projections: x (B,2*hk*dk+H*dv) (or (B,1,C)); a, b (B,H)
    (or (B,1,H)) in x's dtype; conv_w (C,K), A_log, dt_bias (H,) fp32; conv_state (B,C,K-1) fp32
    or None, updated in place; state (B,H,dv,dk) fp32, updated in place.  Returns out (B,H,dv)."""
    lib = load_library()
    _need_cuda(x, a, b, conv_w, A_log, dt_bias, conv_state, state)
    B = x.shape[0]
    K = conv_w.shape[1]
    if out is None:
        out = torch.empty((B, H, dv), dtype=x.dtype, device=x.device)
    d = make_desc(B, 1, H, dk, dv, _dtype_code(x), False, scale, hk)
    _check(lib, lib.gdn_decode_step_prerule(ctypes.byref(d), _ptr(x), _ptr(a), _ptr(b), _ptr(conv_w), int(K),
                                            _ptr(A_log), _ptr(dt_bias), _ptr(conv_state), _ptr(state), _ptr(out),
                                            _stream(stream)))
    return out


def gdn_state_select(step_states, accept, state, *, stream=None):
    """state[b] = step_states[b, accept[b] - 1] where accept[b] > 0 (int32 device tensor)."""
    lib = load_library()
    _need_cuda(step_states, accept, state)
    B, T, H, dv, dk = step_states.shape
    d = make_desc(B, T, H, dk, dv, GDN_F32, False, 1.0)
    _check(lib, lib.gdn_state_select(ctypes.byref(d), _ptr(step_states), _ptr(accept), _ptr(state),
                                     _stream(stream)))
    return state


# ---------------------------------------------------------------------------
# include/gdn_linattn.h: linear attention with a decay for each head, the norm and
# rotation of queries and keys, beam search over recurrent states
# ---------------------------------------------------------------------------

def _where(stream, t, *others):
    """The (device index, raw stream) of a call: the device its tensors are on and `stream`, or the current
    stream of that device.  Tensors that a given stream uses are recorded on it: their memory is not handed
    out again before the call has run."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors (the library has no CPU path)")
    dev = t.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"tensors are on different devices: {t.device} and {o.device}")
    if stream is None:  # (without the Stream object around it: 0.1 us instead of 1.3)
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
    if stream != torch.cuda.current_stream(dev):
        for o in (t,) + others:
            if o is not None:
                o.record_stream(stream)
    return dev, stream.cuda_stream


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """A context in which the device of a call is current, and its stream too (so that what is allocated for it
    belongs to that stream)."""
    if stream is not None:
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev else torch.cuda.device(dev)


def _need(name, t, shape, dtype=None):
    """`t` is a contiguous tensor of `shape` (and `dtype`)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _addr(t):
    return None if t is None else t.data_ptr()


def gdn_linattn_workspace_size(B, T, H, dk, dv, num_seqs, *, dtype=torch.bfloat16, hk=0) -> int:
    lib = _lib or load_library()
    d = make_desc(B, T, H, dk, dv, GDN_F32 if dtype == torch.float32 else GDN_BF16, False, 1.0, hk)
    n = ctypes.c_size_t(0)
    _check(lib, lib.gdn_linattn_workspace_size(ctypes.byref(d), int(num_seqs), ctypes.byref(n)))
    return int(n.value)


def gdn_linattn_chunk_fwd(q, k, v, log_gate, initial_state=None, cu_seqlens=None, *, scale=1.0, snapshot_stride=0,
                          out=None, final_state=True, snapshots=None, workspace=None, stream=None):
    """Linear attention with a decay for each head over prompts: S_t = exp(g_t) S_{t-1} + v_t k_t^T,
    o_t = S_t (scale q_t).  Shapes as gdn_chunk_fwd; log_gate (B,T,H), or (H,) for one fixed decay per head.
    final_state: True to allocate, a tensor to fill (may be initial_state), or None.
    Returns (out, final_state, snapshots).  gdn_chunk_status(workspace) reads the call's device status."""
    lib = _lib or load_library()
    B, T, Hq, dk = q.shape
    H, dv = v.shape[-2], v.shape[-1]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    code = _dtype_code(q)
    _need("q", q, (B, T, Hq, dk))
    _need("k", k, (B, T, Hq, dk), q.dtype)
    _need("v", v, (B, T, H, dv), q.dtype)
    fixed = log_gate.dim() == 1
    _need("log_gate", log_gate, (H,) if fixed else (B, T, H), torch.float32)
    if initial_state is not None:
        _need("initial_state", initial_state, (N, H, dv, dk), torch.float32)
    if cu_seqlens is not None:
        _need("cu_seqlens", cu_seqlens, (N + 1,), torch.int32)
    if out is not None:
        _need("out", out, (B, T, H, dv), q.dtype)
    if isinstance(final_state, torch.Tensor):
        _need("final_state", final_state, (N, H, dv, dk), torch.float32)
    if snapshots is not None and snapshot_stride > 0:
        _need("snapshots", snapshots, (B, T // snapshot_stride, H, dv, dk), torch.float32)
    given = final_state if isinstance(final_state, torch.Tensor) else None
    dev, raw = _where(stream, q, k, v, log_gate, initial_state, cu_seqlens, out, given, snapshots, workspace)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(v)
        if final_state is True:
            final_state = q.new_empty((N, H, dv, dk), dtype=torch.float32)
        elif final_state is False:
            final_state = None
        if snapshot_stride > 0 and snapshots is None:
            snapshots = q.new_empty((B, T // snapshot_stride, H, dv, dk), dtype=torch.float32)
        d = make_desc(B, T, H, dk, dv, code, False, scale, Hq)
        d.gate = GDN_GATE_CONST if fixed else GDN_GATE_HEAD
        if workspace is None:
            n = ctypes.c_size_t(0)
            _check(lib, lib.gdn_linattn_workspace_size(ctypes.byref(d), int(N), ctypes.byref(n)))
            workspace = q.new_empty(max(n.value, 256), dtype=torch.uint8)
        elif not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        st = lib.gdn_linattn_chunk_fwd(ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(),
                                       _addr(initial_state), _addr(cu_seqlens), N, int(snapshot_stride),
                                       out.data_ptr(), _addr(final_state), _addr(snapshots), workspace.data_ptr(),
                                       workspace.numel() * workspace.element_size(), raw)
        if st != GDN_OK:
            _check(lib, st)
    return out, final_state, snapshots


def gdn_linattn_decode_step(q, k, v, log_gate, state, *, scale=1.0, out=None, stream=None):
    """One token of every live sequence of gdn_linattn_chunk_fwd's recurrence; `state` (B,H,dv,dk) fp32 is
    updated in place.  q, k (B,1,hk,dk) or (B,hk,dk); v (B,1,H,dv) or (B,H,dv); log_gate (B,[1,]H) or (H,)."""
    lib = _lib or load_library()
    B, H, dv, dk = state.shape
    hk = q.shape[-2]
    code = _dtype_code(q)
    lead = (B,) if q.dim() == 3 else (B, 1)
    _need("q", q, lead + (hk, dk))
    _need("k", k, lead + (hk, dk), q.dtype)
    _need("v", v, ((B,) if v.dim() == 3 else (B, 1)) + (H, dv), q.dtype)
    fixed = log_gate.dim() == 1
    _need("log_gate", log_gate, (H,) if fixed else ((B,) if log_gate.dim() == 2 else (B, 1)) + (H,), torch.float32)
    _need("state", state, (B, H, dv, dk), torch.float32)
    if out is not None and (out.numel() != B * H * dv or out.dtype != q.dtype or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous (B, 1, H, dv) tensor of {q.dtype}")
    dev, raw = _where(stream, q, k, v, log_gate, state, out)
    d = GdnDesc(B, 1, H, dk, dv, code, GDN_GATE_CONST if fixed else GDN_GATE_HEAD, scale, hk if hk != H else 0)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(v) if v.dim() == 4 else v.new_empty((B, 1, H, dv))
        st = lib.gdn_linattn_decode_step(ctypes.byref(d), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_gate.data_ptr(),
                                         state.data_ptr(), out.data_ptr(), raw)
    if st != GDN_OK:
        _check(lib, st)
    return out


def _token_rows(name, x):
    """(B, T, heads, d) with a token's heads side by side and tokens evenly spaced: the elements from one
    token to the next.  Slices of a wider projection have that form; anything else is refused."""
    B, T, h, d = x.shape
    st = x.stride()
    if (d > 1 and st[3] != 1) or (h > 1 and st[2] != d):
        raise ValueError(f"{name}: a token's heads must lie side by side")
    if B * T <= 1:
        return h * d
    if T > 1:
        if B > 1 and st[0] != T * st[1]:
            raise ValueError(f"{name}: tokens must be evenly spaced over (B, T)")
        return st[1]
    return st[0]


def gdn_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, *, eps=1e-6, weight_offset=0.0,
                     interleaved=False, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head (over its channels, times weight_offset + weight) and the position
    rotation, in one pass.  q (B,T,hq,d), k (B,T,hk,d): dense, or slices of a wider projection (a token's
    heads side by side); positions (B,T) int32; inv_freq (rot/2,) fp32, or None: no rotation; the weights (d,)
    fp32 or None.  Pairs are (i, i + rot/2), or (2i, 2i+1) when `interleaved`.  Returns (q_out, k_out), dense;
    either may be its (dense) input."""
    lib = _lib or load_library()
    B, T, hq, dim = q.shape
    hk = k.shape[2]
    code = _dtype_code(q)
    if k.dtype != q.dtype or tuple(k.shape) != (B, T, hk, dim):
        raise ValueError(f"k must be {(B, T, hk, dim)} of {q.dtype}, got {tuple(k.shape)} of {k.dtype}")
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot:
        _need("inv_freq", inv_freq, (rot // 2,), torch.float32)
        _need("positions", positions, (B, T), torch.int32)
    else:
        positions = None
    if q_weight is not None:
        _need("q_weight", q_weight, (dim,), torch.float32)
    if k_weight is not None:
        _need("k_weight", k_weight, (dim,), torch.float32)
    if q_out is not None:
        _need("q_out", q_out, (B, T, hq, dim), q.dtype)
    if k_out is not None:
        _need("k_out", k_out, (B, T, hk, dim), q.dtype)
    dev, raw = _where(stream, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    d = GdnQkRopeDesc(B * T, hq, hk, dim, rot, 1 if interleaved else 0, code, _token_rows("q", q),
                      _token_rows("k", k) if hk else 0, float(eps), float(weight_offset))
    with _on(dev, stream):
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        st = lib.gdn_qk_norm_rope(ctypes.byref(d), q.data_ptr(), k.data_ptr(), _addr(positions), _addr(inv_freq),
                                  _addr(q_weight), _addr(k_weight), q_out.data_ptr(), k_out.data_ptr(), raw)
    if st != GDN_OK:
        _check(lib, st)
    return q_out, k_out


def gdn_beam_select(logits, scores, K, *, out_scores=None, out_parent=None, out_token=None, workspace=None,
                    stream=None):
    """One step of beam search: for each request the K best of its W x V continuations by
    scores[b, w] + log_softmax(logits[b, w])[t], best first, equals in index order.
    logits (B,W,V) fp32 or bf16 (rows of V values evenly spaced: a padded vocabulary may be sliced off);
    scores (B,W) fp32 or None (zeros).  Returns (scores (B,K) fp32, parent beam (B,K) int32, token (B,K) int32)."""
    lib = _lib or load_library()
    B, W, V = logits.shape
    code = _dtype_code(logits)
    st = logits.stride()
    if V > 1 and st[2] != 1:
        raise ValueError("logits: a row's values must be contiguous")
    if B > 1 and W > 1 and st[0] != W * st[1]:
        raise ValueError("logits: rows must be evenly spaced over (B, W)")
    stride = V if B * W <= 1 else (st[1] if W > 1 else st[0])
    if scores is not None:
        _need("scores", scores, (B, W), torch.float32)
    for name, t, dt in (("out_scores", out_scores, torch.float32), ("out_parent", out_parent, torch.int32),
                        ("out_token", out_token, torch.int32)):
        if t is not None:
            _need(name, t, (B, K), dt)
    dev, raw = _where(stream, logits, scores, out_scores, out_parent, out_token, workspace)
    d = GdnBeamDesc(B, W, V, int(K), code, stride)
    with _on(dev, stream):
        if out_scores is None:
            out_scores = logits.new_empty((B, K), dtype=torch.float32)
        if out_parent is None:
            out_parent = logits.new_empty((B, K), dtype=torch.int32)
        if out_token is None:
            out_token = torch.empty_like(out_parent)
        if workspace is None:
            n = ctypes.c_size_t(0)
            _check(lib, lib.gdn_beam_workspace_size(ctypes.byref(d), ctypes.byref(n)))
            workspace = logits.new_empty(max(n.value, 256), dtype=torch.uint8)
        elif not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        st = lib.gdn_beam_select(ctypes.byref(d), logits.data_ptr(), _addr(scores), out_scores.data_ptr(),
                                 out_parent.data_ptr(), out_token.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), raw)
    if st != GDN_OK:
        _check(lib, st)
    return out_scores, out_parent, out_token


def gdn_state_reorder(state, parent, *, stream=None):
    """Move per-beam states to the beams that go on with them, in place: state row (b, w) becomes row
    (b, parent[b, w]) as it was before the call; a parent outside 0 .. W-1 leaves its row.  `state`: a
    contiguous tensor of any type whose leading dimension is B * W (recurrent states, convolution histories;
    a row is a multiple of 16 bytes); parent (B, W) int32.  Returns state."""
    lib = _lib or load_library()
    B, W = parent.shape
    _need("parent", parent, (B, W), torch.int32)
    if state.dim() < 1 or state.shape[0] != B * W or not state.is_contiguous():
        raise ValueError(f"state must be contiguous with {B * W} rows")
    row_bytes = state.numel() // max(B * W, 1) * state.element_size()
    dev, raw = _where(stream, state, parent)
    with _on(dev, None):
        st = lib.gdn_state_reorder(state.data_ptr(), parent.data_ptr(), B, W, row_bytes, raw)
    if st != GDN_OK:
        _check(lib, st)
    return state


def profile_enable(on: bool = True):
    lib = load_library()
    _check(lib, lib.gdn_profile_enable(1 if on else 0))


def profile_read() -> dict:
    """{kernel name: (launches, total ms)} since the last read (waits for the events)."""
    lib = load_library()
    cap = 64
    arr = (GdnKernelTime * cap)()
    cnt = ctypes.c_int32(0)
    _check(lib, lib.gdn_profile_read(arr, cap, ctypes.byref(cnt)))
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(min(cap, cnt.value))}
