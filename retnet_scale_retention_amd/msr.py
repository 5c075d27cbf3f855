"""Thin ctypes binding of libmsr.so (include/msr.h).

Argument marshalling only: every step of the operation runs in the HIP
kernels behind the C ABI.  PyTorch supplies device memory and the stream:
the current one of the tensors' device, or the torch.cuda.Stream given as
`stream`.  What a call allocates comes from that stream's pool; tensors the
caller brings must be ready on it and stay valid until it has passed the call.
If libmsr.so is missing this module raises on first use -- there is no
fallback implementation.
"""
from __future__ import annotations

import array
import ctypes
import math
import operator
import struct
from pathlib import Path

import numpy as np

import os

LIB_PATH = Path(os.environ.get("MSR_LIB", Path(__file__).resolve().parent / "libmsr.so"))

MSR_OK = 0
MSR_F32, MSR_BF16 = 0, 1
MSR_FLAG_NO_ROTATE, MSR_FLAG_NO_GROUPNORM, MSR_FLAG_DECAY_ROWNORM, MSR_FLAG_SPLIT_SCORES, MSR_FLAG_FUSED = 1, 2, 4, 8, 16
MSR_EXCHANGE_AUTO, MSR_EXCHANGE_OFF, MSR_EXCHANGE_NO_WAIT = 0, 1, 2
MSR_FORM_PARALLEL, MSR_FORM_CHUNKWISE, MSR_FORM_STEP, MSR_FORM_BACKWARD, MSR_FORM_QKV_CHUNKWISE = 0, 1, 2, 3, 4
STATUS = {0: "MSR_OK", -1: "MSR_ERR_INVALID_ARG", -2: "MSR_ERR_SHAPE", -3: "MSR_ERR_DTYPE",
          -4: "MSR_ERR_UNSUPPORTED", -5: "MSR_ERR_WORKSPACE", -6: "MSR_ERR_HIP"}

EXPORTS = ("msr_abi_version", "msr_last_error", "msr_workspace_size", "msr_workspace_bytes", "msr_parallel",
           "msr_chunkwise", "msr_chunkwise_noalloc", "msr_chunkwise_backward", "msr_qkv_projection", "msr_qkv_chunkwise",
           "msr_recurrent_step", "msr_set_kernel_events", "msr_set_exchange",
           "msr_add_rmsnorm", "msr_add_rmsnorm_backward", "msr_add_rmsnorm_backward_workspace", "msr_quantize",
           "msr_scaled_matmul",
           "msr_qk_norm_rotate", "msr_qk_norm_rotate_backward", "msr_qk_norm_rotate_backward_workspace",
           "msr_gated_recurrence", "msr_gated_recurrence_workspace", "msr_gated_recurrence_step",
           "msr_gated_recurrence_backward", "msr_gradient_norm", "msr_gradient_norm_workspace", "msr_clip_gradients")


class MsrError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {what}")


class Problem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("gamma", ctypes.POINTER(ctypes.c_float)), ("theta", ctypes.POINTER(ctypes.c_float)),
        ("scale", ctypes.c_float), ("gn_eps", ctypes.c_float),
        ("pos0", ctypes.c_int64), ("flags", ctypes.c_uint32),
        ("pos_rows", ctypes.c_void_p),
    ]


_lib = None


def load():
    """Load libmsr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m retnet_scale_retention_amd.build`")
    lib = ctypes.CDLL(str(LIB_PATH))
    P = ctypes.POINTER(Problem)
    vp, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_float)
    lib.msr_abi_version.argtypes, lib.msr_abi_version.restype = [], ctypes.c_int
    lib.msr_last_error.argtypes, lib.msr_last_error.restype = [], ctypes.c_char_p
    lib.msr_workspace_size.argtypes = [P, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]
    lib.msr_workspace_size.restype = ctypes.c_int
    lib.msr_workspace_bytes.argtypes = [P, ctypes.c_int32, ctypes.c_int32]
    lib.msr_workspace_bytes.restype = ctypes.c_size_t
    lib.msr_parallel.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.msr_parallel.restype = ctypes.c_int
    lib.msr_chunkwise.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.msr_chunkwise.restype = ctypes.c_int
    lib.msr_chunkwise_noalloc.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp]
    lib.msr_chunkwise_noalloc.restype = ctypes.c_int
    lib.msr_chunkwise_backward.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                           ctypes.c_size_t, vp]
    lib.msr_chunkwise_backward.restype = ctypes.c_int
    lib.msr_qkv_projection.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.msr_qkv_projection.restype = ctypes.c_int
    lib.msr_qkv_chunkwise.argtypes = [P, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp,
                                      ctypes.c_size_t, vp]
    lib.msr_qkv_chunkwise.restype = ctypes.c_int
    lib.msr_recurrent_step.argtypes = [P, vp, vp, vp, vp, vp, vp]
    lib.msr_recurrent_step.restype = ctypes.c_int
    lib.msr_set_kernel_events.argtypes = [vp, vp]
    lib.msr_set_kernel_events.restype = None
    lib.msr_set_exchange.argtypes, lib.msr_set_exchange.restype = [ctypes.c_int32], ctypes.c_int
    i32, i64, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.msr_add_rmsnorm.argtypes = [i64, i32, i32, vp, vp, vp, i32, f32, vp, vp, vp, vp, vp]
    lib.msr_add_rmsnorm.restype = ctypes.c_int
    lib.msr_add_rmsnorm_backward.argtypes = [i64, i32, i32, vp, vp, i32, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.msr_add_rmsnorm_backward.restype = ctypes.c_int
    lib.msr_add_rmsnorm_backward_workspace.argtypes, lib.msr_add_rmsnorm_backward_workspace.restype = [i64, i32], sz
    lib.msr_quantize.argtypes = [i64, i64, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.msr_quantize.restype = ctypes.c_int
    lib.msr_scaled_matmul.argtypes = [i64, i64, i64, vp, vp, vp, vp, i32, i32, vp, vp]
    lib.msr_scaled_matmul.restype = ctypes.c_int
    # msr_problem as bytes (_HEAD_PROBLEM)
    lib.msr_qk_norm_rotate.argtypes = [vp, i32, f32, vp, i64, vp, i64, vp, vp, i32, vp, vp, vp]
    lib.msr_qk_norm_rotate_backward.argtypes = [vp, i32, f32, vp, i64, vp, i64, vp, vp, i32, vp, vp, vp, i64, vp, i64,
                                                vp, vp, vp, sz, vp]
    lib.msr_qk_norm_rotate_backward_workspace.argtypes = [i64, i32, i32, i32]
    lib.msr_gated_recurrence.argtypes = [i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.msr_gated_recurrence_workspace.argtypes = [i64, i64, i64, i32]
    lib.msr_gated_recurrence_step.argtypes = [i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.msr_gated_recurrence_backward.argtypes = [i64, i64, i64, i32, i32, *[vp] * 12, sz, vp]
    lib.msr_gradient_norm.argtypes = [vp, i64, vp, vp, sz, vp]
    lib.msr_gradient_norm_workspace.argtypes = [vp, i64]
    lib.msr_clip_gradients.argtypes = [vp, i64, f32, vp, vp, vp, sz, vp]
    for name in ("msr_qk_norm_rotate", "msr_qk_norm_rotate_backward", "msr_gated_recurrence", "msr_gated_recurrence_step",
                 "msr_gated_recurrence_backward", "msr_gradient_norm", "msr_clip_gradients"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("msr_qk_norm_rotate_backward_workspace", "msr_gated_recurrence_workspace", "msr_gradient_norm_workspace"):
        getattr(lib, name).restype = sz
    del fp
    _lib = lib
    return lib


def _check(status: int):
    if status != MSR_OK:
        raise MsrError(status, load().msr_last_error().decode(errors="replace"))


class _Desc:
    """A Problem plus the host arrays it points to (kept alive)."""

    def __init__(self, B, T, H, dk, dv, dtype, gamma, theta=None, scale=0.0, eps=1e-5, pos0=0, flags=0,
                 pos_rows=None):
        self.gamma = np.ascontiguousarray(gamma, dtype=np.float32)
        if self.gamma.shape != (H,):
            raise ValueError(f"gamma must hold H={H} values")
        self.theta = None if theta is None else np.ascontiguousarray(theta, dtype=np.float32)
        if self.theta is not None and self.theta.shape != (dk // 2,):
            raise ValueError(f"theta must hold dk/2={dk // 2} values")
        fptr = lambda a: (ctypes.POINTER(ctypes.c_float)() if a is None
                          else a.ctypes.data_as(ctypes.POINTER(ctypes.c_float)))
        self.p = Problem(B, T, H, dk, dv, dtype, fptr(self.gamma), fptr(self.theta),
                         float(scale), float(eps), int(pos0), int(flags), pos_rows)

    @property
    def ref(self):
        return ctypes.byref(self.p)


def workspace_size(B, T, H, dk, dv, dtype, gamma, form, chunk=0, **kw) -> int:
    d = _Desc(B, T, H, dk, dv, dtype, gamma, **kw)
    n = ctypes.c_size_t(0)
    _check(load().msr_workspace_size(d.ref, form, chunk, ctypes.byref(n)))
    return int(n.value)


# --------------------------------------------------------------- torch side
def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return MSR_F32
    if t.dtype == torch.bfloat16:
        return MSR_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class _Torch:
    """What the layer's entry points use of torch, looked up once (they are called for every token, and a call's host time
    is most of a small one's cost)."""

    def __init__(self):
        torch = _torch()
        self.f32, self.f8, self.u8, self.empty = torch.float32, torch.float8_e4m3fn, torch.uint8, torch.empty
        self.codes = {torch.float32: MSR_F32, torch.bfloat16: MSR_BF16}
        self.raw_stream, self.device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self.tensor = torch.Tensor


_tc = None


def _setup():
    global _tc
    load()
    _tc = _Torch()
    return _tc


def _handle(stream, index):
    """The stream's handle (None: device `index`'s current stream)."""
    if stream is None:
        return (_tc or _setup()).raw_stream(index)
    if stream.device_index != index:
        raise ValueError(f"stream is of device {stream.device_index}, the tensors are on device {index}")
    return stream.cuda_stream


def _at(index, fn):
    """fn with device `index` the current one while it runs: the library launches on the current device, and the handle of
    a default stream names no device."""
    if (_tc or _setup()).device() == index:
        return fn

    def moved(*args):
        with _torch().cuda.device(index):
            return fn(*args)
    return moved


def _empty(shape, dtype, device, stream, kept=True):
    """Memory that a call on `stream` (None: the current one) writes, taken from that stream's pool: a block of the current
    stream's pool could still be in use there when `stream` writes it, and a workspace of that pool would go back to it on
    return, to be handed out again while `stream` still uses it.  `kept`: the caller gets it, and may drop it while the
    current stream still reads it."""
    tc = _tc or _setup()
    if stream is None:
        return tc.empty(shape, dtype=dtype, device=device)
    torch = _torch()
    with torch.cuda.stream(stream):
        t = tc.empty(shape, dtype=dtype, device=device)
    if kept:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _workspace(workspace, n, like, stream):
    """The caller's workspace where it holds n bytes, or one of the call's own, on the device of `like`; and its bytes."""
    if workspace is not None:
        if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
        size = workspace.nbytes
        if size >= n:
            return workspace, size
    n = max(n, 1)
    return _empty((n,), (_tc or _setup()).u8, like.device, stream, kept=False), n


def _prep(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous device tensor")
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("expected q, k [B, T, H, dk] and v [B, T, H, dv]")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    return (*q.shape, v.shape[3])


def _pos_rows(pos_rows, B, device):
    """Device address of a per-batch-row position tensor (int64 [B]), or None."""
    torch = _torch()
    if pos_rows is None:
        return None
    if (pos_rows.dtype != torch.int64 or tuple(pos_rows.shape) != (B,) or not pos_rows.is_contiguous()
            or pos_rows.device != device):
        raise ValueError(f"pos_rows must be a contiguous int64 [B={B}] tensor on {device}")
    return pos_rows.data_ptr()


def _form(fn, form, q, k, v, gamma, chunk, theta, scale, eps, pos0, flags, state_in,
          return_state, out, state_out, workspace, stream, pos_rows=None):
    torch = _torch()
    B, T, H, dk, dv = _prep(q, k, v)
    code = _dtype_code(q)
    d = _Desc(B, T, H, dk, dv, code, gamma, theta, scale, eps, pos0, flags, _pos_rows(pos_rows, B, q.device))
    n = ctypes.c_size_t(0)
    _check(load().msr_workspace_size(d.ref, form, chunk, ctypes.byref(n)))
    workspace, ws_bytes = _workspace(workspace, n.value, q, stream)
    if out is None:
        out = _empty((B, T, H, dv), q.dtype, q.device, stream)
    if state_in is not None and (state_in.dtype != torch.float32 or not state_in.is_contiguous()
                                 or tuple(state_in.shape) != (B, H, dk, dv)):
        raise ValueError("state_in must be a contiguous float32 [B, H, dk, dv] tensor")
    if state_out is None and return_state:
        state_out = _empty((B, H, dk, dv), torch.float32, q.device, stream)
    args = [d.ref]
    if form == MSR_FORM_CHUNKWISE:
        args.append(int(chunk))
    args += [_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(state_in), _ptr(state_out),
             _ptr(workspace), ws_bytes, _handle(stream, q.get_device())]
    _check(_at(q.get_device(), fn)(*args))
    return out, state_out


def msr_parallel(q, k, v, gamma, *, theta=None, scale=0.0, eps=1e-5, pos0=0, flags=0,
                 state_in=None, return_state=True, out=None, state_out=None, workspace=None,
                 stream=None, pos_rows=None):
    """Parallel form. q, k: [B, T, H, dk]; v: [B, T, H, dv] (float32 or bfloat16,
    on the device); gamma: H host values; pos_rows: optional int64 [B] device
    tensor of per-row start positions (else every row starts at pos0).
    Returns (O, state_out or None)."""
    return _form(load().msr_parallel, MSR_FORM_PARALLEL, q, k, v, gamma, 0, theta, scale, eps,
                 pos0, flags, state_in, return_state, out, state_out, workspace, stream, pos_rows)


def msr_chunkwise(q, k, v, gamma, chunk, *, theta=None, scale=0.0, eps=1e-5, pos0=0, flags=0,
                  state_in=None, return_state=True, out=None, state_out=None, workspace=None,
                  stream=None, pos_rows=None):
    """Chunkwise-recurrent form with chunk size `chunk` (a last chunk shorter
    than `chunk` takes the remaining tokens when chunk does not divide T)."""
    return _form(load().msr_chunkwise, MSR_FORM_CHUNKWISE, q, k, v, gamma, chunk, theta, scale,
                 eps, pos0, flags, state_in, return_state, out, state_out, workspace, stream, pos_rows)


NOALLOC_SCRATCH_BYTES = 64 << 20  # MSR_NOALLOC_SCRATCH_BYTES


def msr_chunkwise_noalloc(q, k, v, gamma, chunk, *, out, state_out=None, theta=None, scale=0.0, eps=1e-5, pos0=0,
                          flags=0, state_in=None, stream=None, pos_rows=None):
    """msr_chunkwise with the library's fixed per-GPU scratch array instead of
    a workspace: allocates nothing (out and state_out are the caller's).
    Returns (O, state_out)."""
    torch = _torch()
    B, T, H, dk, dv = _prep(q, k, v)
    d = _Desc(B, T, H, dk, dv, _dtype_code(q), gamma, theta, scale, eps, pos0, flags,
              _pos_rows(pos_rows, B, q.device))
    if tuple(out.shape) != (B, T, H, dv) or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous [B, T, H, dv] tensor of q's dtype")
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != (B, H, dk, dv)):
            raise ValueError(f"{name} must be a contiguous float32 [B, H, dk, dv] tensor")
    fn = _at(q.get_device(), load().msr_chunkwise_noalloc)
    _check(fn(d.ref, int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(state_in), _ptr(state_out),
              _handle(stream, q.get_device())))
    return out, state_out


def msr_chunkwise_backward(q, k, v, gamma, chunk, grad_out, *, grad_state=None, state_in=None, theta=None,
                           scale=0.0, eps=1e-5, pos0=0, flags=0, pos_rows=None, want_state_grad=True,
                           workspace=None, stream=None):
    """Gradients of the chunkwise (= parallel) form through rotation, scale,
    retention and GroupNorm.  grad_out: dL/dO [B, T, H, dv] (dtype of q);
    grad_state: dL/dstate_out [B, H, dk, dv] float32 or None.  Returns
    (dQ, dK, dV, dstate_in or None), dQ/dK/dV in the dtype of q."""
    torch = _torch()
    B, T, H, dk, dv = _prep(q, k, v)
    if tuple(grad_out.shape) != (B, T, H, dv) or grad_out.dtype != q.dtype or not grad_out.is_contiguous():
        raise ValueError("grad_out must be a contiguous [B, T, H, dv] tensor of q's dtype")
    for name, t in (("state_in", state_in), ("grad_state", grad_state)):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != (B, H, dk, dv)):
            raise ValueError(f"{name} must be a contiguous float32 [B, H, dk, dv] tensor")
    d = _Desc(B, T, H, dk, dv, _dtype_code(q), gamma, theta, scale, eps, pos0, flags,
              _pos_rows(pos_rows, B, q.device))
    n = ctypes.c_size_t(0)
    _check(load().msr_workspace_size(d.ref, MSR_FORM_BACKWARD, chunk, ctypes.byref(n)))
    workspace, ws_bytes = _workspace(workspace, n.value, q, stream)
    dq, dk_, dv_ = (_empty(t.shape, t.dtype, t.device, stream) for t in (q, k, v))
    ds = _empty((B, H, dk, dv), torch.float32, q.device, stream) if want_state_grad else None
    fn = _at(q.get_device(), load().msr_chunkwise_backward)
    _check(fn(d.ref, int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(state_in), _ptr(grad_out), _ptr(grad_state),
              _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(ds), _ptr(workspace), ws_bytes,
              _handle(stream, q.get_device())))
    return dq, dk_, dv_, ds


def _qkv_args(x, wq, wk, wv, H):
    for name, t in (("x", x), ("wq", wq), ("wk", wk), ("wv", wv)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous device tensor")
    if x.dim() != 3 or wq.dim() != 2 or wk.shape != wq.shape or wv.dim() != 2:
        raise ValueError("expected x [B, T, d_model], wq, wk [H dk, d_model], wv [H dv, d_model]")
    B, T, dm = x.shape
    if wq.shape[1] != dm or wv.shape[1] != dm or wq.shape[0] % H or wv.shape[0] % H:
        raise ValueError("weight shapes do not match d_model and H")
    return B, T, dm, wq.shape[0] // H, wv.shape[0] // H


def msr_qkv_projection(x, wq, wk, wv, H, *, theta=None, scale=0.0, pos0=0, flags=0, pos_rows=None,
                       out=None, stream=None):
    """Q = R(x wq^T), K = s R(x wk^T), V = x wv^T as [B, T, H, d] bf16
    (x [B, T, d_model] bf16, weights [H d, d_model]).  Returns (Q, K, V)."""
    B, T, dm, dk, dv = _qkv_args(x, wq, wk, wv, H)
    d = _Desc(B, T, H, dk, dv, _dtype_code(x), np.ones(H, np.float32), theta, scale, 1e-5, pos0, flags,
              _pos_rows(pos_rows, B, x.device))
    if out is None:
        out = tuple(_empty((B, T, H, w), x.dtype, x.device, stream) for w in (dk, dk, dv))
    fn = _at(x.get_device(), load().msr_qkv_projection)
    _check(fn(d.ref, int(dm), _ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), *(_ptr(t) for t in out),
              _handle(stream, x.get_device())))
    return out


def msr_qkv_chunkwise(x, wq, wk, wv, gamma, chunk, *, theta=None, scale=0.0, eps=1e-5, pos0=0, flags=0,
                      state_in=None, return_state=True, out=None, state_out=None, workspace=None,
                      stream=None, pos_rows=None):
    """The projections followed by the chunkwise form: returns (O, state_out
    or None) for the layer input x [B, T, d_model] and weights [H d, d_model]."""
    torch = _torch()
    H = len(np.atleast_1d(gamma))
    B, T, dm, dk, dv = _qkv_args(x, wq, wk, wv, H)
    d = _Desc(B, T, H, dk, dv, _dtype_code(x), gamma, theta, scale, eps, pos0, flags,
              _pos_rows(pos_rows, B, x.device))
    n = ctypes.c_size_t(0)
    _check(load().msr_workspace_size(d.ref, MSR_FORM_QKV_CHUNKWISE, chunk, ctypes.byref(n)))
    workspace, ws_bytes = _workspace(workspace, n.value, x, stream)
    if out is None:
        out = _empty((B, T, H, dv), x.dtype, x.device, stream)
    if state_out is None and return_state:
        state_out = _empty((B, H, dk, dv), torch.float32, x.device, stream)
    fn = _at(x.get_device(), load().msr_qkv_chunkwise)
    _check(fn(d.ref, int(chunk), int(dm), _ptr(x), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(out), _ptr(state_in),
              _ptr(state_out), _ptr(workspace), ws_bytes, _handle(stream, x.get_device())))
    return out, state_out


def msr_recurrent_step(q, k, v, state, gamma, pos, *, theta=None, scale=0.0, eps=1e-5, flags=0,
                       out=None, stream=None):
    """One decode step at absolute position `pos` (an int, or an int64 [B]
    device tensor with one position per batch row); q, k: [B, H, dk],
    v: [B, H, dv]; state [B, H, dk, dv] float32 is updated in place.
    Returns o [B, H, dv]."""
    torch = _torch()
    for name, t in (("q", q), ("k", k), ("v", v), ("state", state)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous device tensor")
    B, H, dk = q.shape
    dv = v.shape[2]
    if state.dtype != torch.float32 or tuple(state.shape) != (B, H, dk, dv):
        raise ValueError("state must be float32 [B, H, dk, dv]")
    if isinstance(pos, torch.Tensor):
        d = _Desc(B, 1, H, dk, dv, _dtype_code(q), gamma, theta, scale, eps, 0, flags,
                  _pos_rows(pos, B, q.device))
    else:
        d = _Desc(B, 1, H, dk, dv, _dtype_code(q), gamma, theta, scale, eps, pos, flags)
    if out is None:
        out = _empty((B, H, dv), q.dtype, q.device, stream)
    fn = _at(q.get_device(), load().msr_recurrent_step)
    _check(fn(d.ref, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(state), _handle(stream, q.get_device())))
    return out


# ------------------------------------------------- the layer around retention
BLOCK = 128  # MSR_BLOCK


def _code(name, t):
    """MSR_F32 or MSR_BF16 of a tensor that has to be a contiguous one on the device."""
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous device tensor")
    code = _tc.codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}; use float32 or bfloat16")
    return code


def _expect(name, t, shape, dtype, index):
    """t's address, t checked to be a contiguous tensor of this shape and type on device `index`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on device {index}")
    return t.data_ptr()


def _weight(weight, d, index):
    if weight is None:
        return None, MSR_F32
    dtype = weight.dtype
    code = _tc.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} of weight; use float32 or bfloat16")
    return _expect("weight", weight, (d,), dtype, index), code


def _rows(shape):
    """Rows of an array [..., d]."""
    return shape[0] if len(shape) == 2 else math.prod(shape[:-1])


def msr_add_rmsnorm(x, weight=None, residual=None, *, eps=1e-6, want_y=True, want_q=False, out=None, stream=None):
    """h = x + residual and its root-mean-square norm n = h / sqrt(mean(h^2) + eps) * weight over the last dimension.
    x, residual: [..., d] float32 or bfloat16; weight: [d] of either type.  Returns (y, sum, q, scale), None where
    not computed: y = n in x's type (want_y); sum = h in x's type (when a residual is given); q, scale (want_q) = n as
    float8_e4m3fn [..., P(d)] (P: the next multiple of 128, zeros there) with a float32 scale per 128 values,
    [..., P(d) / 128].  out: tensors to write, in the same order (sum may be x or residual, y may be x)."""
    tc = _tc or _setup()
    code = _code("x", x)
    shape, dtype, dev = x.shape, x.dtype, x.get_device()
    d = shape[-1] if shape else 0
    y, total, q, scale = out or (None, None, None, None)
    rp = tp = wp = yp = qp = sp = None
    wcode = MSR_F32
    if residual is None:
        total = None
    else:
        rp = _expect("residual", residual, shape, dtype, dev)
        if total is None:
            total = _empty(shape, dtype, x.device, stream)
        tp = _expect("sum", total, shape, dtype, dev)
    if weight is not None:
        wp, wcode = _weight(weight, d, dev)
    if want_y:
        if y is None:
            y = _empty(shape, dtype, x.device, stream)
        yp = _expect("y", y, shape, dtype, dev)
    else:
        y = None
    if want_q:
        blocks = (d + 127) // BLOCK
        qshape, sshape = (*shape[:-1], blocks * BLOCK), (*shape[:-1], blocks)
        if q is None:
            q = _empty(qshape, tc.f8, x.device, stream)
        if scale is None:
            scale = _empty(sshape, tc.f32, x.device, stream)
        qp = _expect("q", q, qshape, tc.f8, dev)
        sp = _expect("scale", scale, sshape, tc.f32, dev)
    else:
        q = scale = None
    fn = _lib.msr_add_rmsnorm if tc.device() == dev else _at(dev, _lib.msr_add_rmsnorm)
    s = fn(_rows(shape), d, code, x.data_ptr(), rp, wp, wcode, eps, tp, yp, qp, sp,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return y, total, q, scale


def msr_add_rmsnorm_backward(h, weight, grad_y, *, grad_sum=None, eps=1e-6, want_weight_grad=True, out=None,
                             workspace=None, stream=None):
    """Gradients of msr_add_rmsnorm: h = the forward call's sum (x when it had no residual), grad_y = dL/dn, grad_sum =
    dL/dsum or None, all [..., d] of one type.  Returns (dx, dweight or None): dx is the gradient of x and of the
    residual, in h's type; dweight is float32 [d].  out: tensors to write, in the same order."""
    tc = _tc or _setup()
    code = _code("h", h)
    shape, dtype, dev = h.shape, h.dtype, h.get_device()
    d, rows = shape[-1] if shape else 0, _rows(shape)
    gp = _expect("grad_y", grad_y, shape, dtype, dev)
    sp = None if grad_sum is None else _expect("grad_sum", grad_sum, shape, dtype, dev)
    wp, wcode = _weight(weight, d, dev)
    dx, dw = out or (None, None)
    if dx is None:
        dx = _empty(shape, dtype, h.device, stream)
    xp, dwp, ws, n = _expect("dx", dx, shape, dtype, dev), None, None, 0
    if want_weight_grad:
        if dw is None:
            dw = _empty((d,), tc.f32, h.device, stream)
        dwp = _expect("dweight", dw, (d,), tc.f32, dev)
        n = _lib.msr_add_rmsnorm_backward_workspace(rows, d)
        if n:
            if workspace is None and stream is None:
                workspace = tc.empty(n, dtype=tc.u8, device=h.device)
            else:
                workspace, n = _workspace(workspace, n, h, stream)
            ws = workspace.data_ptr()
    else:
        dw = None
    fn = _lib.msr_add_rmsnorm_backward if tc.device() == dev else _at(dev, _lib.msr_add_rmsnorm_backward)
    s = fn(rows, d, code, h.data_ptr(), wp, wcode, eps, gp, sp, xp, dwp, ws, n,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return dx, dw


def msr_quantize(x, *, block_rows=1, want_rows=True, want_transposed=False, out=None, stream=None):
    """x [rows, cols] (float32 or bfloat16) in 8 bits: (q, scale, qt, scale_t), None where not wanted.  q:
    float8_e4m3fn [rows, P(cols)] (P: the next multiple of 128, zeros there), qt [cols, P(rows)] its transposed
    counterpart.  block_rows 1: a float32 scale per 128 values of a row of the array written, scale [rows, P(cols) /
    128], scale_t [cols, P(rows) / 128]; block_rows 128: a scale per 128 x 128 square, [P(rows) / 128, P(cols) / 128]
    and its transpose.  out: tensors to write, in the same order."""
    tc = _tc or _setup()
    code = _code("x", x)
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    (R, C), dev = x.shape, x.get_device()
    q, sc, qt, st = out or (None, None, None, None)
    rb, cb, square = (R + 127) // BLOCK, (C + 127) // BLOCK, block_rows == BLOCK
    qp = sp = qtp = stp = None
    if want_rows:
        shape = (rb if square else R, cb)
        if q is None:
            q = _empty((R, cb * BLOCK), tc.f8, x.device, stream)
        if sc is None:
            sc = _empty(shape, tc.f32, x.device, stream)
        qp, sp = _expect("q", q, (R, cb * BLOCK), tc.f8, dev), _expect("scale", sc, shape, tc.f32, dev)
    else:
        q = sc = None
    if want_transposed:
        shape = (cb if square else C, rb)
        if qt is None:
            qt = _empty((C, rb * BLOCK), tc.f8, x.device, stream)
        if st is None:
            st = _empty(shape, tc.f32, x.device, stream)
        qtp, stp = _expect("qt", qt, (C, rb * BLOCK), tc.f8, dev), _expect("scale_t", st, shape, tc.f32, dev)
    else:
        qt = st = None
    fn = _lib.msr_quantize if tc.device() == dev else _at(dev, _lib.msr_quantize)
    s = fn(R, C, code, block_rows, x.data_ptr(), qp, sp, qtp, stp,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return q, sc, qt, st


def msr_scaled_matmul(a, a_scale, b, b_scale, *, out_dtype=None, out=None, stream=None):
    """a b^T of 8-bit operands with a scale for each block of 128: a [..., K] float8_e4m3fn with a_scale [..., K /
    128], b [N, K] with b_scale [N, K / 128] or, per 128 x 128 square, [P(N) / 128, K / 128] (float32; K a multiple
    of 128).  Returns [..., N] of out_dtype: bfloat16 (default) or float32.  A bfloat16 result comes from the 8-bit matrix
    instruction, which drops the bits of each 8 products below 2^-13 of the largest: far below bfloat16's rounding of the
    sum of their magnitudes, but a result that nearly cancels is less accurate than its type.  A float32 result keeps
    fp32's accuracy, and takes up to twice as long."""
    tc = _tc or _setup()
    if not (a.is_cuda and a.is_contiguous()) or not a.dim():
        raise ValueError("a must be a contiguous device tensor")
    if a.dtype is not tc.f8 or b.dtype is not tc.f8:
        raise TypeError("a and b must be float8_e4m3fn")
    shape, dev = a.shape, a.get_device()
    lead, k, n, m = shape[:-1], shape[-1], b.shape[0] if b.dim() else 0, _rows(shape)
    kb = k // BLOCK
    bp = _expect("b", b, (n, k), tc.f8, dev)
    ap = _expect("a_scale", a_scale, (*lead, kb), tc.f32, dev)
    rows = 1 if b_scale.shape == (n, kb) else BLOCK
    sp = _expect("b_scale", b_scale, (n if rows == 1 else (n + 127) // BLOCK, kb), tc.f32, dev)
    if out is None:
        out = _empty((*lead, n), out_dtype or _torch().bfloat16, a.device, stream)
    elif out_dtype is None:
        out_dtype = out.dtype
    code = tc.codes.get(out.dtype)
    if code is None:
        raise TypeError(f"unsupported output dtype {out.dtype}; use float32 or bfloat16")
    op = _expect("out", out, (*lead, n), out_dtype or out.dtype, dev)
    fn = _lib.msr_scaled_matmul if tc.device() == dev else _at(dev, _lib.msr_scaled_matmul)
    s = fn(m, n, k, a.data_ptr(), ap, b.data_ptr(), sp, rows, code, op,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return out


# ------------------------------------------------------- next to retention
_HEAD_PROBLEM = struct.Struct("=6iQQffqI4xQ")  # msr_problem, its pointers as numbers (gamma and dv are not used)


def _heads(name, t, dtype, index):
    """(B, T, H, dk, address, elements from a token to the next) of Q or K: [B, T, H, dk], or [B, H, dk] for one token
    each, the heads of a token packed and the tokens at one distance."""
    shape = t.shape
    if t.get_device() != index or t.dtype is not dtype or index < 0:
        raise ValueError(f"{name} must be a {dtype} tensor on the device of q")
    if len(shape) == 4:
        B, T, H, dk = shape
    elif len(shape) == 3:
        (B, H, dk), T = shape, 1
    else:
        raise ValueError(f"{name} must be [B, T, H, dk] or [B, H, dk]")
    if t.is_contiguous() or B * T == 0:
        return B, T, H, dk, t.data_ptr(), H * dk
    stride = t.stride()
    step = H * dk if B * T == 1 else stride[0] if T == 1 else stride[1]
    if (stride[-1] != 1 and dk > 1) or (stride[-2] != dk and H > 1) or step < H * dk or (
            B > 1 and T > 1 and stride[0] != T * step):
        raise ValueError(f"{name}: the heads of a token must be packed and all tokens at one distance; got strides {stride}")
    return B, T, H, dk, t.data_ptr(), step


def _head_problem(B, T, H, dk, code, theta, scale, pos0, flags, pos_rows, device):
    """msr_problem as bytes, and what it points to."""
    at = 0
    if theta is not None:
        if not (type(theta) is np.ndarray and theta.dtype == np.float32 and theta.flags.c_contiguous):
            theta = np.ascontiguousarray(theta, dtype=np.float32)
        if theta.shape != (dk // 2,):
            raise ValueError(f"theta must hold dk/2={dk // 2} values")
        at = theta.__array_interface__["data"][0]
    return _HEAD_PROBLEM.pack(B, T, H, dk, 4, code, 0, at, scale, 0.0, pos0, flags,
                              0 if pos_rows is None else _pos_rows(pos_rows, B, device)), theta


def _pair_weights(wq, wk, dk, index):
    wqp, qcode = _weight(wq, dk, index)
    wkp, kcode = _weight(wk, dk, index)
    if wqp is not None and wkp is not None and qcode != kcode:
        raise TypeError("wq and wk must share one dtype")
    return wqp, wkp, qcode if wqp is not None else kcode


def msr_qk_norm_rotate(q, k=None, wq=None, wk=None, *, eps=1e-6, theta=None, scale=0.0, pos0=0, flags=0, pos_rows=None,
                       out=None, stream=None):
    """Root-mean-square norms of the query and key heads with the position rotation in the same pass:
    R(pos theta) (q / sqrt(mean(q^2) + eps) * wq), and the same of k times scale (0: dk^-0.5).  q [B, T, H, dk], k
    [B, T, Hk, dk] (or [B, H, dk] for one token each) float32 or bfloat16; views of one fused projection are fine: the
    heads of a token packed, tokens at any one distance.  wq, wk [dk] or None.  pos0 or pos_rows as in the forms,
    MSR_FLAG_NO_ROTATE for the norms alone.  Returns (q', k') packed (out: tensors to write; q' may be q); the forms take
    them with flags=MSR_FLAG_NO_ROTATE and scale=1."""
    tc = _tc or _setup()
    dtype, dev = q.dtype, q.get_device()
    code = tc.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} of q; use float32 or bfloat16")
    B, T, H, dk, qp, qs = _heads("q", q, dtype, dev)
    Hk = ks = 0
    kp = kop = None
    qo, ko = out or (None, None)
    if k is not None:
        Bk, Tk, Hk, dkk, kp, ks = _heads("k", k, dtype, dev)
        if (Bk, Tk, dkk) != (B, T, dk):
            raise ValueError("q and k must share B, T and dk")
        if ko is None:
            ko = _empty(k.shape, dtype, k.device, stream)
        kop = _expect("out of k", ko, k.shape, dtype, dev)
    else:
        ko = wk = None
    if qo is None:
        qo = _empty(q.shape, dtype, q.device, stream)
    qop = _expect("out of q", qo, q.shape, dtype, dev)
    wqp, wkp, wcode = _pair_weights(wq, wk, dk, dev)
    p, keep = _head_problem(B, T, H, dk, code, theta, scale, pos0, flags, pos_rows, q.device)
    fn = _lib.msr_qk_norm_rotate if tc.device() == dev else _at(dev, _lib.msr_qk_norm_rotate)
    s = fn(p, Hk, eps, qp, qs, kp, ks, wqp, wkp, wcode, qop, kop,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return qo, ko


def msr_qk_norm_rotate_backward(q, k, wq, wk, grad_q, grad_k, *, eps=1e-6, theta=None, scale=0.0, pos0=0, flags=0,
                                pos_rows=None, want_weight_grad=True, out=None, workspace=None, stream=None):
    """Gradients of msr_qk_norm_rotate: q, k, weights and the rest as there, grad_q = dL/dq', grad_k = dL/dk' packed.
    Returns (dq, dk, dwq, dwk): dq, dk in q's type, dwq, dwk float32 [dk] (None unless want_weight_grad; that of a weight
    of ones where the weight is None).  out: tensors to write, in the same order; dq and dk may be views like q and k, so
    that they lie side by side in a fused projection's gradient, or grad_q and grad_k themselves."""
    tc = _tc or _setup()
    dtype, dev = q.dtype, q.get_device()
    code = tc.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} of q; use float32 or bfloat16")
    B, T, H, dk, qp, qs = _heads("q", q, dtype, dev)
    gqp = _expect("grad_q", grad_q, q.shape, dtype, dev)
    dq, dkk, dwq, dwk = out or (None, None, None, None)
    if dq is None:
        dq = _empty(q.shape, dtype, q.device, stream)
    elif dq.shape != q.shape:
        raise ValueError("dq must have q's shape")
    dqp, dqs = _heads("dq", dq, dtype, dev)[4:]
    Hk = ks = dks = 0
    kp = gkp = dkp = None
    if k is not None:
        Bk, Tk, Hk, d2, kp, ks = _heads("k", k, dtype, dev)
        if (Bk, Tk, d2) != (B, T, dk):
            raise ValueError("q and k must share B, T and dk")
        gkp = _expect("grad_k", grad_k, k.shape, dtype, dev)
        if dkk is None:
            dkk = _empty(k.shape, dtype, k.device, stream)
        elif dkk.shape != k.shape:
            raise ValueError("dk must have k's shape")
        dkp, dks = _heads("dk", dkk, dtype, dev)[4:]
    else:
        dkk = dwk = wk = None
    wqp, wkp, wcode = _pair_weights(wq, wk, dk, dev)
    p, keep = _head_problem(B, T, H, dk, code, theta, scale, pos0, flags, pos_rows, q.device)
    dwqp = dwkp = ws = None
    n = 0
    if want_weight_grad:
        if dwq is None:
            dwq = _empty((dk,), tc.f32, q.device, stream)
        dwqp = _expect("dwq", dwq, (dk,), tc.f32, dev)
        if k is not None:
            if dwk is None:
                dwk = _empty((dk,), tc.f32, q.device, stream)
            dwkp = _expect("dwk", dwk, (dk,), tc.f32, dev)
        n = _lib.msr_qk_norm_rotate_backward_workspace(B * T, H, Hk, dk)
        workspace, n = _workspace(workspace, n, q, stream)
        ws = workspace.data_ptr()
    else:
        dwq = dwk = None
    fn = _lib.msr_qk_norm_rotate_backward if tc.device() == dev else _at(dev, _lib.msr_qk_norm_rotate_backward)
    s = fn(p, Hk, eps, qp, qs, kp, ks, wqp, wkp, wcode, gqp, gkp, dqp, dqs, dkp, dks, dwqp, dwkp, ws, n,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return dq, dkk, dwq, dwk


GATE_BLOCK = 64  # MSR_GATE_BLOCK


def _gate(x, g, rate, dims):
    code = _code("x", x)
    if x.dim() != dims:
        raise ValueError("x must be [B, T, D]" if dims == 3 else "x must be [B, D]")
    dev = x.get_device()
    return code, dev, _expect("g", g, x.shape, x.dtype, dev), _expect("rate", rate, (x.shape[-1],), _tc.f32, dev)


def msr_gated_recurrence(x, g, rate, *, normalize=True, state_in=None, return_state=True, want_carry=False, out=None,
                         workspace=None, stream=None):
    """A recurrence whose decay depends on the data and the channel: h_t = a_t h_(t-1) + m_t x_t, a_t = exp(-rate
    sigmoid(g_t)), m_t = sqrt(1 - a_t^2) (normalize) or 1.  x, g [B, T, D] float32 or bfloat16, rate [D] float32 >= 0,
    state_in [B, D] float32 or None (zeros).  Returns (h, state, carry), None where not wanted: h in x's type, state
    [B, D] float32 after the last token, carry [B, ceil(T / 64), D] float32: the states before the tokens 0, 64, 128, ...,
    which the backward pass takes.  out: tensors to write, in the same order (state may be state_in)."""
    tc = _tc or _setup()
    code, dev, gp, rp = _gate(x, g, rate, 3)
    B, T, D = shape = x.shape
    h, state, carry = out or (None, None, None)
    if h is None:
        h = _empty(shape, x.dtype, x.device, stream)
    hp = _expect("h", h, shape, x.dtype, dev)
    ip = sp = cp = None
    if state_in is not None:
        ip = _expect("state_in", state_in, (B, D), tc.f32, dev)
    if return_state:
        if state is None:
            state = _empty((B, D), tc.f32, x.device, stream)
        sp = _expect("state", state, (B, D), tc.f32, dev)
    else:
        state = None
    if want_carry:
        cshape = (B, (T + GATE_BLOCK - 1) // GATE_BLOCK, D)
        if carry is None:
            carry = _empty(cshape, tc.f32, x.device, stream)
        cp = _expect("carry", carry, cshape, tc.f32, dev)
    else:
        carry = None
    ws, n = None, _lib.msr_gated_recurrence_workspace(B, T, D, 0)
    if n:
        workspace, n = _workspace(workspace, n, x, stream)
        ws = workspace.data_ptr()
    fn = _lib.msr_gated_recurrence if tc.device() == dev else _at(dev, _lib.msr_gated_recurrence)
    s = fn(B, T, D, code, normalize, x.data_ptr(), gp, rp, ip, hp, sp, cp, ws, n,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return h, state, carry


def msr_gated_recurrence_step(x, g, state, rate, *, normalize=True, state_out=None, out=None, stream=None):
    """One token of msr_gated_recurrence: x, g [B, D]; state [B, D] float32, updated in place unless state_out is given.
    Returns h [B, D]."""
    tc = _tc or _setup()
    code, dev, gp, rp = _gate(x, g, rate, 2)
    B, D = shape = x.shape
    ip = _expect("state", state, shape, tc.f32, dev)
    sp = ip if state_out is None else _expect("state_out", state_out, shape, tc.f32, dev)
    if out is None:
        out = _empty(shape, x.dtype, x.device, stream)
    hp = _expect("out", out, shape, x.dtype, dev)
    fn = _lib.msr_gated_recurrence_step if tc.device() == dev else _at(dev, _lib.msr_gated_recurrence_step)
    s = fn(B, D, code, normalize, x.data_ptr(), gp, rp, ip, sp, hp,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return out


def msr_gated_recurrence_backward(x, g, rate, grad_h, *, normalize=True, state_in=None, carry=None, grad_state=None,
                                  want_rate_grad=True, want_state_grad=True, out=None, workspace=None, stream=None):
    """Gradients of msr_gated_recurrence: x, g, rate, state_in as there, carry the forward call's (None: the forward pass
    runs again for it), grad_h = dL/dh in x's type, grad_state = dL/dstate float32 [B, D] or None.  Returns (dx, dg,
    drate, dstate_in): dx, dg in x's type, drate [D] and dstate_in [B, D] float32, None where not wanted.  out: tensors
    to write, in the same order."""
    tc = _tc or _setup()
    code, dev, gp, rp = _gate(x, g, rate, 3)
    B, T, D = shape = x.shape
    dhp = _expect("grad_h", grad_h, shape, x.dtype, dev)
    dx, dg, drate, dstate = out or (None, None, None, None)
    if dx is None:
        dx = _empty(shape, x.dtype, x.device, stream)
    if dg is None:
        dg = _empty(shape, x.dtype, x.device, stream)
    dxp, dgp = _expect("dx", dx, shape, x.dtype, dev), _expect("dg", dg, shape, x.dtype, dev)
    ip = cp = gsp = drp = dsp = None
    if state_in is not None:
        ip = _expect("state_in", state_in, (B, D), tc.f32, dev)
    if carry is not None:
        cp = _expect("carry", carry, (B, (T + GATE_BLOCK - 1) // GATE_BLOCK, D), tc.f32, dev)
    if grad_state is not None:
        gsp = _expect("grad_state", grad_state, (B, D), tc.f32, dev)
    if want_rate_grad:
        if drate is None:
            drate = _empty((D,), tc.f32, x.device, stream)
        drp = _expect("drate", drate, (D,), tc.f32, dev)
    else:
        drate = None
    if want_state_grad:
        if dstate is None:
            dstate = _empty((B, D), tc.f32, x.device, stream)
        dsp = _expect("dstate_in", dstate, (B, D), tc.f32, dev)
    else:
        dstate = None
    ws, n = None, _lib.msr_gated_recurrence_workspace(B, T, D, 2 if carry is None else 1)
    if n:
        workspace, n = _workspace(workspace, n, x, stream)
        ws = workspace.data_ptr()
    fn = _lib.msr_gated_recurrence_backward if tc.device() == dev else _at(dev, _lib.msr_gated_recurrence_backward)
    s = fn(B, T, D, code, normalize, x.data_ptr(), gp, rp, ip, cp, dhp, gsp, dxp, dgp, drp, dsp, ws, n,
           tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return dx, dg, drate, dstate


_dtype_of = operator.attrgetter("dtype")


def _gradients(grads, out):
    """The C ABI's table of the tensors (msr_gradient: four 64-bit numbers each), and their device.  Column by column: a
    call has many tensors, and this is most of its host time."""
    if not grads:
        raise ValueError("no gradients given")
    T, dev, n = _tc.tensor, grads[0].get_device(), len(grads)
    both = grads if out is None else [*grads, *out]
    if len(both) != (n if out is None else 2 * n):
        raise ValueError("out must hold a tensor for each gradient")
    if dev < 0 or set(map(T.get_device, both)) != {dev} or not all(map(T.is_contiguous, both)):
        raise ValueError("gradients and out must be contiguous tensors on one device")
    codes = list(map(_tc.codes.get, map(_dtype_of, both)))
    if None in codes:
        raise TypeError("unsupported dtype of a gradient; use float32 or bfloat16")
    sizes = list(map(T.numel, both))
    if out is not None and (codes[:n] != codes[n:] or sizes[:n] != sizes[n:]):
        raise ValueError("a tensor of out must have its gradient's type and size")
    at = list(map(T.data_ptr, both))
    table = [0] * (4 * n)
    table[0::4], table[1::4], table[2::4], table[3::4] = at[:n], at[-n:], sizes[:n], codes[:n]
    return array.array("q", table), dev


def msr_gradient_norm(grads, *, out=None, workspace=None, stream=None):
    """The square root of the sum of the squares of all elements of `grads` (contiguous float32 and bfloat16 tensors), a
    float32 scalar on the device (out: the one to write).  Squares and sums are float64, in a fixed order."""
    tc = _tc or _setup()
    grads = list(grads)
    table, dev = _gradients(grads, None)
    at, like = table.buffer_info()[0], grads[0]
    if out is None:
        out = _empty((), tc.f32, like.device, stream)
    op = _expect("out", out, (), tc.f32, dev)
    workspace, n = _workspace(workspace, _lib.msr_gradient_norm_workspace(at, len(grads)), like, stream)
    fn = _lib.msr_gradient_norm if tc.device() == dev else _at(dev, _lib.msr_gradient_norm)
    s = fn(at, len(grads), op, workspace.data_ptr(), n, tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return out


def msr_clip_gradients(grads, max_norm, *, norm=None, out=None, norm_out=None, workspace=None, stream=None):
    """g * min(1, max_norm / norm) for every tensor g of `grads` (contiguous, float32 and bfloat16), in place or to the
    tensors `out`.  norm: a float32 scalar on the device, e.g. one joined over processes; None: that of msr_gradient_norm,
    formed here (norm_out: the scalar to write it to).  Where it is infinite or NaN the gradients stay as they are.
    Returns (out or grads, norm)."""
    tc = _tc or _setup()
    grads = list(grads)
    if out is not None:
        out = list(out)
    table, dev = _gradients(grads, out)
    at, like = table.buffer_info()[0], grads[0]
    np_ = op = ws = None
    n = 0
    if norm is not None:
        if norm_out is not None:
            raise ValueError("norm_out is for the norm that the call forms; norm was given")
        np_ = _expect("norm", norm, (), tc.f32, dev)
    else:
        norm = _empty((), tc.f32, like.device, stream) if norm_out is None else norm_out
        op = _expect("norm_out", norm, (), tc.f32, dev)
        workspace, n = _workspace(workspace, _lib.msr_gradient_norm_workspace(at, len(grads)), like, stream)
        ws = workspace.data_ptr()
    fn = _lib.msr_clip_gradients if tc.device() == dev else _at(dev, _lib.msr_clip_gradients)
    s = fn(at, len(grads), max_norm, np_, op, ws, n, tc.raw_stream(dev) if stream is None else _handle(stream, dev))
    if s:
        _check(s)
    return grads if out is None else out, norm


def set_kernel_events(start=None, stop=None):
    """Measurement hook: record the hipEvent handles `start` / `stop` (ints
    or None) around the main kernel of every later call on this thread."""
    load().msr_set_kernel_events(ctypes.c_void_p(start) if start else None,
                                 ctypes.c_void_p(stop) if stop else None)


def set_exchange(mode: int):
    """Process-wide GroupNorm finishing of the split-row chunk kernel
    (MSR_EXCHANGE_AUTO, MSR_EXCHANGE_OFF or MSR_EXCHANGE_NO_WAIT; include/msr.h)."""
    _check(load().msr_set_exchange(int(mode)))
