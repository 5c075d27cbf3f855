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

import ctypes
import math
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
           "msr_scaled_matmul")


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


def set_kernel_events(start=None, stop=None):
    """Measurement hook: record the hipEvent handles `start` / `stop` (ints
    or None) around the main kernel of every later call on this thread."""
    load().msr_set_kernel_events(ctypes.c_void_p(start) if start else None,
                                 ctypes.c_void_p(stop) if stop else None)


def set_exchange(mode: int):
    """Process-wide GroupNorm finishing of the split-row chunk kernel
    (MSR_EXCHANGE_AUTO, MSR_EXCHANGE_OFF or MSR_EXCHANGE_NO_WAIT; include/msr.h)."""
    _check(load().msr_set_exchange(int(mode)))
