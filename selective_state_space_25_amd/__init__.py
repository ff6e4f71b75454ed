"""libselscan: the selective state-space scan of Mamba on AMD MI355X (gfx950).

Thin Python binding over the C ABI in ``include/selscan.h``.  It only
marshals arguments: torch tensors provide device memory and the current HIP
stream; every step of the scan runs in the HIP kernels of ``libselscan.so``.
There is no fallback: if the library is missing the import of a kernel entry
point raises.

    y, last_state = selscan.fwd(u, delta, A, B, C, D, z, delta_bias, softplus=True)
    y, last_state = selscan.mamba2_fwd(x, dt, A, B, C, D, z, dt_bias, softplus=True)
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libselscan.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_NO_DEVICE, ERR_LAUNCH, ERR_WORKSPACE = range(6)
F32, BF16 = 0, 1

_STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "NO_DEVICE", 4: "LAUNCH", 5: "WORKSPACE"}


class SelscanError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libselscan {_STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Shape(ctypes.Structure):
    """selscan_shape_t (Mamba-1)."""
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("seqlen", ctypes.c_int64), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class M2Shape(ctypes.Structure):
    """selscan_m2_shape_t (Mamba-2)."""
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("ngroups", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


_lib = None

EXPORTED = ("selscan_fwd", "selscan_mamba2_fwd", "selscan_workspace_bytes", "selscan_mamba2_workspace_bytes",
            "selscan_fwd_h0", "selscan_mamba2_fwd_h0", "selscan_step", "selscan_mamba2_step", "selscan_conv1d",
            "selscan_bwd", "selscan_bwd_workspace_bytes", "selscan_fwd_noalloc",
            "selscan_mamba2_bwd", "selscan_mamba2_bwd_workspace_bytes",
            "selscan_delta_fwd", "selscan_delta_workspace_bytes", "selscan_delta_step",
            "selscan_delta_bwd", "selscan_delta_bwd_workspace_bytes",
            "selscan_dropout", "selscan_layer_norm_fwd", "selscan_layer_norm_bwd",
            "selscan_layer_norm_bwd_workspace_bytes",
            "selscan_last_error", "selscan_version", "selscan_timing_enable", "selscan_timing_collect")


class ConvShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("width", ctypes.c_int64), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


class NormShape(ctypes.Structure):
    """selscan_norm_shape_t."""
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("in_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class DropoutShape(ctypes.Structure):
    """selscan_dropout_shape_t."""
    _fields_ = [("n", ctypes.c_int64), ("dtype", ctypes.c_int32), ("p", ctypes.c_double),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_int64), ("total_ms", ctypes.c_double),
                ("min_ms", ctypes.c_double), ("max_ms", ctypes.c_double)]


def lib() -> ctypes.CDLL:
    """The loaded libselscan.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m selective_state_space_25_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, i32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        L.selscan_fwd.argtypes = [ctypes.POINTER(Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, vp, fp, vp]
        L.selscan_fwd.restype = i32
        L.selscan_mamba2_fwd.argtypes = [ctypes.POINTER(M2Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, vp, fp, vp]
        L.selscan_mamba2_fwd.restype = i32
        L.selscan_fwd_h0.argtypes = [ctypes.POINTER(Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, fp, vp, fp, vp]
        L.selscan_fwd_h0.restype = i32
        L.selscan_mamba2_fwd_h0.argtypes = [ctypes.POINTER(M2Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, fp, vp, fp,
                                            vp]
        L.selscan_mamba2_fwd_h0.restype = i32
        L.selscan_fwd_noalloc.argtypes = [ctypes.POINTER(Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, fp, vp, fp,
                                          vp]
        L.selscan_fwd_noalloc.restype = i32
        L.selscan_step.argtypes = [ctypes.POINTER(Shape), fp, vp, vp, fp, vp, vp, fp, vp, fp, i32, vp, vp]
        L.selscan_step.restype = i32
        L.selscan_mamba2_step.argtypes = [ctypes.POINTER(M2Shape), fp, vp, vp, fp, vp, vp, fp, vp, fp, i32, vp, vp]
        L.selscan_mamba2_step.restype = i32
        L.selscan_conv1d.argtypes = [ctypes.POINTER(ConvShape), vp, fp, fp, i32, vp, vp]
        L.selscan_conv1d.restype = i32
        L.selscan_bwd.argtypes = [ctypes.POINTER(Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, fp, vp] + [fp] * 9 + [vp]
        L.selscan_bwd.restype = i32
        L.selscan_mamba2_bwd.argtypes = [ctypes.POINTER(M2Shape), vp, vp, fp, vp, vp, fp, vp, fp, i32, fp, vp] + \
            [fp] * 9 + [vp]
        L.selscan_mamba2_bwd.restype = i32
        L.selscan_mamba2_bwd_workspace_bytes.argtypes = [ctypes.POINTER(M2Shape)]
        L.selscan_mamba2_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.selscan_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Shape)]
        L.selscan_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.selscan_workspace_bytes.argtypes = [ctypes.POINTER(Shape)]
        L.selscan_workspace_bytes.restype = ctypes.c_size_t
        L.selscan_mamba2_workspace_bytes.argtypes = [ctypes.POINTER(M2Shape)]
        L.selscan_mamba2_workspace_bytes.restype = ctypes.c_size_t
        f32 = ctypes.c_float
        L.selscan_delta_workspace_bytes.argtypes = [ctypes.POINTER(M2Shape)]
        L.selscan_delta_workspace_bytes.restype = ctypes.c_size_t
        L.selscan_delta_fwd.argtypes = [ctypes.POINTER(M2Shape), vp, vp, vp, fp, fp, f32, vp, fp, vp, fp, vp]
        L.selscan_delta_fwd.restype = i32
        L.selscan_delta_bwd.argtypes = [ctypes.POINTER(M2Shape), vp, vp, vp, fp, fp, f32, vp, fp, vp, fp, vp, vp, vp] + \
            [fp] * 3 + [vp]
        L.selscan_delta_bwd.restype = i32
        L.selscan_delta_bwd_workspace_bytes.argtypes = [ctypes.POINTER(M2Shape)]
        L.selscan_delta_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.selscan_delta_step.argtypes = [ctypes.POINTER(M2Shape), fp, vp, vp, vp, fp, fp, f32, vp, vp]
        L.selscan_delta_step.restype = i32
        L.selscan_dropout.argtypes = [ctypes.POINTER(DropoutShape), vp, vp, vp]
        L.selscan_dropout.restype = i32
        L.selscan_layer_norm_fwd.argtypes = [ctypes.POINTER(NormShape), vp, vp, fp, fp, vp, vp, fp, fp, vp]
        L.selscan_layer_norm_fwd.restype = i32
        L.selscan_layer_norm_bwd.argtypes = [ctypes.POINTER(NormShape), vp, vp, fp, fp, fp, vp, vp, vp, fp, fp, vp]
        L.selscan_layer_norm_bwd.restype = i32
        L.selscan_layer_norm_bwd_workspace_bytes.argtypes = [ctypes.POINTER(NormShape)]
        L.selscan_layer_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.selscan_last_error.restype = ctypes.c_char_p
        L.selscan_version.restype = ctypes.c_char_p
        L.selscan_timing_enable.argtypes = [i32]
        L.selscan_timing_enable.restype = i32
        L.selscan_timing_collect.argtypes = [ctypes.POINTER(KernelTime), i32]
        L.selscan_timing_collect.restype = i32
        _lib = L
    return _lib


def version() -> str:
    return lib().selscan_version().decode()


def last_error() -> str:
    return lib().selscan_last_error().decode()


def _check(status: int) -> None:
    if status != OK:
        raise SelscanError(status, last_error())


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")


def _ptr(t, name, shape=None, dtype=None, device=None):
    """Device pointer of a dense tensor after checking shape/dtype/device."""
    if t is None:
        return None
    if type(t) is _torch().Tensor and (shape is None or t.shape == shape) and (dtype is None or t.dtype is dtype) \
            and t.is_contiguous() and (device is None or t.device == device):
        return t.data_ptr()
    torch = _torch()   # what is wrong with it, if anything
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _stream_handle(device):
    """The device's current stream as an integer (torch's raw query where it
    has one: the Stream object costs more than the rest of a small call)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None and device.index is not None:
        return raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def m1_shape(batch, dim, dstate, seqlen, in_dtype=BF16, out_dtype=None, workspace=None, workspace_bytes=0):
    return Shape(batch, dim, dstate, seqlen, in_dtype, in_dtype if out_dtype is None else out_dtype,
                 workspace, workspace_bytes)


def fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, out=None, last_state=None,
        return_last_state=True, workspace=None, out_dtype=None, h0=None):
    """Mamba-1 selective scan on the GPU.

    u, delta, z: [batch, dim, L]; B, C: [batch, N, L] (float32 or bfloat16, one
    dtype for all five); A: [dim, N], D, delta_bias: [dim] float32.
    Returns (y [batch, dim, L] float32 unless out_dtype says otherwise,
    last_state [batch, dim, N] float32 or None).  y defaults to float32, the
    precision of the state: a bfloat16 y carries up to 2^-8 relative rounding.
    h0 [batch, dim, N] float32: initial state (None: zero).
    """
    torch = _torch()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selscan.fwd needs tensors on a GPU device")
    batch, dim, L = u.shape
    N = A.shape[1]
    dt = u.dtype
    code = _dtype_code(u)
    odt = (out.dtype if out is not None else torch.float32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, dim, L), dtype=odt, device=dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    s = Shape(batch, dim, N, L, code, _dtype_code(out), ws_ptr, ws_bytes)
    args = (
        _ptr(u, "u", (batch, dim, L), dt, dev), _ptr(delta, "delta", (batch, dim, L), dt, dev),
        _ptr(A, "A", (dim, N), torch.float32, dev), _ptr(B, "B", (batch, N, L), dt, dev),
        _ptr(C, "C", (batch, N, L), dt, dev), _ptr(D, "D", (dim,), torch.float32, dev),
        _ptr(z, "z", (batch, dim, L), dt, dev), _ptr(delta_bias, "delta_bias", (dim,), torch.float32, dev),
        int(bool(softplus)), _ptr(out, "out", (batch, dim, L), odt, dev),
        _ptr(last_state, "last_state", (batch, dim, N), torch.float32, dev), _stream_handle(dev))
    if h0 is None:
        _check(lib().selscan_fwd(ctypes.byref(s), *args))
    else:
        h0p = _ptr(h0, "h0", (batch, dim, N), torch.float32, dev)
        _check(lib().selscan_fwd_h0(ctypes.byref(s), *args[:9], h0p, *args[9:]))
    return out, last_state


def step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, out=None, out_dtype=None):
    """One-token Mamba-1 update (decoding).  state [batch, dim, N] float32 is
    updated in place; u, delta, z [batch, dim]; B, C [batch, N] (float32 or
    bfloat16); A [dim, N], D, delta_bias [dim] float32.  Returns y [batch, dim]
    (float32 unless out_dtype or out says otherwise)."""
    torch = _torch()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selscan.step needs tensors on a GPU device")
    batch, dim = u.shape
    N = A.shape[1]
    dt = u.dtype
    odt = (out.dtype if out is not None else torch.float32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, dim), dtype=odt, device=dev)
    s = Shape(batch, dim, N, 1, _dtype_code(u), _dtype_code(out), None, 0)
    _check(lib().selscan_step(
        ctypes.byref(s), _ptr(state, "state", (batch, dim, N), torch.float32, dev),
        _ptr(u, "u", (batch, dim), dt, dev), _ptr(delta, "delta", (batch, dim), dt, dev),
        _ptr(A, "A", (dim, N), torch.float32, dev), _ptr(B, "B", (batch, N), dt, dev),
        _ptr(C, "C", (batch, N), dt, dev), _ptr(D, "D", (dim,), torch.float32, dev),
        _ptr(z, "z", (batch, dim), dt, dev), _ptr(delta_bias, "delta_bias", (dim,), torch.float32, dev),
        int(bool(softplus)), _ptr(out, "out", (batch, dim), odt, dev), _stream_handle(dev)))
    return out


class _BoundCall:
    """A C-ABI call with its arguments marshalled once: calling it enqueues
    the kernel again on the same buffers (whose contents the caller may
    change in place between calls, as a decoding loop does).  It holds the
    tensors whose addresses it passes, so that their memory stays theirs."""

    def __init__(self, fn, shape, args, tensors):
        self._fn, self._shape, self._args, self._tensors = fn, shape, args, tensors

    def __call__(self):
        st = self._fn(ctypes.byref(self._shape), *self._args)
        if st != OK:
            raise SelscanError(st, last_error())


def bind_step(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, out=None, out_dtype=None):
    """selscan_step with its arguments checked and marshalled once: returns
    (call, y).  Each call() updates `state` in place with the token currently
    held in u, delta, B, C, z and writes y, on the stream that was current at
    binding time."""
    torch = _torch()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selscan.bind_step needs tensors on a GPU device")
    batch, dim = u.shape
    N = A.shape[1]
    dt = u.dtype
    odt = (out.dtype if out is not None else torch.float32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, dim), dtype=odt, device=dev)
    s = Shape(batch, dim, N, 1, _dtype_code(u), _dtype_code(out), None, 0)
    args = (_ptr(state, "state", (batch, dim, N), torch.float32, dev),
            _ptr(u, "u", (batch, dim), dt, dev), _ptr(delta, "delta", (batch, dim), dt, dev),
            _ptr(A, "A", (dim, N), torch.float32, dev), _ptr(B, "B", (batch, N), dt, dev),
            _ptr(C, "C", (batch, N), dt, dev), _ptr(D, "D", (dim,), torch.float32, dev),
            _ptr(z, "z", (batch, dim), dt, dev), _ptr(delta_bias, "delta_bias", (dim,), torch.float32, dev),
            int(bool(softplus)), _ptr(out, "out", (batch, dim), odt, dev), _stream_handle(dev))
    return _BoundCall(lib().selscan_step, s, args, (state, u, delta, A, B, C, D, z, delta_bias, out)), out


def bind_mamba2_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, out=None,
                     out_dtype=None):
    """selscan_mamba2_step with its arguments checked and marshalled once:
    returns (call, y); see bind_step."""
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("selscan.bind_mamba2_step needs tensors on a GPU device")
    batch, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    dtp = x.dtype
    odt = (out.dtype if out is not None else torch.float32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, H, P), dtype=odt, device=dev)
    s = M2Shape(batch, 1, H, P, G, N, _dtype_code(x), _dtype_code(out), None, 0)
    args = (_ptr(state, "state", (batch, H, P, N), torch.float32, dev),
            _ptr(x, "x", (batch, H, P), dtp, dev), _ptr(dt, "dt", (batch, H), dtp, dev),
            _ptr(A, "A", (H,), torch.float32, dev), _ptr(B, "B", (batch, G, N), dtp, dev),
            _ptr(C, "C", (batch, G, N), dtp, dev), _ptr(D, "D", (H,), torch.float32, dev),
            _ptr(z, "z", (batch, H, P), dtp, dev), _ptr(dt_bias, "dt_bias", (H,), torch.float32, dev),
            int(bool(softplus)), _ptr(out, "out", (batch, H, P), odt, dev), _stream_handle(dev))
    return _BoundCall(lib().selscan_mamba2_step, s, args, (state, x, dt, A, B, C, D, z, dt_bias, out)), out


def bwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, dout=None, softplus=True, h0=None,
        want_dh0=False, workspace=None):
    """Gradients of the Mamba-1 scan on the GPU.

    Inputs as for fwd; dout [batch, dim, L] (float32 or bfloat16: the dtype
    of the forward's y) is the gradient of the loss with respect to y.
    Returns a dict of float32 tensors: du, ddelta, dz (when z is given)
    [batch, dim, L]; dA [dim, N]; dB, dC [batch, N, L]; dD (when D is given)
    and ddelta_bias (when delta_bias is given) [dim]; dh0 [batch, dim, N]
    (when h0 is given or want_dh0).
    """
    torch = _torch()
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("selscan.bwd needs tensors on a GPU device")
    if dout is None:
        raise ValueError("dout is required")
    batch, dim, L = u.shape
    N = A.shape[1]
    dt = u.dtype
    f32 = torch.float32
    new = lambda *shape: torch.empty(shape, dtype=f32, device=dev)
    g = {"du": new(batch, dim, L), "ddelta": new(batch, dim, L), "dA": new(dim, N),
         "dB": new(batch, N, L), "dC": new(batch, N, L)}
    if z is not None:
        g["dz"] = new(batch, dim, L)
    if D is not None:
        g["dD"] = new(dim)
    if delta_bias is not None:
        g["ddelta_bias"] = new(dim)
    if h0 is not None or want_dh0:
        g["dh0"] = new(batch, dim, N)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    s = Shape(batch, dim, N, L, _dtype_code(u), _dtype_code(dout), ws_ptr, ws_bytes)
    gp = lambda k: g[k].data_ptr() if k in g else None
    _check(lib().selscan_bwd(
        ctypes.byref(s), _ptr(u, "u", (batch, dim, L), dt, dev), _ptr(delta, "delta", (batch, dim, L), dt, dev),
        _ptr(A, "A", (dim, N), f32, dev), _ptr(B, "B", (batch, N, L), dt, dev), _ptr(C, "C", (batch, N, L), dt, dev),
        _ptr(D, "D", (dim,), f32, dev), _ptr(z, "z", (batch, dim, L), dt, dev),
        _ptr(delta_bias, "delta_bias", (dim,), f32, dev), int(bool(softplus)),
        _ptr(h0, "h0", (batch, dim, N), f32, dev), _ptr(dout, "dout", (batch, dim, L), None, dev),
        gp("du"), gp("ddelta"), gp("dA"), gp("dB"), gp("dC"), gp("dD"), gp("dz"), gp("ddelta_bias"), gp("dh0"),
        _stream_handle(dev)))
    return g


def bwd_workspace_bytes(batch, dim, dstate, seqlen, in_dtype=BF16, out_dtype=None) -> int:
    s = m1_shape(batch, dim, dstate, seqlen, in_dtype, out_dtype)
    return int(lib().selscan_bwd_workspace_bytes(ctypes.byref(s)))


def workspace_bytes(batch, dim, dstate, seqlen, in_dtype=BF16, out_dtype=None) -> int:
    s = m1_shape(batch, dim, dstate, seqlen, in_dtype, out_dtype)
    return int(lib().selscan_workspace_bytes(ctypes.byref(s)))


def mamba2_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, out=None, last_state=None,
               return_last_state=True, workspace=None, out_dtype=None, h0=None):
    """Mamba-2 multi-head selective scan on the GPU.

    x, z: [batch, L, H, P]; dt: [batch, L, H]; B, C: [batch, L, G, N]
    (float32 or bfloat16); A, D, dt_bias: [H] float32.
    Returns (y [batch, L, H, P] float32 unless out_dtype says otherwise,
    last_state [batch, H, P, N] float32 or None).  h0 [batch, H, P, N]
    float32: initial state (None: zero).
    """
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("selscan.mamba2_fwd needs tensors on a GPU device")
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dtp = x.dtype
    odt = (out.dtype if out is not None else torch.float32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, L, H, P), dtype=odt, device=dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, H, P, N), dtype=torch.float32, device=dev)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    s = M2Shape(batch, L, H, P, G, N, _dtype_code(x), _dtype_code(out), ws_ptr, ws_bytes)
    args = (
        _ptr(x, "x", (batch, L, H, P), dtp, dev), _ptr(dt, "dt", (batch, L, H), dtp, dev),
        _ptr(A, "A", (H,), torch.float32, dev), _ptr(B, "B", (batch, L, G, N), dtp, dev),
        _ptr(C, "C", (batch, L, G, N), dtp, dev), _ptr(D, "D", (H,), torch.float32, dev),
        _ptr(z, "z", (batch, L, H, P), dtp, dev), _ptr(dt_bias, "dt_bias", (H,), torch.float32, dev),
        int(bool(softplus)), _ptr(out, "out", (batch, L, H, P), odt, dev),
        _ptr(last_state, "last_state", (batch, H, P, N), torch.float32, dev), _stream_handle(dev))
    if h0 is None:
        _check(lib().selscan_mamba2_fwd(ctypes.byref(s), *args))
    else:
        h0p = _ptr(h0, "h0", (batch, H, P, N), torch.float32, dev)
        _check(lib().selscan_mamba2_fwd_h0(ctypes.byref(s), *args[:9], h0p, *args[9:]))
    return out, last_state


def mamba2_step(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, out=None, out_dtype=None):
    """One-token Mamba-2 update (decoding).  state [batch, H, P, N] float32 is
    updated in place; x, z [batch, H, P]; dt [batch, H]; B, C [batch, G, N]
    (float32 or bfloat16); A, D, dt_bias [H] float32.  Returns y [batch, H, P]."""
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("selscan.mamba2_step needs tensors on a GPU device")
    batch, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    dtp = x.dtype
    odt = (out.dtype if out is not None else torch.float32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, H, P), dtype=odt, device=dev)
    s = M2Shape(batch, 1, H, P, G, N, _dtype_code(x), _dtype_code(out), None, 0)
    _check(lib().selscan_mamba2_step(
        ctypes.byref(s), _ptr(state, "state", (batch, H, P, N), torch.float32, dev),
        _ptr(x, "x", (batch, H, P), dtp, dev), _ptr(dt, "dt", (batch, H), dtp, dev),
        _ptr(A, "A", (H,), torch.float32, dev), _ptr(B, "B", (batch, G, N), dtp, dev),
        _ptr(C, "C", (batch, G, N), dtp, dev), _ptr(D, "D", (H,), torch.float32, dev),
        _ptr(z, "z", (batch, H, P), dtp, dev), _ptr(dt_bias, "dt_bias", (H,), torch.float32, dev),
        int(bool(softplus)), _ptr(out, "out", (batch, H, P), odt, dev), _stream_handle(dev)))
    return out


def mamba2_bwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dout=None, softplus=True, h0=None,
               want_dh0=False, workspace=None):
    """Gradients of the Mamba-2 scan on the GPU (headdim 64).

    Inputs as for mamba2_fwd; dout [batch, L, nheads, headdim] (float32 or
    bfloat16) is the gradient of the loss with respect to y.  Returns a dict
    of float32 tensors: dx, dz (when z is given) [batch, L, nheads, headdim];
    ddt [batch, L, nheads]; dA [nheads]; dB, dC [batch, L, ngroups, N]; dD
    (when D is given) and ddt_bias (when dt_bias is given) [nheads]; dh0
    [batch, nheads, headdim, N] (when h0 is given or want_dh0).
    """
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("selscan.mamba2_bwd needs tensors on a GPU device")
    if dout is None:
        raise ValueError("dout is required")
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dt_ = x.dtype
    f32 = torch.float32
    new = lambda *shape: torch.empty(shape, dtype=f32, device=dev)
    g = {"dx": new(batch, L, H, P), "ddt": new(batch, L, H), "dA": new(H), "dB": new(batch, L, G, N),
         "dC": new(batch, L, G, N)}
    if z is not None:
        g["dz"] = new(batch, L, H, P)
    if D is not None:
        g["dD"] = new(H)
    if dt_bias is not None:
        g["ddt_bias"] = new(H)
    if h0 is not None or want_dh0:
        g["dh0"] = new(batch, H, P, N)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    s = M2Shape(batch, L, H, P, G, N, _dtype_code(x), _dtype_code(dout), ws_ptr, ws_bytes)
    gp = lambda k: g[k].data_ptr() if k in g else None
    _check(lib().selscan_mamba2_bwd(
        ctypes.byref(s), _ptr(x, "x", (batch, L, H, P), dt_, dev), _ptr(dt, "dt", (batch, L, H), dt_, dev),
        _ptr(A, "A", (H,), f32, dev), _ptr(B, "B", (batch, L, G, N), dt_, dev), _ptr(C, "C", (batch, L, G, N), dt_, dev),
        _ptr(D, "D", (H,), f32, dev), _ptr(z, "z", (batch, L, H, P), dt_, dev),
        _ptr(dt_bias, "dt_bias", (H,), f32, dev), int(bool(softplus)),
        _ptr(h0, "h0", (batch, H, P, N), f32, dev), _ptr(dout, "dout", (batch, L, H, P), None, dev),
        gp("dx"), gp("ddt"), gp("dA"), gp("dB"), gp("dC"), gp("dD"), gp("dz"), gp("ddt_bias"), gp("dh0"),
        _stream_handle(dev)))
    return g


def mamba2_bwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype=BF16, out_dtype=None) -> int:
    s = M2Shape(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype, in_dtype if out_dtype is None else out_dtype,
                None, 0)
    return int(lib().selscan_mamba2_bwd_workspace_bytes(ctypes.byref(s)))


def mamba2_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype=BF16, out_dtype=None) -> int:
    s = M2Shape(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype,
                in_dtype if out_dtype is None else out_dtype, None, 0)
    return int(lib().selscan_mamba2_workspace_bytes(ctypes.byref(s)))


def conv1d(x, weight, bias=None, silu=True, out=None, out_dtype=None):
    """Causal depthwise convolution: x [batch, dim, L] (float32 or bfloat16),
    weight [dim, K] and bias [dim] float32.  out[t] = act(bias + sum_k
    weight[k] x[t - (K - 1) + k]), act = silu or identity.  Returns out
    [batch, dim, L] in x's dtype unless out_dtype or out says otherwise."""
    torch = _torch()
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("selscan.conv1d needs tensors on a GPU device")
    batch, dim, L = x.shape
    K = weight.shape[1]
    odt = (out.dtype if out is not None else x.dtype) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, dim, L), dtype=odt, device=dev)
    s = ConvShape(batch, dim, L, K, _dtype_code(x), _dtype_code(out))
    _check(lib().selscan_conv1d(
        ctypes.byref(s), _ptr(x, "x", (batch, dim, L), x.dtype, dev),
        _ptr(weight, "weight", (dim, K), torch.float32, dev), _ptr(bias, "bias", (dim,), torch.float32, dev),
        int(bool(silu)), _ptr(out, "out", (batch, dim, L), odt, dev), _stream_handle(dev)))
    return out


def _ws_arg(workspace, need, device):
    """(pointer, bytes, keep-alive) of a caller's workspace or of one from
    torch's allocator, which is ordered on the current stream."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _torch().empty(need, dtype=_torch().uint8, device=device)
    _ptr(workspace, "workspace", device=device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def delta_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype=BF16, out_dtype=None) -> int:
    s = M2Shape(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype, in_dtype if out_dtype is None else out_dtype,
                None, 0)
    return int(lib().selscan_delta_workspace_bytes(ctypes.byref(s)))


def delta_fwd(q, k, v, g, beta, scale=None, lengths=None, h0=None, out=None, last_state=None, return_last_state=True,
              workspace=None, out_dtype=None):
    """Gated delta rule over a sequence.

    q, k: [batch, L, G, N]; v: [batch, L, H, P] (float32 or bfloat16, one
    dtype), H a multiple of G; g (log decay) and beta (write strength):
    [batch, L, H] float32; scale multiplies the read-out (None: N ** -0.5).
    lengths: [batch] int32 on the GPU, tokens of each row (None: all L);
    h0: [batch, H, P, N] float32 initial state (None: zero).
    Returns (y [batch, L, H, P] float32 unless out_dtype says otherwise,
    last_state [batch, H, P, N] float32 or None).
    """
    torch = _torch()
    f32 = torch.float32
    dev, dt = q.device, q.dtype
    batch, L, G, N = q.shape
    H, P = v.shape[2], v.shape[3]
    odt = (out.dtype if out is not None else f32) if out_dtype is None else out_dtype
    if dev.type != "cuda":
        raise ValueError("selscan.delta_fwd needs tensors on a GPU device")
    if out is None:
        out = torch.empty((batch, L, H, P), dtype=odt, device=dev)
    if last_state is None and return_last_state:
        last_state = torch.empty((batch, H, P, N), dtype=f32, device=dev)
    s = M2Shape(batch, L, H, P, G, N, _dtype_code(q), _dtype_code(out), None, 0)
    args = (_ptr(q, "q", (batch, L, G, N), dt, dev), _ptr(k, "k", (batch, L, G, N), dt, dev),
            _ptr(v, "v", (batch, L, H, P), dt, dev), _ptr(g, "g", (batch, L, H), f32, dev),
            _ptr(beta, "beta", (batch, L, H), f32, dev), N ** -0.5 if scale is None else float(scale),
            _ptr(lengths, "lengths", (batch,), torch.int32, dev), _ptr(h0, "h0", (batch, H, P, N), f32, dev),
            _ptr(out, "out", (batch, L, H, P), odt, dev), _ptr(last_state, "last_state", (batch, H, P, N), f32, dev),
            _stream_handle(dev))
    L_ = lib()
    s.workspace, s.workspace_bytes, ws = _ws_arg(workspace, L_.selscan_delta_workspace_bytes(ctypes.byref(s)), dev)
    _check(L_.selscan_delta_fwd(ctypes.byref(s), *args))
    return out, last_state


def delta_bwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype=BF16, out_dtype=None) -> int:
    s = M2Shape(batch, seqlen, nheads, headdim, ngroups, dstate, in_dtype, in_dtype if out_dtype is None else out_dtype,
                None, 0)
    return int(lib().selscan_delta_bwd_workspace_bytes(ctypes.byref(s)))


def delta_bwd(q, k, v, g, beta, dout, scale=None, lengths=None, h0=None, dlast_state=None, want_dh0=False,
              workspace=None):
    """Gradients of the gated delta rule.

    Inputs as for delta_fwd; dout [batch, L, H, P] (float32 or bfloat16) is
    the gradient of the loss with respect to y, dlast_state [batch, H, P, N]
    float32 that with respect to last_state (None: zero).  Returns a dict: dq,
    dk [batch, L, G, N] and dv [batch, L, H, P] in the inputs' dtype; dg,
    dbeta [batch, L, H] float32; dh0 [batch, H, P, N] float32 (when h0 is
    given or want_dh0).
    """
    torch = _torch()
    f32 = torch.float32
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("selscan.delta_bwd needs tensors on a GPU device")
    batch, L, G, N = q.shape
    H, P = v.shape[2], v.shape[3]
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)
    r = {"dq": new((batch, L, G, N), dt), "dk": new((batch, L, G, N), dt), "dv": new((batch, L, H, P), dt),
         "dg": new((batch, L, H), f32), "dbeta": new((batch, L, H), f32)}
    if h0 is not None or want_dh0:
        r["dh0"] = new((batch, H, P, N), f32)
    s = M2Shape(batch, L, H, P, G, N, _dtype_code(q), _dtype_code(dout), None, 0)
    args = (_ptr(q, "q", (batch, L, G, N), dt, dev), _ptr(k, "k", (batch, L, G, N), dt, dev),
            _ptr(v, "v", (batch, L, H, P), dt, dev), _ptr(g, "g", (batch, L, H), f32, dev),
            _ptr(beta, "beta", (batch, L, H), f32, dev), N ** -0.5 if scale is None else float(scale),
            _ptr(lengths, "lengths", (batch,), torch.int32, dev), _ptr(h0, "h0", (batch, H, P, N), f32, dev),
            _ptr(dout, "dout", (batch, L, H, P), None, dev),
            _ptr(dlast_state, "dlast_state", (batch, H, P, N), f32, dev),
            *(r[n].data_ptr() if n in r else None for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")),
            _stream_handle(dev))
    L_ = lib()
    s.workspace, s.workspace_bytes, ws = _ws_arg(workspace, L_.selscan_delta_bwd_workspace_bytes(ctypes.byref(s)), dev)
    _check(L_.selscan_delta_bwd(ctypes.byref(s), *args))
    return r


def _delta_step_args(state, q, k, v, g, beta, scale, out, out_dtype):
    torch = _torch()
    f32 = torch.float32
    dev, dt = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("selscan.delta_step needs tensors on a GPU device")
    batch, G, N = q.shape
    H, P = v.shape[1], v.shape[2]
    odt = (out.dtype if out is not None else f32) if out_dtype is None else out_dtype
    if out is None:
        out = torch.empty((batch, H, P), dtype=odt, device=dev)
    s = M2Shape(batch, 1, H, P, G, N, _dtype_code(q), _dtype_code(out), None, 0)
    return s, (_ptr(state, "state", (batch, H, P, N), f32, dev), _ptr(q, "q", (batch, G, N), dt, dev),
               _ptr(k, "k", (batch, G, N), dt, dev), _ptr(v, "v", (batch, H, P), dt, dev),
               _ptr(g, "g", (batch, H), f32, dev), _ptr(beta, "beta", (batch, H), f32, dev),
               N ** -0.5 if scale is None else float(scale), _ptr(out, "out", (batch, H, P), odt, dev),
               _stream_handle(dev)), out


def delta_step(state, q, k, v, g, beta, scale=None, out=None, out_dtype=None):
    """One token of the gated delta rule (decoding).  state [batch, H, P, N]
    float32 is updated in place; q, k [batch, G, N]; v [batch, H, P] (float32
    or bfloat16); g, beta [batch, H] float32.  Returns y [batch, H, P]
    (float32 unless out_dtype or out says otherwise)."""
    s, args, out = _delta_step_args(state, q, k, v, g, beta, scale, out, out_dtype)
    _check(lib().selscan_delta_step(ctypes.byref(s), *args))
    return out


def bind_delta_step(state, q, k, v, g, beta, scale=None, out=None, out_dtype=None):
    """selscan_delta_step with its arguments checked and marshalled once:
    returns (call, y); see bind_step."""
    s, args, out = _delta_step_args(state, q, k, v, g, beta, scale, out, out_dtype)
    return _BoundCall(lib().selscan_delta_step, s, args, (state, q, k, v, g, beta, out)), out


def _stream_of_words(seed, offset):
    """seed and offset of a mask: ctypes would keep 64 bits of any integer."""
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError(f"seed and offset must be in [0, 2^64), got {seed} and {offset}")
    return seed, offset


def dropout(x, p, seed, offset=0, out=None):
    """Dropout with a mask that is a function of (seed, offset, element index)
    and is never stored: kept elements times 1 / (1 - p), the others zero.
    The gradient is the same call on the output's gradient.  x: any shape,
    float32 or bfloat16; out: the result (may be x).  seed, offset: integers
    in [0, 2^64)."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("selscan.dropout needs tensors on a GPU device")
    if out is None:
        out = _torch().empty_like(x)
    s = DropoutShape(x.numel(), _dtype_code(x), p, *_stream_of_words(seed, offset))
    _check(lib().selscan_dropout(ctypes.byref(s), _ptr(x, "x"), _ptr(out, "out", x.shape, x.dtype, dev),
                                 _stream_handle(dev)))
    return out


def layer_norm_fwd(x, weight=None, bias=None, residual=None, eps=1e-5, p=0.0, seed=0, offset=0, out=None,
                   out_dtype=None, res_dtype=None):
    """Layer norm of s = dropout(x) + residual over the last dimension.

    x: [..., dim] float32 or bfloat16; residual: the same shape, float32 or
    bfloat16, or None; weight, bias: [dim] float32 or None (1 and 0); p, seed,
    offset: the dropout of x (see dropout).
    Returns (y, s, mean, rstd): y in x's dtype unless out_dtype or out says
    otherwise; s in residual's dtype (x's, or res_dtype, without one; x itself
    when there is neither dropout nor residual, unless out is x's memory); mean
    and rstd [...] float32.
    """
    torch = _torch()
    f32 = torch.float32
    dev, shape = x.device, x.shape
    if dev.type != "cuda":
        raise ValueError("selscan.layer_norm_fwd needs tensors on a GPU device")
    dim = shape[-1]
    odt = (out.dtype if out is not None else x.dtype) if out_dtype is None else out_dtype
    rdt = residual.dtype if residual is not None else (x.dtype if res_dtype is None else res_dtype)
    keep_x = residual is None and p == 0.0 and rdt == x.dtype
    if out is None:
        out = torch.empty(shape, dtype=odt, device=dev)
    elif keep_x and out.untyped_storage().data_ptr() == x.untyped_storage().data_ptr():
        keep_x = False   # y may be written over x
    s = x if keep_x else torch.empty(shape, dtype=rdt, device=dev)
    mean = torch.empty(shape[:-1], dtype=f32, device=dev)
    rstd = torch.empty(shape[:-1], dtype=f32, device=dev)
    sh = NormShape(x.numel() // max(dim, 1), dim, _dtype_code(x), _dtype_code(s), _dtype_code(out), eps, p,
                   *_stream_of_words(seed, offset), None, 0)
    _check(lib().selscan_layer_norm_fwd(
        ctypes.byref(sh), _ptr(x, "x"), _ptr(residual, "residual", shape, rdt, dev),
        _ptr(weight, "weight", (dim,), f32, dev), _ptr(bias, "bias", (dim,), f32, dev),
        _ptr(out, "out", shape, odt, dev), None if s is x else s.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        _stream_handle(dev)))
    return out, s, mean, rstd


def layer_norm_bwd(dy, s, weight=None, mean=None, rstd=None, dresidual=None, p=0.0, seed=0, offset=0, x_dtype=None,
                   workspace=None):
    """Gradients of layer_norm_fwd from the s, mean and rstd that it returned.

    dy: [..., dim] gradient of y; dresidual: gradient of s from its other
    uses, in s's dtype, or None; p, seed, offset as in the forward call.
    Returns a dict: dx in x_dtype (None: s's dtype), dresidual (the gradient
    of residual; the same tensor as dx when there is no dropout and the dtypes
    agree) in s's dtype, dweight and dbias [dim] float32.
    """
    torch = _torch()
    f32 = torch.float32
    dev, shape = dy.device, dy.shape
    if dev.type != "cuda":
        raise ValueError("selscan.layer_norm_bwd needs tensors on a GPU device")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are required")
    dim = shape[-1]
    xdt = s.dtype if x_dtype is None else x_dtype
    ds = torch.empty(shape, dtype=s.dtype, device=dev)
    dx = ds if p == 0.0 and xdt == s.dtype else torch.empty(shape, dtype=xdt, device=dev)
    dw = torch.empty((dim,), dtype=f32, device=dev)
    db = torch.empty((dim,), dtype=f32, device=dev)
    sh = NormShape(dy.numel() // max(dim, 1), dim, _dtype_code(dx), _dtype_code(s), _dtype_code(dy), 0.0, p,
                   *_stream_of_words(seed, offset), None, 0)
    L_ = lib()
    sh.workspace, sh.workspace_bytes, ws = _ws_arg(
        workspace, L_.selscan_layer_norm_bwd_workspace_bytes(ctypes.byref(sh)), dev)
    _check(L_.selscan_layer_norm_bwd(
        ctypes.byref(sh), _ptr(dy, "dy"), _ptr(s, "s", shape, None, dev), _ptr(weight, "weight", (dim,), f32, dev),
        _ptr(mean, "mean", shape[:-1], f32, dev), _ptr(rstd, "rstd", shape[:-1], f32, dev),
        _ptr(dresidual, "dresidual", shape, s.dtype, dev), None if dx is ds else dx.data_ptr(), ds.data_ptr(),
        dw.data_ptr(), db.data_ptr(), _stream_handle(dev)))
    return {"dx": dx, "dresidual": ds, "dweight": dw, "dbias": db}


def timing_enable(on: bool) -> None:
    """Bracket every later kernel launch with HIP events on its own stream."""
    _check(lib().selscan_timing_enable(int(bool(on))))


def timing_collect() -> dict:
    """Wait for the bracketed launches so far; {kernel: {launches, total_ms,
    avg_ms, min_ms, max_ms}} in order of first launch."""
    cap = 32
    buf = (KernelTime * cap)()
    n = lib().selscan_timing_collect(buf, cap)
    if n < 0:
        raise SelscanError(n, "selscan_timing_collect failed")
    res = {}
    for k in buf[:min(n, cap)]:
        res[k.name.decode()] = {"launches": k.launches, "total_ms": k.total_ms,
                                "avg_ms": k.total_ms / max(k.launches, 1), "min_ms": k.min_ms, "max_ms": k.max_ms}
    return res


__all__ = ["delta_fwd", "delta_bwd", "delta_bwd_workspace_bytes", "delta_step", "bind_delta_step", "delta_workspace_bytes", "dropout", "layer_norm_fwd",
           "layer_norm_bwd", "NormShape", "DropoutShape", "bind_step", "bind_mamba2_step", "bwd", "bwd_workspace_bytes", "conv1d", "ConvShape", "step", "mamba2_step", "timing_enable", "timing_collect", "KernelTime", "fwd", "mamba2_fwd", "workspace_bytes", "mamba2_workspace_bytes", "version", "last_error", "lib",
           "SelscanError", "Shape", "M2Shape", "m1_shape", "EXPORTED", "LIB_PATH"]
