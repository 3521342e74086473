"""ctypes binding of the operators around the GEMV: include/gla_scan.h.

Argument marshalling only, as in ``_lib``: the C functions keep their names
and return the C status codes (pointers are addresses as ints or None); the
classes take torch tensors, check them and raise ``GemvError`` on any status
other than GEMV_OK.  There is no fallback.

Scratch.  Where a call needs some, the classes allocate it with torch on the
call's stream and drop it after the launch: torch reuses the memory only for
later work of that stream (and keeps it for a graph that captures the call),
so calls never share scratch.  ``workspace=`` passes a tensor of the caller's
instead.
"""
import ctypes

from . import _lib
from ._lib import (GEMV_ERR_INVALID_ARG, GEMV_ERR_UNSUPPORTED_DTYPE, GEMV_ERR_WRONG_DEVICE, GEMV_OK,
                   Gemv, GemvError, _check_devices, _dtype_code)

# every symbol include/gla_scan.h declares
OPERATOR_EXPORTS = ("gla_scan_workspace_bytes", "gla_scan_forward", "gla_scan_backward",
                    "gla_scan_check_args", "gla_scan_grad_check_args")

_vp, _i32, _i64, _st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
_sz, _f32 = ctypes.c_size_t, ctypes.c_float


class gla_stride_t(ctypes.Structure):
    _fields_ = [("batch", _i64), ("token", _i64), ("head", _i64)]


class gla_scan_t(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("heads", _i64), ("dk", _i64), ("dv", _i64),
                ("dtype", _st), ("gate_f32", _i32), ("scale", _f32),
                ("q", gla_stride_t), ("k", gla_stride_t), ("v", gla_stride_t), ("gk", gla_stride_t),
                ("o", gla_stride_t), ("offsets", _vp), ("rows", _i64)]


class gla_scan_grad_t(ctypes.Structure):
    _fields_ = [("dq", gla_stride_t), ("dk", gla_stride_t), ("dv", gla_stride_t),
                ("dgk", gla_stride_t)]


_ready = None


def load():
    """libgemv.so with these operators' signatures set."""
    global _ready
    if _ready is None:
        lib = _lib.load()
        scan, grad = ctypes.POINTER(gla_scan_t), ctypes.POINTER(gla_scan_grad_t)
        lib.gla_scan_workspace_bytes.argtypes = [scan, _i32]
        lib.gla_scan_workspace_bytes.restype = _sz
        lib.gla_scan_forward.argtypes = [_vp, scan] + [_vp] * 7 + [_vp, _sz, _vp]
        lib.gla_scan_check_args.argtypes = [scan] + [_vp] * 7 + [_vp, _sz]
        lib.gla_scan_backward.argtypes = [_vp, scan, grad] + [_vp] * 12 + [_vp, _sz, _vp]
        lib.gla_scan_grad_check_args.argtypes = [scan, grad] + [_vp] * 12 + [_vp, _sz]
        for name in ("gla_scan_forward", "gla_scan_check_args", "gla_scan_backward",
                     "gla_scan_grad_check_args"):
            getattr(lib, name).restype = _st
        _ready = lib
    return _ready


# ---- the C entry points, same names ------------------------------------------

def gla_scan_workspace_bytes(p, backward=False):
    return load().gla_scan_workspace_bytes(ctypes.byref(p), int(backward))


def gla_scan_forward(h, p, q, k, v, gk, S0, ST, o, workspace=None, workspace_bytes=0, stream=None):
    return load().gla_scan_forward(h, ctypes.byref(p), q, k, v, gk, S0, ST, o, workspace,
                                   workspace_bytes, stream)


def gla_scan_check_args(p, q, k, v, gk, S0, ST, o, workspace=None, workspace_bytes=0):
    return load().gla_scan_check_args(ctypes.byref(p), q, k, v, gk, S0, ST, o, workspace,
                                      workspace_bytes)


def gla_scan_backward(h, p, grad, q, k, v, gk, S0, dout, dST, dq, dk, dv, dgk, dS0, workspace=None,
                      workspace_bytes=0, stream=None):
    return load().gla_scan_backward(h, ctypes.byref(p), ctypes.byref(grad), q, k, v, gk, S0, dout,
                                    dST, dq, dk, dv, dgk, dS0, workspace, workspace_bytes, stream)


def gla_scan_grad_check_args(p, grad, q, k, v, gk, S0, dout, dST, dq, dk, dv, dgk, dS0,
                             workspace=None, workspace_bytes=0):
    return load().gla_scan_grad_check_args(ctypes.byref(p), ctypes.byref(grad), q, k, v, gk, S0,
                                           dout, dST, dq, dk, dv, dgk, dS0, workspace,
                                           workspace_bytes)


# ---- torch tensors -------------------------------------------------------------

def _bad(what):
    return GemvError(GEMV_ERR_INVALID_ARG, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_of(device, stream):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _on_current(device):
    """The library launches on the current device: tensors elsewhere are refused."""
    import torch
    if device.index != torch.cuda.current_device():
        raise GemvError(GEMV_ERR_WRONG_DEVICE, "tensors on %s, current device %d"
                        % (device, torch.cuda.current_device()))


def _scratch(workspace, need, device, stream):
    """(tensor to keep until the launch, address, bytes)."""
    if workspace is not None:
        _check_devices((workspace,), device)
        if not workspace.is_contiguous():
            raise _bad("workspace must be contiguous")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need == 0:
        return None, None, 0
    if stream is not None:
        raise _bad("a call on a stream that is given needs a workspace of %d bytes" % need)
    import torch
    w = torch.empty(need, dtype=torch.uint8, device=device)
    return w, w.data_ptr(), need


def _strides(t):
    b, n, h, _ = t.stride()
    return gla_stride_t(b, n, h)


class GlaScan:
    """GLA over whole sequences (include/gla_scan.h), through a Gemv handle.

    q, k, gk: (b, t, h, dk); v, o: (b, t, h, dv), any strides with dense
    channels (a (b, h, t, d) tensor is passed as ``x.transpose(1, 2)``).
    S0, ST: float32 (b, h, dk, dv).  With ``offsets`` (int32, on the GPU) b is
    1, sequence i is rows offsets[i]..offsets[i+1]-1, states have one entry per
    sequence, and ``longest`` is the longest sequence's length (default: t)."""

    def __init__(self, gemv=None):
        self.g = gemv if gemv is not None else Gemv()

    @staticmethod
    def describe(q, v, gk, o, scale, k=None, offsets=None, longest=None):
        """The gla_scan_t of a call on these tensors (k: strides of q unless given)."""
        import torch
        b, t, h, dk = q.shape
        p = gla_scan_t(b, t, h, dk, v.shape[-1], _dtype_code(q), int(gk.dtype == torch.float32),
                       float(scale), _strides(q), _strides(q if k is None else k), _strides(v),
                       _strides(gk), _strides(o), None, 0)
        if offsets is not None:
            p.batch, p.rows, p.offsets = offsets.numel() - 1, t, offsets.data_ptr()
            p.tokens = t if longest is None else min(int(longest), t)
        return p

    def _check(self, named, states, q, v, gk, offsets):
        import torch
        if q.dim() != 4 or v.dim() != 4:
            raise _bad("q and v must be (b, t, h, d)")
        b, t, h, dk = q.shape
        dv = v.shape[3]
        for name, x, d in named:
            if tuple(x.shape) != (b, t, h, d) or (d > 1 and x.stride(3) != 1):
                raise _bad("%s %s, strides %s" % (name, tuple(x.shape), x.stride()))
        nseq = b
        if offsets is not None:
            if b != 1 or offsets.dim() != 1 or offsets.numel() < 1 or offsets.dtype != torch.int32 or \
                    not offsets.is_contiguous():
                raise _bad("offsets must be dense int32 (n + 1), with b == 1")
            nseq = offsets.numel() - 1
        for name, S in states:
            if S is not None and (tuple(S.shape) != (nseq, h, dk, dv) or not S.is_contiguous()):
                raise _bad("%s must be dense (%d, %d, %d, %d)" % (name, nseq, h, dk, dv))
            if S is not None and S.dtype != torch.float32:
                raise GemvError(GEMV_ERR_UNSUPPORTED_DTYPE, "%s is float32" % name)
        for name, x, _ in named:
            gate = name in ("gk", "dgk")
            if x.dtype != (gk.dtype if gate else q.dtype):
                raise GemvError(GEMV_ERR_UNSUPPORTED_DTYPE, "%s is %s" % (name, x.dtype))
        if gk.dtype not in (q.dtype, torch.float32):
            raise GemvError(GEMV_ERR_UNSUPPORTED_DTYPE, "gk has q's dtype or float32")
        _check_devices([x for _, x, _ in named] + [S for _, S in states] + [offsets], q.device)
        _on_current(q.device)

    def forward(self, q, k, v, gk, o, scale, S0=None, ST=None, offsets=None, longest=None,
                workspace=None, stream=None):
        """o = the outputs, ST = the last state (S0: the first; either may be None)."""
        dk, dv = q.shape[-1], v.shape[-1]
        self._check((("q", q, dk), ("k", k, dk), ("v", v, dv), ("gk", gk, dk), ("o", o, dv)),
                    (("S0", S0), ("ST", ST)), q, v, gk, offsets)
        p = self.describe(q, v, gk, o, scale, k, offsets, longest)
        w, wp, wn = _scratch(workspace, gla_scan_workspace_bytes(p), q.device, stream)
        s = gla_scan_forward(self.g.h, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), gk.data_ptr(),
                             _ptr(S0), _ptr(ST), o.data_ptr(), wp, wn, _stream_of(q.device, stream))
        if s != GEMV_OK:
            raise GemvError(s, "gla_scan_forward")
        return o

    def backward(self, q, k, v, gk, dout, dq, dk, dv, dgk, scale, S0=None, dST=None, dS0=None,
                 offsets=None, longest=None, workspace=None, stream=None):
        """dq, dk, dv, dgk (and dS0) = the gradients of sum(o dout) + sum(ST dST)."""
        nk, nv = q.shape[-1], v.shape[-1]
        self._check((("q", q, nk), ("k", k, nk), ("v", v, nv), ("gk", gk, nk), ("dout", dout, nv),
                     ("dq", dq, nk), ("dk", dk, nk), ("dv", dv, nv), ("dgk", dgk, nk)),
                    (("S0", S0), ("dST", dST), ("dS0", dS0)), q, v, gk, offsets)
        p = self.describe(q, v, gk, dout, scale, k, offsets, longest)
        grad = gla_scan_grad_t(_strides(dq), _strides(dk), _strides(dv), _strides(dgk))
        w, wp, wn = _scratch(workspace, gla_scan_workspace_bytes(p, True), q.device, stream)
        s = gla_scan_backward(self.g.h, p, grad, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                              gk.data_ptr(), _ptr(S0), dout.data_ptr(), _ptr(dST), dq.data_ptr(),
                              dk.data_ptr(), dv.data_ptr(), dgk.data_ptr(), _ptr(dS0), wp, wn,
                              _stream_of(q.device, stream))
        if s != GEMV_OK:
            raise GemvError(s, "gla_scan_backward")
        return dq, dk, dv, dgk
