"""ctypes binding of libmbd_operators.so, the operators around the GEMV
(include/operators.h, gla_scan.h, gemm.h, rmsnorm.h).

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
import os

from ._lib import (GEMV_ERR_INVALID_ARG, GEMV_ERR_UNSUPPORTED_DTYPE, GEMV_ERR_WRONG_DEVICE, GEMV_OK,
                   Gemv, GemvError, _check_devices, _dtype_code)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmbd_operators.so")

# every symbol these headers declare
OPERATOR_EXPORTS = ("operators_prepare", "gla_scan_workspace_bytes", "gla_scan_forward", "gla_scan_backward",
                    "gla_scan_check_args", "gla_scan_grad_check_args", "gemm_workspace_bytes",
                    "gemm_run", "gemm_plan_config", "gemm_check_args", "rmsnorm_run", "rmsnorm_check_args")

GEMM_F16, GEMM_BF16, GEMM_E4M3 = 0, 1, 2
GEMM_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

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


class gemm_t(ctypes.Structure):
    _fields_ = [("m", _i64), ("n", _i64), ("k", _i64), ("lda", _i64), ("ldb", _i64), ("ldc", _i64),
                ("ldr", _i64), ("in_type", _i32), ("dtype", _st), ("act", _i32), ("alpha", _f32),
                ("scale_a", _vp), ("scale_b", _vp), ("bias", _vp), ("residual", _vp)]


class gemm_config_t(ctypes.Structure):
    _fields_ = [("rows", _i32), ("tokens", _i32), ("kind", _i32), ("splits", _i32)]


class rmsnorm_t(ctypes.Structure):
    _fields_ = [("m", _i64), ("n", _i64), ("ldx", _i64), ("ldres", _i64), ("ldsum", _i64),
                ("ldy", _i64), ("dtype", _st), ("out_e4m3", _i32), ("eps", _f32)]


_ready = None


def load():
    """Load libmbd_operators.so (raises if it was not built)."""
    global _ready
    if _ready is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmbd_operators.so is not built (%s); run "
                               "`python -m memory_bound_dense_amd.build_operators`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        lib.operators_prepare.argtypes = [_vp]
        scan, grad = ctypes.POINTER(gla_scan_t), ctypes.POINTER(gla_scan_grad_t)
        lib.gla_scan_workspace_bytes.argtypes = [scan, _i32]
        lib.gla_scan_workspace_bytes.restype = _sz
        lib.gla_scan_forward.argtypes = [_vp, scan] + [_vp] * 7 + [_vp, _sz, _vp]
        lib.gla_scan_check_args.argtypes = [scan] + [_vp] * 7 + [_vp, _sz]
        lib.gla_scan_backward.argtypes = [_vp, scan, grad] + [_vp] * 12 + [_vp, _sz, _vp]
        lib.gla_scan_grad_check_args.argtypes = [scan, grad] + [_vp] * 12 + [_vp, _sz]
        gemm, norm = ctypes.POINTER(gemm_t), ctypes.POINTER(rmsnorm_t)
        lib.gemm_workspace_bytes.argtypes = [gemm]
        lib.gemm_workspace_bytes.restype = _sz
        lib.gemm_run.argtypes = [_vp, gemm, _vp, _vp, _vp, _vp, _sz, _vp]
        lib.gemm_plan_config.argtypes = [gemm, _vp, _vp, ctypes.POINTER(gemm_config_t)]
        lib.gemm_check_args.argtypes = [gemm, _vp, _vp, _vp, _vp, _sz]
        lib.rmsnorm_run.argtypes = [_vp, norm] + [_vp] * 7
        lib.rmsnorm_check_args.argtypes = [norm] + [_vp] * 6
        for name in OPERATOR_EXPORTS:
            if not name.endswith("_bytes"):
                getattr(lib, name).restype = _st
        _ready = lib
    return _ready


# ---- the C entry points, same names ------------------------------------------

def operators_prepare(h):
    """Set the kernels up on the handle's device now (the first call otherwise does)."""
    return load().operators_prepare(h)


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


def gemm_workspace_bytes(p):
    return load().gemm_workspace_bytes(ctypes.byref(p))


def gemm_run(h, p, A, B, C, workspace=None, workspace_bytes=0, stream=None):
    return load().gemm_run(h, ctypes.byref(p), A, B, C, workspace, workspace_bytes, stream)


def gemm_plan_config(p, A=None, B=None):
    """What gemm_run picks for a call, on the host alone (no device); A and B: addresses."""
    cfg = gemm_config_t()
    s = load().gemm_plan_config(ctypes.byref(p), A, B, ctypes.byref(cfg))
    return s, cfg


def gemm_check_args(p, A, B, C, workspace=None, workspace_bytes=0):
    return load().gemm_check_args(ctypes.byref(p), A, B, C, workspace, workspace_bytes)


def rmsnorm_run(h, p, x, residual, w, sum_out, y, scales, stream=None):
    return load().rmsnorm_run(h, ctypes.byref(p), x, residual, w, sum_out, y, scales, stream)


def rmsnorm_check_args(p, x, residual, w, sum_out, y, scales):
    return load().rmsnorm_check_args(ctypes.byref(p), x, residual, w, sum_out, y, scales)


# ---- torch tensors -------------------------------------------------------------

def _handle(gemv):
    """The Gemv whose handle an operator uses, with the operators set up on its device if that
    is the current one (else the first call does it)."""
    g = gemv if gemv is not None else Gemv()
    if g.h is not None:
        s = operators_prepare(g.h)
        if s not in (GEMV_OK, GEMV_ERR_WRONG_DEVICE):
            raise GemvError(s, "operators_prepare")
    return g


def _bad(what):
    return GemvError(GEMV_ERR_INVALID_ARG, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_of(device, stream):
    """The stream's address: the given one, else torch's current one on the device (by torch's
    own short way to it where there is one: 0.1 us instead of 2)."""
    if stream is not None:
        return stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream


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
        self.g = _handle(gemv)

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
            if x.shape != (b, t, h, d) or (d > 1 and x.stride(3) != 1):
                raise _bad("%s %s, strides %s" % (name, tuple(x.shape), x.stride()))
        nseq = b
        if offsets is not None:
            if b != 1 or offsets.dim() != 1 or offsets.numel() < 1 or offsets.dtype != torch.int32 or \
                    not offsets.is_contiguous():
                raise _bad("offsets must be dense int32 (n + 1), with b == 1")
            nseq = offsets.numel() - 1
        for name, S in states:
            if S is not None and (S.shape != (nseq, h, dk, dv) or not S.is_contiguous()):
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


def _rows(name, t, m, n, dtypes):
    """Leading dimension of an (m, n) tensor with dense rows."""
    st = t.stride()
    if t.shape != (m, n) or (n > 1 and st[1] != 1):
        raise _bad("%s %s, strides %s: want dense rows (%d, %d)" % (name, tuple(t.shape), st, m, n))
    if t.dtype not in dtypes:
        raise GemvError(GEMV_ERR_UNSUPPORTED_DTYPE, "%s is %s" % (name, t.dtype))
    return st[0] if m > 1 else max(st[0], n)


def _vector(name, t, n, dtype):
    if t is None:
        return None
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise _bad("%s must be a dense (%d,) tensor" % (name, n))
    if t.dtype != dtype:
        raise GemvError(GEMV_ERR_UNSUPPORTED_DTYPE, "%s is %s" % (name, t.dtype))
    return t.data_ptr()


class Gemm:
    """C = act(alpha * scale_a[:, None] * scale_b * (A @ B.T) + bias) + residual
    (include/gemm.h), through a Gemv handle.  A: (m, k) tokens, B: (n, k)
    weights, both float16, bfloat16 or float8_e4m3fn; C, residual (m, n) and
    bias (n,) of A's dtype (either 16-bit dtype with float8_e4m3fn); scales
    float32.  residual may be C."""

    def __init__(self, gemv=None):
        self.g = _handle(gemv)

    def __call__(self, A, B, C, bias=None, residual=None, act="none", alpha=1.0, scale_a=None,
                 scale_b=None, workspace=None, stream=None):
        import torch
        if A.dim() != 2 or B.dim() != 2:
            raise _bad("A and B must be 2-D")
        if act not in GEMM_ACTS:
            raise _bad("act %r: one of %s" % (act, ", ".join(GEMM_ACTS)))
        (m, k), n = A.shape, B.shape[0]
        e4m3 = A.dtype == torch.float8_e4m3fn
        lda, ldb = _rows("A", A, m, k, (A.dtype,)), _rows("B", B, n, k, (A.dtype,))
        ldc = _rows("C", C, m, n, (torch.float16, torch.bfloat16) if e4m3 else (A.dtype,))
        p = gemm_t(m, n, k, lda, ldb, ldc, 0, GEMM_E4M3 if e4m3 else _dtype_code(A), _dtype_code(C),
                   GEMM_ACTS[act], float(alpha), _vector("scale_a", scale_a, m, torch.float32),
                   _vector("scale_b", scale_b, n, torch.float32), _vector("bias", bias, n, C.dtype))
        if residual is not None:
            p.ldr, p.residual = _rows("residual", residual, m, n, (C.dtype,)), residual.data_ptr()
        _check_devices((B, C, bias, residual, scale_a, scale_b), A.device)
        _on_current(A.device)
        w, wp, wn = _scratch(workspace, gemm_workspace_bytes(p), A.device, stream)
        s = gemm_run(self.g.h, p, A.data_ptr(), B.data_ptr(), C.data_ptr(), wp, wn,
                     _stream_of(A.device, stream))
        if s != GEMV_OK:
            raise GemvError(s, "gemm_run")
        return C


class RmsNorm:
    """Root-mean-square norm over rows (include/rmsnorm.h), through a Gemv
    handle: s = x + residual (stored in sum_out if given), y = s *
    rsqrt(mean(s^2) + eps) * w.  y of x's dtype, or float8_e4m3fn with float32
    ``scales`` (m,)."""

    def __init__(self, gemv=None):
        self.g = _handle(gemv)

    def __call__(self, x, w, y, eps=1e-6, residual=None, sum_out=None, scales=None, stream=None):
        import torch
        if x.dim() != 2:
            raise _bad("x must be 2-D")
        m, n = x.shape
        e4m3 = y.dtype == torch.float8_e4m3fn
        p = rmsnorm_t(m, n, _rows("x", x, m, n, (x.dtype,)), 0, 0,
                      _rows("y", y, m, n, (x.dtype, torch.float8_e4m3fn)), _dtype_code(x), int(e4m3),
                      float(eps))
        if residual is not None:
            p.ldres = _rows("residual", residual, m, n, (x.dtype,))
        if sum_out is not None:
            p.ldsum = _rows("sum_out", sum_out, m, n, (x.dtype,))
        wp, sp = _vector("w", w, n, x.dtype), _vector("scales", scales, m, torch.float32)
        _check_devices((w, y, residual, sum_out, scales), x.device)
        _on_current(x.device)
        s = rmsnorm_run(self.g.h, p, x.data_ptr(), _ptr(residual), wp, _ptr(sum_out), y.data_ptr(),
                        sp, _stream_of(x.device, stream))
        if s != GEMV_OK:
            raise GemvError(s, "rmsnorm_run")
        return y
