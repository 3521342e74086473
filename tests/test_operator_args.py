"""The operators' C entry points without a GPU: declared, exported, and every
bad argument refused with the documented status; the overlap rules; the
formulas of tests/scan_ref.py against differences."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import memory_bound_dense_amd as mbd
import scan_ref
from memory_bound_dense_amd import _lib
from memory_bound_dense_amd import _operators as ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = ["operators.h", "gla_scan.h", "gemm.h", "rmsnorm.h"]
OK, INVALID, DTYPE, MISALIGNED, ALIASING, TOO_LARGE = (
    _lib.GEMV_OK, _lib.GEMV_ERR_INVALID_ARG, _lib.GEMV_ERR_UNSUPPORTED_DTYPE, _lib.GEMV_ERR_MISALIGNED,
    _lib.GEMV_ERR_ALIASING, _lib.GEMV_ERR_TOO_LARGE)
G = 1 << 40          # fake device addresses, far apart: nothing is dereferenced


def at(i):
    return (i + 1) * G


def test_headers_and_library_agree_with_the_binding():
    names = set()
    for h in HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names |= set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**((?:operators|gla_scan|gemm|rmsnorm)_\w+)\s*\(", text,
                                flags=re.M))
    assert sorted(names) == sorted(ops.OPERATOR_EXPORTS)
    lib = ctypes.CDLL(ops.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_headers_compile_as_c(tmp_path):
    """The headers as C99, and every entry point linked from the library by a C program."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "use.c", str(tmp_path / "use")
    src.write_text("#include <stdio.h>\n#include \"operators.h\"\nint main(void) {\n  void* fns[] = {%s};\n"
                   "  gemm_t g = {0};\n  int n = 0;\n"
                   "  for (unsigned i = 0; i < sizeof(fns) / sizeof(fns[0]); ++i) n += fns[i] != NULL;\n"
                   "  printf(\"%%d %%d\", n, (int)gemm_check_args(&g, NULL, NULL, NULL, NULL, 0));\n  return 0;\n}\n"
                   % ", ".join("(void*)&" + n for n in ops.OPERATOR_EXPORTS))
    lib = os.path.dirname(ops.LIB_PATH)
    built = subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-isystem", "/opt/rocm/include", "-D__HIP_PLATFORM_AMD__",
                            "-I", os.path.join(ROOT, "include"), str(src), "-L", lib, "-lmbd_operators",
                            "-Wl,-rpath," + lib, "-o", exe], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert ran.stdout == "%d 0" % len(ops.OPERATOR_EXPORTS), ran.stderr


def test_null_handles():
    assert ops.operators_prepare(None) == _lib.GEMV_ERR_NULL_HANDLE
    p = scan()
    assert ops.gla_scan_forward(None, p, *[at(i) for i in range(7)]) == _lib.GEMV_ERR_NULL_HANDLE
    assert ops.gla_scan_backward(None, p, grads(p), *[at(i) for i in range(12)]) == _lib.GEMV_ERR_NULL_HANDLE
    assert ops.gemm_run(None, gemm(), at(0), at(1), at(2)) == _lib.GEMV_ERR_NULL_HANDLE
    assert ops.rmsnorm_run(None, norm(), at(0), None, at(1), None, at(2), None) == _lib.GEMV_ERR_NULL_HANDLE


# ---- scan ----------------------------------------------------------------------

def dense(b, t, h, d):
    return ops.gla_stride_t(t * h * d, h * d, d)


def scan(b=2, t=40, h=3, dk=16, dv=24, dtype=1, g32=0):
    return ops.gla_scan_t(b, t, h, dk, dv, dtype, g32, 0.5, dense(b, t, h, dk), dense(b, t, h, dk),
                          dense(b, t, h, dv), dense(b, t, h, dk), dense(b, t, h, dv), None, 0)


def grads(p):
    return ops.gla_scan_grad_t(p.q, p.k, p.v, p.gk)


def fwd(p, ptr=None, ws=None, wn=None, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), gk=at(3), S0=at(4), ST=at(5), o=at(6))
    a.update(kw)
    need = ops.gla_scan_workspace_bytes(p)
    return ops.gla_scan_check_args(p, a["q"], a["k"], a["v"], a["gk"], a["S0"], a["ST"], a["o"],
                                   at(20) if ws is None else ws, need if wn is None else wn)


def bwd(p, gr=None, ws=None, wn=None, **kw):
    names = ("q", "k", "v", "gk", "S0", "dout", "dST", "dq", "dk", "dv", "dgk", "dS0")
    a = {n: at(i) for i, n in enumerate(names)}
    a.update(kw)
    need = ops.gla_scan_workspace_bytes(p, True)
    return ops.gla_scan_grad_check_args(p, gr or grads(p), *[a[n] for n in names],
                                        at(20) if ws is None else ws, need if wn is None else wn)


def test_scan_accepts():
    for p in (scan(), scan(t=4000), scan(dtype=0, g32=1), scan(dk=256, dv=256), scan(1, 1, 1, 1, 1)):
        assert fwd(p) == OK and bwd(p) == OK
    assert fwd(scan(dv=65536)) == OK
    assert fwd(scan(), S0=None, ST=None) == OK
    assert bwd(scan(), S0=None, dST=None, dS0=None) == OK
    assert fwd(scan(), S0=at(5)) == OK                     # the state in place
    for zero in ("batch", "heads", "dk", "dv"):
        p = scan()
        setattr(p, zero, 0)
        assert fwd(p, q=None, k=None, v=None, gk=None, o=None) == OK
    p = scan(t=0)
    assert fwd(p, q=None, k=None, v=None, gk=None, o=None) == OK


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(gate_f32=2), DTYPE), (dict(batch=-1), INVALID),
    (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(dk=-1), INVALID), (dict(dv=-1), INVALID),
    (dict(dk=257), TOO_LARGE), (dict(dv=65537), TOO_LARGE), (dict(tokens=1 << 31), TOO_LARGE),
    (dict(batch=1 << 20, heads=2), TOO_LARGE)])
def test_scan_sizes_refused(change, status):
    p = scan()
    for n, x in change.items():
        setattr(p, n, x)
    assert fwd(p) == status and bwd(p) == status
    assert ops.gla_scan_workspace_bytes(p) == 0


def test_scan_backward_width():
    assert bwd(scan(dv=257)) == TOO_LARGE and fwd(scan(dv=257)) == OK


@pytest.mark.parametrize("name", ["q", "k", "v", "gk", "o"])
def test_scan_pointers_and_strides(name):
    assert fwd(scan(), **{name: None}) == INVALID
    assert fwd(scan(), **{name: at(9) + 1}) == MISALIGNED
    if name == "gk":
        assert fwd(scan(g32=1), gk=at(9) + 2) == MISALIGNED
    width = 24 if name in ("v", "o") else 16
    for st, status in ((0, INVALID), (width - 1, INVALID), (-width, INVALID), ((1 << 24) + 1, INVALID)):
        p = scan()
        s = getattr(p, name)
        setattr(p, name, ops.gla_stride_t(s.batch, st, s.head))
        assert fwd(p) == status, st
    for bad in (ops.gla_stride_t(-1, 100, 16), ops.gla_stride_t(0, 100, -16), ops.gla_stride_t(1 << 41, 100, 16)):
        p = scan()
        setattr(p, name, bad)
        assert fwd(p) == INVALID
    # a broadcast input is fine, a broadcast output is not
    p = scan()
    s = getattr(p, name)
    setattr(p, name, ops.gla_stride_t(0, s.token, 0))
    assert fwd(p) == (ALIASING if name == "o" else OK)


def test_scan_states_and_scratch():
    assert fwd(scan(), S0=at(4) + 2) == MISALIGNED and fwd(scan(), ST=at(4) + 2) == MISALIGNED
    assert bwd(scan(), dS0=at(4) + 2) == MISALIGNED and bwd(scan(), dST=at(4) + 1) == MISALIGNED
    p = scan(t=4000)
    need = ops.gla_scan_workspace_bytes(p)
    assert need > 0
    assert fwd(p, ws=0) == INVALID and fwd(p, wn=need - 1) == INVALID and fwd(p, ws=at(20) + 8) == MISALIGNED
    need = ops.gla_scan_workspace_bytes(p, True)
    assert bwd(p, ws=0) == INVALID and bwd(p, wn=need - 1) == INVALID and bwd(p, ws=at(20) + 4) == MISALIGNED
    # scratch on an input or output
    assert fwd(p, ws=at(6)) == ALIASING and bwd(p, ws=at(2) - 256) == ALIASING


def test_scan_overlaps():
    p = scan()
    for n in ("q", "k", "v", "gk"):
        assert fwd(p, o=at({"q": 0, "k": 1, "v": 2, "gk": 3}[n])) == ALIASING
        assert bwd(p, dq=at({"q": 0, "k": 1, "v": 2, "gk": 3}[n])) == ALIASING
    assert fwd(p, q=at(1)) == OK                            # inputs may share
    assert fwd(p, o=at(5)) == ALIASING                      # o in ST
    assert fwd(p, ST=at(4) + 4) == ALIASING                 # ST partly over S0
    assert bwd(p, dk=at(7)) == ALIASING                     # dq and dk
    assert bwd(p, dS0=at(6)) == ALIASING                    # dS0 over dST
    assert bwd(p, dS0=at(4)) == ALIASING                    # dS0 over S0


def fused(b, t, h, dk, dv):
    """Strides of q, k, v, g, o as slices of one (b, t, h, 3 dk + 2 dv) tensor, and their offsets."""
    w = 3 * dk + 2 * dv
    return ops.gla_stride_t(t * h * w, h * w, w), [2 * x for x in (0, dk, 2 * dk, 2 * dk + dv, 3 * dk + dv)]


def test_scan_fused_slices():
    p = scan()
    st, off = fused(2, 40, 3, 16, 24)
    for n in ("q", "k", "v", "gk", "o"):
        setattr(p, n, st)
    base = at(0)
    ptr = dict(q=base + off[0], k=base + off[1], v=base + off[2], gk=base + off[3], o=base + off[4])
    assert fwd(p, **ptr) == OK
    assert fwd(p, **dict(ptr, o=base + off[4] - 2)) == ALIASING       # one channel into g
    assert fwd(p, **dict(ptr, o=base + off[2])) == ALIASING
    # (b, t, 3, h, d): k behind q within a token; the output takes the third place
    w = 3 * 3 * 16
    q = scan(dv=16)
    for n in ("q", "k", "v", "gk", "o"):
        setattr(q, n, ops.gla_stride_t(40 * w, w, 16))
    assert fwd(q, q=base, k=base + 2 * 48, v=base, gk=base, o=base + 4 * 48) == OK
    assert fwd(q, q=base, k=base + 2 * 48, v=base, gk=base, o=base + 2 * 48) == ALIASING
    assert fwd(q, q=base, k=base + 2 * 48, v=base, gk=base, o=base + 4 * 48 - 2 * 16) == ALIASING


def test_scan_packed():
    p = scan(b=1)
    p.offsets, p.rows, p.batch, p.tokens = at(15), 100, 5, 40
    assert fwd(p) == OK and bwd(p) == OK
    p.offsets = at(15) + 2
    assert fwd(p) == MISALIGNED
    p.offsets, p.rows = at(15), -1
    assert fwd(p) == INVALID
    p.rows = 1 << 31
    assert fwd(p) == TOO_LARGE
    p.rows = 100
    assert fwd(p, o=at(15)) == ALIASING


# ---- product ---------------------------------------------------------------------

def gemm(m=40, n=50, k=64, **kw):
    p = ops.gemm_t(m, n, k, k, k, n, n, 1, 1, 0, 1.0)
    for name, x in kw.items():
        setattr(p, name, x)
    return p


def gcheck(p, A=at(0), B=at(1), C=at(2), ws=at(9), wn=None):
    return ops.gemm_check_args(p, A, B, C, ws, ops.gemm_workspace_bytes(p) if wn is None else wn)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(m=0), OK), (dict(n=0), OK), (dict(in_type=3), DTYPE), (dict(in_type=-1), DTYPE),
    (dict(dtype=2), DTYPE), (dict(in_type=0), DTYPE), (dict(in_type=2), OK), (dict(in_type=2, dtype=0), OK),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(m=-1), INVALID), (dict(n=-1), INVALID),
    (dict(k=-1), INVALID), (dict(lda=63), INVALID), (dict(ldb=63), INVALID), (dict(ldc=49), INVALID),
    (dict(residual=at(5), ldr=49), INVALID), (dict(ldr=0), OK), (dict(lda=(1 << 22) + 1), TOO_LARGE),
    (dict(ldb=1 << 23), TOO_LARGE), (dict(in_type=2, ldb=1 << 23), OK), (dict(ldc=(1 << 30) + 1), TOO_LARGE),
    (dict(m=(1 << 30) + 1), TOO_LARGE), (dict(bias=at(4) + 1), MISALIGNED),
    (dict(scale_a=at(4) + 2), MISALIGNED), (dict(scale_b=at(4) + 1), MISALIGNED),
    (dict(residual=at(4) + 1), MISALIGNED), (dict(bias=at(2)), ALIASING), (dict(scale_a=at(2) + 4), ALIASING),
    (dict(residual=at(2) + 2), ALIASING), (dict(residual=at(2)), OK), (dict(residual=at(2), ldr=51), ALIASING)])
def test_gemm_checks(kw, status):
    assert gcheck(gemm(**kw)) == status


def test_gemm_pointers():
    p = gemm()
    assert gcheck(p, A=None) == INVALID and gcheck(p, B=None) == INVALID and gcheck(p, C=None) == INVALID
    assert gcheck(gemm(k=0, lda=0, ldb=0), A=None, B=None) == OK
    assert gcheck(p, A=at(0) + 1) == MISALIGNED and gcheck(gemm(in_type=2), A=at(0) + 1) == OK
    assert gcheck(p, C=at(2) + 1) == MISALIGNED
    assert gcheck(p, C=at(0)) == ALIASING and gcheck(p, C=at(1) + 10) == ALIASING
    # C between the columns of a wider A
    assert gcheck(gemm(lda=200, ldc=200), C=at(0) + 2 * 64) in (OK, ALIASING)


def test_gemm_scratch():
    p = gemm(m=16, n=64, k=65536, lda=65536, ldb=65536)
    need = ops.gemm_workspace_bytes(p)
    assert need > 0 and gcheck(p) == OK
    assert gcheck(p, ws=0) == INVALID and gcheck(p, wn=need // 64) == INVALID
    assert gcheck(p, ws=at(9) + 8) == MISALIGNED
    assert gcheck(p, ws=at(1)) == ALIASING and gcheck(p, ws=at(2)) == ALIASING
    for m in (1, 16, 33, 64, 65, 300, 5000):
        for n in (1, 16, 1000, 70000):
            for k in (0, 1, 64, 5000):
                q = gemm(m, n, k)
                assert gcheck(q) == OK, (m, n, k)
    bad = gemm(lda=3)
    assert ops.gemm_workspace_bytes(bad) == 0


# ---- norm -------------------------------------------------------------------------

def norm(m=5, n=32, e4m3=0, **kw):
    p = ops.rmsnorm_t(m, n, n, n, n, n, 1, e4m3, 1e-6)
    for name, x in kw.items():
        setattr(p, name, x)
    return p


def ncheck(p, x=at(0), res=None, w=at(1), s=None, y=at(2), sc=None):
    return ops.rmsnorm_check_args(p, x, res, w, s, y, sc)


def test_norm_checks():
    p, q = norm(), norm(e4m3=1)
    r, s, sc = at(3), at(4), at(5)
    assert ncheck(p) == OK and ncheck(p, res=r) == OK and ncheck(p, res=r, s=s) == OK
    assert ncheck(q, sc=sc) == OK
    assert ncheck(norm(dtype=2)) == DTYPE and ncheck(norm(out_e4m3=2)) == DTYPE
    assert ncheck(norm(m=-1)) == INVALID and ncheck(norm(m=0), x=None, w=None, y=None) == OK
    assert ncheck(norm(n=-1)) == INVALID
    assert ncheck(norm(m=(1 << 21) + 1)) == TOO_LARGE and ncheck(norm(ldx=(1 << 30) + 1)) == TOO_LARGE
    assert ncheck(norm(n=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25)) == TOO_LARGE
    assert ncheck(norm(ldx=31)) == INVALID and ncheck(norm(ldy=31)) == INVALID
    assert ncheck(norm(ldres=31), res=r) == INVALID and ncheck(norm(ldsum=31), res=r, s=s) == INVALID
    for n in ("x", "w", "y"):
        assert ncheck(p, **{n: None}) == INVALID
        assert ncheck(p, **{n: at(7) + 1}) == MISALIGNED
    assert ncheck(q, sc=sc, y=at(7) + 1) == OK and ncheck(q, sc=sc + 2) == MISALIGNED
    assert ncheck(q) == INVALID and ncheck(p, sc=sc) == INVALID        # scales exactly with e4m3
    assert ncheck(p, s=s) == INVALID                                   # a sum without a residual
    assert ncheck(p, res=r, s=at(0)) == OK and ncheck(p, res=r, s=r) == OK and ncheck(p, y=at(0)) == OK
    assert ncheck(p, res=r, s=at(0), y=at(0)) == ALIASING
    assert ncheck(p, res=r, s=at(0) + 2) == ALIASING and ncheck(p, y=at(0) + 2) == ALIASING
    assert ncheck(p, res=r, y=r) == ALIASING and ncheck(p, y=at(1)) == ALIASING
    assert ncheck(q, y=at(0), sc=sc) == ALIASING and ncheck(q, sc=at(0)) == ALIASING
    assert ncheck(norm(ldsum=40), res=r, s=at(0)) == ALIASING          # in place needs the same rows


# ---- the binding --------------------------------------------------------------------

def test_binding_refuses_before_the_library():
    g = mbd.Gemv.__new__(mbd.Gemv)
    g.h, g.ws = None, None
    bf = torch.bfloat16
    q, v = torch.zeros(1, 4, 2, 8, dtype=bf), torch.zeros(1, 4, 2, 6, dtype=bf)

    def status(f):
        with pytest.raises(mbd.GemvError) as e:
            f()
        return e.value.status

    sc = mbd.GlaScan(g)
    assert status(lambda: sc.forward(q, q, v, q, v.clone(), 1.0)) == INVALID                 # on the CPU
    assert status(lambda: sc.forward(q[0], q, v, q, v, 1.0)) == INVALID
    assert status(lambda: sc.forward(q, q[..., :4], v, q, v, 1.0)) == INVALID
    assert status(lambda: sc.forward(q, q, v, q, v.half(), 1.0)) == DTYPE
    assert status(lambda: sc.forward(q, q, v, q.double(), v, 1.0)) == DTYPE
    assert status(lambda: sc.forward(q, q, v.transpose(1, 3), q, v, 1.0)) == INVALID
    S = torch.zeros(1, 2, 8, 6)
    assert status(lambda: sc.forward(q, q, v, q, v, 1.0, S0=S[:, :1])) == INVALID
    assert status(lambda: sc.forward(q, q, v, q, v, 1.0, ST=S.double())) == DTYPE
    off = torch.zeros(3, dtype=torch.int32)
    assert status(lambda: sc.forward(q, q, v, q, v, 1.0, S0=S, offsets=off)) == INVALID      # two sequences
    assert status(lambda: sc.forward(q, q, v, q, v, 1.0, offsets=off.long())) == INVALID
    assert status(lambda: sc.backward(q, q, v, q, v, q, q, v, q.float(), 1.0)) == DTYPE
    mm = mbd.Gemm(g)
    A, B, C = torch.zeros(3, 8, dtype=bf), torch.zeros(5, 8, dtype=bf), torch.zeros(3, 5, dtype=bf)
    assert status(lambda: mm(A, B, C)) == INVALID
    assert status(lambda: mm(A, B[:, :4], C)) == INVALID and status(lambda: mm(A, B, C.t())) == INVALID
    assert status(lambda: mm(A, B, C, act="swish")) == INVALID
    assert status(lambda: mm(A, B.half(), C)) == DTYPE and status(lambda: mm(A, B, C.half())) == DTYPE
    assert status(lambda: mm(A, B, C, bias=torch.zeros(4, dtype=bf))) == INVALID
    assert status(lambda: mm(A, B, C, scale_a=torch.zeros(3, dtype=bf))) == DTYPE
    assert status(lambda: mm(A.float(), B.float(), C.float())) == DTYPE
    nm = mbd.RmsNorm(g)
    w = torch.ones(8, dtype=bf)
    assert status(lambda: nm(A, w, torch.zeros_like(A))) == INVALID
    assert status(lambda: nm(A, w[:4], torch.zeros_like(A))) == INVALID
    assert status(lambda: nm(A, w.float(), torch.zeros_like(A))) == DTYPE
    assert status(lambda: nm(A, w, torch.zeros_like(A).half())) == DTYPE
    assert status(lambda: nm(A[0], w, A)) == INVALID


def test_structs_have_the_headers_layout():
    """Field order and sizes of the binding's structs against the headers' text."""
    c = {"int64_t": 8, "int32_t": 4, "gemv_dtype_t": 4, "float": 4, "const float*": 8, "const void*": 8,
         "const int32_t*": 8, "gla_stride_t": 24}
    for header, name, cls in (("gla_scan.h", "gla_scan_t", ops.gla_scan_t),
                              ("gla_scan.h", "gla_scan_grad_t", ops.gla_scan_grad_t),
                              ("gemm.h", "gemm_t", ops.gemm_t), ("rmsnorm.h", "rmsnorm_t", ops.rmsnorm_t)):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
        body = re.search(r"typedef struct \{([^}]*)\}\s*%s;" % name, text).group(1)
        fields = []
        for line in body.split(";"):
            m = re.match(r"\s*((?:const )?\w+\*?)\s+(.*)", line.strip(), flags=re.S)
            if m:
                fields += [(f.strip(), c[m.group(1)]) for f in m.group(2).split(",")]
        got = [(f[0], ctypes.sizeof(f[1])) for f in cls._fields_]
        assert got == fields, name


# ---- the reference's gradients against differences -----------------------------------

def test_reference_gradients_against_differences():
    rng = np.random.default_rng(3)
    t, h, dk, dv, scale = 7, 2, 3, 4, 0.7
    x = {n: rng.standard_normal((t, h, d)) for n, d in (("q", dk), ("k", dk), ("v", dv))}
    x["g"] = -rng.random((t, h, dk))
    S0, do, dST = rng.standard_normal((h, dk, dv)), rng.standard_normal((t, h, dv)), rng.standard_normal((h, dk, dv))

    def loss(x, S0):
        o, ST, _, _ = scan_ref.forward(x["q"], x["k"], x["v"], x["g"], scale, S0)
        return (o * do).sum() + (ST * dST).sum()

    got, _ = scan_ref.backward(x["q"], x["k"], x["v"], x["g"], do, scale, S0, dST)
    e = 1e-5
    for name in ("q", "k", "v", "g", "S0"):
        base = S0 if name == "S0" else x[name]
        for _ in range(12):
            i = tuple(rng.integers(0, s) for s in base.shape)
            up, dn = base.copy(), base.copy()
            up[i] += e
            dn[i] -= e
            f = (lambda b: loss(x, b)) if name == "S0" else (lambda b: loss(dict(x, **{name: b}), S0))
            diff = (f(up) - f(dn)) / (2 * e)
            # central differences: e^2 / 6 times a third derivative of order 10, and 1e-16 / e of rounding
            assert abs(diff - got["d" + name][i]) < 1e-8 * (1 + abs(diff)), (name, i)
