"""GPU: root-mean-square norm with residual addition (include/rmsnorm.h)
against float64.

s is one rounding of an exact sum of two 16-bit values (their fp32 sum rounds
once more only where it is inexact in 24 bits, which can move s by one unit in
a tie: compared with the same two roundings).  y: the sum of squares of n terms
passes through at most n / 512 + 24 roundings per term in the widest form, the
root halves that; products, division and root add 8: |y - y64| <= (n / 512 + 40)
u |y| before the one rounding to 16 bits (eps / 2) or, in 8 bits, to a step of
e4m3: 2^-4 relative, 2^-10 scale absolute below its normal range (2^-6)."""
import pytest
import torch

import memory_bound_dense_amd as mbd

pytestmark = pytest.mark.gpu
BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module")
def norm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    g = mbd.Gemv()
    yield mbd.RmsNorm(g)
    g.close()


def make(m, n, dt, residual, seed=0):
    gen = torch.Generator().manual_seed(seed + n)
    x = torch.randn(m, n, generator=gen).mul(2).to(dt)
    r = torch.randn(m, n, generator=gen).mul(4).to(dt) if residual else None
    w = (1 + 0.2 * torch.randn(n, generator=gen)).to(dt)
    return x, r, w


def want(x, r, w, eps):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    d = s.double()
    return s, d / torch.sqrt((d * d).mean(1, keepdim=True) + eps) * w.double()


def check16(y, z, n):
    got = y.double().cpu()
    f = torch.finfo(y.dtype)
    e = (n / 512 + 40) * U * z.abs()
    assert ((got - z).abs() <= e + f.eps / 2 * (z.abs() + e) + f.smallest_normal * f.eps / 2).all()


def check8(y, scales, z, n):
    sc = z.abs().amax(1) / 448
    got_s = scales.double().cpu()
    assert ((got_s - sc).abs() <= (n / 512 + 40) * U * sc).all()
    got = y.float().double().cpu() * sc[:, None]
    e = (n / 512 + 40) * U * z.abs()
    assert ((got - z).abs() <= e + torch.maximum(2.0 ** -4 * z.abs(), 2.0 ** -10 * sc[:, None]) * (1 + 1e-6)).all()


SIZES = [(1, 1), (3, 7), (2, 8), (5, 512), (4, 520), (7, 1024), (3, 2048), (2, 4096), (3, 7168), (2, 7169),
         (2, 16384), (2, 32768), (1, 40000)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
def test_matches(norm, m, n, dt, residual):
    x, r, w = make(m, n, dt, residual)
    s, z = want(x, r, w, 1e-6)
    xd, wd, rd = x.cuda(), w.cuda(), None if r is None else r.cuda()
    for e4m3 in (False, True):
        y = torch.full((m, n), float("nan"), device="cuda").to(E4 if e4m3 else dt)
        sc = torch.full((m,), float("nan"), device="cuda") if e4m3 else None
        so = torch.full((m, n), float("nan"), dtype=dt, device="cuda") if residual else None
        norm(xd, wd, y, eps=1e-6, residual=rd, sum_out=so, scales=sc)
        torch.cuda.synchronize()
        if residual:
            assert torch.equal(so.cpu(), s)
        if e4m3:
            check8(y, sc, z, n)
        else:
            check16(y, z, n)


@pytest.mark.parametrize("n", [64, 333, 7168])
def test_in_place_and_strided(norm, n):
    """sum_out = x, sum_out = residual and y = x give the same bits as separate
    tensors; rows of a wider tensor, and what lies beside them stays."""
    m = 5
    x, r, w = (t.cuda() for t in make(m, n, BF, True))
    y0, s0 = torch.empty_like(x), torch.empty_like(x)
    norm(x, w, y0, residual=r, sum_out=s0)
    for which in ("x", "residual"):
        a, b, y = x.clone(), r.clone(), torch.empty_like(x)
        norm(a, w, y, residual=b, sum_out=a if which == "x" else b)
        assert torch.equal(y, y0) and torch.equal(a if which == "x" else b, s0)
    a, s = x.clone(), torch.empty_like(x)
    norm(a, w, a, residual=r, sum_out=s)
    assert torch.equal(a, y0) and torch.equal(s, s0)
    a = x.clone()
    norm(a, w, a, residual=r)
    assert torch.equal(a, y0)
    wide = torch.full((m, n + 24), 7.0, dtype=BF, device="cuda")
    wide[:, 8:n + 8] = x
    big = torch.full((m, n + 24), 5.0, dtype=BF, device="cuda")
    norm(wide[:, 8:n + 8], w, big[:, 16:n + 16], residual=r)
    torch.cuda.synchronize()
    assert torch.equal(big[:, 16:n + 16], y0)
    assert (big[:, :16] == 5).all() and (big[:, n + 16:] == 5).all()


@pytest.mark.parametrize("n", [64, 333])
def test_zero_and_special_rows(norm, n):
    x = torch.randn(6, n).to(BF)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 3] = float("inf")
    w = torch.ones(n, dtype=BF)
    y, sc = torch.empty(6, n, device="cuda").to(E4), torch.empty(6, device="cuda")
    norm(x.cuda(), w.cuda(), y, scales=sc)
    y16 = torch.empty(6, n, dtype=BF, device="cuda")
    norm(x.cuda(), w.cuda(), y16)
    torch.cuda.synchronize()
    back = (y.float() * sc[:, None]).cpu()
    assert (back[0] == 0).all() and (y16[0] == 0).all() and sc[0] == 0
    assert torch.isnan(back[1]).all() and torch.isnan(y16[1]).all()
    for b in (back[2], y16[2].float().cpu()):
        assert torch.isnan(b[3]) and (b[torch.arange(n) != 3] == 0).all()
    s, z = want(x[3:], None, w, 1e-6)
    check8(y[3:], sc[3:], z, n)


@pytest.mark.parametrize("n", [64, 333])
def test_tiny_rows(norm, n):
    """s w near 2^-124: 448 over the row's largest is beyond float32."""
    gen = torch.Generator().manual_seed(n)
    x, w = torch.randn(3, n, generator=gen).mul(2.0 ** -60).to(BF), torch.full((n,), 2.0 ** -64, dtype=BF)
    x[:, ::5] = 0
    _, z = want(x, None, w, 1e-6)
    y, sc = torch.empty(3, n, device="cuda").to(E4), torch.empty(3, device="cuda")
    norm(x.cuda(), w.cuda(), y, scales=sc)
    torch.cuda.synchronize()
    check8(y, sc, z, n)


def test_empty(norm):
    w = torch.empty(0, dtype=BF, device="cuda")
    norm(torch.empty(3, 0, dtype=BF, device="cuda"), w, torch.empty(3, 0, dtype=BF, device="cuda"))
    w = torch.ones(8, dtype=BF, device="cuda")
    norm(torch.empty(0, 8, dtype=BF, device="cuda"), w, torch.empty(0, 8, dtype=BF, device="cuda"))
