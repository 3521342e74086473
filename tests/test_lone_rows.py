"""A product or norm of one row, and a scan of one token, take it from anywhere:
its leading dimension or token stride is never used, so it is neither limited nor
chooses a kernel."""
import pytest
import torch

import memory_bound_dense_amd as mbd
import test_gemm
import test_gla_scan as tg
from memory_bound_dense_amd import _operators as ops
from test_operator_args import INVALID, OK, TOO_LARGE, at, bwd, fwd, gcheck, gemm, grads, ncheck, norm, scan

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def test_leading_dimensions_of_single_rows_are_not_limited():
    far = 1 << 40
    assert gcheck(gemm(m=1, lda=far, ldc=far)) == OK
    assert gcheck(gemm(m=1, lda=far, ldc=far, residual=at(5), ldr=far + 1)) == OK
    assert gcheck(gemm(m=1, residual=at(2), ldr=far)) == OK                     # in place
    assert gcheck(gemm(n=1, ldb=far)) == OK and gcheck(gemm(m=1, n=1, lda=far, ldb=far)) == OK
    for p in (gemm(m=2, lda=far), gemm(n=2, ldb=far), gemm(m=2, ldc=far)):
        assert gcheck(p) == TOO_LARGE
    assert gcheck(gemm(m=1, lda=63)) == INVALID and gcheck(gemm(n=1, ldb=63)) == INVALID
    # a row itself is still limited to 2^23 bytes
    k = (1 << 22) + 8
    assert gcheck(gemm(m=1, n=1, k=k, lda=k, ldb=k)) == TOO_LARGE
    r, s = at(3), at(4)
    assert ncheck(norm(m=1, ldx=far, ldres=far, ldsum=far, ldy=far), res=r, s=s) == OK
    assert ncheck(norm(m=1, ldsum=far), res=r, s=at(0)) == OK                   # in place
    assert ncheck(norm(m=2, ldx=far)) == TOO_LARGE and ncheck(norm(m=1, ldx=31)) == INVALID


def test_the_token_stride_of_one_token_is_not_limited():
    for packed in (False, True):
        for st in (0, 1 << 25, 1 << 40):
            p = scan(b=1 if packed else 2, t=1)
            for n in ("q", "k", "v", "gk", "o"):
                s = getattr(p, n)
                setattr(p, n, ops.gla_stride_t(s.batch, st, s.head))
            if packed:
                p.offsets, p.rows = at(15), 1
            assert fwd(p) == OK and bwd(p, grads(p)) == OK
            p.tokens = p.rows = 2
            assert fwd(p) == INVALID


@pytest.fixture(scope="module")
def h():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    g = mbd.Gemv()
    yield g
    g.close()


def alone(x, stride, shift=0):
    """A (1, n) view of the same values with that stride of its row."""
    room = torch.empty(x.shape[1] + shift, device="cuda").to(x.dtype)
    room[shift:] = x[0]
    return torch.as_strided(room, (1, x.shape[1]), (stride, 1), shift)


@pytest.mark.gpu
@pytest.mark.parametrize("a", [BF, HF, E4], ids=["bf16", "f16", "e4m3"])
def test_last_token_of_a_long_sequence(h, a):
    """hidden[:, -1] of 2048 tokens of width 4096, 2^23 elements apart."""
    hidden = torch.randn(1, 2048, 4096, device="cuda").to(a)
    x = hidden[:, -1]
    assert x.stride(0) == 1 << 23
    out = BF if a == E4 else a
    y = {n: None if t is None else t.cuda() for n, t in test_gemm.make(1, 1000, 4096, a, out, 1, True, True, False).items()}
    C, D = torch.empty(1, 1000, dtype=out, device="cuda"), torch.empty(1, 2048, 1000, dtype=out, device="cuda")[:, -1]
    gemm = mbd.Gemm(h)
    gemm(x.clone(), y["B"].contiguous(), C, bias=y["bias"], residual=y["residual"].contiguous(), act="silu")
    gemm(x, y["B"].contiguous(), D, bias=y["bias"], residual=alone(y["residual"], 1 << 33), act="silu")
    torch.cuda.synchronize()
    assert torch.equal(C, D)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("stride", [40, 41, 1 << 33])
def test_single_rows_of_any_stride(h, stride, shift):
    """One row of A, of B, of both: the bits of dense rows at the same alignment."""
    gemm, norm_ = mbd.Gemm(h), mbd.RmsNorm(h)
    for m, n in ((1, 30), (70, 1), (1, 1), (300, 1)):
        x = test_gemm.make(m, n, 40, BF, BF, 3, False, False, False)
        A, B = x["A"].contiguous().cuda(), x["B"].contiguous().cuda()
        got = []
        for st in (40, stride):
            C = torch.empty(m, n, dtype=BF, device="cuda")
            gemm(alone(A, st, shift) if m == 1 else A, alone(B, st, shift) if n == 1 else B, C)
            got.append(C)
        torch.cuda.synchronize()
        assert torch.equal(*got), (m, n)
    x, w = torch.randn(1, 40, device="cuda").to(BF), torch.ones(40, dtype=BF, device="cuda")
    got = []
    for st in (40, stride):
        y, s = (alone(torch.empty_like(x), st, shift) for _ in range(2))
        norm_(alone(x, st, shift), w, y, residual=alone(x, st, shift), sum_out=s)
        got.append(torch.cat([y, s]))
    torch.cuda.synchronize()
    assert torch.equal(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("stride", [1 << 25, 1 << 33])
def test_one_token_of_a_far_stride(h, stride):
    """The first token of (tokens, batch, ...) tensors whose tokens are far apart."""
    x = tg.cuda(tg.inputs(2, 1, 3, 64, 40, BF, BF, seed=2))
    sc = mbd.GlaScan(h)
    got = []
    for far in (False, True):
        like = lambda t: torch.as_strided(t, t.shape, (t.stride(0), stride, t.stride(2), 1)) if far else t
        o, ST, dS0 = torch.empty_like(x["v"]), torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
        r = [torch.empty_like(x[n]) for n in ("q", "k", "v", "g")]
        y = [like(x[n]) for n in ("q", "k", "v", "g", "do")]
        sc.forward(*y[:4], like(o), x["scale"], S0=x["S0"], ST=ST)
        sc.backward(*y, *[like(t) for t in r], x["scale"], S0=x["S0"], dST=x["dST"], dS0=dS0)
        got.append([o, ST, dS0] + r)
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
