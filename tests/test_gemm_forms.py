"""Every form of the product: sizes that the plan gives to each tile and type,
with k in one piece and split, of whole slabs (128 bytes) and not, and to each
number of rows and tokens of the few-token kernel.  The plan is asked, so a new
cost in it that leaves a form without a size here fails on the CPU."""
import pytest
import torch

import memory_bound_dense_amd as mbd
import test_gemm
from memory_bound_dense_amd import _operators as ops
from test_operator_args import gemm

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(0, HF), (1, BF), (2, E4)]
TIDS = ["f16", "bf16", "e4m3"]

# rows of A and B on 16-byte boundaries or not; kind, rows, tokens; m, n, slabs; whether k is split
FORMS = [
    (True, 1, 64, 64, 65, 64, 5, False), (True, 1, 64, 64, 130, 100, 64, True),
    (True, 1, 64, 128, 200, 14000, 5, False), (True, 1, 64, 128, 65, 4096, 128, True),
    (True, 2, 128, 128, 520, 14000, 1, False), (True, 2, 128, 128, 520, 14000, 6, False),
    (True, 2, 128, 128, 4096, 300, 128, True),
    (True, 2, 256, 128, 260, 14000, 1, False), (True, 2, 256, 128, 260, 14000, 2, False),
    (True, 2, 256, 128, 260, 14000, 3, False), (True, 2, 256, 128, 260, 14000, 6, False),
    (True, 2, 256, 128, 65, 11008, 64, True),
    (True, 2, 256, 256, 2500, 5000, 1, False), (True, 2, 256, 256, 2500, 5000, 5, False),
    (True, 2, 256, 256, 130, 11008, 128, True),
    (False, 1, 64, 64, 65, 64, 5, False), (False, 1, 64, 64, 130, 100, 64, True),
    (False, 1, 64, 128, 200, 14000, 5, False), (False, 1, 64, 128, 65, 6000, 32, True),
    (False, 1, 128, 128, 260, 14000, 3, False), (False, 1, 128, 128, 65, 11008, 64, True),
    (False, 1, 256, 256, 2500, 5000, 5, False), (False, 1, 256, 256, 130, 11008, 64, True)]
# rows, tokens: m, n
FEW = [(rows, tokens, tokens - 7, n) for tokens in (16, 32, 64) for rows, n in ((16, 100), (32, 4100), (48, 8203), (64, 12300))]


def depth(t, slabs, tail):
    """k of so many slabs; with a tail the last one is cut within a 16-byte piece."""
    return slabs * 128 // (1 if t == 2 else 2) - (5 if tail else 0)


def strides(t, whole, k):
    """A leading dimension on 16-byte boundaries, or off them."""
    return (k + 15) // 16 * 16 if whole else (k + 15) // 16 * 16 + (3 if t == 2 else 1)


def plan(t, m, n, k, ld):
    return ops.gemm_plan_config(gemm(m, n, k, in_type=t, dtype=1 if t == 2 else t, lda=ld, ldb=ld), 0, 0)


@pytest.mark.parametrize("t", [0, 1, 2], ids=TIDS)
@pytest.mark.parametrize("tail", [False, True], ids=["whole", "tail"])
def test_the_sizes_take_their_forms(t, tail):
    seen = set()
    for whole, kind, rows, tokens, m, n, slabs, split in FORMS:
        k = depth(t, slabs, tail)
        s, c = plan(t, m, n, k, strides(t, whole, k))
        assert s == mbd.GEMV_OK and (c.kind, c.rows, c.tokens, c.splits > 1) == (kind, rows, tokens, split), (m, n, k)
        seen.add((whole, kind, rows, tokens, split))
    assert len(seen) == 18
    for rows, tokens, m, n in FEW:
        s, c = plan(t, m, n, depth(t, 9, tail), 8192)
        assert s == mbd.GEMV_OK and (c.kind, c.rows, c.tokens, c.splits) == (0, rows, tokens, 1)
        s, c = plan(t, m, 100, depth(t, 300, tail), 1 << 20)
        assert (c.kind, c.rows, c.tokens) == (0, 16, tokens) and c.splits > 1


def test_plan_refusals():
    cfg = ops.gemm_config_t()
    lib = ops.load()
    assert lib.gemm_plan_config(None, None, None, cfg) == ops.GEMV_ERR_INVALID_ARG
    assert lib.gemm_plan_config(gemm(), None, None, None) == ops.GEMV_ERR_INVALID_ARG
    assert ops.gemm_plan_config(gemm(lda=3))[0] == ops.GEMV_ERR_INVALID_ARG
    s, c = ops.gemm_plan_config(gemm(m=0))
    assert s == mbd.GEMV_OK and (c.rows, c.tokens, c.kind, c.splits) == (0, 0, 0, 0)


@pytest.fixture(scope="module")
def h():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    g = mbd.Gemv()
    yield g
    g.close()


def rows_in(x, ld):
    """The same rows in a wider tensor whose other columns are NaN."""
    wide = torch.full((x.shape[0], ld), float("nan"), device=x.device).to(x.dtype)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def check(h, t, dt, m, n, k, ld):
    """Integers, whose sums are exact, over the whole output; random values against float64 in 24 rows
    and 200 columns."""
    mm = mbd.Gemm(h)
    out = BF if dt == E4 else dt
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    A = torch.randint(-3, 4, (m, k), generator=gen, device="cuda").float()
    B = torch.randint(-1, 2, (n, k), generator=gen, device="cuda").float()
    C = torch.full((m, n), float("nan"), dtype=out, device="cuda")
    mm(rows_in(A.to(dt), ld), rows_in(B.to(dt), ld), C)
    want = A @ B.t().contiguous()       # below 2^24: exact in float32, whatever the order
    assert torch.equal(C, want.to(out))
    A = torch.randn(m, k, generator=gen, device="cuda").to(dt)
    B = torch.randn(n, k, generator=gen, device="cuda").mul((4.0 if dt == E4 else 1.0) / k ** 0.5).to(dt)
    bias, res = torch.randn(n, generator=gen, device="cuda").to(out), torch.randn(m, n, generator=gen, device="cuda").to(out)
    sa, sb = (torch.rand(i, generator=gen, device="cuda") + 0.1 for i in (m, n))
    mm(rows_in(A, ld), rows_in(B, ld), C, bias=bias, residual=res, act="gelu", alpha=0.5, scale_a=sa, scale_b=sb)
    torch.cuda.synchronize()
    cpu = torch.Generator().manual_seed(n)
    i = torch.cat([torch.randint(m, (22,), generator=cpu), torch.tensor([0, m - 1])])
    j = torch.cat([torch.randint(n, (198,), generator=cpu), torch.tensor([0, n - 1])])
    A, B, bias, res, sa, sb = (x.cpu() for x in (A, B, bias, res, sa, sb))
    x = dict(A=A[i], B=B[j], bias=bias[j], residual=res[i][:, j], sa=sa[i], sb=sb[j])
    z, err = test_gemm.want(x, "gelu", 0.5)
    test_gemm.check(C.cpu()[i][:, j], z, err)
    assert torch.isfinite(C).all()


@pytest.mark.gpu
@pytest.mark.parametrize("t,dt", TYPES, ids=TIDS)
@pytest.mark.parametrize("tail", [False, True], ids=["whole", "tail"])
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "%s_%d_%dx%d_%d%s" % (
    "aligned" if f[0] else "any", f[1], f[2], f[3], f[6], "_split" if f[7] else ""))
def test_every_form(h, form, tail, t, dt):
    whole, _, _, _, m, n, slabs, _ = form
    k = depth(t, slabs, tail)
    check(h, t, dt, m, n, k, strides(t, whole, k))


@pytest.mark.gpu
@pytest.mark.parametrize("t,dt", TYPES, ids=TIDS)
@pytest.mark.parametrize("rows,tokens,m,n", FEW)
def test_every_form_of_few_tokens(h, rows, tokens, m, n, t, dt):
    for tail in (False, True):
        k = depth(t, 9, tail)
        check(h, t, dt, m, n, k, strides(t, False, k))
        check(h, t, dt, m, n, k, (k + 127) // 128 * 128)
    k = depth(t, 300, True)
    check(h, t, dt, m, 100, k, strides(t, False, k))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(16, 300, 4096), (64, 100, 9000), (300, 1000, 2048), (2048, 4096, 328)])
def test_bits_go_by_sizes_and_alignment_alone(h, m, n, k):
    """Rows on 16-byte boundaries at any leading dimension, and rows off them at any: the same bits
    each; up to 64 tokens all the same."""
    mm = mbd.Gemm(h)
    A, B = (torch.randn(r, k, generator=torch.Generator().manual_seed(r)).to(BF).cuda() for r in (m, n))
    got = []
    for ld in (k, k + 8, k + 200, k + 1, k + 6):
        C = torch.empty(m, n, dtype=BF, device="cuda")
        mm(rows_in(A, ld), rows_in(B, ld), C)
        got.append(C)
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2]) and torch.equal(got[3], got[4])
    if m <= 64:
        assert torch.equal(got[0], got[3])
