"""GPU: the root-mean-square norm with eps = 0: rows of zeros keep scale 0 and
codes 0, other rows and rows with a NaN are what they are."""
import pytest
import torch

import memory_bound_dense_amd as mbd
import test_rmsnorm
from test_rmsnorm import norm  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("n", [64, 333, 7168])
def test_rows_of_zeros(norm, n):  # noqa: F811
    x, _, w = test_rmsnorm.make(5, n, BF, False)
    x[1] = 0
    x[3] = 0
    x[3, n // 2] = float("nan")
    y, sc = torch.empty(5, n, device="cuda").to(E4), torch.empty(5, device="cuda")
    norm(x.cuda(), w.cuda(), y, eps=0.0, scales=sc)
    torch.cuda.synchronize()
    assert sc[1] == 0 and (y[1].float() == 0).all()
    assert torch.isnan(sc[3])
    rows = [0, 2, 4]
    _, z = test_rmsnorm.want(x[rows], None, w, 0.0)
    test_rmsnorm.check8(y.float()[rows], sc[rows], z, n)
