"""The product's size limits on the host: what the checks accept has scratch and
a grid that are worked out without overflow (no handle, no GPU)."""
import pytest

from memory_bound_dense_amd import _operators as ops
from test_operator_args import INVALID, OK, TOO_LARGE, gemm

FAR = 1 << 56          # fake addresses, further apart than any tensor


def check(p, ws=4 * FAR, wn=1 << 62):
    return ops.gemm_check_args(p, FAR, 2 * FAR, 3 * FAR, ws, wn)


def rows(m, n, k, t):
    ld = (k + 15) // 16 * 16
    return gemm(m, n, k, in_type=t, dtype=1 if t == 2 else t, lda=ld, ldb=ld)


@pytest.mark.parametrize("m,n", [(1 << 30, 1 << 30), (1 << 30, (1 << 8) + 1), (1 << 20, 1 << 20), (5, 1 << 29),
                                 (64, (1 << 28) + 64), (1, 1 << 30)])
@pytest.mark.parametrize("k", [1, 4096])
def test_refused(m, n, k):
    p = rows(m, n, k, 1)
    assert check(p) == TOO_LARGE
    if m * n > 1 << 38:
        assert ops.gemm_workspace_bytes(p) == 0


@pytest.mark.parametrize("t", [0, 1, 2])
def test_scratch_is_what_it_says(t):
    """Sizes up to the limits: accepted with the scratch that is asked for, a float32 sum an
    output and split; without it refused where aligned rows need it."""
    asked = 0
    for m in (1, 40, 64, 65, 1000, 1 << 16, 1 << 22, 1 << 28, 1 << 30):
        for n in (1, 48, 1000, 1 << 16, 1 << 24, 1 << 28, 1 << 30):
            for k in (0, 1, 4096, 1 << 21):
                p = rows(m, n, k, t)
                need = ops.gemm_workspace_bytes(p)
                if m * n > 1 << 36 or (m <= 64 and n > 1 << 28):
                    assert check(p) in (OK, TOO_LARGE)
                    continue
                splits = 256 if m <= 64 else 8
                assert 0 <= need <= splits * 4 * m * (n + 15), (m, n, k)
                assert check(p, wn=need) == OK, (m, n, k)
                if need:
                    asked += check(p, wn=0) == INVALID
    assert asked > 10
