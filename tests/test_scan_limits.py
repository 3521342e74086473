"""The scan's checks refuse what its launches cannot take (no handle, no GPU)."""
from test_operator_args import OK, TOO_LARGE, bwd, fwd, scan


def test_workgroups_of_the_outputs():
    for dv, status in ((1024, OK), (1025, TOO_LARGE), (65536, TOO_LARGE)):
        assert fwd(scan(b=1 << 10, t=1, h=1 << 10, dk=1, dv=dv), S0=None, ST=None) == status
    assert fwd(scan(b=16, t=1, h=1 << 10, dk=1, dv=65536), S0=None, ST=None) == OK
    assert bwd(scan(b=1 << 10, t=1, h=1 << 10, dk=256, dv=256), S0=None, dST=None, dS0=None) == OK
