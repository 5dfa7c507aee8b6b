"""Shapes at the limits of include/mcc1d_ssm.h, by their workspace sizes (no GPU
needed)."""
import pytest

import test_ssm_abi_host as abi
from test_ssm_abi_host import OK, SHAPE, lib, scan_args, scan_bwd_args, size  # noqa: F401


def grouped(S, B, G, N, **kw):
    return scan_args(S=S, B=B, H=G, G=G, N=N, B_strides=(B * G * N, G * N, N), C_strides=(B * G * N, G * N, N),
                     u_strides=(B * G, G), delta_strides=(B * G, G), **kw)


@pytest.mark.parametrize("S,B,G,N", [(1 << 20, 1, 4096, 1), (1 << 20, 1, 4096, 64), (1 << 26, 1, 64, 16), (1 << 16, 64, 1024, 16)])
def test_many_group_rows_are_the_backwards_limit_only(S, B, G, N):
    """S B G = 2^32: each row of B and C is an input like any other to the forward."""
    assert size("scan", grouped(S, B, G, N))[0] == OK
    padded = 4
    while padded < N:
        padded *= 2
    st = size("scan_bwd", scan_bwd_args(grouped(S, B, G, N, y=None)))[0]
    assert st == (OK if S * B * G * padded < 1 << 37 else SHAPE)


def test_the_smallest_refused():
    assert size("scan_bwd", scan_bwd_args(grouped(1 << 20, 1, 2048, 64, y=None))) == (SHAPE, 12345)
    assert size("scan_bwd", scan_bwd_args(grouped(1 << 20, 1, 2047, 64, y=None)))[0] == OK
    assert abi.in_phase("scan_bwd", scan_bwd_args(grouped(1 << 20, 1, 2048, 64, y=None))) == SHAPE
