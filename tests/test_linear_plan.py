"""Which kernel linear takes (gdit_debug_linear_plan): host logic, no GPU."""

import ctypes

import pytest

import flow_matching_dit_b200 as fm
from flow_matching_dit_b200 import _lib
from tests.test_ops_host import L, linear_args  # noqa: F401


@pytest.mark.parametrize("m, n, k, aligned, bn", [
    (16384, 8192, 2048, True, 256), (4100, 4104, 2048, True, 256), (4100, 4103, 2048, False, 256),
    (4100, 1032, 520, True, 128), (4100, 1030, 520, False, 128), (16384, 16, 64, True, 0), (1, 4096, 1024, True, 0),
    (136, 1024, 4096, True, 0), (5, 72, 128, True, 0), (200, 264, 192, True, 0), (1, 1, 8, True, 0),
])
@pytest.mark.parametrize("dtype", [fm.GDIT_F32, fm.GDIT_BF16])
@pytest.mark.parametrize("residual", [False, True])
def test_kernels_of_sizes(m, n, k, aligned, bn, dtype, residual):
    """The tile width of the kernel on pairs of CTAs, 0 for the one that cuts K."""
    p = fm.debug_linear_plan(m, n, k, dtype, residual, aligned)
    assert (p["bn"] if p["pair"] else 0) == bn
    assert not p["pair"] or p["splits"] == 1


@pytest.mark.parametrize("m, n, k", [(1, 4096, 1024), (17, 1024, 1024), (136, 1024, 4096), (1, 16, 8), (3, 50, 8192), (100, 8192, 64)])
@pytest.mark.parametrize("sms", [8, 132, 148])
def test_parts_of_k_are_never_empty(m, n, k, sms):
    p = fm.debug_linear_plan(m, n, k, num_sms=sms)
    assert p["bn"] in (32, 64, 128, 256) and 1 <= p["splits"] <= 8
    assert p["splits"] == 1 or 2 * p["splits"] <= -(-k // 64)


def test_refusals(L):  # noqa: F811
    out = [ctypes.byref(ctypes.c_int()) for _ in range(3)]
    for args, sms in ((linear_args(k=60), 148), (linear_args(m=0), 148), (linear_args(x=None), 148), (linear_args(), -1), (linear_args(), 7)):
        assert L.gdit_debug_linear_plan(ctypes.byref(args), sms, *out) == _lib.GDIT_EINVAL
    assert L.gdit_debug_linear_plan(ctypes.byref(linear_args()), 148, None, *out[1:]) == _lib.GDIT_EINVAL
