"""Calls of the operators that are refused, beside those of test_ops_host.  No GPU."""

import ctypes

import pytest

from flow_matching_dit_b200 import _lib
from tests.test_ops_host import L, attention_args  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, -3e38])
def test_attention_scales_whose_base_2_form_overflows(L, scale):  # noqa: F811
    """Scores are exponentiated to the base 2: scale log2(e) has to be a float, too."""
    assert L.gdit_attention(ctypes.byref(attention_args(scale=scale)), None) == _lib.GDIT_EINVAL
    assert "scale" in L.gdit_last_error(None).decode()


@pytest.mark.parametrize("limit_ns", [0, 999, 1_000_000_001])
def test_wait_expiry_limits(L, limit_ns):  # noqa: F811
    assert L.gdit_debug_op_wait_expiry(0, limit_ns) == _lib.GDIT_EINVAL
