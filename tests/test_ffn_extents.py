"""The gated block's largest extents and the workspace of its backward pass, as
include/bmm.h states them (CPU: nothing is launched)."""
import ctypes

import pytest

import bf16_matrix_multiply_amd as bmm

EINVAL = -1


def workspace(batch, M, F, K, ld_x=None, ld_h=None, dtype=1, act=0):
    """Bytes, or < 0, through the C entry point."""
    d = bmm.GatedDesc(batch, M, F, K, K if ld_x is None else ld_x, F if ld_h is None else ld_h,
                      dtype, act)
    return bmm.lib().bmm_gated_backward_workspace_bytes(ctypes.byref(d))


def error():
    return bmm.lib().bmm_last_error().decode()


def test_widest_block():
    """K up to 2^21 and F up to 2^20 are taken; past either the message names it."""
    assert workspace(1, 3, 8, 1 << 21) > 0
    assert workspace(1, 3, 1 << 20, 16) > 0
    assert workspace(1, 3, 8, (1 << 21) + 16) == EINVAL
    assert "K <= 2^21" in error()
    assert workspace(1, 3, (1 << 20) + 8, 16) == EINVAL
    assert "F <= 2^20" in error()


@pytest.mark.parametrize("K", [(1 << 21) + 16, (1 << 22) - 16])
def test_too_wide_for_any_entry_point(K):
    d = bmm.GatedDesc(1, 3, 8, K, K, 8, 1, 0)
    p = [ctypes.c_void_p((i + 1) << 40) for i in range(10)]
    assert bmm.lib().bmm_gated(p[0], None, None, p[1], p[2], p[3], ctypes.byref(d), None) == EINVAL
    assert "K <= 2^21" in error()
    assert bmm.lib().bmm_gated_backward(*p[:9], ctypes.byref(d), p[9], 1 << 40, None) == EINVAL
    assert "K <= 2^21" in error()
