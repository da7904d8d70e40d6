"""Limits of the feed-forward operators' extents, refused before any launch (CPU)."""
import ctypes

import pytest

import bf16_matrix_multiply_amd as bmm

BF16 = bmm.ELEM_TYPES["bf16"]


def mma(ld):
    p = [ctypes.c_void_p(4096 * (i + 1)) for i in range(5)]
    return bmm.lib().bmm_mx4_mma(p[0], p[1], p[2], p[3], p[4], 1, 4, 64, 64, ld, BF16, None)


@pytest.mark.parametrize("ld", [(1 << 21) + 8, 1 << 30])
def test_mx4_output_rows_too_far_apart(ld):
    assert mma(ld) == -1, bmm.lib().bmm_last_error()
    assert b"2^21" in bmm.lib().bmm_last_error()


def test_workspace_grows_with_nothing_else_than_the_extents():
    """The same extents ask for the same workspace, and it holds [dG | dU]."""
    for M, F, K in ((1, 8, 16), (45, 1368, 528), (32773, 1024, 512), (8192, 8192, 4096)):
        need = bmm.gated_backward_workspace_bytes(1, M, F, K)
        assert need == bmm.gated_backward_workspace_bytes(1, M, F, K)
        assert need >= M * 2 * F * 2
