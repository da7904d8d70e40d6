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


SIZES = [  # (batch, M, F, K): one tile, split dX, split dW, dX in two launches, batches, nothing
    (1, 5, 24, 32), (1, 300, 520, 336), (1, 12000, 1032, 1040), (1, 32773, 1024, 512),
    (1, 8229, 1032, 2048), (1, 4783, 3064, 3888), (3, 129, 200, 144), (1, 8192, 8192, 4096),
    (2, 0, 24, 32), (2, 5, 0, 32), (0, 5, 24, 32),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_workspace_depends_on_the_extents_alone(size):
    """Row strides, type and activation ask for the same bytes."""
    batch, M, F, K = size
    need = bmm.gated_backward_workspace_bytes(batch, M, F, K)
    for ld_x in (K, K + 8, K + 4096):
        for ld_h in (F, F + 8, 3 * F + 24):
            for dtype in (0, 1):
                for act in range(4):
                    assert workspace(batch, M, F, K, ld_x, ld_h, dtype, act) == need


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_workspace_is_what_its_parts_take(size):
    """[dG | dU] in 16 bits, each half padded to 32 values; a word for the scale and one
    for each of its peaks (one for 256 x 8 values, 1024 at most), to 256 bytes; and the
    float32 parts of the largest of the products, which come one after another."""
    batch, M, F, K = size
    wide = 2 * (-(-F // 32) * 32)
    dgu = batch * M * wide * 2
    peaks = min(-(-batch * M * F // 2048), 1024)
    base = -(-(dgu + (4 * (1 + peaks) if peaks else 0)) // 256) * 256

    def parts(product, rows):
        _, splits = bmm.ffn_plan(product, batch, M, F, K)
        return splits * batch * rows * K * 4 if splits > 1 else 0
    need = bmm.gated_backward_workspace_bytes(batch, M, F, K)
    dw = parts("gated_dw", wide)
    if bmm.ffn_plan("gated_dx_rest", batch, M, F, K)[0] == "none":
        assert need == base + max(dw, parts("gated_dx", M))
    else:   # (where dX's rows part is not told; the first launch has most of them)
        assert base + dw <= need <= base + max(dw, parts("gated_dx", M), parts("gated_dx_rest", M // 2))
