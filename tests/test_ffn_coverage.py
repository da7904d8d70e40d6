"""The shapes of the feed-forward operators' GPU tests reach every tile that the plan
can choose, in every element type (CPU: the plan is host code)."""
import ctypes

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import test_gpu_ffn_large as large
from tests import test_gpu_ffn_tiles as tiles
from tests import test_gpu_gated as gated
from tests import test_gpu_mx4 as mx4

BF, HF = torch.bfloat16, torch.float16
TILES = ["128x128", "256x128", "256x192", "256x256"]


def reached(product):
    """{(tile, whether its sum is split, dtype)} of the test shapes; 4 bits: dtype None."""
    if product == "gated":
        shapes = [(s[:4], (BF, HF)) for s in gated.SHAPES] + [(s[:4], s[5:6]) for s in large.GATED] + \
            [((1, *s), (BF, HF)) for s in tiles.GATED]
    elif product.startswith("gated"):
        shapes = [(s[:4], (BF, HF)) for s in gated.BACK] + [(s[:4], s[5:6]) for s in large.BACK] + \
            [((1, *s), (BF, HF)) for s in tiles.BACK]
    else:
        lists = (large.PRODUCTS, mx4.PRODUCTS) if product == "mx4_mma" else (large.MX4_GATED, mx4.GATED)
        shapes = [((max(s[0], 1), *s[1:4]), (None,)) for l in lists for s in l] + \
            [((1, *s), (None,)) for s in (tiles.PRODUCTS if product == "mx4_mma" else tiles.MX4_GATED)]
    out = set()
    for shape, dtypes in shapes:
        tile, splits = bmm.ffn_plan(product, *shape)
        out |= {(tile, splits > 1, d) for d in dtypes}
    return out


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_gated(dtype):
    got = reached("gated")
    for tile in TILES + ["few_rows"]:
        assert (tile, False, dtype) in got, tile


@pytest.mark.parametrize("product", ["mx4_mma", "mx4_gated"])
def test_four_bits(product):
    got = reached(product)
    for tile in TILES + ["few_rows"]:
        assert (tile, False, None) in got, tile


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("product", ["gated_dx", "gated_dw"])
def test_gated_backward(product, dtype):
    got = reached(product)
    for tile in TILES:
        for split in (False, True):
            assert (tile, split, dtype) in got, (tile, split)


def test_second_launch_of_dx():
    got = reached("gated_dx_rest")
    for tile in ("none", "128x128", "256x128", "256x192"):
        assert any(tile == t for t, _, _ in got), tile


def test_plan_of_nothing_and_refusals():
    assert bmm.ffn_plan("gated", 1, 0, 8, 16) == ("none", 1)
    assert bmm.ffn_plan("gated", 1, 5, 0, 16) == ("none", 1)
    assert bmm.ffn_plan("gated", 1, 5, 8, 0)[0] == "few_rows"     # zeros are written
    assert bmm.ffn_plan("gated_dw", 1, 0, 8, 16)[0] != "none"     # and here
    assert bmm.ffn_plan("gated_dx", 1, 5, 8, 0) == ("none", 1)
    assert bmm.ffn_plan("mx4_mma", 0, 5, 8, 32) == ("none", 1)
    for product, F, K, needle in (("gated", 12, 16, "multiple of 8"), ("gated_dx", 8, 24, "multiple of 16"),
                                  ("mx4_mma", 12, 32, "multiple of 8"),
                                  ("mx4_gated", 8, 48, "multiple of 32"),
                                  ("mx4_mma", 8, 1 << 22, "too large"), ("gated", -8, 16, "negative"),
                                  ("mx4_mma", -8, 32, "negative"), ("mx4_gated", 8, -32, "negative")):
        with pytest.raises(bmm.BmmError, match=needle):
            bmm.ffn_plan(product, 1, 5, F, K)
    for product in (-1, 6):
        assert bmm.lib().bmm_ffn_plan(product, 1, 5, 8, 32, None) == -1
        assert b"bmm_ffn_product" in bmm.lib().bmm_last_error()
    splits = ctypes.c_int32(-7)
    assert bmm.lib().bmm_ffn_plan(0, 1, 5, 8, 32, ctypes.byref(splits)) == 4 and splits.value == 1
