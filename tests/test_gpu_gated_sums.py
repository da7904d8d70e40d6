"""Long sums of the gated block's gradients on the GPU: in the norm and, on whole
numbers, bit for bit (tests/ffn_sums.py)."""
import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import ffn_sums as sums
from tests.test_gpu_ffn_large import BACK as LARGE
from tests.test_gpu_ffn_large import block, normal
from tests.test_gpu_ffn_tiles import BACK as TILES

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
SHAPES = [s[:4] for s in LARGE] + [(1, *s) for s in TILES] + [(1, 32773, 1024, 512)]
IDS = ["x".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_norm(i, dtype):
    batch, M, F, K = SHAPES[i]
    act = sorted(bmm.ACTS)[i % 4]
    gen, x, wg, wu = block(800 + i, batch, M, F, K, dtype, 8 * (i % 2))
    dh, g, u = (normal(gen, batch, M, F).to(dtype) for _ in range(3))
    got = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act=act)
    sums.check_norm(got, sums.gradients(dh, g, u, x, wg, wu, act), act)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_whole_numbers(i, dtype):
    batch, M, F, K = SHAPES[i]
    blocks = [sums.whole_block(10 * i + b, M, F, K, dtype, "cuda") for b in range(batch)]
    dh, g, u, x, wg, wu = (torch.stack(t) for t in zip(*blocks))
    got = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act="relu")
    sums.check_whole(got, sums.gradients(dh, g, u, x, wg, wu, "relu"), "relu")
