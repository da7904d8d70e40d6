"""What lies in the padding of 4-bit operands (codes of K values past the matrix,
rows past its last one) reaches no result, whichever kernel makes the product."""
import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def operand(seed, rows, K):
    """A 4-bit operand of one scale (1), as the format pads it (zeros) and with other
    codes, and NaN scales for the rows past the last one, in its padding; and its
    float64 values."""
    gen = torch.Generator().manual_seed(seed)
    code = torch.randint(0, 16, (rows, K), generator=gen)
    byte = torch.full((rows, K // 32), 127)
    up, wide = -(-rows // 16) * 16, -(-K // 128) * 128
    full = torch.randint(1, 8, (up, wide), generator=gen)     # codes of values above 0
    full[:rows, :K] = code
    scale = torch.full((up, wide // 32), 127)                 # padded K values count, if they do
    scale[rows:] = 255
    clean = bmm.Mx4Operand(*(t.cuda() for t in ref.mx4_layout(code, byte)), rows, K)
    dirty = bmm.Mx4Operand(*(t.cuda() for t in ref.mx4_layout(full, scale)), rows, K)
    assert dirty.codes.shape == clean.codes.shape and dirty.scales.shape == clean.scales.shape
    return clean, dirty, ref.mx4_values(code, byte)


@pytest.mark.parametrize("M", [1, 7, 23, 40, 64, 65, 150, 300])
@pytest.mark.parametrize("N,K", [(72, 32), (264, 160), (520, 1056)])
def test_product(M, N, K):
    """Every sum is a multiple of 1/4 below 2^22, so the product is exact."""
    a_clean, a_dirty, a = operand(M + K, M, K)
    b_clean, b_dirty, b = operand(N + K, N, K)
    want = a @ b.t()
    for A, B in ((a_clean, b_clean), (a_dirty, b_clean), (a_clean, b_dirty), (a_dirty, b_dirty)):
        assert torch.equal(bmm.mx4_mma(A, B, F32).double().cpu(), want)


@pytest.mark.parametrize("M", [1, 7, 23, 40, 64, 65, 150, 300])
@pytest.mark.parametrize("F,K", [(72, 32), (264, 160), (520, 1056)])
def test_gated(M, F, K):
    x_clean, x_dirty, x = operand(M + K, M, K)
    g_clean, g_dirty, g = operand(F + K, F, K)
    u_clean, u_dirty, u = operand(F + K + 1, F, K)
    want = (torch.clamp(x @ g.t(), min=0) * (x @ u.t())).to(F32).to(BF)
    for X, G, U in ((x_clean, g_clean, u_clean), (x_dirty, g_dirty, u_dirty)):
        got = bmm.mx4_gated(X, G, U, act="relu", dtype=BF)
        # exact projections; their product is rounded to float32 and then to bf16
        assert torch.equal(got.cpu(), want)
