"""The checks of tests/ffn_sums.py see mistakes that a split sum, its last slab or its
last rows could bring, planted here in weight gradients made on the CPU."""
import pytest
import torch

from tests import ffn_ref as ref
from tests import ffn_sums as sums

BF, HF = torch.bfloat16, torch.float16
M, F, K = 20011, 40, 48


def weight_gradient(d, x, mistake):
    """d^T x in float64 as the kernel sums it (slabs of 32 rows), with a mistake."""
    if mistake == "tail":            # the 11 rows after the last whole slab
        d, x = d[:M // 32 * 32], x[:M // 32 * 32]
    out = d.t().contiguous() @ x
    slab = slice(9600, 9632)
    if mistake == "lost slab":
        out -= d[slab].t().contiguous() @ x[slab]
    if mistake == "slab twice":
        out += d[slab].t().contiguous() @ x[slab]
    if mistake == "lost row":
        out -= d[77:78].t().contiguous() @ x[77:78]
    return out


MISTAKES = ["tail", "lost slab", "slab twice", "lost row"]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_norm(dtype):
    gen = torch.Generator().manual_seed(1)
    dh, g, u = (torch.randn(M, F, generator=gen).to(dtype) for _ in range(3))
    x = torch.randn(M, K, generator=gen).to(dtype)
    a, slope = ref.act(g.double(), "silu")
    for d in (dh.double() * u.double() * slope, dh.double() * a):
        exact, rounded = d.t().contiguous() @ x.double(), d.to(dtype).double()
        assert sums.norm_ratio(weight_gradient(rounded, x.double(), None).to(dtype), exact) < 0.8
        for mistake in MISTAKES:
            got = weight_gradient(rounded, x.double(), mistake).to(dtype)
            assert sums.norm_ratio(got, exact) > 1, mistake


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_whole_numbers(dtype):
    dh, g, u, x, wg, wu = sums.whole_block(2, M, F, K, dtype, "cpu")
    want = sums.gradients(dh, g, u, x, wg, wu, "relu")
    d = dh.double() * u.double() * (g > 0)
    assert torch.equal(d.to(dtype).double(), d)
    assert (d.abs().t().contiguous() @ x.double().abs()).max() < 2 ** 24
    sums.check_whole((want[0].to(dtype), weight_gradient(d, x.double(), None).to(dtype)), want, "")
    for mistake in MISTAKES:
        with pytest.raises(AssertionError, match="differ"):
            sums.check_whole((want[0].to(dtype), weight_gradient(d, x.double(), mistake).to(dtype)),
                             want, mistake)
