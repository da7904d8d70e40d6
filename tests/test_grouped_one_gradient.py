"""One gradient of a product by groups where it, or everything, is empty: a step whose
batch has no rows, or a width of zero. Only a call that leaves out what there is to
compute is refused."""
import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import grouped_ref as gref
from tests.test_ffn_refuse import EINVAL, L, err  # noqa: F401
from tests.test_grouped_refuse import gated_backward, mma_backward

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("kw", [dict(T=0), dict(N=0, ld_y=0), dict(T=0, N=0, ld_y=0),
                                dict(K=0, ld_x=0)], ids=str)
def test_empty_gradients_have_no_address(L, kw):  # noqa: F811
    """(an empty tensor's data pointer is null)"""
    assert mma_backward(L, dX=0, dW=0, **kw) == 0, err(L)
    assert gated_backward(L, dX=0, dWg=0, dWu=0, **kw) == 0, err(L)


def test_nothing_wanted(L):  # noqa: F811
    assert mma_backward(L, dX=0, dW=0) == EINVAL and "no gradient" in err(L)
    assert gated_backward(L, dX=0, dWg=0, dWu=0) == EINVAL and "no gradient" in err(L)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,N", [(0, 24), (5, 0), (0, 0)])
def test_each_alone(T, N, dtype):
    K, ends = 32, gref.ends_of([T - T // 2, T // 2]).cuda()
    x = torch.ones(T, K, dtype=dtype, device="cuda")
    dy = torch.ones(T, N, dtype=dtype, device="cuda")
    w = torch.zeros(2, N // 8, K // 16, 8, 8, dtype=torch.int32, device="cuda")
    for dx in (True, False):
        got = bmm.grouped_mma_backward(dy, x, w, ends, need_dx=dx, need_dw=not dx)
        more = bmm.grouped_gated_backward(dy, dy, dy, x, w, w, ends, need_dx=dx, need_dw=not dx)
        for t, shape in zip((*got, *more), [(T, K) if dx else None, None if dx else (2, N, K)] +
                            [(T, K) if dx else None] + 2 * [None if dx else (2, N, K)]):
            assert t is None if shape is None else t.shape == shape and (t == 0).all()
