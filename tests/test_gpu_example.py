"""The feed-forward example: training lowers the error, and its gradients and its
4-bit form are those of the block."""
import pytest
import torch

from examples import feed_forward as ff

pytestmark = pytest.mark.gpu


def test_training_and_four_bits():
    """Adam on a realisable target brings the error to about half in 60 steps (in
    plain float32 arithmetic 0.72 -> 0.35); 0.7 leaves room for bf16. 4 bits hold
    a normal value to about 12% (steps of a quarter to a half of an octave); of the
    eight such factors of an output's terms (two operands in each of three products,
    one of them through a gate) independent errors add up to about a third."""
    losses, error = ff.run(steps=60, dim=256, width=512, tokens=512)
    assert losses[-1] < 0.7 * losses[0]
    assert error < 0.5


def test_gradients_against_autograd():
    gen = torch.Generator(device="cuda").manual_seed(1)
    block = ff.Block(128, 256, gen)
    x = torch.randn(64, 128, generator=gen, device="cuda").to(ff.BF16)
    r = torch.randn(64, 128, generator=gen, device="cuda").to(ff.BF16)
    y, kept = block.forward(x)
    dx, grads = block.backward(r.float(), kept)
    leaves = [t.detach().double().requires_grad_() for t in (x, *block.halves())]
    X, wg, wu, wd = leaves
    Y = (torch.nn.functional.silu(X @ wg.t()) * (X @ wu.t())) @ wd.t()
    # H, dH, dG and dU are rounded to bf16 on the way: relative errors of a few half
    # steps (2^-8), independent from term to term
    assert (y.double() - Y).norm() < 4 * 2 ** -8 * Y.norm()
    (Y * r.double()).sum().backward()
    for got, leaf in zip((dx, *grads), leaves):
        assert (got.double() - leaf.grad).norm() < 6 * 2 ** -8 * leaf.grad.norm()
