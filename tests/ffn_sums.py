"""Checks of the gated block's gradients that see a mistake in a long sum.

A bound on each element that adds the half steps of all its terms grows with their
number, the gradient only like its root, so over many rows such a bound no longer
sees a few lost ones. Two checks that do:

- in the norm, against gradients whose dG and dU are not rounded. Those two are off
  by independent roundings, which give a gradient the relative error of one (below
  half a step, 0.42 of it in the root mean square), and its own rounding as much
  again: together below half a step of its norm. One lost row of M makes 1 / sqrt(M).
- bit for bit, on whole numbers: with relu, small whole dH, G, U, X and weights, dG
  and dU are whole numbers that 16 bits hold and every partial sum one that float32
  holds, so only the gradient's own rounding is left."""
import torch

from tests import ffn_ref as ref


def gradients(dh, g, u, x, wg, wu, act):
    """(dX, dWg, dWu) in float64; nothing is rounded on the way."""
    dh, g, u, x, wg, wu = (t.double() for t in (dh, g, u, x, wg, wu))
    a, slope = ref.act(g, act)
    dg, du = dh * u * slope, dh * a
    return (dg @ wg + du @ wu, dg.transpose(-1, -2).contiguous() @ x,
            du.transpose(-1, -2).contiguous() @ x)


def norm_ratio(got, want):
    """The error's norm over half a step of the gradient's; at most 1."""
    return ((got.double() - want).norm() / (ref.half_step(got.dtype) * want.norm())).item()


def check_norm(got, want, what):
    for o, r, name in zip(got, want, ("dX", "dWg", "dWu")):
        ratio = norm_ratio(o, r)
        assert ratio <= 1, f"{what} {name}: {ratio}"


def whole_block(seed, M, F, K, dtype, device):
    """dH, G, U, X, Wg, Wu of whole numbers from -2 to 2, X and the weights from -3 to
    3. dG and dU are at most 4, so a sum of n terms is at most 12 n: below 2^24 for n
    up to 10^6."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def whole(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=gen, device=device).to(dtype)
    return (whole(2, M, F), whole(2, M, F), whole(2, M, F), whole(3, M, K), whole(3, F, K),
            whole(3, F, K))


def check_whole(got, want, what):
    for o, r, name in zip(got, want, ("dX", "dWg", "dWu")):
        off = o != r.to(o.dtype)
        assert not off.any(), f"{what} {name}: {int(off.sum())} of {off.numel()} differ"
