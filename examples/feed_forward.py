"""A gated feed-forward block, y = Wd (silu(Wg x) * (Wu x)): trained in bf16, then
held in 4 bits and used a token at a time.

    python -m examples.feed_forward [--steps 60] [--dim 512] [--width 1024]

Training runs the block forward with its projections kept (``gated``), the down
projection and its gradients on packed operands (``pack_operand``, ``mma_tile``)
and the block's backward pass (``gated_backward``); the optimiser keeps float32
weights. Then all three weights go to 4 bits (``mx4_quantize``) and single tokens
through ``mx4_gated`` and ``mx4_mma``.
"""
import argparse
import math

import torch

import bf16_matrix_multiply_amd as bmm

BF16 = torch.bfloat16


def pack_b(w: torch.Tensor) -> torch.Tensor:
    """A row-major bf16 weight (rows, K) as a packed B operand."""
    return bmm.pack_operand(w.view(torch.int16), 8)


def product(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    """Row-major float32 a b^T of packed operands: mma_tile's atoms, laid out."""
    d = bmm.mma_tile(a, b, None, 0.0, "bf16")
    _, m, n = d.shape[:3]
    return d.permute(0, 1, 3, 2, 4).reshape(m * 16, n * 8)


class Block:
    """The three weights in float32, and their bf16 forms of the current step."""

    def __init__(self, dim: int, width: int, gen: torch.Generator):
        def init(rows, cols):
            return torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)
        self.weights = [init(width, dim), init(width, dim), init(dim, width)]

    def halves(self):
        return [w.to(BF16) for w in self.weights]

    def forward(self, x: torch.Tensor):
        """y and what the backward pass takes."""
        wg, wu, wd = self.halves()
        gate, up = pack_b(wg), pack_b(wu)
        h, g, u = bmm.gated(x, gate, up, save=True)
        y = product(bmm.pack_operand(h.view(torch.int16), 16), pack_b(wd))
        return y, (x, gate, up, wd, h, g, u)

    @staticmethod
    def backward(dy: torch.Tensor, kept):
        """Gradients of the input and of the three weights."""
        x, gate, up, wd, h, g, u = kept
        dy = dy.to(BF16)
        # dH = dY Wd, dWd = dY^T H: the operands whose summed axis runs across rows
        # are packed from there
        dh = product(bmm.pack_operand(dy.view(torch.int16), 16),
                     bmm.pack_operand_kmajor(wd.view(torch.int16), 8)).to(BF16)
        dwd = product(bmm.pack_operand_kmajor(dy.view(torch.int16), 16),
                      bmm.pack_operand_kmajor(h.view(torch.int16), 8))
        dx, dwg, dwu = bmm.gated_backward(dh, g, u, x, gate, up)
        return dx, [dwg.float(), dwu.float(), dwd]


class FourBit:
    """The block with its weights in 4 bits, for tokens being decoded."""

    def __init__(self, block: Block):
        self.wg, self.wu, self.wd = (bmm.mx4_quantize(w) for w in block.halves())

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        h = bmm.mx4_gated(bmm.mx4_quantize(x), self.wg, self.wu)
        return bmm.mx4_mma(bmm.mx4_quantize(h), self.wd, dtype=BF16)


def train(block: Block, target: Block, steps: int, tokens: int, rate: float, gen: torch.Generator):
    """Fits block to target's outputs by Adam; the mean squared error of each step."""
    first = [torch.zeros_like(w) for w in block.weights]
    second = [torch.zeros_like(w) for w in block.weights]
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, block.weights[0].shape[1], generator=gen, device="cuda").to(BF16)
        y, kept = block.forward(x)
        off = y - target.forward(x)[0]
        losses.append(off.square().mean())
        _, grads = block.backward(off * (2 / tokens), kept)
        for w, g, m, v in zip(block.weights, grads, first, second):
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.02)
            w -= rate * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.98 ** step)).sqrt() + 1e-8)
    return [float(l) for l in losses]


def run(steps=60, dim=512, width=1024, tokens=1024, rate=3e-3, seed=0):
    """The losses, and the 4-bit block's relative error over 8 tokens one by one."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    target, block = Block(dim, width, gen), Block(dim, width, gen)
    losses = train(block, target, steps, tokens, rate, gen)
    x = torch.randn(16, dim, generator=gen, device="cuda").to(BF16)
    want = block.forward(x)[0][:8]
    small = FourBit(block)
    got = torch.cat([small(x[i:i + 1]) for i in range(8)]).float()
    return losses, float((got - want).norm() / want.norm())


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--dim", type=int, default=512, help="a multiple of 32")
    parser.add_argument("--width", type=int, default=1024, help="a multiple of 32")
    args = parser.parse_args()
    losses, error = run(args.steps, args.dim, args.width)
    print(f"mean squared error: step 1 {losses[0]:.4f}, step {len(losses)} {losses[-1]:.4f}")
    print(f"4-bit weights and activations, one token at a time: {100 * error:.1f}% off")


if __name__ == "__main__":
    main()
