"""A mixture of experts, y = sum over a token's experts of p Wd_e (silu(Wg_e x) * (Wu_e x)):
trained in bf16, then held in 8 bits and used a few tokens at a time.

    python -m examples.experts [--steps 60] [--dim 256] [--width 512] [--experts 8]

A token's ``top`` experts are those with the largest router logits, weighted by the
softmax over them. Its copies are sorted by expert and the experts' block runs on the
sorted rows (``grouped_gated``, ``grouped_mma``, and their backward passes); where an
expert's rows end is a tensor on the GPU, so no step waits for the host. Then the
weights go to 8 bits (``i8_quantize``, ``i8_pack``) and tokens through ``i8_gated`` and
``i8_mma``.
"""
import argparse
import math

import torch

import bf16_matrix_multiply_amd as bmm

BF16 = torch.bfloat16


def pack_b(w: torch.Tensor) -> torch.Tensor:
    """Row-major bf16 weights (experts, rows, K) as packed B operands."""
    return bmm.pack_operand(w.view(torch.int16), 8)


class Route:
    """A token's experts and their weights; the copies' order by expert and its ends."""

    def __init__(self, logits: torch.Tensor, top: int):
        tokens, n = logits.shape
        value, expert = logits.topk(top, dim=1)
        self.weight = value.softmax(1)                                   # (tokens, top)
        self.order = expert.reshape(-1).argsort(stable=True)             # sorted row -> copy
        self.token = self.order // top                                   # sorted row -> token
        self.ends = torch.zeros(n, dtype=torch.int32, device=logits.device).scatter_add_(
            0, expert.reshape(-1), torch.ones_like(self.order, dtype=torch.int32)).cumsum(
                0, dtype=torch.int32)
        self.row_weight = self.weight.reshape(-1)[self.order][:, None]   # of the sorted rows

    def gather(self, x):
        return x[self.token]

    def combine(self, rows):
        """Each token's rows, weighted and added in float32."""
        out = torch.empty_like(rows, dtype=torch.float32)
        out[self.order] = rows.float() * self.row_weight
        return out.reshape(*self.weight.shape, -1).sum(1)


class Experts:
    """The experts' weights in float32, and their bf16 forms of the current step."""

    def __init__(self, n: int, dim: int, width: int, gen: torch.Generator):
        def init(rows, cols):
            return torch.randn(n, rows, cols, generator=gen, device="cuda") / math.sqrt(cols)
        self.weights = [init(width, dim), init(width, dim), init(dim, width)]

    def forward(self, x: torch.Tensor, route: Route):
        """y (float32) and what the backward pass takes."""
        gate, up, down = (pack_b(w.to(BF16)) for w in self.weights)
        rows = route.gather(x)
        h, g, u = bmm.grouped_gated(rows, gate, up, route.ends, save=True)
        y = bmm.grouped_mma(h, down, route.ends)
        return route.combine(y), (rows, gate, up, down, h, g, u)

    @staticmethod
    def backward(dy: torch.Tensor, route: Route, kept):
        """Gradients of the three weights (and of x's sorted rows)."""
        rows, gate, up, down, h, g, u = kept
        d_rows = (route.gather(dy) * route.row_weight).to(BF16)
        dh, d_down = bmm.grouped_mma_backward(d_rows, h, down, route.ends)
        dx, d_gate, d_up = bmm.grouped_gated_backward(dh, g, u, rows, gate, up, route.ends)
        return dx, [d_gate.float(), d_up.float(), d_down.float()]


class EightBit:
    """The experts with their weights in 8 bits, for tokens being decoded."""

    def __init__(self, experts: Experts):
        self.gate, self.up, self.down = (bmm.i8_pack(bmm.i8_quantize(w)) for w in experts.weights)

    def __call__(self, x: torch.Tensor, route: Route) -> torch.Tensor:
        h = bmm.i8_gated(bmm.i8_quantize(route.gather(x)), self.gate, self.up, route.ends)
        return route.combine(bmm.i8_mma(bmm.i8_quantize(h), self.down, route.ends, dtype=BF16))


def gradient_error(experts: Experts, x, route: Route, dy) -> float:
    """The largest relative error (in the norm) of the weights' gradients against float64."""
    _, kept = experts.forward(x, route)
    _, grads = experts.backward(dy, route, kept)
    ws = [w.to(BF16).double().requires_grad_() for w in experts.weights]
    rows, start, loss = route.gather(x).double(), 0, 0.0
    d_rows = route.gather(dy).double() * route.row_weight.double()
    for e, end in enumerate(route.ends.tolist()):
        r = slice(start, end)
        g, u = rows[r] @ ws[0][e].t(), rows[r] @ ws[1][e].t()
        loss = loss + ((g * torch.sigmoid(g) * u) @ ws[2][e].t() * d_rows[r]).sum()
        start = end
    loss.backward()
    return max(float((got.double() - w.grad).norm() / w.grad.norm()) for got, w in zip(grads, ws))


def run(steps=60, dim=256, width=512, n_experts=8, tokens=512, top=2, rate=3e-3, seed=0):
    """The losses; the 8-bit experts' relative error over 8 tokens; the gradients' error."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    router = torch.randn(dim, n_experts, generator=gen, device="cuda") / math.sqrt(dim)
    target, experts = (Experts(n_experts, dim, width, gen) for _ in range(2))
    first = [torch.zeros_like(w) for w in experts.weights]
    second = [torch.zeros_like(w) for w in experts.weights]
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, dim, generator=gen, device="cuda").to(BF16)
        route = Route(x.float() @ router, top)
        y, kept = experts.forward(x, route)
        off = y - target.forward(x, route)[0]
        losses.append(off.square().mean())
        _, grads = experts.backward(off * (2 / tokens), route, kept)
        for w, g, m, v in zip(experts.weights, grads, first, second):
            m.lerp_(g, 0.1)
            v.lerp_(g * g, 0.02)
            w -= rate * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.98 ** step)).sqrt() + 1e-8)
    grad = gradient_error(experts, x, route, off)
    x = torch.randn(8, dim, generator=gen, device="cuda").to(BF16)
    route = Route(x.float() @ router, top)
    want = experts.forward(x, route)[0]
    got = EightBit(experts)(x, route)
    return [float(l) for l in losses], float((got - want).norm() / want.norm()), grad


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--dim", type=int, default=256, help="a multiple of 32")
    parser.add_argument("--width", type=int, default=512, help="a multiple of 32")
    parser.add_argument("--experts", type=int, default=8)
    args = parser.parse_args()
    losses, error, grad = run(args.steps, args.dim, args.width, args.experts)
    print(f"mean squared error: step 1 {losses[0]:.4f}, step {len(losses)} {losses[-1]:.4f}")
    print(f"gradients against float64: {100 * grad:.2f}% off")
    print(f"8-bit weights and activations, 8 tokens: {100 * error:.1f}% off")


if __name__ == "__main__":
    main()
