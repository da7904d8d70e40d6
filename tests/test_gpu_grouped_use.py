"""The products by groups and of 8-bit integers as programs use them: a block of experts
forward and backward, the same served in 8 bits, captured in graphs, on other streams,
with more than 2^31 elements, and the example."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


class Block:
    """Experts' weights in one 16-bit type, packed for the kernels."""

    def __init__(self, E, dim, width, dtype, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.wg, self.wu = (gref.weights(gen, E, width, dim, dtype, "cuda") for _ in range(2))
        self.wd = gref.weights(gen, E, dim, width, dtype, "cuda")
        self.packed = [ref.pack(w) for w in (self.wg, self.wu, self.wd)]

    def forward(self, x, ends, act):
        g, u, d = self.packed
        H, G, U = bmm.grouped_gated(x, g, u, ends, act=act, save=True)
        return bmm.grouped_mma(H, d, ends), (H, G, U)

    def backward(self, dy, x, ends, act, kept):
        g, u, d = self.packed
        H, G, U = kept
        dH, dWd = bmm.grouped_mma_backward(dy, H, d, ends)
        dX, dWg, dWu = bmm.grouped_gated_backward(dH, G, U, x, g, u, ends, act=act)
        return dX, dWg, dWu, dWd, dH


def check(got, want, what, dtype=BF):
    """Both (value, bound), the value in float64 on the CPU."""
    ref.check(got, want[0], want[1], dtype, what)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_block(dtype):
    """Each operator's output against 64 bits from the 16-bit values that it was given, so
    that a stage's own error is all that its bound holds."""
    counts, act = [70, 0, 129, 3, 200], "silu"
    T, dim, width = sum(counts) + 9, 256, 400
    block = Block(5, dim, width, dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, dim, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(T, dim, generator=gen, device="cuda").to(dtype)
    ends = gref.ends_of(counts).cuda()
    y, kept = block.forward(x, ends, act)
    grads = block.backward(dy, x, ends, act, kept)
    c = lambda t: t.double().cpu()
    wg, wu, wd = c(block.wg), c(block.wu), c(block.wd)
    for got, want, what in zip(kept, gref.gated(c(x), wg, wu, counts, act), "HGU"):
        check(got, want, what, dtype)
    check(y, gref.mma(c(kept[0]), wd, counts), "Y", dtype)
    dX, dWg, dWu, dWd, dH = grads
    want_dh, want_dwd = gref.mma_backward(c(dy), c(kept[0]), wd, counts)
    check(dH, want_dh, "dH", dtype)
    check(dWd, want_dwd, "dWd", dtype)
    want = gref.gated_backward(c(dH), c(kept[1]), c(kept[2]), c(x), wg, wu, counts, act, dtype)
    for got, w, what in zip((dX, dWg, dWu), want, ("dX", "dWg", "dWu")):
        check(got, w, what, dtype)


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [60, 0, 75, 300]], ids=["decode", "prompt"])
def test_served_in_8_bits(counts):
    """X and H quantised a token, weights a channel; each stage from the codes it was given."""
    T, dim, width = sum(counts), 256, 416
    block = Block(4, dim, width, BF)
    gate, up, down = (bmm.i8_pack(bmm.i8_quantize(w)) for w in (block.wg, block.wu, block.wd))
    rows = [bmm.i8_quantize(w) for w in (block.wg, block.wu, block.wd)]
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, dim, generator=gen, device="cuda").to(BF)
    ends = gref.ends_of(counts).cuda()
    q = bmm.i8_quantize(x)
    h = bmm.i8_gated(q, gate, up, ends, act="gelu")
    p = bmm.i8_quantize(h)
    y = bmm.i8_mma(p, down, ends, dtype=BF)
    for got, (codes, scales) in ((q, gref.i8_quantize(x.cpu())), (p, gref.i8_quantize(h.cpu()))):
        assert torch.equal(got.codes.cpu().long(), codes) and torch.equal(got.scales.cpu(), scales)
    for e, r in gref.groups(counts):
        def product(a, w):
            return gref.i8_mma(a.codes[r], a.scales[r], w.codes[e], w.scales[e], torch.float32)
        gv, uv = product(q, rows[0]).double(), product(q, rows[1]).double()
        want = ref.act(gv, "gelu")[0] * uv
        ref.check(h[r], want, want.abs() * ref.act_rel(gv, "gelu"), BF, "H")
        assert torch.equal(y[r], product(p, rows[2]).to(BF))
    # and the whole block next to 16 bits: codes are off by half of 1 / 127 of the row's
    # largest value at most, some 3.5 of its root mean square, so by 3.5 / 254 / sqrt(3) =
    # 0.8% of that, for x, both weights of a product and H: well below 4 of them together
    full = block.forward(x, ends, "gelu")[0].float()
    assert (y.float() - full).norm() < 4 * 2 * 0.008 * full.norm()


def test_graph_takes_other_groups():
    """Forward, backward and the 8-bit forms captured once, replayed with other rows and
    other groups in the same buffers, with eager work between the replays."""
    E, T, dim, width, act = 6, 200, 128, 288, "silu"
    block = Block(E, dim, width, BF)
    gate, up, down = (bmm.i8_pack(bmm.i8_quantize(w)) for w in (block.wg, block.wu, block.wd))
    x, dy = (torch.zeros(T, dim, dtype=BF, device="cuda") for _ in range(2))
    ends = torch.zeros(E, dtype=torch.int32, device="cuda")

    def step():
        y, kept = block.forward(x, ends, act)
        grads = block.backward(dy, x, ends, act, kept)
        h = bmm.i8_gated(bmm.i8_quantize(x), gate, up, ends, act=act)
        return (y, *kept, *grads, h, bmm.i8_mma(bmm.i8_quantize(h), down, ends, dtype=BF))

    def load(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, dim, generator=gen, device="cuda"))
        dy.copy_(torch.randn(T, dim, generator=gen, device="cuda"))
        counts = [[200, 0, 0, 0, 0, 0], [0] * 6, [30, 40, 1, 0, 100, 9], [1, 1, 1, 1, 1, 1],
                  [0, 0, 0, 0, 0, 200]][seed % 5]
        ends.copy_(gref.ends_of(counts))

    load(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (0, 1, 2, 3, 4, 7):
        load(seed)
        for o in outs:
            o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (seed, i)


def test_two_graphs_share_nothing():
    """Two captured backward passes replayed in turns, each with its own workspace; and one
    workspace serves both where they run one after the other."""
    counts = [[100, 0, 60], [0, 150, 10]]
    block = Block(3, 96, 144, HF)
    gen = torch.Generator(device="cuda").manual_seed(5)
    made, shared = [], torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    for c in counts:
        x, dy = (torch.randn(160, n, generator=gen, device="cuda").to(HF) for n in (96, 96))
        ends = gref.ends_of(c).cuda()
        _, kept = block.forward(x, ends, "gelu")
        want = block.backward(dy, x, ends, "gelu", kept)
        g, u, d = block.packed

        def both(x=x, dy=dy, ends=ends, kept=kept):
            H, G, U = kept
            dH, dWd = bmm.grouped_mma_backward(dy, H, d, ends, workspace=shared)
            return (*bmm.grouped_gated_backward(dH, G, U, x, g, u, ends, act="gelu", workspace=shared),
                    dWd, dH)
        both()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = both()
        made.append((graph, out, want, both))   # (both: its inputs have to live on)
    for _ in range(3):
        for graph, out, _, _ in made:
            for o in out:
                o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in made:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_other_streams():
    """Two blocks at once on two streams that are not the current one."""
    counts = [120, 7, 0, 333]
    ends = gref.ends_of(counts).cuda()
    blocks = [Block(4, 160, 272, BF, seed) for seed in range(2)]
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, dy = (torch.randn(460, 160, generator=gen, device="cuda").to(BF) for _ in range(2))

    def run(block):
        y, kept = block.forward(x, ends, "relu")
        return (y, *block.backward(dy, x, ends, "relu", kept))
    want = [run(b) for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    got = [None, None]
    for _ in range(4):
        for i, (s, b) in enumerate(zip(streams, blocks)):
            with torch.cuda.stream(s):
                got[i] = run(b)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for t, r in zip(a, b):
            assert torch.equal(t, r)


def test_rows_past_2_to_the_31_elements():
    """T * K and T * N past 2^32 bytes and 2^31 elements: rows near the end, and a group's
    sum that starts there."""
    T, K, N = (1 << 20) + 300, 2064, 8
    x = torch.zeros(T, K, dtype=BF, device="cuda")
    x[-200:] = torch.randint(-2, 3, (200, K), device="cuda").to(BF)
    counts = [1000, T - 1000 - 150, 0, 150]
    ends = gref.ends_of(counts).cuda()
    w = torch.randint(-2, 3, (4, N, K), device="cuda").to(BF)
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    want[-200:-150] = x[-200:-150].double() @ w[1].double().t()
    want[-150:] = x[-150:].double() @ w[3].double().t()
    assert torch.equal(bmm.grouped_mma(x, ref.pack(w), ends), want.to(BF))
    dy = torch.zeros(T, N, dtype=BF, device="cuda")
    dy[-200:] = torch.randint(-2, 3, (200, N), device="cuda").to(BF)
    dx, dw = bmm.grouped_mma_backward(dy, x, ref.pack(w), ends)
    assert not dx[:-200].any()
    assert torch.equal(dx[-200:-150], (dy[-200:-150].double() @ w[1].double()).to(BF))
    assert torch.equal(dx[-150:], (dy[-150:].double() @ w[3].double()).to(BF))
    assert not dw[0].any() and not dw[2].any()
    assert torch.equal(dw[1], (dy[-200:-150].double().t().contiguous() @ x[-200:-150].double()).to(BF))
    assert torch.equal(dw[3], (dy[-150:].double().t().contiguous() @ x[-150:].double()).to(BF))
    del dx, dy, want
    # 8 bits: codes past 2^31, the same rows
    Tq = (1 << 21) + 100
    a = torch.zeros(Tq, 1056, dtype=torch.int8, device="cuda")
    a[-100:] = torch.randint(-128, 128, (100, 1056), device="cuda").to(torch.int8)
    sa = torch.rand(Tq, device="cuda")
    b = torch.randint(-128, 128, (1, 8, 1056), device="cuda").to(torch.int8)
    sb = torch.rand(1, 8, device="cuda")
    D = bmm.i8_mma(bmm.I8Operand(a, sa), bmm.I8Operand(gref.i8_pack(b), sb))
    assert not D[:-100].any()
    assert torch.equal(D[-100:], gref.i8_mma(a[-100:], sa[-100:], b[0], sb[0], torch.float32))


def test_norm_of_long_sums():
    """A lost row shows: over many rows the gradients stay within one half step of their
    norm (each element's own rounding; sums in float32 add some 1e-6 of it)."""
    counts = [3000, 0, 12345, 1]
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(sum(counts), 64, generator=gen, device="cuda").to(BF)
    dy = torch.randn(sum(counts), 128, generator=gen, device="cuda").to(BF)
    w = gref.weights(gen, 4, 128, 64, BF, "cuda")
    _, dw = bmm.grouped_mma_backward(dy, x, ref.pack(w), gref.ends_of(counts).cuda())
    for e, r in gref.groups(counts):
        want = dy[r].double().t().contiguous() @ x[r].double()
        assert (dw[e].double() - want).norm() <= ref.half_step(BF) * want.norm()
        assert math.isfinite(want.norm().item())


def test_example():
    from examples import experts
    losses, error, grad = experts.run(steps=4, dim=64, width=96, n_experts=4, tokens=64, top=2)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
    # gradients against float64 autograd of the same 16-bit weights: H, G, U, dH, dG and dU and
    # the results are each rounded to bf16, half a step of relative error each, 7 at most
    assert grad <= 7 * ref.half_step(BF), grad
    # 8-bit codes of x, H and the weights: each off by 0.8% of its size (3.5 / 254 / sqrt 3),
    # five of them, and bf16's own
    assert error < 5 * 0.008 * 2, error
