"""The f16 backward pass where dG and dU leave f16's range, against 64-bit
gradients whose dG and dU are not rounded.

Bounds in the norm: dG and dU are off by independent roundings, each at most half
a step and a third of that squared in the mean, and so is every gradient's own
rounding; together less than half a step of the gradients' norm. A gradient below
2^-14 is off by at most half the smallest f16 besides."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
HF = torch.float16
TINY = 2.0 ** -14            # smallest normal f16


def block(seed, M, F, K, dh=1.0, g=1.0, u=1.0, x=1.0, w=1.0, batch=1):
    """dH, G, U, X, Wg, Wu in f16, normal values times the given sizes."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(size, *shape):
        return (torch.randn(batch, *shape, generator=gen, device="cuda") * size).to(HF)
    w /= math.sqrt(K)
    return (normal(dh, M, F), normal(g, M, F), normal(u, M, F), normal(x, M, K),
            normal(w, F, K), normal(w, F, K))


def run(ts, act="silu", **kw):
    dh, g, u, x, wg, wu = ts
    return bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act=act, **kw)


def exact(ts, act):
    dh, g, u, x, wg, wu = (t.double() for t in ts)
    a, slope = ref.act(g, act)
    dg, du = dh * u * slope, dh * a
    return (dg @ wg + du @ wu, dg.transpose(1, 2).contiguous() @ x,
            du.transpose(1, 2).contiguous() @ x)


def check_norm(got, want, what):
    for o, r, name in zip(got, want, ("dX", "dWg", "dWu")):
        assert torch.isfinite(o).all(), f"{what} {name}"
        off = (o.double() - r).norm().item()
        bound = ref.half_step(HF) * r.norm().item() + ref.half_tiny(HF) * math.sqrt(r.numel())
        assert off <= bound, f"{what} {name}: {off} > {bound}"


SMALL = [  # (M, F, K, sizes of dH and U): one tile and several, splits, two launches of dX
    (8192, 264, 272, 1e-5, 1.0), (8192, 264, 272, 1e-5, 0.03), (8229, 1032, 2048, 1e-4, 0.01),
    (45, 1368, 528, 1e-5, 0.1), (700, 2056, 2048, 1e-6, 1.0),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("i", range(len(SMALL)), ids=[str(s) for s in SMALL])
def test_small_gradients(i, act):
    M, F, K, dh, u = SMALL[i]
    ts = block(i, M, F, K, dh=dh, u=u)
    check_norm(run(ts, act), exact(ts, act), act)


@pytest.mark.parametrize("M,F,K", [(70, 136, 96), (8192, 264, 272)])
def test_products_above_the_largest_f16(M, F, K):
    """dG and dU of up to 10^7, gradients back in range by small weights and X."""
    ts = block(20, M, F, K, dh=2000.0, u=1000.0, g=100.0, x=1e-5, w=1e-4)
    want = exact(ts, "gelu_tanh")
    assert max(r.abs().max().item() for r in want) < 60000
    check_norm(run(ts, "gelu_tanh"), want, "large")


def test_a_power_of_two_passes_through():
    """Gradients of 2^-10 dH are those of dH times 2^-10, bit for bit where neither
    leaves the normal numbers; relu keeps every value of dG and dU a product of f16
    numbers."""
    ts = block(30, 2050, 264, 528, dh=8.0, u=4.0, x=4.0, w=16.0)
    ts = (torch.where(ts[0].abs() < 2.0 ** -4, torch.zeros_like(ts[0]), ts[0]), *ts[1:])
    one = run(ts, "relu")
    two = run((ts[0] * 2.0 ** -10, *ts[1:]), "relu")
    for p, q in zip(one, two):
        assert torch.isfinite(p).all()
        normal = (p == 0) | (p.abs() >= 1024 * TINY)
        assert normal.float().mean() > 0.9
        assert torch.equal(p[normal].float() * 2.0 ** -10, q[normal].float())


def test_nothing_and_infinities_stay_in_their_rows():
    """No gradient at all gives zeros. A NaN and an infinity in two rows of dH reach
    those rows of dX only, and the other rows' scale stays that of the finite values."""
    ts = block(40, 150, 264, 96, dh=1e-5)
    zero = torch.zeros_like(ts[0])
    assert not any(o.any() for o in run((zero, *ts[1:])))
    quiet, loud = ts[0].clone(), ts[0].clone()
    quiet[0, [7, 140]] = 0
    loud[0, 7], loud[0, 140] = float("nan"), float("inf")
    loud[0, 7, 5:], loud[0, 140, 9:] = 0, 0
    want = run((quiet, *ts[1:]), need_dw=False)[0]
    got = run((loud, *ts[1:]), need_dw=False)[0]
    keep = [r for r in range(150) if r not in (7, 140)]
    assert torch.equal(got[0, keep], want[0, keep])
    assert torch.isnan(got[0, 7]).all() and not torch.isfinite(got[0, 140]).any()


def test_batches_and_strides():
    """Batched, with dH, G and U column groups of one buffer: the same bits as apart."""
    dh, g, u, x, wg, wu = block(50, 130, 200, 64, dh=1e-5, batch=2)
    buf = torch.cat([dh, g, u], 2)
    parts = [buf[:, :, 200 * i:200 * (i + 1)] for i in range(3)]
    got = run((*parts, x, wg, wu))
    check_norm(got, exact((dh, g, u, x, wg, wu), "silu"), "batched")
    for p, q in zip(got, run((dh, g, u, x, wg, wu))):
        assert torch.equal(p, q)


def test_graph_replays_follow_the_scale():
    """Captured once; every replay, on values of another size and with eager work in
    between, equals the eager result."""
    ts = block(60, 515, 136, 272)
    dh, packed = ts[0], (ref.pack(ts[4]), ref.pack(ts[5]))
    ws = torch.empty(bmm.gated_backward_workspace_bytes(1, 515, 136, 272), dtype=torch.uint8,
                     device="cuda")

    def step():
        return bmm.gated_backward(*ts[:4], *packed, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i, size in enumerate((1e-5, 100.0, 1.0, 1e-3)):
        gen = torch.Generator().manual_seed(i)
        dh.copy_((torch.randn(dh.shape, generator=gen) * size).to(HF))
        graph.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in outs]
        for k, e in zip(kept, step()):
            assert torch.equal(k, e), i
        check_norm(kept, exact(ts, "silu"), str(size))
        torch.cuda.synchronize()
