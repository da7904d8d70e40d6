"""The gated feed-forward block on the GPU, forward and backward, against 64-bit
references with derived bounds (tests/ffn_ref.py)."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
ACTS = sorted(bmm.ACTS)


def inputs(seed, batch, M, F, K, dtype, pad=0, scale=1.0):
    """x (batch, M, K) with K + pad elements between rows, weights and their
    packed forms, on the CPU and the GPU."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(batch, M, K + pad, generator=gen) * scale).to(dtype)
    wg, wu = ((torch.randn(batch, F, K, generator=gen) / math.sqrt(max(K, 1))).to(dtype)
              for _ in range(2))
    return x.cuda()[:, :, :K], wg.cuda(), wu.cuda()


def poison(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


SHAPES = [  # (batch, M, F, K, pad): one row, ragged tiles and slabs, odd counts, several tiles
    (1, 1, 8, 16, 0), (1, 1, 136, 512, 0), (1, 3, 24, 48, 8), (2, 17, 72, 80, 0),
    (1, 16, 64, 32, 0), (3, 5, 40, 1040, 24), (1, 33, 264, 272, 0), (1, 64, 512, 256, 0),
    (1, 65, 88, 96, 0), (1, 129, 136, 144, 40), (2, 130, 200, 64, 0), (1, 300, 520, 336, 0),
    (1, 257, 1160, 2064, 0), (1, 700, 2056, 48, 8),
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=[str(s) for s in SHAPES])
def test_gated(i, dtype):
    batch, M, F, K, pad = SHAPES[i]
    act = ACTS[i % 4]
    x, wg, wu = inputs(i, batch, M, F, K, dtype, pad)
    (h, eh), (g, eg), (u, eu) = ref.gated(x.double().cpu(), wg.double().cpu(), wu.double().cpu(), act)
    H, G, U = bmm.gated(x, ref.pack(wg), ref.pack(wu), act=act, save=True)
    ref.check(H, h, eh, dtype, "H")
    ref.check(G, g, eg, dtype, "G")
    ref.check(U, u, eu, dtype, "U")
    # without the projections: the same bits, in rows wider than F, the rest untouched
    wide = poison(batch, M, F + 16, dtype=dtype)
    out = bmm.gated(x, ref.pack(wg), ref.pack(wu), act=act, out=wide[:, :, :F])
    assert torch.equal(out, H)
    assert torch.isnan(wide[:, :, F:]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_gated_activation_range(act, dtype):
    """Projections from far negative to far positive: X is a column of values,
    the weights pick it (gate) and 1 (up), so G is X exactly and H = act(X)."""
    v = torch.cat([torch.linspace(-40, 40, 2001), torch.tensor([0.0, -0.0, 1e-3, -1e-3, 3e4, -3e4])])
    v = v.to(dtype)
    x = torch.zeros(1, v.numel(), 16, dtype=dtype)
    x[0, :, 0], x[0, :, 1] = v, 1
    wg, wu = torch.zeros(1, 8, 16, dtype=dtype), torch.zeros(1, 8, 16, dtype=dtype)
    wg[:, :, 0], wu[:, :, 1] = 1, 1
    H = bmm.gated(x.cuda(), ref.pack(wg).cuda(), ref.pack(wu).cuda(), act=act)
    a, _ = ref.act(v.double(), act)
    a = a[None, :, None].expand(1, -1, 8)
    ref.check(H, a, a.abs() * ref.act_rel(v.double()[None, :, None], act), dtype, act)


def test_gated_two_dimensional_and_one_row_slice():
    x, wg, wu = inputs(3, 1, 9, 40, 64, BF, pad=8)
    a, b = ref.pack(wg), ref.pack(wu)
    full = bmm.gated(x, a, b)
    assert torch.equal(bmm.gated(x[0], a, b), full[0])
    assert torch.equal(bmm.gated(x[0, 4:5], a, b), full[0, 4:5])
    assert torch.equal(bmm.gated(x[0, 1::2], a, b), full[0, 1::2])   # every other row


def test_gated_empty():
    x, wg, wu = inputs(4, 1, 4, 16, 32, BF)
    a, b = ref.pack(wg), ref.pack(wu)
    assert bmm.gated(x[0, :0], a, b).shape == (0, 16)
    none = torch.empty(1, 2, 0, 8, 8, dtype=torch.int32, device="cuda")   # K = 0: the empty sum
    H, G, U = bmm.gated(torch.empty(5, 0, dtype=BF, device="cuda"), none, none, save=True)
    assert H.shape == (5, 16) and not H.any() and not G.any() and not U.any()
    none = torch.empty(1, 0, 2, 8, 8, dtype=torch.int32, device="cuda")   # F = 0
    assert bmm.gated(x, none, none).shape == (1, 4, 0)


def test_gated_keeps_rows_apart():
    """A NaN and an infinity in two rows of X reach those rows only."""
    x, wg, wu = inputs(5, 1, 150, 48, 96, BF)
    clean = bmm.gated(x, ref.pack(wg), ref.pack(wu))
    x = x.clone()
    x[0, 7, 3], x[0, 140, 95] = float("nan"), float("inf")
    H = bmm.gated(x, ref.pack(wg), ref.pack(wu))
    assert torch.isnan(H[0, 7]).all() and not torch.isfinite(H[0, 140]).any()
    keep = [r for r in range(150) if r not in (7, 140)]
    assert torch.equal(H[0, keep], clean[0, keep])


BACK = [  # (batch, M, F, K, pad)
    (1, 1, 8, 16, 0), (1, 1, 136, 512, 0), (1, 3, 24, 48, 8), (2, 17, 72, 80, 0),
    (1, 16, 64, 32, 0), (3, 5, 40, 1040, 24), (1, 33, 264, 272, 0), (1, 64, 512, 256, 0),
    (1, 130, 88, 96, 0), (2, 129, 200, 144, 40), (1, 300, 520, 336, 0), (1, 1025, 40, 48, 0),
    (1, 5003, 72, 80, 8), (1, 70, 1160, 528, 0), (1, 40, 4104, 64, 0),
]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(BACK)), ids=[str(s) for s in BACK])
def test_gated_backward(i, dtype):
    batch, M, F, K, pad = BACK[i]
    act = ACTS[i % 4]
    x, wg, wu = inputs(100 + i, batch, M, F, K, dtype, pad)
    gen = torch.Generator().manual_seed(i)
    dh, g, u = (torch.randn(batch, M, F, generator=gen).to(dtype).cuda() for _ in range(3))
    want = ref.gated_backward(*(t.double().cpu() for t in (dh, g, u, x, wg, wu)), act, dtype)
    got = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act=act)
    for o, (r, e), name in zip(got, want, ("dX", "dWg", "dWu")):
        ref.check(o, r, e, dtype, name)
    # one gradient at a time: the same bits
    dx, none, _ = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act=act, need_dw=False)
    assert none is None and torch.equal(dx, got[0])
    none, dwg, dwu = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act=act,
                                        need_dx=False)
    assert none is None and torch.equal(dwg, got[1]) and torch.equal(dwu, got[2])


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
def test_gated_backward_mean_error(dtype):
    """Over many independent terms the errors add up like their roots: those of
    dG and dU (each below a half step, root mean square below half a step over
    sqrt(2)) give every gradient that relative error, and its own rounding
    as much again; together below a half step of the gradients' norm."""
    x, wg, wu = inputs(50, 1, 300, 520, 336, dtype)
    gen = torch.Generator().manual_seed(50)
    dh, g, u = (torch.randn(1, 300, 520, generator=gen).to(dtype).cuda() for _ in range(3))
    want = ref.gated_backward(*(t.double().cpu() for t in (dh, g, u, x, wg, wu)), "silu", dtype)
    got = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu))
    for o, (r, _), name in zip(got, want, ("dX", "dWg", "dWu")):
        off = (o.double().cpu() - r).norm().item()
        assert off <= ref.half_step(dtype) * r.norm().item(), name


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_slopes(act):
    """Slopes over the whole range: with X = 1 in one column, dWg of single rows
    is dG of that row, so each row's slope is seen through its own rounding."""
    v = torch.cat([torch.linspace(-30, 30, 1016), torch.tensor([0.0, -0.0, 1e-3, -1e-3, 3e4, -3e4,
                                                                1e-6, -1e-6])]).to(BF)
    F = v.numel()
    x = torch.zeros(1, 1, 16, dtype=BF)
    x[0, 0, 0] = 1
    g, one = v[None, None].cuda(), torch.ones(1, 1, F, dtype=BF, device="cuda")
    w = ref.pack(torch.zeros(1, F, 16, dtype=BF)).cuda()
    _, dwg, dwu = bmm.gated_backward(one, g, one, x.cuda(), w, w, act=act)
    gd = v.double()
    a, slope = ref.act(gd, act)
    rel = ref.act_rel(gd, act)
    ref.check(dwg[0, :, 0], slope, (slope.abs() + gd.abs().clamp(max=64) + 1) * rel, BF, "slope")
    ref.check(dwu[0, :, 0], a, a.abs() * rel, BF, "value")
    assert not dwg[0, :, 1:].any() and not dwu[0, :, 1:].any()


def test_gated_backward_against_differences():
    """The gradients of sum(H * R) against central differences of the float64
    forward pass, in random directions."""
    x, wg, wu = inputs(11, 1, 40, 72, 64, BF)
    r = torch.randn(1, 40, 72, generator=torch.Generator().manual_seed(1)).to(BF)
    _, G, U = bmm.gated(x, ref.pack(wg), ref.pack(wu), act="gelu", save=True)
    grads = bmm.gated_backward(r.cuda(), G, U, x, ref.pack(wg), ref.pack(wu), act="gelu")
    leaves = [t.double().cpu() for t in (x, wg, wu)]

    def loss(ts):
        return (ref.gated(*ts, "gelu")[0][0] * r.double()).sum().item()

    gen = torch.Generator().manual_seed(2)
    for i in range(3):
        d = torch.randn(leaves[i].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        up = loss([t + step * d if k == i else t for k, t in enumerate(leaves)])
        down = loss([t - step * d if k == i else t for k, t in enumerate(leaves)])
        want = (up - down) / (2 * step)
        have = (grads[i].double().cpu() * d).sum().item()
        # each gradient element is off by at most a few half steps (its own
        # rounding, dG and dU, and the kept G and U) of independent sign
        spread = 6 * ref.half_step(BF) * (grads[i].double().cpu() * d).norm().item()
        assert abs(have - want) <= 4 * spread, (i, have, want, spread)


def test_gated_backward_empty():
    x, wg, wu = inputs(6, 1, 4, 16, 32, BF)
    a, b = ref.pack(wg), ref.pack(wu)
    h = torch.empty(0, 16, dtype=BF, device="cuda")
    dx, dwg, dwu = bmm.gated_backward(h, h, h, x[0, :0], a, b)     # no rows: weight gradients are 0
    assert dx.shape == (0, 32) and dwg.shape == (16, 32) and not dwg.any() and not dwu.any()
    none = torch.empty(1, 0, 2, 8, 8, dtype=torch.int32, device="cuda")
    h = torch.empty(1, 4, 0, dtype=BF, device="cuda")
    dx, dwg, _ = bmm.gated_backward(h, h, h, x, none, none)        # F = 0: dX is 0
    assert dwg.shape == (1, 0, 32) and not dx.any()


def test_gated_backward_strided_projections():
    """dH, G and U as column groups of one buffer."""
    x, wg, wu = inputs(7, 1, 37, 48, 64, HF)
    gen = torch.Generator().manual_seed(7)
    buf = torch.randn(1, 37, 3 * 48, generator=gen).to(HF).cuda()
    parts = [buf[:, :, 48 * i:48 * (i + 1)] for i in range(3)]
    a, b = ref.pack(wg), ref.pack(wu)
    got = bmm.gated_backward(*parts, x, a, b)
    want = bmm.gated_backward(*(p.contiguous() for p in parts), x, a, b)
    for o, w in zip(got, want):
        assert torch.equal(o, w)


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32 (X 4.6 GB apart, [dG | dU] 4.9 GB)."""
    M, ld, K, F = 72000, 32768, 16, 40
    buf = torch.empty(M, ld, dtype=BF, device="cuda")
    x = buf[:, :K]
    gen = torch.Generator(device="cuda").manual_seed(8)
    x.copy_(torch.randn(M, K, device="cuda", generator=gen).to(BF))
    _, wg, wu = inputs(8, 1, 1, F, K, BF)
    a, b = ref.pack(wg), ref.pack(wu)
    got, want = bmm.gated(x, a, b), bmm.gated(x.contiguous(), a, b)
    assert torch.equal(got, want)
    rows = torch.tensor([0, 1, 65535, 65536, M - 1])
    (h, eh), _, _ = ref.gated(x[rows].double().cpu(), wg[0].double().cpu(), wu[0].double().cpu(),
                              "silu")
    ref.check(got[rows], h, eh, BF, "H")
    dh = torch.randn(M, F, device="cuda", generator=gen).to(BF)
    _, G, U = bmm.gated(x, a, b, save=True)
    one = bmm.gated_backward(dh, G, U, x, a, b)
    two = bmm.gated_backward(dh, G, U, x.contiguous(), a, b)
    for p, q in zip(one, two):
        assert torch.equal(p, q)
    del buf, x, one, two
    M, F = 300000, 4096
    x = torch.randn(M, K, device="cuda", generator=gen).to(BF)
    _, wg, wu = inputs(9, 1, 1, F, K, BF)
    a, b = ref.pack(wg), ref.pack(wu)
    _, G, U = bmm.gated(x, a, b, save=True)
    dx, _, _ = bmm.gated_backward(G, G, U, x, a, b, need_dw=False)
    rows = torch.tensor([0, 131071, 131072, 262143, 262144, M - 1])
    G, U = G[rows], U[rows]
    want, _, _ = ref.gated_backward(*(t.double().cpu() for t in (G, G, U, x[rows], wg[0], wu[0])),
                                    "silu", BF)
    ref.check(dx[rows], *want, BF, "dX")


def test_another_stream_and_repeated_calls():
    """Work on a side stream, and the same bits from every call."""
    x, wg, wu = inputs(12, 1, 2050, 264, 528, BF)
    a, b = ref.pack(wg), ref.pack(wu)
    H, G, U = bmm.gated(x, a, b, save=True)
    first = bmm.gated_backward(H, G, U, x, a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            H2, G2, U2 = bmm.gated(x, a, b, save=True)
            again = bmm.gated_backward(H2, G2, U2, x, a, b)
    side.synchronize()
    assert torch.equal(H, H2)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_graph_replays():
    """Forward and backward captured in a HIP graph; every replay, with eager
    work in between, equals the eager result on the inputs of the moment."""
    x, wg, wu = inputs(13, 1, 515, 136, 272, BF)
    x = x.contiguous()
    a, b = ref.pack(wg), ref.pack(wu)
    ws = torch.empty(bmm.gated_backward_workspace_bytes(1, 515, 136, 272), dtype=torch.uint8,
                     device="cuda")

    def step():
        H, G, U = bmm.gated(x, a, b, save=True)
        return (H, *bmm.gated_backward(H, G, U, x, a, b, workspace=ws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in outs]
        for k, e in zip(kept, step()):
            assert torch.equal(k, e), i
        torch.cuda.synchronize()


def test_binding_refuses_on_the_gpu():
    x, wg, wu = inputs(14, 1, 4, 16, 32, BF)
    a, b = ref.pack(wg), ref.pack(wu)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        bmm.gated(x.float(), a, b)
    with pytest.raises(ValueError, match="unit innermost stride"):
        bmm.gated(x.transpose(1, 2), a, b)
    with pytest.raises(ValueError, match="disagree"):
        bmm.gated(x[:, :, :16], a, b)
    with pytest.raises(ValueError, match="differ in shape"):
        bmm.gated(x, a, b[:, :1].contiguous())
    with pytest.raises(ValueError, match="packed words"):
        bmm.gated(x, a[..., :4], b)
    with pytest.raises(ValueError, match="out must be"):
        bmm.gated(x, a, b, out=torch.empty(1, 4, 24, dtype=BF, device="cuda"))
    h = bmm.gated(x, a, b)
    with pytest.raises(ValueError, match="dH must be"):
        bmm.gated_backward(h[:, :3], h, h, x, a, b)
    with pytest.raises(bmm.BmmError, match="workspace_bytes"):
        bmm.gated_backward(h, h, h, x, a, b, workspace=torch.empty(16, dtype=torch.uint8,
                                                                   device="cuda"))
