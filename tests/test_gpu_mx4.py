"""4-bit floats on the GPU: quantisation and back bit for bit against the
format's definition in 64 bits, products and the gated block within derived
bounds (tests/ffn_ref.py)."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
F32, BF, HF = torch.float32, torch.bfloat16, torch.float16
NAMES = {F32: "f32", BF: "bf16", HF: "f16"}


def assert_operand(op, x64):
    """Codes and scales, padding included, equal the definition's."""
    code, byte = ref.mx4_quantize(x64)
    codes, scales = ref.mx4_layout(code, byte)
    assert torch.equal(op.scales.cpu(), scales)
    assert torch.equal(op.codes.cpu(), codes)
    return code, byte


@pytest.mark.parametrize("dtype", [F32, BF, HF], ids=NAMES.get)
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (1, 16384, 0), (3, 96, 8), (16, 128, 0),
                                        (17, 160, 24), (33, 544, 0), (130, 2080, 0)])
def test_quantize(rows, K, pad, dtype):
    gen = torch.Generator().manual_seed(rows * K)
    x = torch.randn(rows, K + pad, generator=gen)
    x *= torch.exp2(torch.randint(-12, 9, (rows, 1), generator=gen))
    x = torch.where(torch.rand(x.shape, generator=gen) < 0.1, 0.0, x).to(dtype)
    x[:, :32][rows // 2] = 0
    dev = x.cuda()[:, :K]
    op = bmm.mx4_quantize(dev)
    code, byte = assert_operand(op, dev.double().cpu())
    for to in (F32, BF, HF):
        wide = torch.full((rows, K + 8), 7.0, dtype=to, device="cuda")
        got = bmm.mx4_dequantize(op, to, out=wide[:, :K])
        assert torch.equal(got.cpu(), ref.mx4_values(code, byte).to(to))
        assert (wide[:, K:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=NAMES.get)
def test_quantize_every_16_bit_value(dtype):
    """Each of the 65536 values beside a maximum that makes it meet every step:
    as the block's largest, and under larger ones."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = torch.zeros(65536, 64, dtype=dtype)
    x[:, 5] = bits
    x[:, 40] = bits
    x[:, 32] = bits * 4       # the same block, its largest value four times this one
    op = bmm.mx4_quantize(x.cuda())
    code, byte = assert_operand(op, x.double())
    got = bmm.mx4_dequantize(op, F32).cpu()
    want = ref.mx4_values(code, byte).to(F32)
    assert torch.equal(got.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


def test_quantize_float32_edges():
    """Ties, values next to them, the largest and the smallest scales,
    subnormals, and blocks with NaN and infinities."""
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9999995])
    near = torch.cat([grid, torch.nextafter(grid, grid * 0), torch.nextafter(grid, grid * 2)])
    rows = []
    for e in (-149, -140, -130, -129, -128, -127, -126, -60, 0, 60, 120, 124):
        block = torch.zeros(32)
        block[:30] = near
        block[30] = 4.0
        rows.append(torch.ldexp(block.double(), torch.tensor(e)).float() * torch.tensor([1, -1] * 16))
    special = torch.zeros(7, 32)
    special[0, 3] = float("nan")
    special[1, 31] = float("inf")
    special[2, 0] = -float("inf")
    special[3] = torch.finfo(F32).max
    special[4, 9] = torch.finfo(F32).smallest_normal / 4
    special[5] = -0.0
    x = torch.cat([torch.stack(rows), special])
    op = bmm.mx4_quantize(x.cuda())
    code, byte = assert_operand(op, x.double())
    got = bmm.mx4_dequantize(op, F32).cpu()
    want = ref.mx4_values(code, byte).to(F32)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(want).any()
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


def test_quantize_batched_and_empty():
    x = torch.randn(3, 20, 160, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    op = bmm.mx4_quantize(x)
    for b in range(3):
        one = bmm.mx4_quantize(x[b])
        assert torch.equal(op.codes[b], one.codes[0]) and torch.equal(op.scales[b], one.scales[0])
    assert torch.equal(bmm.mx4_dequantize(op, BF)[1], bmm.mx4_dequantize(bmm.mx4_quantize(x[1]), BF))
    none = bmm.mx4_quantize(x[0, :0])
    assert none.codes.numel() == 0 and bmm.mx4_dequantize(none).shape == (0, 160)
    none = bmm.mx4_quantize(x[0, :, :0])
    assert bmm.mx4_dequantize(none).shape == (20, 0)


def operand(seed, rows, K, batch=0):
    """A random 4-bit operand on the GPU and its float64 values."""
    gen = torch.Generator().manual_seed(seed)
    n = max(batch, 1)
    code = torch.randint(0, 16, (n, rows, K), generator=gen)
    byte = torch.randint(118, 132, (n, rows, K // 32), generator=gen)
    parts = [ref.mx4_layout(code[b], byte[b]) for b in range(n)]
    op = bmm.Mx4Operand(torch.cat([p[0] for p in parts]).cuda(),
                        torch.cat([p[1] for p in parts]).cuda(), rows, K, batch > 0)
    v = torch.stack([ref.mx4_values(code[b], byte[b]) for b in range(n)])
    return op, v if batch else v[0]


PRODUCTS = [  # (batch, M, N, K)
    (0, 1, 8, 32), (0, 1, 136, 512), (0, 3, 24, 96), (2, 17, 72, 160), (0, 16, 64, 128),
    (3, 5, 40, 2080), (0, 33, 264, 544), (0, 64, 512, 256), (0, 65, 88, 1120), (0, 130, 136, 640),
    (2, 129, 200, 64), (0, 300, 520, 672), (0, 257, 1160, 4128), (0, 700, 2056, 96),
]


@pytest.mark.parametrize("i", range(len(PRODUCTS)), ids=[str(s) for s in PRODUCTS])
def test_product(i):
    batch, M, N, K = PRODUCTS[i]
    A, a = operand(i, M, K, batch)
    B, b = operand(1000 + i, N, K, batch)
    want, e = a @ b.transpose(-1, -2), ref.sum_error(a, b)
    for dtype in (F32, BF, HF):
        wide = torch.full((*a.shape[:-1], N + 8), 7.0, dtype=dtype, device="cuda")
        got = bmm.mx4_mma(A, B, dtype, out=wide[..., :N])
        ref.check(got, want, e, dtype, NAMES[dtype])
        assert (wide[..., N:] == 7).all()


def test_product_is_exact_on_one_scale():
    """With one scale for all blocks every partial sum is a multiple of 1/4
    below 2^22: float32 holds them all, so the product is exact."""
    gen = torch.Generator().manual_seed(5)
    ca, cb = (torch.randint(0, 16, (n, 1056), generator=gen) for n in (200, 264))
    one = torch.full((264, 33), 127)
    A = bmm.Mx4Operand(*(t.cuda() for t in ref.mx4_layout(ca, one[:200])), 200, 1056)
    B = bmm.Mx4Operand(*(t.cuda() for t in ref.mx4_layout(cb, one)), 264, 1056)
    want = ref.mx4_values(ca, one[:200]) @ ref.mx4_values(cb, one).t()
    assert torch.equal(bmm.mx4_mma(A, B).double().cpu(), want)


@pytest.mark.parametrize("M", [7, 150])
def test_product_nan_blocks(M):
    """A NaN scale reaches its row of D (or column) and no other."""
    A, a = operand(1, M, 256)
    B, b = operand(2, 72, 256)
    a, b = a.clone(), b.clone()
    A.scales[0, 0, 0, 2, 5, 1] = 255      # row 5, K values 192 ..
    B.scales[0, 4, 0, 0, 2, 0] = 255      # row 66, K values 0 ..
    got = bmm.mx4_mma(A, B).cpu()
    want = a @ b.t()
    nan = torch.zeros(M, 72, dtype=torch.bool)
    nan[5], nan[:, 66] = True, True
    assert torch.equal(torch.isnan(got), nan)
    e = ref.sum_error(a, b)
    assert ((got.double() - want).abs() <= ref.rounded(want, e, F32))[~nan].all()


GATED = [(0, 1, 8, 32), (0, 1, 136, 512), (2, 17, 72, 160), (0, 7, 520, 1024), (0, 64, 264, 544),
         (0, 65, 88, 1120), (2, 129, 200, 64), (0, 257, 1160, 2080)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=NAMES.get)
@pytest.mark.parametrize("i", range(len(GATED)), ids=[str(s) for s in GATED])
def test_mx4_gated(i, dtype):
    batch, M, F, K = GATED[i]
    act = sorted(bmm.ACTS)[i % 4]
    X, x = operand(i, M, K, batch)
    (Wg, wg), (Wu, wu) = (operand(s + i, F, K, batch) for s in (100, 200))
    # weights scaled so that the projections are of order 1
    shift = int(round(math.log2(math.sqrt(K)))) + 2
    for w in (Wg, Wu):
        w.scales.copy_(torch.where(w.scales > 0, w.scales - shift, w.scales))
    wg, wu = wg * 2.0 ** -shift, wu * 2.0 ** -shift
    (h, eh), _, _ = ref.gated(x, wg, wu, act)
    wide = torch.full((*x.shape[:-1], F + 8), 7.0, dtype=dtype, device="cuda")
    got = bmm.mx4_gated(X, Wg, Wu, act=act, dtype=dtype, out=wide[..., :F])
    ref.check(got, h, eh, dtype, act)
    assert (wide[..., F:] == 7).all()


def test_products_of_nothing():
    A, _ = operand(1, 4, 64)
    B, _ = operand(2, 16, 64)
    nil = bmm.Mx4Operand(A.codes[:, :0], A.scales[:, :0], 0, 64)
    assert bmm.mx4_mma(nil, B).shape == (0, 16) and bmm.mx4_mma(A, nil).shape == (4, 0)
    k0 = [bmm.Mx4Operand(torch.empty(1, 1, 0, 4, 16, 16, dtype=torch.uint8, device="cuda"),
                         torch.empty(1, 1, 0, 4, 16, 4, dtype=torch.uint8, device="cuda"), r, 0)
          for r in (4, 16)]
    assert not bmm.mx4_mma(*k0).any() and bmm.mx4_mma(*k0).shape == (4, 16)
    assert not bmm.mx4_gated(k0[0], k0[1], k0[1]).any()


def test_chain_in_a_graph():
    """Quantise, gate, quantise, multiply: captured once, replayed on changing
    inputs with eager work in between."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(70, 256, generator=gen).to(BF).cuda()
    Wg, Wu, Wd = (bmm.mx4_quantize((torch.randn(n, k, generator=gen) / math.sqrt(k)).to(BF).cuda())
                  for n, k in ((96, 256), (96, 256), (256, 96)))

    def step():
        h = bmm.mx4_gated(bmm.mx4_quantize(x), Wg, Wu)
        return h, bmm.mx4_mma(bmm.mx4_quantize(h), Wd, BF)

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
