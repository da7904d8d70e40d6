"""The feed-forward operators at sizes that take the large tiles, their ragged
edges, the splits of a long sum and the kernel for few rows, against 64-bit
references on the GPU with derived bounds (tests/ffn_ref.py)."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def block(seed, batch, M, F, K, dtype, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = normal(gen, batch, M, K + pad).to(dtype)[:, :, :K]
    wg, wu = ((normal(gen, batch, F, K) / math.sqrt(K)).to(dtype) for _ in range(2))
    return gen, x, wg, wu


GATED = [  # (batch, M, F, K, pad, dtype, act)
    (1, 1003, 5464, 2048, 64, HF, "gelu_tanh"), (1, 500, 8200, 4112, 0, BF, "silu"),
    (2, 1030, 4104, 2064, 8, BF, "gelu"), (1, 2051, 4104, 1040, 0, HF, "relu"),
    (1, 17, 1160, 2064, 0, BF, "silu"), (1, 49, 2056, 1040, 24, HF, "gelu"),
    (3, 64, 520, 272, 0, BF, "gelu_tanh"), (1, 2, 4104, 4112, 0, BF, "relu"),
    (1, 2000, 1544, 4112, 0, BF, "gelu"),
]


@pytest.mark.parametrize("i", range(len(GATED)), ids=[str(s[:4]) for s in GATED])
def test_gated(i):
    batch, M, F, K, pad, dtype, act = GATED[i]
    _, x, wg, wu = block(i, batch, M, F, K, dtype, pad)
    (h, eh), (g, eg), (u, eu) = ref.gated(x.double(), wg.double(), wu.double(), act)
    wide = torch.full((batch, M, F + 8), float("nan"), dtype=dtype, device="cuda")
    out = bmm.gated(x, ref.pack(wg), ref.pack(wu), act=act, out=wide[:, :, :F])
    ref.check(out, h, eh, dtype, "H")
    assert torch.isnan(wide[:, :, F:]).all()
    H, G, U = bmm.gated(x, ref.pack(wg), ref.pack(wu), act=act, save=True)
    assert torch.equal(H, out)
    ref.check(G, g, eg, dtype, "G")
    ref.check(U, u, eu, dtype, "U")


BACK = [  # (batch, M, F, K, pad, dtype, act)
    (1, 3001, 3080, 2064, 8, BF, "silu"), (1, 6000, 1032, 2064, 0, HF, "gelu"),
    (1, 12000, 1032, 1040, 0, BF, "gelu_tanh"), (2, 1500, 1032, 784, 0, HF, "relu"),
    (1, 20011, 264, 272, 24, BF, "silu"), (1, 700, 2056, 2048, 0, BF, "gelu"),
    # dX in two launches: whole rounds of large tiles, and the rows left
    (1, 8229, 1032, 2048, 8, HF, "silu"), (1, 4111, 1032, 4096, 0, BF, "gelu_tanh"),
    # tiles of 192 columns, with and without splits
    (1, 5000, 1408, 2048, 0, BF, "relu"), (1, 3000, 4104, 1536, 0, HF, "silu"),
]


@pytest.mark.parametrize("i", range(len(BACK)), ids=[str(s[:4]) for s in BACK])
def test_gated_backward(i):
    batch, M, F, K, pad, dtype, act = BACK[i]
    gen, x, wg, wu = block(100 + i, batch, M, F, K, dtype, pad)
    dh, g, u = (normal(gen, batch, M, F).to(dtype) for _ in range(3))
    want = ref.gated_backward(*(t.double() for t in (dh, g, u, x, wg, wu)), act, dtype)
    packed = ref.pack(wg), ref.pack(wu)
    got = bmm.gated_backward(dh, g, u, x, *packed, act=act)
    for o, (r, e), name in zip(got, want, ("dX", "dWg", "dWu")):
        ref.check(o, r, e, dtype, name)
    again = bmm.gated_backward(dh, g, u, x, *packed, act=act)
    for o, a in zip(got, again):
        assert torch.equal(o, a)


def operand(gen, rows, K, batch, spread=6):
    """A random 4-bit operand and its float64 values, both on the GPU."""
    n = max(batch, 1)
    code = torch.randint(0, 16, (n, rows, K), generator=gen, device="cuda")
    byte = torch.randint(125 - spread, 125 + spread, (n, rows, K // 32), generator=gen, device="cuda")
    parts = [ref.mx4_layout(code[b].cpu(), byte[b].cpu()) for b in range(n)]
    op = bmm.Mx4Operand(torch.cat([p[0] for p in parts]).cuda(),
                        torch.cat([p[1] for p in parts]).cuda(), rows, K, batch > 0)
    v = torch.stack([ref.mx4_values(code[b].cpu(), byte[b].cpu()) for b in range(n)]).cuda()
    return op, v if batch else v[0]


PRODUCTS = [  # (batch, M, N, K)
    (0, 1503, 8200, 4128), (0, 2051, 4104, 1056), (2, 1030, 2056, 544), (0, 40, 4104, 4128),
    (0, 64, 520, 160), (2, 23, 1160, 2080), (0, 13, 4104, 8224), (0, 1003, 10920, 4128),
]


@pytest.mark.parametrize("i", range(len(PRODUCTS)), ids=[str(s) for s in PRODUCTS])
def test_mx4_product(i):
    batch, M, N, K = PRODUCTS[i]
    gen = torch.Generator(device="cuda").manual_seed(200 + i)
    A, a = operand(gen, M, K, batch)
    B, b = operand(gen, N, K, batch)
    want, e = a @ b.transpose(-1, -2).contiguous(), ref.sum_error(a, b)
    for dtype in (torch.float32, BF, HF):
        wide = torch.full((*a.shape[:-1], N + 8), 7.0, dtype=dtype, device="cuda")
        ref.check(bmm.mx4_mma(A, B, dtype, out=wide[..., :N]), want, e, dtype, str(dtype))
        assert (wide[..., N:] == 7).all()


MX4_GATED = [  # (batch, M, F, K, dtype, act)
    (0, 1003, 8200, 2080, BF, "silu"), (0, 4095, 2056, 1056, HF, "gelu_tanh"),
    (2, 530, 1032, 288, BF, "gelu"), (0, 50, 2056, 4128, HF, "silu"), (0, 7, 4104, 4128, BF, "relu"),
    (0, 1003, 5464, 4128, BF, "gelu"),
]


@pytest.mark.parametrize("i", range(len(MX4_GATED)), ids=[str(s[:4]) for s in MX4_GATED])
def test_mx4_gated(i):
    batch, M, F, K, dtype, act = MX4_GATED[i]
    gen = torch.Generator(device="cuda").manual_seed(300 + i)
    X, x = operand(gen, M, K, batch, spread=2)
    shift = int(round(math.log2(math.sqrt(K)))) + 1      # projections of order 1
    ops = [operand(gen, F, K, batch, spread=2) for _ in range(2)]
    for w, _ in ops:
        w.scales.copy_(torch.where(w.scales > 0, w.scales - shift, w.scales))
    wg, wu = (v * 2.0 ** -shift for _, v in ops)
    (h, eh), _, _ = ref.gated(x, wg, wu, act)
    ref.check(bmm.mx4_gated(X, ops[0][0], ops[1][0], act=act, dtype=dtype), h, eh, dtype, act)


def test_nan_stays_in_its_row_and_column():
    """Rows of X with NaN and infinities in a large tile reach no other row, a
    NaN among the weights only its column."""
    _, x, wg, wu = block(7, 1, 1100, 2600, 2064, BF)
    clean = bmm.gated(x, ref.pack(wg), ref.pack(wu))
    x, wu = x.clone(), wu.clone()
    x[0, 255, 2063], x[0, 256, 0], x[0, 1099, 1000] = float("nan"), float("inf"), -float("inf")
    wu[0, 127, 5] = float("nan")
    H = bmm.gated(x, ref.pack(wg), ref.pack(wu))
    rows = [r for r in range(1100) if r not in (255, 256, 1099)]
    cols = [c for c in range(2600) if c != 127]
    assert torch.isnan(H[0, :, 127]).all() and torch.isnan(H[0, 255]).all()
    assert torch.equal(H[0][rows][:, cols], clean[0][rows][:, cols])
