"""Every tile that the feed-forward products can be made by, with ragged edges, in
every element type, against 64-bit references on the GPU (tests/ffn_ref.py). That the
lists reach every tile is tests/test_ffn_coverage.py's matter."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests.test_gpu_ffn_large import block, normal, operand

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
ACTS = sorted(bmm.ACTS)


def ids(shapes):
    return ["x".join(map(str, s)) for s in shapes]


GATED = [(641, 5400, 816), (905, 5928, 432), (6321, 1224, 304), (4095, 5464, 2064)]  # (M, F, K)


@TYPES
@pytest.mark.parametrize("i", range(len(GATED)), ids=ids(GATED))
def test_gated(i, dtype):
    M, F, K = GATED[i]
    act = ACTS[i % 4]
    _, x, wg, wu = block(400 + i, 1, M, F, K, dtype, 8 * (i % 2))
    (h, eh), (g, eg), (u, eu) = ref.gated(x.double(), wg.double(), wu.double(), act)
    wide = torch.full((1, M, F + 8), float("nan"), dtype=dtype, device="cuda")
    out = bmm.gated(x, ref.pack(wg), ref.pack(wu), act=act, out=wide[:, :, :F])
    ref.check(out, h, eh, dtype, "H")
    assert torch.isnan(wide[:, :, F:]).all()
    H, G, U = bmm.gated(x, ref.pack(wg), ref.pack(wu), act=act, save=True)
    assert torch.equal(H, out)
    ref.check(G, g, eg, dtype, "G")
    ref.check(U, u, eu, dtype, "U")


@TYPES
def test_nan_stays_in_its_row_and_column(dtype):
    """As the test of that name, on the largest tile: faults in the rows on both sides
    of a tile's edge and in the last one, in the last summed value, and in the columns
    on both sides of a tile's edge."""
    M, F, K = 4095, 5464, 2064
    assert bmm.ffn_plan("gated", 1, M, F, K)[0] == "256x256"
    _, x, wg, wu = block(7, 1, M, F, K, dtype)
    clean = bmm.gated(x, ref.pack(wg), ref.pack(wu))
    x, wg, wu = x.clone(), wg.clone(), wu.clone()
    x[0, 255, K - 1], x[0, 256, 0], x[0, M - 1, 1000] = float("nan"), float("inf"), -float("inf")
    wu[0, 127, 5], wg[0, 128, K - 1] = float("nan"), float("nan")
    H = bmm.gated(x, ref.pack(wg), ref.pack(wu))
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(F, dtype=torch.bool)
    rows[[255, 256, M - 1]], cols[[127, 128]] = False, False
    assert torch.isnan(H[0, :, [127, 128]]).all() and torch.isnan(H[0, 255]).all()
    assert torch.equal(H[0][rows.cuda()][:, cols.cuda()], clean[0][rows.cuda()][:, cols.cuda()])


BACK = [  # (M, F, K)
    # dWg and dWu by each tile, with one sum and with split ones
    (759, 8168, 400), (5515, 2632, 144), (321, 4568, 1296), (8713, 2696, 144), (225, 2936, 2768),
    (6609, 8856, 208),
    # dX so
    (8161, 392, 912), (133, 5352, 2576), (8847, 264, 1200), (6029, 3960, 144), (8841, 248, 1552),
    (8929, 3272, 400),
    # dX in two launches
    (5087, 600, 4048), (4881, 936, 3280), (6065, 440, 4080), (5271, 1800, 3504), (6977, 792, 3856),
]


@TYPES
@pytest.mark.parametrize("i", range(len(BACK)), ids=ids(BACK))
def test_gated_backward(i, dtype):
    M, F, K = BACK[i]
    act = ACTS[i % 4]
    gen, x, wg, wu = block(500 + i, 1, M, F, K, dtype, 8 * (i % 2))
    dh, g, u = (normal(gen, 1, M, F).to(dtype) for _ in range(3))
    want = ref.gated_backward(*(t.double() for t in (dh, g, u, x, wg, wu)), act, dtype)
    got = bmm.gated_backward(dh, g, u, x, ref.pack(wg), ref.pack(wu), act=act)
    for o, (r, e), name in zip(got, want, ("dX", "dWg", "dWu")):
        ref.check(o, r, e, dtype, name)


PRODUCTS = [(1187, 6328, 3232), (8695, 1304, 1568), (5253, 3048, 1184)]   # (M, N, K)


@pytest.mark.parametrize("i", range(len(PRODUCTS)), ids=ids(PRODUCTS))
def test_mx4_product(i):
    M, N, K = PRODUCTS[i]
    gen = torch.Generator(device="cuda").manual_seed(600 + i)
    A, a = operand(gen, M, K, 0)
    B, b = operand(gen, N, K, 0)
    want, e = a @ b.t().contiguous(), ref.sum_error(a, b)
    for dtype in (torch.float32, BF, HF):
        wide = torch.full((M, N + 8), 7.0, dtype=dtype, device="cuda")
        ref.check(bmm.mx4_mma(A, B, dtype, out=wide[:, :N]), want, e, dtype, str(dtype))
        assert (wide[:, N:] == 7).all()


MX4_GATED = [(417, 8136, 3232), (1459, 3928, 1696), (975, 8104, 1184)]    # (M, F, K)


@pytest.mark.parametrize("i", range(len(MX4_GATED)), ids=ids(MX4_GATED))
def test_mx4_gated(i):
    M, F, K = MX4_GATED[i]
    act = ACTS[i % 4]
    gen = torch.Generator(device="cuda").manual_seed(700 + i)
    X, x = operand(gen, M, K, 0, spread=2)
    shift = int(round(math.log2(math.sqrt(K)))) + 1      # projections of order 1
    ops = [operand(gen, F, K, 0, spread=2) for _ in range(2)]
    for w, _ in ops:
        w.scales.copy_(torch.where(w.scales > 0, w.scales - shift, w.scales))
    wg, wu = (v * 2.0 ** -shift for _, v in ops)
    (h, eh), _, _ = ref.gated(x, wg, wu, act)
    for dtype in (BF, HF):
        wide = torch.full((M, F + 8), 7.0, dtype=dtype, device="cuda")
        got = bmm.mx4_gated(X, ops[0][0], ops[1][0], act=act, dtype=dtype, out=wide[:, :F])
        ref.check(got, h, eh, dtype, act)
        assert (wide[:, F:] == 7).all()
