"""Products by groups and of 8-bit integers at shapes that take every tile, unsplit and
split, and every way in which the rows' tiles are laid out: on whole numbers, bit for
bit. With operands of a few small whole numbers every partial sum is one that float32
holds, so only the result's own rounding is left (tests/ffn_sums.py)."""
import random

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16

# (groups, rows with the tail's, width, K)
MMA = [(4, 130, 128, 32), (4, 200, 48, 64), (1, 7000, 1080, 832), (1, 4100, 2832, 512),
       (3, 5000, 2984, 384), (24, 9000, 2984, 160)]
GATED = [(3, 130, 64, 32), (2, 130, 112, 32), (1, 1500, 2632, 864), (2, 5000, 1096, 512),
         (1, 3300, 2352, 352), (24, 9000, 1400, 160)]
MMA_BACK = [(24, 200, 56, 64), (2, 5000, 48, 32), (6, 5000, 488, 2080), (1, 4100, 400, 3808),
            (24, 130, 2272, 1344), (1, 7000, 1952, 1312), (24, 130, 1872, 960), (3, 130, 936, 32),
            (1, 2600, 752, 3104), (2, 4100, 504, 2720), (1, 5000, 232, 3328), (70, 9000, 520, 1360)]
GATED_BACK = [(8, 300, 40, 32), (3, 3300, 32, 32), (6, 7000, 200, 2016), (1, 7000, 1712, 288),
              (24, 130, 2248, 160), (1, 7000, 2400, 544), (24, 130, 616, 1472), (1, 130, 648, 32),
              (2, 4100, 440, 1824), (6, 7000, 2872, 160), (4, 7000, 296, 1440), (6, 7000, 2912, 288),
              (1, 5000, 144, 3328)]
I8_GROUPS = [(16, 130, 32, 32), (2, 300, 40, 96), (1, 5000, 1632, 1664), (2, 4100, 2864, 928),
             (2, 5000, 2976, 768), (24, 9000, 2984, 320)]
I8 = [(130, 32, 32), (300, 32, 32), (3300, 2320, 1664), (7000, 1696, 800), (7000, 2256, 640)]
I8_GATED_GROUPS = [(24, 200, 72, 32), (2, 130, 56, 160), (1, 2000, 2032, 1696), (1, 2600, 2248, 896),
                   (1, 2600, 3152, 544), (24, 9000, 1400, 320)]
I8_GATED = [(130, 112, 32), (2000, 2040, 1536), (2000, 3056, 800), (5000, 1480, 704)]


def counts_of(E, T, seed):
    """Groups of very different sizes, one in five without rows, and a tail of a few."""
    rng = random.Random(seed)
    tail = rng.choice([0, 3]) if T > 8 else 0
    chosen = [e for e in range(E) if E == 1 or rng.random() < 0.8] or [0]
    counts = [0] * E
    for e in rng.choices(chosen, [rng.random() ** 2 + 0.02 for _ in chosen], k=T - tail):
        counts[e] += 1
    return counts, tail


def whole(gen, top, *shape, dtype):
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").to(dtype)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def same(got, want, what):
    off = got != want.to(got.dtype)
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} differ"


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", MMA, ids=str)
def test_mma(shape, dtype):
    E, T, N, K = shape
    for seed in range(3):
        counts, tail = counts_of(E, T, seed)
        gen = gen_of(seed)
        x, w = whole(gen, 2, T, K, dtype=dtype), whole(gen, 2, E, N, K, dtype=dtype)
        want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        for e, r in gref.groups(counts):
            want[r] = x[r].double() @ w[e].double().t()
        same(bmm.grouped_mma(x, ref.pack(w), gref.ends_of(counts).cuda()), want, f"Y {seed}")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated(shape, dtype):
    E, T, F, K = shape
    for seed in range(2):
        counts, tail = counts_of(E, T, seed)
        gen = gen_of(seed)
        x = whole(gen, 1, T, K, dtype=dtype)
        wg, wu = (whole(gen, 1, E, F, K, dtype=dtype) for _ in range(2))
        g = torch.zeros(T, F, dtype=torch.float64, device="cuda")
        u = torch.zeros_like(g)
        for e, r in gref.groups(counts):
            g[r], u[r] = x[r].double() @ wg[e].double().t(), x[r].double() @ wu[e].double().t()
        H, G, U = bmm.grouped_gated(x, ref.pack(wg), ref.pack(wu), gref.ends_of(counts).cuda(),
                                    act="relu", save=True)
        same(G, g, "G")
        same(U, u, "U")
        same(H, g.float().clamp(min=0) * u.float(), "H")   # the product rounded to float32 first


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", MMA_BACK, ids=str)
def test_mma_backward(shape, dtype):
    E, T, N, K = shape
    for seed in range(2):
        counts, tail = counts_of(E, T, seed)
        gen = gen_of(seed)
        x, dy = whole(gen, 2, T, K, dtype=dtype), whole(gen, 2, T, N, dtype=dtype)
        w = whole(gen, 2, E, N, K, dtype=dtype)
        dx = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
        for e, r in gref.groups(counts):
            dx[r] = dy[r].double() @ w[e].double()
            dw[e] = dy[r].double().t().contiguous() @ x[r].double()
        args = dy, x, ref.pack(w), gref.ends_of(counts).cuda()
        dX, dW = bmm.grouped_mma_backward(*args)
        same(dX, dx, "dX")
        same(dW, dw, "dW")
        same(bmm.grouped_mma_backward(*args, need_dw=False)[0], dx, "dX alone")
        same(bmm.grouped_mma_backward(*args, need_dx=False)[1], dw, "dW alone")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", GATED_BACK, ids=str)
def test_gated_backward(shape, dtype):
    E, T, F, K = shape
    counts, tail = counts_of(E, T, 1)
    gen = gen_of(1)
    dh, g, u = (whole(gen, 2, T, F, dtype=dtype) for _ in range(3))
    x = whole(gen, 1, T, K, dtype=dtype)
    wg, wu = (whole(gen, 1, E, F, K, dtype=dtype) for _ in range(2))
    dg, du = (dh * u * (g > 0)).double(), (dh * g.clamp(min=0)).double()
    dx = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    dwg = torch.zeros(E, F, K, dtype=torch.float64, device="cuda")
    dwu = torch.zeros_like(dwg)
    for e, r in gref.groups(counts):
        dx[r] = dg[r] @ wg[e].double() + du[r] @ wu[e].double()
        dwg[e] = dg[r].t().contiguous() @ x[r].double()
        dwu[e] = du[r].t().contiguous() @ x[r].double()
    args = dh, g, u, x, ref.pack(wg), ref.pack(wu), gref.ends_of(counts).cuda()
    for kw in ({}, {"need_dw": False}, {"need_dx": False}):
        got = bmm.grouped_gated_backward(*args, act="relu", **kw)
        for o, want, what in zip(got, (dx, dwg, dwu), ("dX", "dWg", "dWu")):
            if o is not None:
                same(o, want, f"{what} {kw}")


def codes(seed, *shape):
    gen = gen_of(seed)
    q = torch.randint(-128, 128, shape, generator=gen, device="cuda").to(torch.int8)
    return q, torch.exp2(torch.randn(shape[:-1], generator=gen, device="cuda")) / 127


@pytest.mark.parametrize("dtype", [BF, HF, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", I8_GROUPS, ids=str)
def test_i8_groups(shape, dtype):
    E, T, N, K = shape
    counts, tail = counts_of(E, T, 2)
    (a, sa), (b, sb) = codes(1, T, K), codes(2, E, N, K)
    want = torch.zeros(T, N, dtype=dtype, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = gref.i8_mma(a[r], sa[r], b[e], sb[e], dtype)
    got = bmm.i8_mma(bmm.I8Operand(a, sa), bmm.I8Operand(gref.i8_pack(b), sb),
                     gref.ends_of(counts).cuda(), dtype=dtype)
    same(got, want, "D")


@pytest.mark.parametrize("dtype", [BF, HF, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", I8, ids=str)
def test_i8(shape, dtype):
    M, N, K = shape
    (a, sa), (b, sb) = codes(3, M, K), codes(4, 1, N, K)
    got = bmm.i8_mma(bmm.I8Operand(a, sa), bmm.I8Operand(gref.i8_pack(b), sb), dtype=dtype)
    same(got, gref.i8_mma(a, sa, b[0], sb[0], dtype), "D")


def i8_relu(a, sa, g, sg, u, su, dtype):
    gv, uv = (gref.i8_mma(a, sa, w, s, torch.float32) for w, s in ((g, sg), (u, su)))
    return (gv.clamp(min=0) * uv).to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", I8_GATED_GROUPS, ids=str)
def test_i8_gated_groups(shape, dtype):
    E, T, F, K = shape
    counts, tail = counts_of(E, T, 3)
    (a, sa), (g, sg), (u, su) = codes(5, T, K), codes(6, E, F, K), codes(7, E, F, K)
    sa = sa / K
    want = torch.zeros(T, F, dtype=dtype, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = i8_relu(a[r], sa[r], g[e], sg[e], u[e], su[e], dtype)
    got = bmm.i8_gated(bmm.I8Operand(a, sa), bmm.I8Operand(gref.i8_pack(g), sg),
                       bmm.I8Operand(gref.i8_pack(u), su), gref.ends_of(counts).cuda(), act="relu",
                       dtype=dtype)
    same(got, want, "H")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", I8_GATED, ids=str)
def test_i8_gated(shape, dtype):
    M, F, K = shape
    (a, sa), (g, sg), (u, su) = codes(8, M, K), codes(9, 1, F, K), codes(10, 1, F, K)
    sa = sa / K
    got = bmm.i8_gated(bmm.I8Operand(a, sa), bmm.I8Operand(gref.i8_pack(g), sg),
                       bmm.I8Operand(gref.i8_pack(u), su), act="relu", dtype=dtype)
    same(got, i8_relu(a, sa, g[0], sg[0], u[0], su[0], dtype), "H")


# Rows by group whose tiles are laid out in each way that the kernel knows (the host's
# copy of that rule and what each list takes: test_grouped_coverage.py).
LAYOUTS = [   # (rows of each group, width, K)
    ([1274, 1154, 1274], 2048, 1024), ([3070, 614], 2048, 1024), ([1228, 4096, 6274], 2048, 1024),
    ([512, 512, 0, 156, 253, 762], 4096, 1024), ([1478, 4196], 2048, 512),
    ([3, 514, 115, 484, 384, 676], 4096, 1024), ([210, 250, 0, 460, 1180, 1180], 4096, 512),
    ([1018, 762, 642, 403, 768, 0, 642, 156, 1018, 153], 4096, 1024),
    ([2298, 2048, 130, 3322, 2048, 130], 4096, 512), ([700, 100, 703, 800, 213, 700], 4096, 512),
    ([1274, 1666, 1154, 407, 250, 307, 1024, 437, 1636, 1536], 4096, 512),
    ([512, 512, 0, 403, 130, 153, 0, 250, 768, 153, 283, 515, 403, 253, 100, 768], 4096, 1024),
    ([703, 700, 340, 830, 3, 100, 1300, 800, 800, 1053], 4096, 512), ([129, 127] * 11, 4096, 512),
    ([8548], 4096, 512), ([634, 484, 676, 484, 576, 384], 4096, 512),
]


@pytest.mark.parametrize("counts,n,K", LAYOUTS, ids=lambda c: f"{len(c)}x{sum(c)}" if isinstance(c, list) else str(c))
def test_layouts(counts, n, K):
    """By tiles of 256 rows: every row made once, whatever the groups are."""
    E, T = len(counts), sum(counts) + 7
    gen = gen_of(E)
    x, w = whole(gen, 1, T, K, dtype=BF), whole(gen, 1, E, n, K, dtype=BF)
    want = torch.zeros(T, n, dtype=torch.float64, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = x[r].double() @ w[e].double().t()
    out = torch.full((T, n), float("nan"), dtype=BF, device="cuda")
    ends = gref.ends_of(counts).cuda()
    bmm.grouped_mma(x, ref.pack(w), ends, out=out)
    same(out[:-7], want[:-7], "Y")
    assert torch.isnan(out[-7:]).all()
    same(bmm.grouped_mma(x, ref.pack(w), ends), want, "Y, fresh")


# ---- sums of groups without rows ----

def some(E, filled, T):
    """T rows in `filled` of E groups, the last and the first without rows where they can be."""
    rng = random.Random(E + filled)
    chosen = rng.sample(range(1, E - 1), filled) if filled < E - 1 else range(filled)
    counts = [0] * E
    for e in [*chosen, *rng.choices(chosen, k=T - filled)][:T]:
        counts[e] += 1
    return counts


# (groups, those with rows, rows, N, K): a group's sums are less than, exactly and more than
# the 64 KB that are filled at a time
EMPTY = [(3, 1, 5, 128, 256), (64, 3, 40, 40, 48), (64, 63, 700, 40, 48), (65, 2, 2, 264, 272),
         (130, 40, 300, 264, 272), (130, 130, 300, 40, 48), (200, 199, 600, 24, 32),
         (9, 2, 4000, 264, 272), (1000, 5, 30, 264, 32)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", EMPTY, ids=str)
def test_empty_groups(shape, dtype):
    E, filled, T, N, K = shape
    counts = some(E, filled, T)
    gen, ends = gen_of(E + T), gref.ends_of(counts).cuda()
    x, dy = whole(gen, 2, T, K, dtype=dtype), whole(gen, 2, T, N, dtype=dtype)
    g, u = whole(gen, 1, T, N, dtype=dtype), whole(gen, 1, T, N, dtype=dtype)
    w = bmm.pack_operand(whole(gen, 2, E, N, K, dtype=dtype), 8)
    want, want_g, want_u = (torch.zeros(E, N, K, device="cuda") for _ in range(3))
    on = (g > 0).float()   # relu: dG = dH U there, dU = dH G
    for e, r in gref.groups(counts):
        xt = x[r].float().t().contiguous().t()
        want[e] = dy[r].float().t() @ xt
        want_g[e] = (dy[r].float() * u[r].float() * on[r]).t() @ xt
        want_u[e] = (dy[r].float() * g[r].float() * on[r]).t() @ xt
    for _ in range(2):   # (what an allocation held before)
        dirt = [torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda") for _ in range(3)]
        del dirt
        dw = bmm.grouped_mma_backward(dy, x, w, ends, need_dx=False)[1]
        same(dw, want, "dW")
        dirt = [torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda") for _ in range(3)]
        del dirt, dw
        _, dwg, dwu = bmm.grouped_gated_backward(dy, g, u, x, w, w, ends, act="relu", need_dx=False)
        same(dwg, want_g, "dWg")
        same(dwu, want_u, "dWu")


# (groups, rows, width, K): both gradients in one launch, whose tiles find room side by side
# (dX's few or long) or not
SIDE = [(16, 610, 512, 768), (8, 500, 768, 2048), (41, 216, 1352, 128), (24, 900, 640, 1024),
        (95, 105, 120, 1040)]


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", SIDE, ids=str)
def test_gradients_side_by_side(shape, dtype):
    for kind in ("mma", "gated"):
        E, T, N, K = shape
        assert all(bmm.group_plan(f"grouped_{kind}_{p}", E, T, N, K)[0] == "128x128"
                   for p in ("dx", "dw"))
    test_mma_backward(shape, dtype)
    test_gated_backward(shape, dtype)


# ---- the ends of the ranges ----

# (groups, rows, width, K)
ENDS = [(4096, 5000, 16, 32), (4096, 1, 8, 16), (2, 3, 8, 1 << 21), (2, 200, 8, 1 << 21),
        (3, 40, 1 << 20, 32), (2, 300, 1 << 20, 16)]


@pytest.mark.parametrize("shape", ENDS, ids=str)
def test_ends_of_the_ranges(shape):
    test_mma(shape, BF)
    test_mma_backward(shape, HF)
    test_gated(shape, HF)
    test_gated_backward(shape, BF)


def test_ends_of_the_ranges_in_8_bits():
    test_i8_groups((4096, 5000, 16, 32), BF)
    test_i8_groups((3, 40, 1 << 20, 32), torch.float32)
    test_i8((5, 1 << 20, 32), HF)
    test_i8_gated((200, 1 << 20, 32), BF)


@pytest.mark.parametrize("E,T,N,K", [(2, 300, 128, 64), (1, 4100, 2832, 512)])
def test_widest_rows(E, T, N, K):
    """Rows 2^21 elements apart, the most there may be: inputs and outputs."""
    counts, _ = counts_of(E, T, 0)
    ends, gen, wide = gref.ends_of(counts).cuda(), gen_of(7), 1 << 21

    def spread(t):
        out = torch.empty(T, wide, dtype=t.dtype, device="cuda")[:, 64:64 + t.shape[1]]
        return out.copy_(t)
    x, dy = whole(gen, 2, T, K, dtype=BF), whole(gen, 2, T, N, dtype=BF)
    w = ref.pack(whole(gen, 2, E, N, K, dtype=BF))
    far = spread(x)
    y = bmm.grouped_mma(x, w, ends, out=torch.full((T, N), 9, dtype=BF, device="cuda"))
    same(bmm.grouped_mma(far, w, ends, out=spread(torch.full((T, N), 9, dtype=BF, device="cuda"))),
         y.float(), "Y")
    h = bmm.grouped_gated(x, w, w, ends, act="relu")
    same(bmm.grouped_gated(far, w, w, ends, act="relu"), h.float(), "H")
    want = bmm.grouped_mma_backward(dy, x, w, ends)
    far_y = spread(dy)
    for a, b in zip(bmm.grouped_mma_backward(far_y, far, w, ends), want):
        same(a, b.float(), "gradients")
    want = bmm.grouped_gated_backward(dy, dy, dy, x, w, w, ends, act="relu")
    for a, b in zip(bmm.grouped_gated_backward(far_y, far_y, far_y, far, w, w, ends, act="relu"), want):
        same(a, b.float(), "gated gradients")
    del far, far_y
    q, s = codes(8, T, K)
    b, sb = codes(9, E, N, K)
    far = torch.empty(T, 2 * wide, dtype=torch.int8, device="cuda")[:, 64:64 + K].copy_(q)
    packed = bmm.i8_pack(bmm.I8Operand(b, sb))
    d = bmm.i8_mma(bmm.I8Operand(q, s), packed, ends)
    same(bmm.i8_mma(bmm.I8Operand(far, s), packed, ends), d, "8 bits")
