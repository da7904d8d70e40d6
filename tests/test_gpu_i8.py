"""8-bit integers on the GPU: codes, scales and products bit for bit against the
definitions (tests/grouped_ref.py), the gated block against 64 bits."""
import math

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = sorted(bmm.ACTS)


def same_bits(got, want):
    got, want = got.cpu(), want.cpu()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and \
        torch.equal(got.nan_to_num(0), want.nan_to_num(0))


# ---- quantisation ----

@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,K,pad", [
    (1, 32, 0), (1, 4096, 0), (3, 4128, 0), (5, 64, 8), (67, 288, 24), (2, 16384, 0), (3, 16416, 0),
    (1, 65536, 0), (2, 65568, 8), (1, 131072, 0), (258, 1056, 0)])
def test_quantize(rows, K, pad, dtype):
    gen = torch.Generator().manual_seed(rows + K)
    x = torch.randn(rows, K + pad, generator=gen) * torch.exp2(
        torch.randint(-6, 7, (rows, 1), generator=gen).float())
    x[:, ::7] = x.abs().amax(1, keepdim=True) / 2       # 63.5 exactly, or next to it
    x[:, 3] = 0
    x = x.to(dtype)
    codes, scales = gref.i8_quantize(x[:, :K])
    got = bmm.i8_quantize(x.cuda()[:, :K])
    assert got.codes.dtype == torch.int8 and got.codes.shape == (rows, K)
    assert torch.equal(got.codes.cpu().long(), codes)
    assert same_bits(got.scales, scales)


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "f16", "f32"])
def test_quantize_every_half(dtype):
    """Values at and next to every border between two codes."""
    top = torch.tensor([1.0, 127.0, 254.0, 1.9921875, 3.0, 100.0])[:, None]
    k = torch.arange(127).double()[None]
    half = (k + 0.5) * top.double() / 127
    near = half.to(dtype)
    steps = [near]
    for sign in (1, -1):
        bits = near.view(torch.int32 if dtype == F32 else torch.int16) + sign
        steps.append(bits.view(dtype))
    x = torch.cat([top.to(dtype), *steps, -near, torch.zeros(6, 416 - 1 - 4 * 127 + 128, dtype=dtype)], 1)
    x = torch.cat([x, torch.zeros(6, -x.shape[1] % 32, dtype=dtype)], 1).contiguous()
    codes, scales = gref.i8_quantize(x)
    got = bmm.i8_quantize(x.cuda())
    assert torch.equal(got.codes.cpu().long(), codes) and same_bits(got.scales, scales)


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "f16", "f32"])
def test_quantize_range(dtype):
    """Rows of the largest and the smallest numbers, of zeros, and with NaN and infinities."""
    info = torch.finfo(dtype)
    gen = torch.Generator().manual_seed(5)
    x = torch.rand(8, 64, generator=gen) * 2 - 1
    tiny = info.smallest_normal * info.eps
    scale = torch.tensor([info.max, info.max / 3, info.smallest_normal, info.smallest_normal * 5, 1.0,
                          1.0, 1.0, 1.0])
    x = (x.double() * scale.double()[:, None]).to(dtype)
    x[0, 0] = info.max
    x[4] = 0
    x[5, 9], x[6, 10], x[7, 11] = float("nan"), float("inf"), float("-inf")
    small = torch.zeros(2, 64, dtype=dtype)          # subnormal numbers
    small[0, :9] = (torch.arange(9).double() * tiny).to(dtype)
    small[1, 5] = tiny
    x = torch.cat([x, small, -small])
    codes, scales = gref.i8_quantize(x)
    got = bmm.i8_quantize(x.cuda())
    assert torch.equal(got.codes.cpu().long(), codes)
    assert same_bits(got.scales, scales)


def test_quantize_batched_and_empty():
    x = torch.randn(3, 5, 64).to(BF).cuda()
    got = bmm.i8_quantize(x)
    assert got.codes.shape == (3, 5, 64) and got.scales.shape == (3, 5)
    one = bmm.i8_quantize(x[1])
    assert torch.equal(got.codes[1], one.codes) and torch.equal(got.scales[1], one.scales)
    assert bmm.i8_quantize(x[:, :0]).codes.shape == (3, 0, 64)
    assert (bmm.i8_quantize(x[0, :, :0]).scales == 0).all()


def test_pack():
    q = bmm.i8_quantize(torch.randn(2, 24, 96, device="cuda"))
    w = bmm.i8_pack(q)
    assert torch.equal(w.codes, gref.i8_pack(q.codes)) and w.scales.shape == (2, 24)
    one = bmm.i8_pack(bmm.I8Operand(q.codes[1], q.scales[1]))
    assert torch.equal(one.codes[0], w.codes[1]) and one.scales.shape == (1, 24)


# ---- products ----

def operand(seed, *shape, device="cpu"):
    """Codes and scales, the extremes -128 and 127 among the codes."""
    gen = torch.Generator(device=device).manual_seed(seed)
    codes = torch.randint(-128, 128, shape, generator=gen, device=device).to(torch.int8)
    scales = torch.exp2(torch.randn(shape[:-1], generator=gen, device=device)) / 127
    return codes, scales


PRODUCTS = [  # (batch or 0, M, N, K)
    (0, 1, 8, 32), (0, 1, 136, 1024), (0, 3, 24, 64), (2, 17, 72, 96), (0, 16, 64, 32),
    (3, 5, 40, 1056), (0, 33, 264, 288), (0, 64, 512, 256), (0, 65, 88, 96), (0, 129, 136, 160),
    (2, 130, 200, 64), (0, 300, 520, 352), (0, 257, 1160, 2080), (0, 700, 2056, 64),
]


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("i", range(len(PRODUCTS)), ids=[str(s) for s in PRODUCTS])
def test_mma(i, dtype):
    batch, M, N, K = PRODUCTS[i]
    a, sa = operand(i, max(batch, 1), M, K)
    b, sb = operand(i + 50, max(batch, 1), N, K)
    want = torch.stack([gref.i8_mma(*t, dtype) for t in zip(a, sa, b, sb)])
    B = bmm.I8Operand(gref.i8_pack(b.cuda()), sb.cuda())
    A = bmm.I8Operand(*((a.cuda(), sa.cuda()) if batch else (a[0].cuda(), sa[0].cuda())))
    D = bmm.i8_mma(A, B, dtype=dtype)
    assert D.shape == ((batch, M, N) if batch else (M, N))
    assert torch.equal(D.cpu().reshape(want.shape), want)
    # rows of codes and of D further apart
    wide_a = torch.full((*a.shape[:2], K + 16), 99, dtype=torch.int8, device="cuda")
    wide_a[:, :, :K] = a.cuda()
    wide = torch.full((*want.shape[:2], N + 16), float("nan"), dtype=dtype, device="cuda")
    if not batch:
        wide_a, wide = wide_a[0], wide[0]
    bmm.i8_mma(bmm.I8Operand(wide_a[..., :K], A.scales), B, dtype=dtype, out=wide[..., :N])
    assert torch.equal(wide[..., :N], D) and torch.isnan(wide[..., N:]).all()


@pytest.mark.parametrize("M", [1, 20, 64, 200])
def test_longest_sum(M):
    """Every product the largest there is: the sum stays below 2^31."""
    K, N = 131040, 24
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(M, device="cuda")
    D = bmm.i8_mma(bmm.I8Operand(a, one), bmm.I8Operand(gref.i8_pack(b), torch.ones(1, N, device="cuda")))
    assert (D == float(torch.tensor(128 * 128 * K).float())).all()


GATED = [(0, 1, 8, 32), (0, 7, 136, 1024), (2, 17, 72, 96), (0, 33, 264, 288), (0, 64, 64, 64),
         (0, 129, 136, 160), (2, 130, 200, 64), (0, 300, 520, 352), (0, 700, 1032, 64)]


def gated_reference(a, sa, g, sg, u, su, act):
    """(h, bound) from the projections as stated, bit for bit, and the activation in 64 bits."""
    gv, uv = gref.i8_mma(a, sa, g, sg, F32).double(), gref.i8_mma(a, sa, u, su, F32).double()
    h = ref.act(gv, act)[0] * uv
    return h, h.abs() * ref.act_rel(gv, act)


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(GATED)), ids=[str(s) for s in GATED])
def test_gated(i, dtype):
    batch, M, F, K = GATED[i]
    act = ACTS[i % 4]
    (a, sa), (g, sg), (u, su) = (operand(i + 10 * j, max(batch, 1), n, K)
                                 for j, n in enumerate((M, F, F)))
    sa = sa / math.sqrt(K)
    refs = [gated_reference(*t, act) for t in zip(a, sa, g, sg, u, su)]
    X = bmm.I8Operand(*((a.cuda(), sa.cuda()) if batch else (a[0].cuda(), sa[0].cuda())))
    ws = [bmm.I8Operand(gref.i8_pack(w.cuda()), s.cuda()) for w, s in ((g, sg), (u, su))]
    H = bmm.i8_gated(X, *ws, act=act, dtype=dtype)
    want, err = (torch.stack([r[j] for r in refs]) for j in range(2))
    ref.check(H.reshape(want.shape), want, err, dtype, "H")
    wide = torch.full((*H.shape[:-1], F + 8), float("nan"), dtype=dtype, device="cuda")
    assert torch.equal(bmm.i8_gated(X, *ws, act=act, dtype=dtype, out=wide[..., :F]), H)
    assert torch.isnan(wide[..., F:]).all()


GROUPS = [  # (rows of each group, rows behind the last, N, K)
    ([1], 0, 8, 32), ([0, 1, 0], 2, 136, 512), ([3, 0, 17, 1, 0], 0, 72, 96), ([16, 15, 17], 5, 64, 32),
    ([1] * 70, 1, 40, 96), ([5, 0, 33, 64, 1], 0, 264, 288), ([40, 0, 30, 64, 33], 3, 104, 160), ([60, 0, 64, 129, 2], 3, 104, 160),
    ([21, 18, 0, 25] * 5, 1, 264, 160), ([127, 128, 129, 0, 256, 1], 30, 136, 160),
    ([1000, 3, 0, 40], 77, 520, 352), ([300, 500, 2, 600], 0, 1160, 544),
]
GROUP_IDS = [f"{len(s[0])}x{sum(s[0])}+{s[1]}_{s[2]}x{s[3]}" for s in GROUPS]


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("i", range(len(GROUPS)), ids=GROUP_IDS)
def test_groups(i, dtype):
    counts, tail, N, K = GROUPS[i]
    T, E = sum(counts) + tail, len(counts)
    a, sa = operand(i, T, K)
    sa[sum(counts):] = float("nan")
    b, sb = operand(i + 50, E, N, K)
    want = torch.zeros(T, N, dtype=dtype)
    for e, r in gref.groups(counts):
        want[r] = gref.i8_mma(a[r], sa[r], b[e], sb[e], dtype)
    A, B = bmm.I8Operand(a.cuda(), sa.cuda()), bmm.I8Operand(gref.i8_pack(b.cuda()), sb.cuda())
    ends = gref.ends_of(counts).cuda()
    assert torch.equal(bmm.i8_mma(A, B, ends, dtype=dtype).cpu(), want)
    out = torch.full((T, N), float("nan"), dtype=dtype, device="cuda")
    bmm.i8_mma(A, B, ends, dtype=dtype, out=out)
    assert torch.equal(out[:sum(counts)].cpu(), want[:sum(counts)])
    assert torch.isnan(out[sum(counts):]).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(GROUPS)), ids=GROUP_IDS)
def test_gated_groups(i, dtype):
    counts, tail, F, K = GROUPS[i]
    T, E, act = sum(counts) + tail, len(counts), ACTS[(i + 1) % 4]
    a, sa = operand(i, T, K)
    sa = sa / math.sqrt(K)
    sa[sum(counts):] = float("inf")
    (g, sg), (u, su) = operand(i + 20, E, F, K), operand(i + 30, E, F, K)
    want, err = torch.zeros(T, F, dtype=torch.float64), torch.zeros(T, F, dtype=torch.float64)
    for e, r in gref.groups(counts):
        want[r], err[r] = gated_reference(a[r], sa[r], g[e], sg[e], u[e], su[e], act)
    ws = [bmm.I8Operand(gref.i8_pack(w.cuda()), s.cuda()) for w, s in ((g, sg), (u, su))]
    H = bmm.i8_gated(bmm.I8Operand(a.cuda(), sa.cuda()), *ws, gref.ends_of(counts).cuda(), act=act,
                     dtype=dtype)
    ref.check(H, want, err, dtype, "H")
    assert (H[sum(counts):] == 0).all()


def test_nan_scales_and_empty():
    a, sa = operand(1, 5, 64, device="cuda")
    b, sb = operand(2, 1, 24, 64, device="cuda")
    sa[2] = float("nan")
    B = bmm.I8Operand(gref.i8_pack(b), sb)
    D = bmm.i8_mma(bmm.I8Operand(a, sa), B)
    assert torch.isnan(D[2]).all() and torch.isfinite(D[[0, 1, 3, 4]]).all()
    assert bmm.i8_mma(bmm.I8Operand(a[:0], sa[:0]), B).shape == (0, 24)
    none = bmm.I8Operand(torch.empty(1, 3, 0, 8, 8, dtype=torch.int32, device="cuda"), sb)
    D = bmm.i8_mma(bmm.I8Operand(a[:, :0], torch.ones(5, device="cuda")), none)
    assert D.shape == (5, 24) and (D == 0).all()


def test_one_row_and_every_other_row():
    a, sa = operand(3, 9, 64, device="cuda")
    b, sb = operand(4, 1, 40, 64, device="cuda")
    B = bmm.I8Operand(gref.i8_pack(b), sb)
    full = bmm.i8_mma(bmm.I8Operand(a, sa), B)
    assert torch.equal(bmm.i8_mma(bmm.I8Operand(a[4:5], sa[4:5]), B), full[4:5])
    assert torch.equal(bmm.i8_mma(bmm.I8Operand(a[1::2], sa[1::2].contiguous()), B), full[1::2])


def test_quantize_rows_of_many_launches():
    """2^26 + 5 rows: more threads than one launch may have. Row r holds r % 251 + 1."""
    rows, K = (1 << 26) + 5, 32
    index = torch.arange(rows, device="cuda", dtype=torch.int32) % 251
    value = (index + 1).to(torch.bfloat16)
    codes, scales = bmm.i8_quantize(value[:, None].expand(rows, K).contiguous())
    assert bool((codes.view(torch.int32) == 0x7f7f7f7f).all())
    # (divided on the CPU: on the GPU a number as divisor is multiplied by its reciprocal)
    want = (torch.arange(1, 252, dtype=torch.float32) / torch.tensor(127.0)).cuda()
    assert torch.equal(scales, want[index])
