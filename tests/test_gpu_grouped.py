"""Products by groups of rows on the GPU, forward and backward, against 64-bit
references with derived bounds (tests/grouped_ref.py, tests/ffn_ref.py)."""
import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
ACTS = sorted(bmm.ACTS)


def spread(E, each, last=0):
    """E groups of about so many rows, odd and different."""
    return [each + (7 * e) % 5 - 2 if each > 2 else each for e in range(E - 1)] + [last]


SHAPES = [  # (rows of each group, rows behind the last, N, K, columns beside X)
    ([1], 0, 8, 16, 0),                                  # one row of one group
    ([0, 1, 0], 0, 136, 512, 0),
    ([0, 0], 3, 24, 48, 8),                              # nothing but the tail
    ([3, 0, 17, 1, 0], 2, 72, 80, 0),
    ([16, 15, 17], 0, 64, 32, 24),                       # at the few-rows blocks' edges
    ([5, 0, 33, 64, 1], 9, 264, 272, 0),
    ([1] * 70, 1, 40, 96, 8),                            # more groups than lanes
    (spread(130, 3, 40), 0, 24, 48, 0),
    ([0] * 63 + [9] + [0] * 63 + [2], 5, 56, 64, 0),
    ([127, 128, 129, 0, 256, 1], 30, 136, 144, 40),      # at the tiles' edges
    ([255, 257, 300], 0, 200, 64, 0),
    ([40, 0, 30, 64, 33], 3, 104, 160, 8),
    ([60, 0, 64, 129, 2], 3, 104, 160, 0),               # few rows in blocks of 64
    (spread(20, 20, 33), 1, 264, 144, 0),
    ([1000, 3, 0, 40], 77, 520, 336, 0),                 # one group much larger
    ([300, 500, 2, 600], 0, 1160, 528, 0),
    ([700, 0, 690], 130, 2056, 48, 8),
]
IDS = [f"{len(s[0])}x{sum(s[0])}+{s[1]}_{s[2]}x{s[3]}" for s in SHAPES]


def inputs(seed, shape, dtype, n_weights=1):
    counts, tail, N, K, pad = shape
    gen = torch.Generator().manual_seed(seed)
    x = gref.matrix(gen, sum(counts) + tail, K, pad, dtype)
    x[sum(counts):] = float("nan")                       # nothing there is read
    return x, [gref.weights(gen, len(counts), N, K, dtype) for _ in range(n_weights)], gen


def clean(x, counts):
    """float64, with zeros in the tail's place."""
    x = x.double()
    x[sum(counts):] = 0
    return x


def poison(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_mma(i, dtype):
    counts, tail, N, K, pad = SHAPES[i]
    x, (w,), _ = inputs(i, SHAPES[i], dtype)
    y, e = gref.mma(clean(x, counts), w.double(), counts)
    X, W, ends = x.cuda(), ref.pack(w.cuda()), gref.ends_of(counts).cuda()
    Y = bmm.grouped_mma(X, W, ends)
    ref.check(Y, y, e, dtype, "Y")
    assert (Y[sum(counts):] == 0).all()
    # the same bits in rows wider than N; what is beside them and behind the groups stays
    wide = poison(sum(counts) + tail, N + 16, dtype=dtype)
    out = bmm.grouped_mma(X, W, ends, out=wide[:, :N])
    assert torch.equal(out[:sum(counts)], Y[:sum(counts)])
    assert torch.isnan(wide[:, N:]).all() and torch.isnan(wide[sum(counts):]).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_gated(i, dtype):
    counts, tail, F, K, pad = SHAPES[i]
    act = ACTS[i % 4]
    x, (wg, wu), _ = inputs(i + 100, SHAPES[i], dtype, 2)
    want = gref.gated(clean(x, counts), wg.double(), wu.double(), counts, act)
    X, A, B, ends = x.cuda(), ref.pack(wg.cuda()), ref.pack(wu.cuda()), gref.ends_of(counts).cuda()
    H, G, U = bmm.grouped_gated(X, A, B, ends, act=act, save=True)
    for got, (r, e), what in zip((H, G, U), want, "HGU"):
        ref.check(got, r, e, dtype, what)
        assert (got[sum(counts):] == 0).all()
    wide = poison(sum(counts) + tail, F + 8, dtype=dtype)
    out = bmm.grouped_gated(X, A, B, ends, act=act, out=wide[:, :F])
    assert torch.equal(out[:sum(counts)], H[:sum(counts)])
    assert torch.isnan(wide[:, F:]).all() and torch.isnan(wide[sum(counts):]).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_mma_backward(i, dtype):
    counts, tail, N, K, pad = SHAPES[i]
    x, (w,), gen = inputs(i + 200, SHAPES[i], dtype)
    dy = gref.matrix(gen, sum(counts) + tail, N, pad, dtype)
    dy[sum(counts):] = float("nan")
    want = gref.mma_backward(clean(dy, counts), clean(x, counts), w.double(), counts)
    args = dy.cuda(), x.cuda(), ref.pack(w.cuda()), gref.ends_of(counts).cuda()
    dX, dW = bmm.grouped_mma_backward(*args)
    for got, (r, e), what in zip((dX, dW), want, ("dX", "dW")):
        ref.check(got, r, e, dtype, what)
    assert (dX[sum(counts):] == 0).all()
    # one of them alone, in a workspace that held something else
    need = bmm.grouped_mma_backward_workspace_bytes(len(counts), sum(counts) + tail, N, K)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    one, none = bmm.grouped_mma_backward(*args, need_dw=False, workspace=ws[:need])
    assert none is None and torch.equal(one, dX)
    none, one = bmm.grouped_mma_backward(*args, need_dx=False, workspace=ws[:need])
    assert none is None and torch.equal(one, dW)
    assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("i", range(len(SHAPES)), ids=IDS)
def test_gated_backward(i, dtype):
    counts, tail, F, K, pad = SHAPES[i]
    act = ACTS[(i + 1) % 4]
    x, (wg, wu), gen = inputs(i + 300, SHAPES[i], dtype, 2)
    dh, g, u = (gref.matrix(gen, sum(counts) + tail, F, pad, dtype) for _ in range(3))
    dh[sum(counts):], g[sum(counts):], u[sum(counts):] = float("inf"), float("nan"), float("inf")
    want = gref.gated_backward(*(clean(t, counts) for t in (dh, g, u, x)), wg.double(), wu.double(),
                               counts, act, dtype)
    args = (dh.cuda(), g.cuda(), u.cuda(), x.cuda(), ref.pack(wg.cuda()), ref.pack(wu.cuda()),
            gref.ends_of(counts).cuda())
    got = bmm.grouped_gated_backward(*args, act=act)
    for o, (r, e), what in zip(got, want, ("dX", "dWg", "dWu")):
        ref.check(o, r, e, dtype, what)
    assert (got[0][sum(counts):] == 0).all()
    need = bmm.grouped_gated_backward_workspace_bytes(len(counts), sum(counts) + tail, F, K)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    dx, *none = bmm.grouped_gated_backward(*args, act=act, need_dw=False, workspace=ws[:need])
    assert none == [None, None] and torch.equal(dx, got[0])
    none, *dw = bmm.grouped_gated_backward(*args, act=act, need_dx=False, workspace=ws[:need])
    assert none is None and torch.equal(dw[0], got[1]) and torch.equal(dw[1], got[2])
    assert (ws[need:] == 0xFF).all()


def test_empty_sums():
    """K = 0 and N = 0: zeros where there is something to write."""
    ends = gref.ends_of([3, 2]).cuda()
    x = torch.ones(5, 0, dtype=BF, device="cuda")
    w = torch.empty(2, 3, 0, 8, 8, dtype=torch.int32, device="cuda")
    assert (bmm.grouped_mma(x, w, ends) == 0).all()
    assert (bmm.grouped_gated(x, w, w, ends) == 0).all()
    x = torch.ones(5, 32, dtype=BF, device="cuda")
    w = torch.empty(2, 0, 2, 8, 8, dtype=torch.int32, device="cuda")
    dy = torch.empty(5, 0, dtype=BF, device="cuda")
    dx, dw = bmm.grouped_mma_backward(dy, x, w, ends)
    assert dx.shape == (5, 32) and (dx == 0).all() and dw.shape == (2, 0, 32)
    dx, dwg, _ = bmm.grouped_gated_backward(dy, dy, dy, x, w, w, ends)
    assert (dx == 0).all() and dwg.shape == (2, 0, 32)


def test_no_rows():
    ends = gref.ends_of([0, 0]).cuda()
    x = torch.empty(0, 32, dtype=BF, device="cuda")
    w = ref.pack(torch.ones(2, 24, 32, dtype=BF, device="cuda"))
    dy = torch.empty(0, 24, dtype=BF, device="cuda")
    assert bmm.grouped_mma(x, w, ends).shape == (0, 24)
    assert [t.shape[0] for t in bmm.grouped_gated(x, w, w, ends, save=True)] == [0, 0, 0]
    dx, dw = bmm.grouped_mma_backward(dy, x, w, ends)
    assert dx.shape == (0, 32) and dw.shape == (2, 24, 32) and (dw == 0).all()
    _, dwg, dwu = bmm.grouped_gated_backward(dy, dy, dy, x, w, w, ends)
    assert (dwg == 0).all() and (dwu == 0).all()


@pytest.mark.parametrize("counts", [[5, 0, 4], [200, 0, 129]], ids=["few", "many"])
def test_nan_stays_in_its_group(counts):
    """A NaN or an infinity in one group's rows or weight reaches no other group."""
    x, (w,), gen = inputs(7, (counts, 0, 72, 64, 0), BF)
    dy = gref.matrix(gen, sum(counts), 72, 0, BF)
    x[0, 3], w[1], dy[1, 5] = float("nan"), float("inf"), float("inf")
    X, W, ends, dY = x.cuda(), ref.pack(w.cuda()), gref.ends_of(counts).cuda(), dy.cuda()
    n = counts[0]
    Y = bmm.grouped_mma(X, W, ends)
    assert torch.isnan(Y[0]).all() and torch.isfinite(Y[1:]).all()
    dX, dW = bmm.grouped_mma_backward(dY, X, W, ends)
    assert torch.isfinite(dX[n:]).all() and torch.isfinite(dW[2]).all() and (dW[1] == 0).all()
    assert torch.isnan(dW[0][:, 3]).all()
    H = bmm.grouped_gated(X, W, W, ends)
    assert torch.isnan(H[0]).all() and torch.isfinite(H[1:]).all()
