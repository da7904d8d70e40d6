"""The shapes of the GPU tests of the products by groups and of 8-bit integers reach every
tile that the plan can choose and every layout of the rows' tiles (CPU: the plan is host
code; the layout's rule is written out here a second time); and the 64-bit references'
gradients against differences."""
import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref
from tests import test_gpu_grouped as small
from tests import test_gpu_grouped_tiles as tiles

TILES = ["128x128", "256x128", "256x192", "256x256"]


def reached(product, shapes):
    return {bmm.group_plan(product, *s)[0] for s in shapes}, \
        {(t, n > 1) for t, n in (bmm.group_plan(product, *s) for s in shapes)}


@pytest.mark.parametrize("product,shapes", [
    ("grouped_mma", tiles.MMA), ("grouped_gated", tiles.GATED), ("i8_mma", tiles.I8_GROUPS),
    ("i8_mma", [(0, *s) for s in tiles.I8]), ("i8_gated", tiles.I8_GATED_GROUPS),
    ("i8_gated", [(0, *s) for s in tiles.I8_GATED])], ids=lambda p: p if isinstance(p, str) else "")
def test_forward(product, shapes):
    got, _ = reached(product, shapes)
    more = [] if shapes[0][0] == 0 else ["few_rows"]   # (one 8-bit weight: test_gpu_i8.py)
    assert set(TILES + more) <= got, got


@pytest.mark.parametrize("product,shapes", [
    ("grouped_mma_dx", tiles.MMA_BACK), ("grouped_mma_dw", tiles.MMA_BACK),
    ("grouped_gated_dx", tiles.GATED_BACK), ("grouped_gated_dw", tiles.GATED_BACK)],
    ids=lambda p: p if isinstance(p, str) else "")
def test_backward(product, shapes):
    got, split = reached(product, shapes)
    assert set(TILES) <= got, got
    assert any(s for _, s in split) and any(not s for _, s in split)


def test_few_rows_blocks_and_one_launch():
    """Blocks of 16 and 64 rows; both gradients in one launch, dX split and unsplit."""
    for kind in ("mma", "gated"):
        blocks = set()
        for counts, tail, N, K, _ in small.SHAPES:
            T, E = sum(counts) + tail, len(counts)
            if T and bmm.group_plan(f"grouped_{kind}", E, T, N, K)[0] == "few_rows":
                some = min(E, T)
                wide = some * -(-N // (16 if kind == "gated" else 32))
                blocks.add(16 if T // some <= 16 or (T // some <= 48 and wide <= 128) else 64)
        assert blocks == {16, 64}, kind
    both = set()
    for E, T, N, K in tiles.MMA_BACK + tiles.GATED_BACK:
        for kind in ("mma", "gated"):
            dx, dw = (bmm.group_plan(f"grouped_{kind}_{p}", E, T, N, K) for p in ("dx", "dw"))
            if dx[0] == dw[0] == "128x128":
                both.add((dx[1] > 1, dw[1] > 1))
    assert (False, False) in both and (True, False) in both and (False, True) in both


def layout(counts, NT):
    """How 256-row tiles of these groups lie: (small ones among the others, small ones last,
    tiles of the last round in halves)."""
    full = sum((n + 127) // 256 for n in counts)
    small_ones = sum(0 < n % 256 <= 128 for n in counts)
    mixed = 4 * small_ones >= full
    n = (full + (small_ones if mixed else 0)) * NT
    last = 0 if mixed else small_ones * NT
    over = n % 256
    cut = not mixed and 0 < over <= 128 and 2 * over + last <= 256
    return mixed and small_ones > 0, last > 0, cut, n // 256 > 1


def test_layouts():
    got = set()
    for counts, n, K in tiles.LAYOUTS:
        tile, _ = bmm.group_plan("grouped_mma", len(counts), sum(counts) + 7, n, K)
        if tile.startswith("256"):
            got.add(layout(counts, -(-n // int(tile[4:]))))
    for i, what in enumerate(("mixed", "small last", "halves", "rounds")):
        assert {g[i] for g in got} == {False, True}, what
    assert any(g[1] and g[2] for g in got), "small ones and halves together"


@pytest.mark.parametrize("act", sorted(bmm.ACTS))
def test_reference_gradients_against_differences(act):
    """dL for L = sum(R * out) along random directions: central differences of the float64
    forward, whose error is of the order of step^2 and 2^-52 / step (relu: no row near 0)."""
    torch.manual_seed(3)
    counts, T = [4, 0, 7], 13
    x = torch.randn(T, 16, dtype=torch.float64)
    wg, wu = torch.randn(3, 8, 16, dtype=torch.float64), torch.randn(3, 8, 16, dtype=torch.float64)
    r = torch.randn(T, 8, dtype=torch.float64)
    r[11:] = 0

    def forward(x, wg, wu):
        return gref.gated(x, wg, wu, counts, act)
    (h, _), (g, _), (u, _) = forward(x, wg, wu)
    grads = gref.gated_backward(r, g, u, x, wg, wu, counts, act, torch.float64)
    for i, (t, (grad, _)) in enumerate(zip((x, wg, wu), grads)):
        v = torch.randn_like(t)
        step = 1e-5
        args = [[x, wg, wu] for _ in range(2)]
        args[0][i], args[1][i] = t + step * v, t - step * v
        diff = sum(s * (r * forward(*a)[0][0]).sum() for s, a in zip((1, -1), args)) / (2 * step)
        assert abs(diff - (grad * v).sum()) < 1e-6 * (1 + abs(diff)), i
    w = torch.randn(3, 8, 16, dtype=torch.float64)
    (dx, _), (dw, _) = gref.mma_backward(r, x, w, counts)
    vx, vw = torch.randn_like(x), torch.randn_like(w)
    loss = lambda a, b: (r * gref.mma(a, b, counts)[0]).sum()
    for grad, v, f in ((dx, vx, lambda s: loss(x + s * vx, w)), (dw, vw, lambda s: loss(x, w + s * vw))):
        diff = (f(1e-3) - f(-1e-3)) / 2e-3          # linear in each: exact but for rounding
        assert abs(diff - (grad * v).sum()) < 1e-9 * (1 + abs(diff))


def test_i8_reference():
    x = torch.tensor([[2.0, 1.0, -1.0, 0.0, 0.5, 2 * 63.49 / 127, -2 * 1.5625 / 127]])
    codes, scale = gref.i8_quantize(x)
    assert codes.tolist() == [[127, 64, -64, 0, 32, 63, -2]]   # 63.5 to 64, 31.75 to 32
    assert scale.item() == pytest.approx(2 / 127)
    assert torch.isnan(gref.i8_quantize(torch.tensor([[1.0, float("inf")]]))[1]).all()
    assert ref.half_step(torch.bfloat16) == 2 ** -8
