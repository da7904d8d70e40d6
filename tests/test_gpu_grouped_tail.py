"""Rows behind the last group, many of them: by every tile, sums whole and in parts. They
are not read (they hold NaN), become zero in fresh outputs and stay in given ones."""
import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref
from tests.test_gpu_grouped_tiles import GATED, GATED_BACK, I8_GROUPS, MMA, MMA_BACK, counts_of, gen_of, \
    same, whole

pytestmark = pytest.mark.gpu
BF, HF, NAN = torch.bfloat16, torch.float16, float("nan")
SHARES = [(0, 1), (1, 8), (3, 5), (19, 20)]   # of the rows that belong to a group


def rows_of(E, T, share):
    n = T * share[0] // share[1]
    return counts_of(E, n, n)[0] if n else [0] * E


def checked(call, want, n, what):
    """A fresh output and a given one."""
    fresh = call(None)
    same(fresh[:n], want[:n], what)
    assert not fresh[n:].any(), what
    given = torch.full_like(fresh, NAN)
    call(given)
    same(given[:n], want[:n], what)
    assert torch.isnan(given[n:]).all(), what


def with_tail(t, n, value=NAN):
    t = t.clone()
    t[n:] = value
    return t


@pytest.mark.parametrize("share", SHARES, ids=str)
@pytest.mark.parametrize("shape", MMA, ids=str)
def test_mma(shape, share):
    E, T, N, K = shape
    counts = rows_of(E, T, share)
    n, gen, ends = sum(counts), gen_of(T), gref.ends_of(counts).cuda()
    x, w = whole(gen, 2, T, K, dtype=BF), whole(gen, 2, E, N, K, dtype=BF)
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = x[r].double() @ w[e].double().t()
    x, w = with_tail(x, n), ref.pack(w)
    checked(lambda out: bmm.grouped_mma(x, w, ends, out=out), want, n, "Y")


@pytest.mark.parametrize("share", SHARES, ids=str)
@pytest.mark.parametrize("shape", GATED, ids=str)
def test_gated(shape, share):
    E, T, F, K = shape
    counts = rows_of(E, T, share)
    n, gen, ends = sum(counts), gen_of(T), gref.ends_of(counts).cuda()
    x, wg, wu = (whole(gen, 1, *s, dtype=HF) for s in ((T, K), (E, F, K), (E, F, K)))
    g, u = (torch.zeros(T, F, dtype=torch.float64, device="cuda") for _ in range(2))
    for e, r in gref.groups(counts):
        g[r], u[r] = x[r].double() @ wg[e].double().t(), x[r].double() @ wu[e].double().t()
    x, wg, wu = with_tail(x, n), ref.pack(wg), ref.pack(wu)
    checked(lambda out: bmm.grouped_gated(x, wg, wu, ends, act="relu", out=out),
            g.float().clamp(min=0) * u.float(), n, "H")
    for got, want in zip(bmm.grouped_gated(x, wg, wu, ends, act="relu", save=True)[1:], (g, u)):
        same(got, want, "projections")


@pytest.mark.parametrize("share", SHARES, ids=str)
@pytest.mark.parametrize("shape", MMA_BACK, ids=str)
def test_mma_dx(shape, share):
    E, T, N, K = shape
    counts = rows_of(E, T, share)
    n, gen, ends = sum(counts), gen_of(T), gref.ends_of(counts).cuda()
    x, dy, w = (whole(gen, 2, *s, dtype=BF) for s in ((T, K), (T, N), (E, N, K)))
    want = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = dy[r].double() @ w[e].double()
    for need_dw in (False, True):
        same(bmm.grouped_mma_backward(with_tail(dy, n), with_tail(x, n), ref.pack(w), ends,
                                      need_dw=need_dw)[0], want, "dX")


@pytest.mark.parametrize("share", SHARES, ids=str)
@pytest.mark.parametrize("shape", GATED_BACK, ids=str)
def test_gated_dx(shape, share):
    E, T, F, K = shape
    counts = rows_of(E, T, share)
    n, gen, ends = sum(counts), gen_of(T), gref.ends_of(counts).cuda()
    dh, g, u = (whole(gen, 2, T, F, dtype=HF) for _ in range(3))
    x, wg, wu = (whole(gen, 1, *s, dtype=HF) for s in ((T, K), (E, F, K), (E, F, K)))
    dg, du = (dh * u * (g > 0)).double(), (dh * g.clamp(min=0)).double()
    want = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = dg[r] @ wg[e].double() + du[r] @ wu[e].double()
    same(bmm.grouped_gated_backward(*(with_tail(t, n) for t in (dh, g, u, x)), ref.pack(wg), ref.pack(wu),
                                    ends, act="relu", need_dw=False)[0], want, "dX")


@pytest.mark.parametrize("share", SHARES, ids=str)
@pytest.mark.parametrize("shape", I8_GROUPS, ids=str)
def test_i8(shape, share):
    E, T, N, K = shape
    counts = rows_of(E, T, share)
    n, gen, ends = sum(counts), gen_of(T), gref.ends_of(counts).cuda()
    a, b = whole(gen, 127, T, K, dtype=torch.int8), whole(gen, 127, E, N, K, dtype=torch.int8)
    sa, sb = (torch.rand(*s, generator=gen, device="cuda") for s in ((T,), (E, N)))
    want = torch.zeros(T, N, device="cuda")
    for e, r in gref.groups(counts):
        want[r] = gref.i8_mma(a[r], sa[r], b[e], sb[e], torch.float32)
    A, B = bmm.I8Operand(a, with_tail(sa, n)), bmm.I8Operand(gref.i8_pack(b), sb)
    checked(lambda out: bmm.i8_mma(A, B, ends, out=out), want, n, "D")
