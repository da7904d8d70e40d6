"""64-bit references of the products by groups, group by group, with the bounds of
ffn_ref; and inputs whose groups are chosen."""
import math

import torch

from tests import ffn_ref as ref


def ends_of(counts):
    return torch.tensor(counts, dtype=torch.int64).cumsum(0).to(torch.int32)


def groups(counts):
    """(group, its rows) of the groups that have rows."""
    start = 0
    for e, n in enumerate(counts):
        if n:
            yield e, slice(start, start + n)
        start += n


def matrix(gen, rows, cols, pad, dtype, device="cpu"):
    """(rows, cols) normal values with cols + pad elements between rows."""
    return torch.randn(rows, cols + pad, generator=gen, device=device).to(dtype)[:, :cols]


def weights(gen, E, N, K, dtype, device="cpu"):
    w = torch.empty(E, N, K, dtype=dtype, device=device)
    for e in range(E):
        w[e] = (torch.randn(N, K, generator=gen, device=device) / math.sqrt(max(K, 1))).to(dtype)
    return w


def mma(x, w, counts):
    """(y, bound) of float64 inputs; zeros behind the last group."""
    y = x.new_zeros(x.shape[0], w.shape[1])
    e_y = torch.zeros_like(y)
    for e, r in groups(counts):
        y[r], e_y[r] = x[r] @ w[e].t(), ref.sum_error(x[r], w[e])
    return y, e_y


def mma_backward(dy, x, w, counts):
    """((dx, bound), (dw, bound))."""
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    ex, ew = torch.zeros_like(dx), torch.zeros_like(dw)
    for e, r in groups(counts):
        wt, dyt, xt = (t.t().contiguous() for t in (w[e], dy[r], x[r]))
        dx[r], ex[r] = dy[r] @ wt.t(), ref.sum_error(dy[r], wt)
        dw[e], ew[e] = dyt @ xt.t(), ref.sum_error(dyt, xt)
    return (dx, ex), (dw, ew)


def gated(x, wg, wu, counts, act):
    """((h, bound), (g, bound), (u, bound))."""
    out = [[x.new_zeros(x.shape[0], wg.shape[1]) for _ in range(2)] for _ in range(3)]
    for e, r in groups(counts):
        for o, got in zip(out, ref.gated(x[r], wg[e], wu[e], act)):
            o[0][r], o[1][r] = got
    return [tuple(o) for o in out]


def gated_backward(dh, g, u, x, wg, wu, counts, act, dtype):
    """((dx, bound), (dwg, bound), (dwu, bound))."""
    dx = [torch.zeros_like(x) for _ in range(2)]
    dw = [[torch.zeros_like(wg) for _ in range(2)] for _ in range(2)]
    for e, r in groups(counts):
        a, b, c = ref.gated_backward(dh[r], g[r], u[r], x[r], wg[e], wu[e], act, dtype)
        dx[0][r], dx[1][r] = a
        for o, got in zip(dw, (b, c)):
            o[0][e], o[1][e] = got
    return tuple(dx), tuple(dw[0]), tuple(dw[1])


# ---- 8-bit integers ----

def i8_quantize(x):
    """(codes int64, scales float32) of x (rows, K) on the CPU, from the definition:
    the code next to 127 |x| / max, of two as near the even one. Everything is taken
    in 64 bits, where the comparison of 2 * 127 |x| with (2 c + 1) max is exact."""
    x = x.double()
    bad = ~torch.isfinite(x).all(1, keepdim=True)
    top = torch.where(bad, 0.0, x.abs().amax(1, keepdim=True) if x.shape[1] else x.new_zeros(x.shape[0], 1))
    one = torch.where(top > 0, top, 1.0)
    a = torch.where(bad, 0.0, 127 * x.abs())
    low = torch.floor(a / one)
    low -= (low * one > a).double()          # (the quotient may round up to a whole number)
    twice = 2 * a - (2 * low + 1) * one
    code = low + ((twice > 0) | ((twice == 0) & (low % 2 == 1))).double()
    scale = (top.float() / 127)[:, 0]
    return (torch.sign(x) * code).nan_to_num(0).long(), \
        torch.where(bad[:, 0], float("nan"), scale)


def i8_pack(codes):
    """Row-major int8 codes (batch, rows, K) as packed words, by reshaping."""
    b, n, k = codes.shape
    words = codes.contiguous().view(torch.int32).reshape(b, n // 8, 8, k // 32, 8)
    return words.permute(0, 1, 3, 2, 4).contiguous()


def i8_mma(a, sa, b, sb, dtype):
    """The product as stated, bit for bit: exact sums, rounded to float32, times the
    row's scale, times the column's, rounded. (Sums below 2^53: exact in float64.)"""
    d = (a.double() @ b.double().t()).float() * sa[:, None]
    return (d * sb[None]).to(dtype)
