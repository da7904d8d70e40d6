"""64-bit references and error bounds of the feed-forward operators.

Every bound is built from the arithmetic the operators state: products of
exact inputs summed in float32 (each addition off by at most 2^-23 of the
running magnitude, whatever the order), activations in float32, and one rounding of
half a step, eps / 2, wherever a value is rounded to 16 bits (plus half the
smallest subnormal)."""
import math

import torch

U32 = 2.0 ** -23            # one float32 addition, rounded or cut
LIPSCHITZ = 1.13            # largest slope of the four activations


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def half_tiny(dtype):
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def act(g, name):
    """(value, slope) in the type of g (float64)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        p = torch.special.erfc(-g * math.sqrt(0.5)) / 2   # accurate in the far tail
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        z = 2 * c * (g + 0.044715 * g ** 3)
        s = 1 / (1 + torch.exp(-z))      # (1 + tanh(z / 2)) / 2, without its cancellation
        q = 1 / (1 + torch.exp(z))       # 1 - s
        return g * s, s + g * s * q * 2 * c * (1 + 3 * 0.044715 * g * g)
    return torch.where(g > 0, g, 0.0), (g > 0).to(g.dtype)


def act_rel(g, name):
    """Relative error of a float32 activation: a few roundings, and the
    exponential's argument, whose last bit is worth its size."""
    size = {"silu": g.abs(), "gelu": g * g / 2,
            "gelu_tanh": 1.6 * (g.abs() + 0.044715 * g.abs() ** 3), "relu": 0 * g}[name]
    return (8 + 4 * torch.clamp(size, max=128)) * U32


def sum_error(a, b):
    """Bound on a float32 sum of the products of a (.., M, K) and b (.., N, K)."""
    return (a.shape[-1] + 2) * U32 * (a.abs() @ b.abs().transpose(-1, -2))


def rounded(ref, err, dtype):
    """Bound on a value with error `err` after rounding to dtype."""
    return err + half_step(dtype) * (ref.abs() + err) + half_tiny(dtype)


def gated(x, wg, wu, name):
    """((h, bound), (g, bound), (u, bound)) of float64 inputs."""
    g, u = x @ wg.transpose(-1, -2), x @ wu.transpose(-1, -2)
    eg, eu = sum_error(x, wg), sum_error(x, wu)
    a, _ = act(g, name)
    h = a * u
    eh = LIPSCHITZ * eg * (u.abs() + eu) + a.abs() * eu + h.abs() * act_rel(g, name)
    return (h, eh), (g, eg), (u, eu)


def gated_backward(dh, g, u, x, wg, wu, name, dtype):
    """((dx, bound), (dwg, bound), (dwu, bound)): float64 inputs whose dG and dU
    are rounded to dtype on the way."""
    a, slope = act(g, name)
    dg, du = dh * u * slope, dh * a
    rel = act_rel(g, name)
    eg = rounded(dg, (dh * u).abs() * (slope.abs() + g.abs() + 1) * rel, dtype)
    eu = rounded(du, du.abs() * rel, dtype)
    dgu, egu = torch.cat([dg, du], -1), torch.cat([eg, eu], -1)
    w = torch.cat([wg, wu], -2)
    n = U32 * (dgu.shape[-1] + 32 + 2)
    dx = dgu @ w
    ex = egu @ w.abs() + n * ((dgu.abs() + egu) @ w.abs())
    n = U32 * (x.shape[-2] + 32 + 2)
    dw = dgu.transpose(-1, -2) @ x
    ew = egu.transpose(-1, -2) @ x.abs() + n * ((dgu.abs() + egu).transpose(-1, -2) @ x.abs())
    F = g.shape[-1]
    return (dx, ex), (dw[..., :F, :], ew[..., :F, :]), (dw[..., F:, :], ew[..., F:, :])


def check(got, ref, err, dtype, what):
    """Every element within its bound; the worst ratio in the message."""
    got = got.double().cpu()
    ref, bound = ref.cpu(), rounded(ref, err, dtype).cpu()
    assert got.shape == ref.shape, what
    assert not torch.isnan(got).any(), f"{what}: unwritten or NaN outputs"
    # past the type's largest value (and a half step) rounding gives an infinity
    limit = torch.finfo(dtype).max * (1 + half_step(dtype) / 2)
    over = torch.isinf(got) & (torch.sign(got) == torch.sign(ref)) & (ref.abs() + err.cpu() >= limit)
    must = ref.abs() - err.cpu() > limit
    bad = torch.where(over | must, ~over, (got - ref).abs() > bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"{got[i].item()} for {ref[i].item()} +- {bound[i].item()}")


def pack(w):
    """(batch, rows, K) 16-bit weights as packed B words, by reshaping."""
    b, n, k = w.shape
    atoms = w.view(torch.int16).reshape(b, n // 8, 8, k // 16, 16).permute(0, 1, 3, 2, 4)
    return atoms.contiguous().view(torch.int32)


# ---- 4-bit floats, from the format's definition ----

def mx4_quantize(x):
    """x (rows, K) float64 -> (codes (rows, K) int, scale bytes (rows, K / 32) int)."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    expo = torch.where(torch.isfinite(top) & (top > 0), torch.frexp(top)[1] - 1, -1000)
    byte = torch.clamp(expo - 2 + 127, 0, 254)
    v = torch.where(bad[:, :, None], 0.0, b) * torch.exp2(127.0 - byte.double())[:, :, None]
    # 1 bit of mantissa: steps of 0.5 below 2, then 1, then 2; ties to even
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    m = torch.clamp(torch.round(m / step) * step, max=6.0)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    code = torch.searchsorted(grid, m.contiguous()) + 8 * torch.signbit(v).long()
    code = torch.where(bad[:, :, None], 0, code)
    return code.reshape(x.shape), torch.where(bad, 255, byte)


def mx4_layout(code, byte):
    """Codes (rows, K) and scale bytes (rows, K / 32) in the operand's layout."""
    rows, K = code.shape
    r, s, q = -(-rows // 16), -(-K // 128), -(-K // 512)
    c = torch.zeros(r * 16, s * 128, dtype=torch.int64)
    c[:rows, :K] = code
    c = c.reshape(r, 16, s, 4, 16, 2).permute(0, 2, 3, 1, 4, 5)
    e = torch.zeros(r * 16, q * 16, dtype=torch.int64)
    e[:rows, :K // 32] = byte
    e = e.reshape(r, 16, q, 4, 4).permute(0, 2, 4, 1, 3)
    return ((c[..., 0] + 16 * c[..., 1]).to(torch.uint8).contiguous()[None],
            e.to(torch.uint8).contiguous()[None])


def mx4_values(code, byte):
    """float64 values of codes (rows, K) and scale bytes."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    v = grid[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    s = torch.where(byte == 255, float("nan"), torch.exp2(byte.double() - 127))
    return v * s.repeat_interleave(32, 1)
