"""The experts' operators and the 8-bit products on real work: inputs, plain
forms and exact values.

A block of experts keeps E weights of one shape. Its rows (a token times each of
its experts) are sorted by expert; expert e has the rows from ends[e - 1] up to
ends[e] (the first from 0), any number of them, also none. Rows from ends[E - 1]
on belong to no expert (a batch padded to a fixed size): their outputs are zero.

- ``grouped_mma``             Y = X W_e^T for the rows of each expert e;
- ``grouped_mma_backward``    dX = dY W_e and dW_e = dY^T X over its rows;
- ``grouped_gated``           H = act(X Wg_e^T) * (X Wu_e^T), the projections
                              kept for the backward pass where a training step
                              asks for them;
- ``grouped_gated_backward``  dX, dWg and dWu of that block from dH and the kept
                              projections;
- ``i8_mma``                  D = X W^T in 8-bit integers: a scale for each row
                              of X, which is quantised on the way in, and one for
                              each row of W; one weight, or one for each expert;
- ``i8_gated``                the gated block's projections in 8-bit integers.

``run`` computes them in elementary torch operations in 32 bits, rounded once at
the end, or, with ``own`` set, through the package's entry points. ``exact``
computes the same outputs in 64 bits from the definitions.

Weights of a program are kept packed (8 rows x 32 bytes an atom: 16 values of 16
bits or 32 of 8) beside the row-major matrix that the plain forms read. 8-bit
weights are codes -127 .. 127 and a scale for each row.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GROUPED = ("grouped_mma", "grouped_mma_backward", "grouped_gated", "grouped_gated_backward")


# ---- cases ----
#
# E experts (0: one weight, no groups), ``active`` of which have rows; ``rows`` rows
# in all and ``tail`` behind them that belong to none; K values a row in, N out (the
# gated block: F). ``skew`` spreads the experts' popularity: exp(skew * normal).

def listed():
    """Twelve cases: the smallest calls, ordinary ones and the largest."""
    return [
        # one token through its six experts of 64 narrow ones
        dict(name="mma_token", op="grouped_mma", E=64, rows=6, active=6, tail=0, K=1408, N=2048,
             dtype="bf16", pad=0, skew=0.0),
        # a long prompt through two of eight wide experts a token, some far more popular
        dict(name="mma_prompt", op="grouped_mma", E=8, rows=16384, active=8, tail=0, K=8192,
             N=4096, dtype="bf16", pad=0, skew=0.7),
        # a short sequence through a few small experts, one without rows, X a column slice
        dict(name="mma_backward_short_f16", op="grouped_mma_backward", E=5, rows=777, active=4,
             tail=0, K=528, N=1000, dtype="f16", pad=8, skew=0.5),
        # a training step's tokens, six of 64 narrow experts each
        dict(name="mma_backward_train", op="grouped_mma_backward", E=64, rows=24576, active=64,
             tail=0, K=1408, N=2048, dtype="bf16", pad=0, skew=0.4),
        # 32 tokens decoded together, two of eight wide experts each, in a batch padded to 40
        dict(name="gated_decode", op="grouped_gated", E=8, rows=64, active=8, tail=16, K=4096,
             F=8192, dtype="bf16", pad=0, skew=0.3, act="silu", save=False),
        # the forward pass of a training step through 64 narrow experts, projections kept
        dict(name="gated_train_f16", op="grouped_gated", E=64, rows=24576, active=64, tail=0,
             K=2048, F=1408, dtype="f16", pad=0, skew=0.4, act="gelu_tanh", save=True),
        # a short sequence, two experts without rows, padded to a fixed length
        dict(name="gated_backward_short", op="grouped_gated_backward", E=8, rows=301, active=6,
             tail=83, K=1024, F=776, dtype="bf16", pad=0, skew=0.5, act="gelu"),
        # the backward pass of a training step through 16 experts
        dict(name="gated_backward_train", op="grouped_gated_backward", E=16, rows=16384, active=16,
             tail=0, K=2048, F=4096, dtype="bf16", pad=0, skew=0.5, act="silu"),
        # one token through a 16384 x 16384 8-bit layer
        dict(name="i8_token", op="i8_mma", E=0, rows=1, active=1, tail=0, K=16384, N=16384,
             dtype="bf16", pad=0, skew=0.0, out="bf16"),
        # a full batch through an 8192 x 8192 8-bit layer
        dict(name="i8_square", op="i8_mma", E=0, rows=8192, active=1, tail=0, K=8192, N=8192,
             dtype="bf16", pad=0, skew=0.0, out="bf16"),
        # seven tokens decoded together, two of eight wide 8-bit experts each
        dict(name="i8_gated_decode", op="i8_gated", E=8, rows=14, active=7, tail=0, K=4096, F=8192,
             dtype="bf16", pad=0, skew=0.0, act="silu", out="bf16"),
        # a prompt through an 8-bit gated block
        dict(name="i8_gated_prompt_f16", op="i8_gated", E=0, rows=4095, active=1, tail=0, K=4096,
             F=8192, dtype="f16", pad=0, skew=0.0, act="gelu_tanh", out="f16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(GROUPED + ("i8_mma", "i8_gated"))
    eight = op not in GROUPED
    E = 0 if eight and rng.random() < 0.5 else _log_int(rng, 2, 128)
    K = (32 if eight else 16) * _log_int(rng, 4, 256)
    wide = 8 * _log_int(rng, 8, 1024)
    E = min(E, (1 << 27) // (K * wide))    # at most 2^27 weights a matrix
    rows = _log_int(rng, 1, max(1, min(16384, (1 << 37) // (K * wide))))
    active = 1
    if E:
        active = min(E, rows) if rng.random() < 0.6 else rng.randint(1, min(E, rows))
    case = dict(op=op, E=E, rows=rows, active=active,
                tail=rng.choice([0, 0, 5, 130]) if E else 0, K=K)
    case["F" if "gated" in op else "N"] = wide
    case.update(dtype=rng.choice(["bf16", "f16"]), pad=rng.choice([0, 0, 8, 64]),
                skew=rng.choice([0.0, 0.5, 1.5]))
    if "gated" in op:
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "grouped_gated":
        case["save"] = rng.random() < 0.5
    if eight:
        case["out"] = rng.choice(["bf16", "f16", "f32"]) if op == "i8_mma" else case["dtype"]
    return case


# ---- inputs ----

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _rows(gen, rows, cols, pad, dtype):
    """(rows, cols) activations; with pad, a column slice of a wider buffer."""
    return _normal(gen, rows, cols + pad).to(dtype)[:, :cols]


def _packed(w):
    """Row-major (E, N, bytes / size) weights as packed words (E, N/8, bytes/32, 8, 8)."""
    words = w.view(torch.int32)
    e, n, k = words.shape
    return words.reshape(e, n // 8, 8, k // 8, 8).permute(0, 1, 3, 2, 4).contiguous()


def _counts(case, seed):
    """Rows of each expert: one for each active expert, the others by popularity."""
    rng = random.Random(seed)
    chosen = sorted(rng.sample(range(case["E"]), case["active"]))
    weights = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in chosen]
    counts = [0] * case["E"]
    for e in chosen:
        counts[e] = 1
    for e in rng.choices(chosen, weights, k=case["rows"] - case["active"]):
        counts[e] += 1
    return counts


def _weight(gen, E, rows, K, dtype):
    """Expert by expert, so that the 32-bit draws need little room."""
    w = torch.empty(E, rows, K, dtype=dtype, device="cuda")
    for e in range(E):
        w[e] = _normal(gen, rows, K).div_(math.sqrt(K)).to(dtype)
    return w


def _weight_i8(gen, E, rows, K):
    """8-bit weights as a checkpoint holds them: codes (E, rows, K) and scales (E, rows)."""
    codes = torch.empty(E, rows, K, dtype=torch.int8, device="cuda")
    scales = torch.empty(E, rows, device="cuda")
    for e in range(E):
        w = _normal(gen, rows, K).div_(math.sqrt(K))
        scales[e] = w.abs().amax(1) / 127
        codes[e] = torch.round(w / scales[e][:, None]).to(torch.int8)
    return codes, scales


def prepare(case, seed):
    """The inputs of one pass, made from the seed alone."""
    gen, dtype, op = _generator(seed), DTYPES[case["dtype"]], case["op"]
    E, K, T = case["E"], case["K"], case["rows"] + case["tail"]
    s = dict(case=case, op=op)
    s["counts"] = _counts(case, seed) if E else [case["rows"]]
    if E:
        s["ends"] = torch.tensor(s["counts"]).cumsum(0).to(torch.int32).cuda()
    s["x"] = _rows(gen, T, K, case["pad"], dtype)
    width = case["F"] if "gated" in op else case["N"]
    names = ("wg", "wu") if "gated" in op else ("w",)
    if op in GROUPED:
        for name in names:
            s[name] = _weight(gen, E, width, K, dtype)
            s[name + "_packed"] = _packed(s[name])
    else:
        # tokens of different sizes, a few channels larger than the others
        s["x"] *= torch.exp2(torch.randint(-3, 4, (T, 1), generator=gen, device="cuda"))
        s["x"][:, ::61] *= 4
        for name in names:
            codes, scales = _weight_i8(gen, max(E, 1), width, K)
            s[name], s[name + "_scales"] = codes, scales
            s[name + "_packed"] = _packed(codes)
    if op == "grouped_mma_backward":
        s["dy"] = _rows(gen, T, width, case["pad"], dtype)
    if op == "grouped_gated_backward":
        s["g"], s["u"] = (torch.zeros(T, width, dtype=dtype, device="cuda") for _ in range(2))
        for e, rows in _groups(s):
            s["g"][rows] = s["x"][rows] @ s["wg"][e].t()
            s["u"][rows] = s["x"][rows] @ s["wu"][e].t()
        s["dh"] = (_normal(gen, T, width) / 8).to(dtype)
    return s


def _groups(s):
    """(expert, its rows as a slice) for each expert."""
    start = 0
    for e, n in enumerate(s["counts"]):
        yield e, slice(start, start + n)
        start += n


# ---- plain forms ----

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _act(g, act):
    if act == "silu":
        return g * _sigmoid(g)
    if act == "gelu":
        return 0.5 * g * torch.erfc(-g * math.sqrt(0.5))   # no cancellation for g < 0
    if act == "gelu_tanh":   # 0.5 (1 + tanh z) = sigmoid(2 z)
        return g * _sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    return torch.where(g > 0, g, torch.zeros_like(g))


def _act_slope(g, act):
    if act == "silu":
        s = _sigmoid(g)
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return (0.5 * torch.erfc(-g * math.sqrt(0.5))
                + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = _sigmoid(2 * c * (g + 0.044715 * g * g * g))
        return s + g * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * g * g)
    return (g > 0).to(g.dtype)


def _by_row(s, x, w, out):
    """out[rows of e] = x[rows of e] w_e^T, in 32 bits, rounded to out's type."""
    for e, rows in _groups(s):
        if rows.stop > rows.start:
            out[rows] = (x[rows].float() @ w[e].float().t()).to(out.dtype)
    return out


def _i8_codes(x):
    """(codes, scale) of each row: 127 x / max |x| rounded to nearest, ties to even,
    and max |x| / 127. The quotient is taken in 64 bits: in 32, one next to a half
    may round onto it."""
    top = x.float().abs().amax(1, keepdim=True)
    q = torch.round(127 * x.double() / torch.where(top > 0, top, 1).double())
    return q.float(), top / 127


def _plain(s):
    case, op = s["case"], s["op"]
    dtype, T = s["x"].dtype, case["rows"] + case["tail"]
    new = s["x"].new_zeros
    if op == "grouped_mma":
        return _by_row(s, s["x"], s["w"], new(T, case["N"]))
    if op == "grouped_mma_backward":
        dx, dw = new(T, case["K"]), new(s["w"].shape)
        for e, rows in _groups(s):
            if rows.stop > rows.start:
                dy = s["dy"][rows].float()
                dx[rows] = (dy @ s["w"][e].float()).to(dtype)
                dw[e] = (dy.t() @ s["x"][rows].float()).to(dtype)
        return dx, dw
    if op == "grouped_gated":
        h, g, u = (new(T, case["F"]) for _ in range(3))
        for e, rows in _groups(s):
            if rows.stop > rows.start:
                x = s["x"][rows].float()
                ge, ue = x @ s["wg"][e].float().t(), x @ s["wu"][e].float().t()
                h[rows] = (_act(ge, case["act"]) * ue).to(dtype)
                g[rows], u[rows] = ge.to(dtype), ue.to(dtype)
        return (h, g, u) if case["save"] else h
    if op == "grouped_gated_backward":
        dx, dwg, dwu = new(T, case["K"]), new(s["wg"].shape), new(s["wu"].shape)
        for e, rows in _groups(s):
            if rows.stop > rows.start:
                x, g, u, dh = (s[n][rows].float() for n in ("x", "g", "u", "dh"))
                dg, du = dh * u * _act_slope(g, case["act"]), dh * _act(g, case["act"])
                dx[rows] = (dg @ s["wg"][e].float() + du @ s["wu"][e].float()).to(dtype)
                dwg[e], dwu[e] = (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)
        return dx, dwg, dwu
    codes, scale = _i8_codes(s["x"])
    out = DTYPES[case["out"]]
    d = new(T, case["N"] if op == "i8_mma" else case["F"], dtype=out)
    for e, rows in _groups(s):
        if rows.stop > rows.start:
            def product(name):
                return codes[rows] @ s[name][e].float().t() * scale[rows] * s[name + "_scales"][e]
            if op == "i8_mma":
                d[rows] = product("w").to(out)
            else:
                d[rows] = (_act(product("wg"), case["act"]) * product("wu")).to(out)
    return d


def _own(s):
    import bf16_matrix_multiply_amd as bmm

    case, op, ends = s["case"], s["op"], s.get("ends")
    if op == "grouped_mma":
        return bmm.grouped_mma(s["x"], s["w_packed"], ends)
    if op == "grouped_mma_backward":
        return bmm.grouped_mma_backward(s["dy"], s["x"], s["w_packed"], ends)
    if op == "grouped_gated":
        return bmm.grouped_gated(s["x"], s["wg_packed"], s["wu_packed"], ends, act=case["act"],
                                 save=case["save"])
    if op == "grouped_gated_backward":
        return bmm.grouped_gated_backward(s["dh"], s["g"], s["u"], s["x"], s["wg_packed"],
                                          s["wu_packed"], ends, act=case["act"])
    x, dtype = bmm.i8_quantize(s["x"]), DTYPES[case["out"]]
    if op == "i8_mma":
        return bmm.i8_mma(x, bmm.I8Operand(s["w_packed"], s["w_scales"]), ends, dtype=dtype)
    return bmm.i8_gated(x, bmm.I8Operand(s["wg_packed"], s["wg_scales"]),
                        bmm.I8Operand(s["wu_packed"], s["wu_scales"]), ends, act=case["act"],
                        dtype=dtype)


def run(state):
    """One pass through the case's operator."""
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    """Bytes (each input read once, each output written once) and operations."""
    op, E, K, rows = case["op"], max(case["E"], 1), case["K"], case["rows"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    b, active, T = size[case["dtype"]], case["active"], case["rows"] + case["tail"]
    if op == "grouped_mma":
        n = case["N"]
        return dict(bytes=b * (rows * K + active * n * K + T * n), flops=2 * rows * n * K)
    if op == "grouped_mma_backward":
        n = case["N"]
        return dict(bytes=b * (rows * (n + K) + active * n * K + T * K + E * n * K),
                    flops=4 * rows * n * K)
    if op == "grouped_gated":
        f = case["F"]
        outs = 3 if case["save"] else 1
        return dict(bytes=b * (rows * K + 2 * active * f * K + outs * T * f),
                    flops=4 * rows * f * K)
    if op == "grouped_gated_backward":
        f = case["F"]
        return dict(bytes=b * (3 * rows * f + rows * K + 2 * active * f * K + T * K
                               + 2 * E * f * K), flops=8 * rows * f * K)
    cols = case["N"] if op == "i8_mma" else case["F"]
    n = cols if op == "i8_mma" else 2 * cols
    return dict(bytes=b * rows * K + active * n * (K + 4) + size[case["out"]] * T * cols,
                flops=2 * rows * n * K)


# ---- exact values ----

def _exact_act(g, act):
    """(act(g), act'(g)) in 64 bits, from the functions' definitions."""
    if act == "silu":
        s = torch.special.expit(g)
        return g * s, s + g * s * torch.special.expit(-g)
    if act == "gelu":
        phi = torch.special.erfc(-g * math.sqrt(0.5)) / 2
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t * t) * c * (1 + 0.134145 * g * g)
    return torch.clamp(g, min=0), torch.heaviside(g, torch.zeros_like(g))


def _exact_i8(x):
    """The values that a row's codes and scale stand for, in 64 bits: of the two
    neighbouring codes the nearer one, of two as near the even one."""
    top = x.double().abs().amax(1, keepdim=True)
    top = torch.where(top > 0, top, torch.ones_like(top))
    a = 127 * x.double().abs()
    low = torch.floor(a / top)
    twice = 2 * a - (2 * low + 1) * top          # whole multiples of the inputs: exact
    up = (twice > 0) | ((twice == 0) & (low % 2 == 1))
    return torch.sign(x.double()) * (low + up) * (top / 127)


def exact(case, seed):
    """The outputs of ``run`` for the case's inputs, in 64 bits."""
    s = prepare(case, seed)
    op, T, E = case["op"], case["rows"] + case["tail"], max(case["E"], 1)
    width = case["F"] if "gated" in op else case["N"]

    def new(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")
    starts = [0]
    for n in s["counts"]:
        starts.append(starts[-1] + n)
    if op not in GROUPED:
        s["x"] = _exact_i8(s["x"])

    def weight(name, e):
        w = s[name][e].double()
        return w if op in GROUPED else w * s[name + "_scales"][e].double()[:, None]
    outs = {"grouped_mma": 1, "i8_mma": 1, "i8_gated": 1, "grouped_mma_backward": 2,
            "grouped_gated_backward": 3}.get(op) or (3 if case["save"] else 1)
    if "backward" in op:
        out = [new(T, case["K"])] + [new(E, width, case["K"]) for _ in range(outs - 1)]
    else:
        out = [new(T, width) for _ in range(outs)]
    for e in range(E):
        a, b = starts[e], starts[e + 1]
        if a == b:
            continue
        x = s["x"][a:b].double()
        if op in ("grouped_mma", "i8_mma"):
            out[0][a:b] = x.mm(weight("w", e).t())
        elif op == "grouped_mma_backward":
            dy = s["dy"][a:b].double()
            out[0][a:b] = dy.mm(weight("w", e))
            out[1][e] = dy.t().contiguous().mm(x)
        elif op == "grouped_gated_backward":
            g, u, dh = (s[n][a:b].double() for n in ("g", "u", "dh"))
            h, slope = _exact_act(g, case["act"])
            dg, du = dh * u * slope, dh * h
            both = torch.cat([weight("wg", e), weight("wu", e)])
            out[0][a:b] = torch.cat([dg, du], 1).mm(both)
            out[1][e], out[2][e] = dg.t().contiguous().mm(x), du.t().contiguous().mm(x)
        else:
            g, u = x.mm(weight("wg", e).t()), x.mm(weight("wu", e).t())
            out[0][a:b] = _exact_act(g, case["act"])[0] * u
            if outs == 3:
                out[1][a:b], out[2][a:b] = g, u
    return out[0] if outs == 1 else tuple(out)
