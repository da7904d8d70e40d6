"""The feed-forward operators on real work: inputs, plain forms and exact values.

Five operators, each over the sizes that a program meets:

- ``gated``           H = act(X Wg^T) * (X Wu^T), both projections of a gated
                      feed-forward block, with the projections kept for the
                      backward pass where a training step asks for them;
- ``gated_backward``  dX, dWg and dWu of that block from dH and the kept
                      projections;
- ``mx4_quantize``    values to microscaled 4-bit floats (blocks of 32 along
                      K, one power-of-two scale each) and back;
- ``mx4_mma``         D = X W^T with W held in 4 bits and X quantised on the
                      way in;
- ``mx4_gated``       the gated block's projections with 4-bit operands.

``run`` computes them in elementary torch operations in 32 bits, rounded once
at the end, or, with ``own`` set, through the package's entry points.
``exact`` computes the same outputs in 64 bits from the definitions.

Weights of the bf16/f16 operators are kept in the package's packed B layout
(8 rows x 16 K values an atom) beside the row-major matrix; 4-bit weights are
kept as codes and scales only, in the layout of ``mx4_values`` below.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# The eight magnitudes of a 4-bit float (2 exponent bits, 1 mantissa bit).
MX4_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ----

def listed():
    """Twelve cases: the smallest calls, ordinary ones and the largest."""
    return [
        # one token through a block whose weights (2 x 64 MiB) stream from memory
        dict(name="gated_token", op="gated", M=1, K=4096, F=8192, dtype="bf16", act="silu",
             pad=0, save=False),
        # a ragged chunk of tokens, X a column slice of a wider buffer
        dict(name="gated_chunk_f16", op="gated", M=1003, K=2048, F=5464, dtype="f16",
             act="gelu_tanh", pad=64, save=False),
        # the forward pass of a training step, projections kept
        dict(name="gated_train", op="gated", M=8192, K=4096, F=8192, dtype="bf16", act="silu",
             pad=0, save=True),
        # a short sequence through a small block
        dict(name="backward_short_f16", op="gated_backward", M=45, K=528, F=1368, dtype="f16",
             act="gelu", pad=0),
        # many tokens through a small block: the weight gradients sum over all of them
        dict(name="backward_long", op="gated_backward", M=32773, K=512, F=1024, dtype="bf16",
             act="silu", pad=0),
        # the backward pass of a training step
        dict(name="backward_train", op="gated_backward", M=8192, K=4096, F=8192, dtype="bf16",
             act="silu", pad=0),
        # one token's activations, on their way into a 4-bit product
        dict(name="mx4_quantize_token", op="mx4_quantize", rows=1, K=16384, dtype="bf16", pad=0),
        # a weight matrix brought to 4 bits once, and read back
        dict(name="mx4_quantize_weight", op="mx4_quantize", rows=8192, K=8192, dtype="bf16",
             pad=0),
        # one token through a 16384 x 16384 4-bit layer (128 MiB of codes)
        dict(name="mx4_token", op="mx4_mma", M=1, N=16384, K=16384, dtype="bf16", out="bf16"),
        # a full batch through an 8192 x 8192 4-bit layer
        dict(name="mx4_square", op="mx4_mma", M=8192, N=8192, K=8192, dtype="bf16", out="bf16"),
        # a few tokens decoded together through a 4-bit gated block
        dict(name="mx4_gated_decode", op="mx4_gated", M=7, K=4096, F=8192, dtype="bf16",
             act="silu", out="bf16"),
        # a prompt through a 4-bit gated block
        dict(name="mx4_gated_prompt_f16", op="mx4_gated", M=4095, K=4096, F=8192, dtype="f16",
             act="gelu_tanh", out="f16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["gated", "gated_backward", "mx4_quantize", "mx4_mma", "mx4_gated"])
    half = rng.choice(["bf16", "f16"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
    if op == "mx4_quantize":
        return dict(op=op, rows=_log_int(rng, 1, 8192), K=32 * _log_int(rng, 1, 256),
                    dtype=rng.choice(["bf16", "f16", "f32"]), pad=rng.choice([0, 8, 96]))
    if op == "mx4_mma":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=8 * _log_int(rng, 8, 1024),
                    K=32 * _log_int(rng, 2, 256), dtype=half,
                    out=rng.choice(["bf16", "f16", "f32"]))
    if op == "mx4_gated":
        return dict(op=op, M=_log_int(rng, 1, 4096), K=32 * _log_int(rng, 2, 128),
                    F=8 * _log_int(rng, 8, 1024), dtype=half, act=act, out=half)
    # tokens up to 8192 in a wide block, up to 32768 in a narrow one
    K, F = 16 * _log_int(rng, 4, 256), 8 * _log_int(rng, 8, 1024)
    M = _log_int(rng, 1, 32768 if K * F <= 1 << 20 else 8192)
    case = dict(op=op, M=M, K=K, F=F, dtype=half, act=act, pad=rng.choice([0, 8, 64]))
    if op == "gated":
        case["save"] = rng.random() < 0.5
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
    """A row-major (N, K) weight as packed B words (1, N/8, K/16, 8, 8)."""
    n, k = w.shape
    atoms = w.view(torch.int16).reshape(1, n // 8, 8, k // 16, 16).permute(0, 1, 3, 2, 4)
    return atoms.contiguous().view(torch.int32)


def _mx4_weight(gen, rows, K):
    """A 4-bit weight as a checkpoint holds it: (codes, scales) in the layout
    of mx4_values. Codes have the histogram of normal values, scales vary by
    a few powers of two around 1 / sqrt(K)."""
    r16, s128, s512 = -(-rows // 16), -(-K // 128), -(-K // 512)
    v = _normal(gen, r16 * 16, s128 * 128).abs_() * 2
    code = torch.bucketize(v, torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.], device="cuda"))
    code = code + 8 * (_normal(gen, r16 * 16, s128 * 128) < 0)
    code = code.to(torch.uint8)
    code[rows:] = 0
    code[:, K:] = 0
    code = code.reshape(1, r16, 16, s128, 4, 16, 2).permute(0, 1, 3, 4, 2, 5, 6)
    codes = (code[..., 0] + 16 * code[..., 1]).contiguous()
    mid = 127 - int(round(math.log2(math.sqrt(K)))) - 1
    scale = torch.randint(mid - 2, mid + 2, (r16 * 16, s512 * 16), generator=gen, device="cuda")
    scale[rows:] = 0
    scale[:, K // 32:] = 0
    scales = scale.to(torch.uint8).reshape(1, r16, 16, s512, 4, 4).permute(0, 1, 3, 5, 2, 4)
    return codes, scales.contiguous()


def prepare(case, seed):
    """The inputs of one pass, made from the seed alone."""
    gen, dtype = _generator(seed), DTYPES[case["dtype"]]
    s = dict(case=case, op=case["op"])
    if s["op"] in ("gated", "gated_backward"):
        M, K, F = case["M"], case["K"], case["F"]
        s["x"] = _rows(gen, M, K, case["pad"], dtype)
        for name in ("wg", "wu"):
            w = (_normal(gen, F, K) / math.sqrt(K)).to(dtype)
            s[name], s[name + "_packed"] = w, _packed(w)
        if s["op"] == "gated_backward":
            s["g"], s["u"] = s["x"] @ s["wg"].t(), s["x"] @ s["wu"].t()
            s["dh"] = (_normal(gen, M, F) / 8).to(dtype)
    elif s["op"] == "mx4_quantize":
        # rows of different sizes, some blocks all zero, some with an outlier
        x = _normal(gen, case["rows"], case["K"] + case["pad"])
        x *= torch.exp2(torch.randint(-6, 7, (case["rows"], 1), generator=gen, device="cuda"))
        pick = torch.randint(0, 64, x.shape, generator=gen, device="cuda")
        x = torch.where(pick == 0, x * 16, x)
        zero = torch.randint(0, 16, (case["rows"], x.shape[1] // 8 + 1), generator=gen,
                             device="cuda") == 0
        x = torch.where(zero.repeat_interleave(8, 1)[:, :x.shape[1]], 0.0, x)
        s["x"] = x.to(dtype)[:, :case["K"]]
    else:
        s["x"] = _rows(gen, case["M"], case["K"], 0, dtype)
        for name in ("w",) if s["op"] == "mx4_mma" else ("wg", "wu"):
            s[name] = _mx4_weight(gen, case["N" if s["op"] == "mx4_mma" else "F"], case["K"])
    return s


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


def _mx4_round(x):
    """x (rows, K) to the nearest values that 4 bits and a block's scale hold."""
    rows, K = x.shape
    b = x.float().reshape(rows, K // 32, 32)
    top = b.abs().amax(2, keepdim=True)
    # the scale 2^e: the largest power of two at or below the block's largest
    # magnitude, less two, so that this magnitude lands in [4, 8)
    e = torch.clamp(torch.frexp(top).exponent - 3, -127, 127)
    e = torch.where(top > 0, e, torch.zeros_like(e))
    v = torch.ldexp(b, -e)
    m = v.abs()
    q = (0.5 * (m > 0.25) + 0.5 * (m >= 0.75) + 0.5 * (m > 1.25) + 0.5 * (m >= 1.75)
         + 1.0 * (m > 2.5) + 1.0 * (m >= 3.5) + 2.0 * (m > 5.0))
    return torch.ldexp(torch.where(v < 0, -q, q), e).reshape(rows, K)


def mx4_values(codes, scales, rows, K, dtype=torch.float32):
    """The (rows, K) values of a 4-bit operand.

    codes  (1, rows/16, K/128, 4, 16, 16) bytes: [.., r, s, g, i, j] holds row
           16 r + i, K values 128 s + 32 g + 2 j (low half) and the next one
           (high half): a sign bit and an index into MX4_MAGNITUDES.
    scales (1, rows/16, K/512, 4, 16, 4) bytes: [.., r, q, g, i, t] is 127 plus
           the exponent of row 16 r + i, K values 512 q + 128 t + 32 g and on.
    """
    table = torch.tensor(MX4_MAGNITUDES + tuple(-m for m in MX4_MAGNITUDES), device=codes.device,
                         dtype=dtype)
    _, r16, s128 = codes.shape[:3]
    c = codes.permute(0, 1, 4, 2, 3, 5).reshape(r16 * 16, s128 * 64)
    v = torch.stack([table[(c & 15).long()], table[(c >> 4).long()]], 2)
    v = v.reshape(r16 * 16, s128 * 4, 32)
    e = scales.permute(0, 1, 4, 2, 5, 3).reshape(r16 * 16, -1)[:, :s128 * 4]
    v = v * torch.exp2(e.to(dtype) - 127)[:, :, None]
    return v.reshape(r16 * 16, s128 * 128)[:rows, :K]


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "gated":
        dtype = s["x"].dtype
        x = s["x"].float()
        g, u = x @ s["wg"].float().t(), x @ s["wu"].float().t()
        h = (_act(g, case["act"]) * u).to(dtype)
        return (h, g.to(dtype), u.to(dtype)) if case["save"] else h
    if op == "gated_backward":
        dtype = s["x"].dtype
        g, u, dh, x = s["g"].float(), s["u"].float(), s["dh"].float(), s["x"].float()
        dg, du = dh * u * _act_slope(g, case["act"]), dh * _act(g, case["act"])
        dx = dg @ s["wg"].float() + du @ s["wu"].float()
        return dx.to(dtype), (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)
    if op == "mx4_quantize":
        return _mx4_round(s["x"]).to(s["x"].dtype)
    x, out = _mx4_round(s["x"]), DTYPES[case["out"]]
    if op == "mx4_mma":
        return (x @ mx4_values(*s["w"], case["N"], case["K"]).t()).to(out)
    g = x @ mx4_values(*s["wg"], case["F"], case["K"]).t()
    u = x @ mx4_values(*s["wu"], case["F"], case["K"]).t()
    return (_act(g, case["act"]) * u).to(out)


def _own(s):
    import bf16_matrix_multiply_amd as bmm

    case, op = s["case"], s["op"]
    if op == "gated":
        return bmm.gated(s["x"], s["wg_packed"], s["wu_packed"], act=case["act"],
                         save=case["save"])
    if op == "gated_backward":
        return bmm.gated_backward(s["dh"], s["g"], s["u"], s["x"], s["wg_packed"], s["wu_packed"],
                                  act=case["act"])
    x = bmm.mx4_quantize(s["x"])
    if op == "mx4_quantize":
        return bmm.mx4_dequantize(x, dtype=s["x"].dtype)
    if op == "mx4_mma":
        w = bmm.Mx4Operand(*s["w"], case["N"], case["K"])
        return bmm.mx4_mma(x, w, dtype=DTYPES[case["out"]])
    wg = bmm.Mx4Operand(*s["wg"], case["F"], case["K"])
    wu = bmm.Mx4Operand(*s["wu"], case["F"], case["K"])
    return bmm.mx4_gated(x, wg, wu, act=case["act"], dtype=DTYPES[case["out"]])


def run(state):
    """One pass through the case's operator."""
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    """Bytes (each input read once, each output written once) and operations."""
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    b = size[case["dtype"]]
    if op == "gated":
        M, K, F = case["M"], case["K"], case["F"]
        outs = 3 if case["save"] else 1
        return dict(bytes=b * (M * K + 2 * F * K + outs * M * F), flops=4 * M * F * K)
    if op == "gated_backward":
        M, K, F = case["M"], case["K"], case["F"]
        return dict(bytes=b * (3 * M * F + 2 * M * K + 4 * F * K), flops=8 * M * F * K)
    if op == "mx4_quantize":
        n = case["rows"] * case["K"]   # values in and out, codes and scales out and in
        return dict(bytes=2 * b * n + 2 * (n // 2 + n // 32), flops=4 * n)
    M, K, out = case["M"], case["K"], size[case["out"]]
    n = case["N"] if op == "mx4_mma" else 2 * case["F"]
    cols = case["N"] if op == "mx4_mma" else case["F"]
    return dict(bytes=b * M * K + n * K // 2 + n * K // 32 + out * M * cols, flops=2 * M * n * K)


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


def _exact_mx4(x):
    """The 4-bit rounding of x in 64 bits: half steps of even parity."""
    b = x.double().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top)), torch.zeros_like(top))
    # log2 may round up to a whole number just below a power of two
    e = torch.where(torch.exp2(e) > top, e - 1, e)
    scale = torch.exp2(torch.clamp(torch.where(top > 0, e - 2, e), -127, 127))
    v = b / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
    return (torch.clamp(torch.round(v / step) * step, -6, 6) * scale).reshape(x.shape)


def _exact_weight(weight, rows, K):
    """(rows, K) values of codes and scales, decoded field by field."""
    codes, scales = (t[0].cpu() for t in weight)
    low, high = codes & 15, codes >> 4
    c = torch.stack([low, high], -1).flatten(-2)            # (r, s, g, i, 32)
    c = c.permute(0, 3, 1, 2, 4).flatten(0, 1).flatten(1)   # (row, K)
    sign, expo, man = c >> 3, (c >> 1) & 3, (c & 1).double()
    expo = expo.double()
    v = torch.where(expo == 0, man / 2, (1 + man / 2) * torch.exp2(expo - 1))
    v = torch.where(sign == 1, -v, v)
    e = scales.permute(0, 3, 1, 4, 2).flatten(0, 1).flatten(1).double()   # (row, K / 32)
    v = v[:rows, :K] * torch.exp2(e - 127).repeat_interleave(32, 1)[:rows, :K]
    return v.cuda()


def exact(case, seed):
    """The outputs of ``run`` for the case's inputs, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        x = s["x"].double()
        g, u = x.mm(s["wg"].double().t()), x.mm(s["wu"].double().t())
        h = _exact_act(g, case["act"])[0] * u
        return (h, g, u) if case["save"] else h
    if op == "gated_backward":
        g, u, dh = s["g"].double(), s["u"].double(), s["dh"].double()
        a, slope = _exact_act(g, case["act"])
        dg, du, x = dh * u * slope, dh * a, s["x"].double()
        dx = torch.cat([dg, du], 1).mm(torch.cat([s["wg"], s["wu"]]).double())
        return dx, dg.t().contiguous().mm(x), du.t().contiguous().mm(x)
    q = _exact_mx4(s["x"])
    if op == "mx4_quantize":
        return q
    if op == "mx4_mma":
        return q.mm(_exact_weight(s["w"], case["N"], case["K"]).t())
    g = q.mm(_exact_weight(s["wg"], case["F"], case["K"]).t())
    u = q.mm(_exact_weight(s["wu"], case["F"], case["K"]).t())
    return _exact_act(g, case["act"])[0] * u
