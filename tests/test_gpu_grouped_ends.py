"""Ends that no groups have: negative, falling, behind the last row. They are held to
0 .. T and to be no smaller than the ones before, and nothing outside of the matrices is
touched: every output and the workspace lie in a larger buffer, whose rest stays. The
outputs are those of the ends as they are held, bit for bit."""
import ctypes
import random

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
GUARD = 1 << 15   # bytes on either side

# (groups, rows, width, K): few rows and tiles, sums whole and in parts (asserted below), up
# to 64 groups and more
SHAPES = [(3, 20, 24, 32), (70, 150, 40, 96), (3, 600, 264, 272), (130, 300, 24, 48),
          (24, 9000, 1400, 160), (2, 5000, 48, 32), (70, 9000, 520, 1360), (1, 4100, 400, 3808),
          (1, 130, 936, 32)]


def wild(E, T, seed):
    """Ends of groups of T rows, one in four of them replaced; the last one by a large one
    in seed 0, by a small one in seed 1."""
    rng = random.Random(seed)
    ends = sorted(rng.randrange(T) for _ in range(E))
    for i in range(E):
        if rng.random() < 0.25:
            ends[i] = rng.choice([-2 ** 31, -1, 0, rng.randrange(T)])
    if E > 8:
        ends[E - 2] = rng.choice([T, T + 1, ends[E - 2]])
    if seed == 0:
        ends[-1] = rng.choice([T + 1, 2 ** 31 - 1])
    if seed == 1:
        ends[-1] = -5
    return ends


def held(ends, T):
    out, top = [], 0
    for x in ends:
        top = max(top, min(x, T))
        out.append(top)
    return out


class Guarded:
    """Buffers of a pattern around what a call may write."""

    def __init__(self):
        self.all = []

    def new(self, shape, dtype):
        n = torch.Size(shape).numel() * dtype.itemsize
        raw = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, n))
        return raw[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        for raw, n in self.all:
            assert (raw[:GUARD] == 0xA5).all() and (raw[GUARD + n:] == 0xA5).all()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def test_shapes():
    for kind in ("mma", "gated"):
        dx = [bmm.group_plan(f"grouped_{kind}_dx", *s) for s in SHAPES]
        dw = [bmm.group_plan(f"grouped_{kind}_dw", *s) for s in SHAPES]
        for plans in (dx, dw):
            assert {n > 1 for _, n in plans} == {False, True}
        assert {a[0] == b[0] == "128x128" for a, b in zip(dx, dw)} == {False, True}
        assert {bmm.group_plan(f"grouped_{kind}", *s)[0] == "few_rows" for s in SHAPES} == {False, True}


@pytest.mark.parametrize("dtype", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_wild_ends(shape, dtype):
    E, T, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(E + T)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)
    x, dy, g, u = rand(T, K), rand(T, N), rand(T, N), rand(T, N)
    w = ref.pack(rand(E, N, K) * 0.1)
    q, v = bmm.i8_quantize(rand(T, 32)), bmm.i8_pack(bmm.i8_quantize(rand(E, N, 32)))
    L, p, code = bmm.lib(), lambda t: t.data_ptr(), bmm._HALF_DTYPES[dtype]
    for seed in range(4):
        bad = wild(E, T, seed)
        good = held(bad, T)

        def run(ends, zero_tail):
            guard = Guarded()
            ends = torch.tensor(ends, dtype=torch.int64).to(torch.int32).cuda()
            y, h, hg, hu = (guard.new((T, N), dtype) for _ in range(4))
            d8, h8 = guard.new((T, N), torch.float32), guard.new((T, N), dtype)
            dx, dw, dx2, dwg, dwu = (guard.new(s, dtype) for s in
                                     ((T, K), (E, N, K), (T, K), (E, N, K), (E, N, K)))

            def d(act=0):
                return ctypes.byref(bmm.GroupedDesc(E, T, N, K, K, N, code, act, zero_tail))
            need = L.bmm_grouped_mma_backward_workspace_bytes(d())
            ws = guard.new((need,), torch.uint8)
            need2 = L.bmm_grouped_gated_backward_workspace_bytes(d(1))
            ws2 = guard.new((need2,), torch.uint8)
            elem = bmm._ELEM_DTYPES[dtype]
            i8 = ctypes.byref(bmm.I8Desc(E, T, N, 32, 32, N, bmm.ELEM_TYPES["f32"], 0, zero_tail))
            i8g = ctypes.byref(bmm.I8Desc(E, T, N, 32, 32, N, elem, 1, zero_tail))
            s = stream()
            for rc in (
                    L.bmm_grouped_mma(p(y), p(x), p(w), p(ends), d(), s),
                    L.bmm_grouped_gated(p(h), p(hg), p(hu), p(x), p(w), p(w), p(ends), d(1), s),
                    L.bmm_i8_mma(p(d8), p(q.codes), p(q.scales), p(v.codes), p(v.scales), p(ends), i8, s),
                    L.bmm_i8_gated(p(h8), p(q.codes), p(q.scales), p(v.codes), p(v.scales), p(v.codes),
                                   p(v.scales), p(ends), i8g, s),
                    L.bmm_grouped_mma_backward(p(dx), p(dw), p(dy), p(x), p(w), p(ends), d(), p(ws), need, s),
                    L.bmm_grouped_gated_backward(p(dx2), p(dwg), p(dwu), p(dy), p(g), p(u), p(x), p(w),
                                                 p(w), p(ends), d(1), p(ws2), need2, s)):
                assert rc == 0, L.bmm_last_error()
            torch.cuda.synchronize()
            guard.check()
            return y, h, hg, hu, d8, h8, dw, dx, dx2, dwg, dwu

        for zero_tail in (0, 1):
            for i, (a, b) in enumerate(zip(run(bad, zero_tail), run(good, zero_tail))):
                assert same(a, b), (seed, zero_tail, i)
