"""The counts of the products by groups (csrc/group_counts.h: the arithmetic that the
kernels use) against Python's whole numbers, up to 2^31 - 1 rows (CPU); and products of
that many rows on the GPU, which one launch of fewer than 2^32 threads has to hold."""
import ctypes
import gc
import os
import random
import subprocess

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests import ffn_ref as ref
from tests import grouped_ref as gref
from tests import test_gpu_grouped_tiles as tiles
from tests import test_grouped_coverage as coverage
from tests.test_ffn_refuse import L, P, err  # noqa: F401
from tests.test_grouped_refuse import i8

BF = torch.bfloat16
TOP = 2 ** 31 - 1
CSRC = os.path.join(os.path.dirname(bmm.__file__), "csrc")
SOURCE = """
#include "group_counts.h"
using namespace bmm::ffn;
extern "C" {
int full(int tm, int n) {
  return tm == 16 ? full_tiles<16>(n) : tm == 64 ? full_tiles<64>(n)
       : tm == 128 ? full_tiles<128>(n) : full_tiles<256>(n);
}
int small(int tm, int n) { return tm == 128 ? small_tiles<128>(n) : small_tiles<256>(n); }
void layout256(unsigned full, unsigned small, unsigned NT, unsigned splits, unsigned* out) {
  const auto l = row_layout<256>(full, small, NT, splits);
  out[0] = l.full;
  out[1] = l.last;
  out[2] = l.mixed;
  out[3] = l.cut;
}
void band(unsigned v, unsigned k, unsigned NT, unsigned* out) {
  const auto t = band_tile(v, k, NT);
  out[0] = t.row;
  out[1] = t.col;
}
int64_t most(int64_t T, int64_t E, int64_t tm) { return most_row_tiles(T, E, tm); }
void range32(int K, int values, unsigned split, unsigned splits, int* out) {
  const auto r = slab_range(int32_t(K), values, split, splits);
  out[0] = r.first;
  out[1] = r.end;
}
void range64(int64_t K, int values, unsigned split, unsigned splits, int64_t* out) {
  const auto r = slab_range(K, values, split, splits);
  out[0] = r.first;
  out[1] = r.end;
}
}
"""


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    here = tmp_path_factory.mktemp("counts")
    (here / "counts.cpp").write_text(SOURCE)
    out = str(here / "counts.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined",
                           "-fno-sanitize-recover=undefined", "-static-libubsan", "-shared", "-fPIC",
                           f"-I{CSRC}", str(here / "counts.cpp"), "-o", out])
    lib = ctypes.CDLL(out)
    lib.most.restype = ctypes.c_int64
    lib.most.argtypes = [ctypes.c_int64] * 3
    lib.range64.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_uint, ctypes.c_void_p]
    return lib


ROWS = sorted({n for c in (0, 16, 64, 128, 256, 512, 1 << 20, TOP) for d in range(-300, 301)
               for n in [c + d] if 0 <= n <= TOP})


@pytest.mark.parametrize("tm", [16, 64, 128, 256])
def test_row_tiles(counts, tm):
    for n in ROWS:
        small = int(tm == 256 and 0 < n % 256 <= 128)
        assert counts.full(tm, n) == -(-n // tm) - small, n
        if tm >= 128:
            assert counts.small(tm, n) == small, n
        for E in (1, 4096):   # all rows in one group, the others empty
            assert counts.most(n, E, tm) >= -(-n // tm)


@pytest.mark.parametrize("splits", [1, 2, 3, 12, 32])
def test_slabs(counts, splits):
    """Every slab is in one part, in order; a part starts at an even slab and may end one
    behind the last, which reads as zeros."""
    for out, fn in (((ctypes.c_int * 2)(), counts.range32), ((ctypes.c_int64 * 2)(), counts.range64)):
        for K in ROWS if splits == 1 else ROWS[::3]:
            slabs, at = -(-K // 32), 0
            for s in range(splits):
                fn(K, 32, s, splits, out)
                first, end = out
                assert 0 <= first <= slabs + 1 and first % 2 == 0 and end <= slabs + 1, (K, s)
                if end > first:
                    assert first == at, (K, s)
                    at = end
            assert at in (slabs, slabs + slabs % 2), (K, at)


def row_layout(counts, groups, NT):
    """The kernel's layout of these groups' 256-row tiles, as test_grouped_coverage's."""
    out = (ctypes.c_uint * 4)()
    full = sum(counts.full(256, n) for n in groups)
    counts.layout256(full, sum(counts.small(256, n) for n in groups), NT, 1, out)
    tiles, last, mixed, cut = out
    some = any(0 < n % 256 <= 128 for n in groups)
    return bool(mixed) and some, last > 0, cut > 0, tiles * NT // 256 > 1


def test_layouts_are_the_kernels(counts):
    """The copy of the rule by which the layouts' coverage is asserted gives what the kernel
    does, for the shapes there and others."""
    rng = random.Random(1)
    for groups, n, _ in tiles.LAYOUTS:
        for tn in (128, 192, 256):
            NT = -(-n // tn)
            assert row_layout(counts, groups, NT) == coverage.layout(groups, NT)
    for _ in range(3000):
        groups = [rng.choice([0, rng.randrange(700), 256 * rng.randrange(9), 256 * rng.randrange(9) + 3])
                  for _ in range(rng.randrange(1, 30))]
        NT = rng.randrange(1, 33)
        if any(groups):
            assert row_layout(counts, groups, NT) == coverage.layout(groups, NT), (groups, NT)


def test_every_tile_of_a_group_once(counts):
    out = (ctypes.c_uint * 2)()
    for k in (1, 2, 5, 6, 7, 11, 12, 13, 18, 19, 64, 100):
        for NT in (1, 3, 16):
            got = []
            for v in range(k * NT):
                counts.band(v, k, NT, out)
                got.append(tuple(out))
            assert sorted(got) == [(r, c) for r in range(k) for c in range(NT)]


def workgroups(tile, splits, T, N, E=1):
    tm, tn = map(int, tile.split("x"))
    return (T + (E + 1) * (tm - 1)) // tm * -(-N // tn) * splits + 128


@pytest.mark.parametrize("groups,T", [(1, TOP), (7, TOP), (4096, TOP), (4096, TOP - 600000)])
@pytest.mark.parametrize("product,N,K", [
    ("grouped_mma", 8, 16), ("grouped_mma", 48, 32), ("grouped_mma_dx", 8, 16), ("grouped_mma_dx", 64, 48),
    ("grouped_gated", 8, 16), ("grouped_gated_dx", 8, 16), ("i8_mma", 8, 32), ("i8_gated", 16, 32)])
def test_most_rows_in_one_launch(product, groups, T, N, K):
    tile, splits = bmm.group_plan(product, groups, T, N, K)
    width = K if product.endswith("dx") else 2 * N if "gated" in product else N
    assert workgroups(tile, splits, T, width, groups) < 1 << 24, tile


@pytest.mark.parametrize("M", [(1 << 31) - 128, 1 << 31, (1 << 32) - 40000])
def test_most_rows_of_one_weight(M):
    for tile, splits in (bmm.group_plan("i8_mma", 0, min(M, TOP), 8, 32), bmm.ffn_plan("gated", 1, M, 8, 16),
                         bmm.ffn_plan("mx4_mma", 1, M, 64, 32)):
        assert tile.startswith("256"), tile


def test_more_tiles_than_a_launch_holds(L):  # noqa: F811
    """Refused on the host, with the reason."""
    assert i8(L, D=1 << 62, M=1 << 33, N=8, K=32, ld_a=32, ld_d=8) < 0
    assert "more tiles than one launch may have" in err(L)


@pytest.fixture
def much_memory():
    """Up to 160 GiB, given back at the end."""
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_weight_gradient_of_the_most_rows(much_memory):
    """2^31 - 1 rows in one group, and in three; all of them zeros but a few at the ends of
    the groups and of the sums' parts."""
    K, N = 16, 8
    x = torch.zeros(TOP, K, dtype=BF, device="cuda")
    dy = torch.zeros(TOP, N, dtype=BF, device="cuda")
    at = torch.tensor([0, 1, 5000, TOP // 2, TOP // 2 + 1, TOP - 300, TOP - 32, TOP - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x[at] = torch.randint(-2, 3, (len(at), K), generator=gen, device="cuda").to(BF)
    dy[at] = torch.randint(-2, 3, (len(at), N), generator=gen, device="cuda").to(BF)
    for rows in ([TOP], [1, TOP - 301, 300], [TOP // 2 + 1, 0, TOP - TOP // 2 - 1]):
        E = len(rows)
        w = ref.pack(torch.zeros(E, N, K, dtype=BF, device="cuda"))
        _, dw = bmm.grouped_mma_backward(dy, x, w, gref.ends_of(rows).cuda(), need_dx=False)
        for e, r in gref.groups(rows):
            mine = at[(at >= r.start) & (at < r.stop)]
            want = dy[mine].double().t().contiguous() @ x[mine].double()
            assert torch.equal(dw[e].double(), want), (rows, e)
        assert all((dw[e] == 0).all() for e in range(E) if rows[e] == 0)


@pytest.mark.gpu
def test_products_of_the_most_rows(much_memory):
    """Forward product and dX of 2^31 - 1 rows, zeros but for a few; every output written."""
    K, N = 16, 8
    at = torch.tensor([0, 255, 256, 5000, TOP // 2, TOP - 257, TOP - 256, TOP - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    rows = [5000, TOP - 5257, 0, 257]
    ends = gref.ends_of(rows).cuda()
    w = torch.randint(-2, 3, (4, N, K), generator=gen, device="cuda").to(BF)
    group = torch.bucketize(at, ends.long(), right=True)

    def only(t, want):
        """t is `want` in the rows `at` and zero elsewhere."""
        assert torch.equal(t[at].double(), want)
        t[at] = 0
        assert not any(part.any() for part in t.split(1 << 27))
    x = torch.zeros(TOP, K, dtype=BF, device="cuda")
    x[at] = torch.randint(-2, 3, (len(at), K), generator=gen, device="cuda").to(BF)
    y = torch.full((TOP, N), float("nan"), dtype=BF, device="cuda")
    bmm.grouped_mma(x, ref.pack(w), ends, out=y)
    only(y, (w[group].double() * x[at].double()[:, None]).sum(2))
    y[at] = torch.randint(-2, 3, (len(at), N), generator=gen, device="cuda").to(BF)
    dx, _ = bmm.grouped_mma_backward(y, x, ref.pack(w), ends, need_dw=False)
    only(dx, (w[group].double() * y[at].double()[:, :, None]).sum(1))
