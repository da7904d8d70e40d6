"""Refusals of the products by groups and of 8-bit integers, on the CPU: every invalid
argument is rejected on the host before any HIP call, and empty problems are no-ops."""
import ctypes

import pytest
import torch

import bf16_matrix_multiply_amd as bmm
from tests.test_devices import BF, I32, empty, gpus  # noqa: F401 (a fixture)
from tests.test_ffn_refuse import EALIGN, EINVAL, EOVERLAP, L, P, err  # noqa: F401

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer")
ENDS = P[11]


def desc(groups=3, T=5, N=24, K=32, ld_x=32, ld_y=24, dtype=1, act=0, zero_tail=1):
    return ctypes.byref(bmm.GroupedDesc(groups, T, N, K, ld_x, ld_y, dtype, act, zero_tail))


def mma(L, Y=P[0], X=P[3], W=P[4], ends=ENDS, **kw):
    return L.bmm_grouped_mma(Y, X, W, ends, desc(**kw), None)


def gated(L, H=P[0], G=0, U=0, X=P[3], Wg=P[4], Wu=P[5], ends=ENDS, **kw):
    return L.bmm_grouped_gated(H, G, U, X, Wg, Wu, ends, desc(**kw), None)


def mma_backward(L, dX=P[0], dW=P[1], dY=P[2], X=P[3], W=P[4], ends=ENDS, ws=P[6], ws_bytes=1 << 30,
                 **kw):
    return L.bmm_grouped_mma_backward(dX, dW, dY, X, W, ends, desc(**kw), ws, ws_bytes, None)


def gated_backward(L, dX=P[0], dWg=P[1], dWu=P[2], dH=P[7], G=P[8], U=P[9], X=P[3], Wg=P[4], Wu=P[5],
                   ends=ENDS, ws=P[6], ws_bytes=1 << 30, **kw):
    return L.bmm_grouped_gated_backward(dX, dWg, dWu, dH, G, U, X, Wg, Wu, ends, desc(**kw), ws,
                                        ws_bytes, None)


DESC = [
    (dict(dtype=2), EINVAL, "dtype"),
    (dict(act=-1), EINVAL, "act"),
    (dict(zero_tail=2), EINVAL, "zero_tail"),
    (dict(groups=-1), EINVAL, "negative"),
    (dict(T=-1), EINVAL, "negative"),
    (dict(groups=0), EINVAL, "must be a group"),
    (dict(groups=4097), EINVAL, "too large"),
    (dict(T=1 << 31), EINVAL, "too large"),
    (dict(N=(1 << 20) + 8, ld_y=1 << 21), EINVAL, "too large"),
    (dict(K=1 << 22, ld_x=1 << 22), EINVAL, "too large"),
    (dict(groups=4096, N=1 << 20, K=1 << 20, ld_x=1 << 20, ld_y=1 << 20), EINVAL, "too large"),
    (dict(N=20), EINVAL, "multiple of 8"),
    (dict(K=24), EINVAL, "multiple of 16"),
    (dict(ld_x=16), EINVAL, "ld_x"),
    (dict(ld_y=16), EINVAL, "ld_y"),
    (dict(ld_x=(1 << 21) + 8), EINVAL, "2^21"),
    (dict(ld_x=36), EALIGN, "multiples of 8"),
    (dict(ld_y=28), EALIGN, "multiples of 8"),
]


@pytest.mark.parametrize("fn", [mma, gated, mma_backward, gated_backward])
@pytest.mark.parametrize("kw,code,needle", DESC)
def test_extents(L, fn, kw, code, needle):  # noqa: F811
    assert fn(L, **kw) == code, err(L)
    assert needle in err(L)


@pytest.mark.parametrize("fn,kw,code,needle", [
    (mma, dict(act=1), EINVAL, "without a gate"),
    (mma_backward, dict(act=2), EINVAL, "without a gate"),
    (gated, dict(act=4), EINVAL, "bmm_act"),
    (mma, dict(ends=0), EINVAL, "ends is null"),
    (gated, dict(ends=0), EINVAL, "ends is null"),
    (mma_backward, dict(ends=0), EINVAL, "ends is null"),
    (gated_backward, dict(ends=0), EINVAL, "ends is null"),
    (mma, dict(ends=ENDS + 2), EALIGN, "ends must be"),
    (mma, dict(Y=0), EINVAL, "Y is null"),
    (mma, dict(X=0), EINVAL, "X is null"),
    (mma, dict(W=0), EINVAL, "W is null"),
    (gated, dict(Wu=0), EINVAL, "Wu is null"),
    (gated, dict(G=P[1]), EINVAL, "both or neither"),
    (mma, dict(Y=P[0] + 8), EALIGN, "Y must be"),
    (mma, dict(X=P[3] + 2), EALIGN, "X must be"),
    (gated, dict(Wu=P[5] + 4), EALIGN, "Wu must be"),
    (mma, dict(Y=P[3] + 64), EOVERLAP, "Y overlaps X"),
    (mma, dict(Y=P[4]), EOVERLAP, "Y overlaps W"),
    (mma, dict(Y=ENDS), EOVERLAP, "Y overlaps ends"),
    (gated, dict(G=P[0], U=P[2]), EOVERLAP, "H overlaps G"),
    (mma_backward, dict(dX=0, dW=0), EINVAL, "no gradient"),
    (gated_backward, dict(dX=0, dWg=0, dWu=0), EINVAL, "no gradient"),
    (gated_backward, dict(dWu=0), EINVAL, "both or neither"),
    (mma_backward, dict(dY=0), EINVAL, "dY is null"),
    (gated_backward, dict(G=0), EINVAL, "G is null"),
    (mma_backward, dict(W=0), EINVAL, "W is null"),
    (mma_backward, dict(X=0), EINVAL, "X is null"),
    (gated_backward, dict(ws_bytes=8), EINVAL, "workspace_bytes"),
    (gated_backward, dict(ws=0), EINVAL, "workspace is null"),
    (gated_backward, dict(ws=P[6] + 8), EALIGN, "workspace must be"),
    (gated_backward, dict(ws=P[7]), EOVERLAP, "overlaps"),
    (mma_backward, dict(dX=P[1]), EOVERLAP, "dX overlaps dW"),
    (mma_backward, dict(dW=P[3]), EOVERLAP, "dW overlaps X"),
])
def test_arguments(L, fn, kw, code, needle):  # noqa: F811
    assert fn(L, **kw) == code, err(L)
    assert needle in err(L)


def test_null_descriptors(L):  # noqa: F811
    for call in (lambda: L.bmm_grouped_mma(P[0], P[1], P[2], ENDS, None, None),
                 lambda: L.bmm_grouped_gated(P[0], 0, 0, P[1], P[2], P[3], ENDS, None, None),
                 lambda: L.bmm_grouped_mma_backward_workspace_bytes(None),
                 lambda: L.bmm_grouped_gated_backward_workspace_bytes(None),
                 lambda: L.bmm_i8_mma(P[0], P[1], P[2], P[3], P[4], None, None, None)):
        assert call() == EINVAL and "descriptor" in err(L)


def test_empty_is_noop(L):  # noqa: F811
    for kw in (dict(T=0), dict(N=0, ld_y=0)):
        assert mma(L, Y=0, X=0, W=0, **kw) == 0 and gated(L, H=0, X=0, Wg=0, Wu=0, **kw) == 0
    for kw in (dict(K=0, ld_x=0), dict(T=0, N=0, ld_y=0)):
        assert mma_backward(L, dY=0, X=0, W=0, ws=0, ws_bytes=0, **kw) == 0
        assert gated_backward(L, dH=0, G=0, U=0, X=0, Wg=0, Wu=0, ws=0, ws_bytes=0, **kw) == 0


@pytest.mark.parametrize("shape", [(1, 1, 8, 16), (5, 777, 1000, 528), (64, 24576, 1408, 2048), (3, 0, 24, 32),
                                   (4096, 7, 24, 32), (8, 384, 776, 1024), (2, 5000, 48, 32)])
def test_workspaces_hold_their_parts(shape):
    """[dG | dU] and its peaks, and the partial sums of a split product (of both where one
    launch makes them)."""
    E, T, N, K = shape
    for gated_too in (False, True):
        name = "grouped_gated" if gated_too else "grouped_mma"
        need = getattr(bmm, name + "_backward_workspace_bytes")(E, T, N, K)
        width = 2 * (-(-N // 32) * 32) if gated_too else N
        slopes = 2 * T * width if gated_too else 0
        dx_tile, dx = bmm.group_plan(name + "_dx", E, T, N, K)
        dw_tile, dw = bmm.group_plan(name + "_dw", E, T, N, K)
        parts = [4 * dx * T * K if dx > 1 else 0, 4 * dw * E * width * K if dw > 1 else 0]
        both = dx_tile == dw_tile == "128x128"
        assert need >= slopes + (sum(parts) if both else max(parts))
        assert need <= slopes + sum(parts) + 8192


# ---- 8-bit integers ----

def i8(L, D=P[0], A=P[1], sa=P[2], B=P[3], sb=P[4], ends=0, batch=1, M=5, N=24, K=64, ld_a=64,  # noqa: F811
       ld_d=24, et=3, act=0, zero_tail=0):
    d = bmm.I8Desc(batch, M, N, K, ld_a, ld_d, et, act, zero_tail)
    return L.bmm_i8_mma(D, A, sa, B, sb, ends, ctypes.byref(d), None)


def i8_gated(L, D=P[0], A=P[1], sa=P[2], B=P[3], sb=P[4], C=P[5], sc=P[6], ends=0, batch=1, M=5,  # noqa: F811
             N=24, K=64, ld_a=64, ld_d=24, et=3, act=0, zero_tail=0):
    d = bmm.I8Desc(batch, M, N, K, ld_a, ld_d, et, act, zero_tail)
    return L.bmm_i8_gated(D, A, sa, B, sb, C, sc, ends, ctypes.byref(d), None)


@pytest.mark.parametrize("fn", [i8, i8_gated])
@pytest.mark.parametrize("kw,code,needle", [
    (dict(et=0), EINVAL, "elem_type"),
    (dict(et=4), EINVAL, "elem_type"),
    (dict(act=-1), EINVAL, "act"),
    (dict(zero_tail=-1), EINVAL, "zero_tail"),
    (dict(batch=-1), EINVAL, "negative"),
    (dict(M=-1), EINVAL, "negative"),
    (dict(N=20), EINVAL, "multiple of 8"),
    (dict(K=48), EINVAL, "multiple of 32"),
    (dict(K=1 << 17, ld_a=1 << 17), EINVAL, "too large"),
    (dict(N=(1 << 20) + 8, ld_d=1 << 21), EINVAL, "too large"),
    (dict(M=1 << 41), EINVAL, "too large"),
    (dict(M=1 << 31, ends=ENDS), EINVAL, "too large"),
    (dict(batch=4097, ends=ENDS), EINVAL, "too large"),
    (dict(batch=0, ends=ENDS), EINVAL, "must be a group"),
    (dict(ld_a=32), EINVAL, "ld_a"),
    (dict(ld_d=16), EINVAL, "ld_d"),
    (dict(ld_a=(1 << 22) + 16), EINVAL, "2^22"),
    (dict(ld_a=72), EALIGN, "multiple of 16"),
    (dict(ld_d=28), EALIGN, "of 8"),
    (dict(D=0), EINVAL, "is null"),
    (dict(A=0), EINVAL, "is null"),
    (dict(sa=0), EINVAL, "scales is null"),
    (dict(B=0), EINVAL, "is null"),
    (dict(sb=0), EINVAL, "scales is null"),
    (dict(A=P[1] + 8), EALIGN, "must be 16-byte"),
    (dict(sb=P[4] + 4), EALIGN, "must be 16-byte"),
    (dict(sa=P[2] + 2), EALIGN, "must be 4-byte"),
    (dict(ends=ENDS + 1), EALIGN, "ends must be"),
    (dict(D=P[1]), EOVERLAP, "overlaps"),
    (dict(D=P[2]), EOVERLAP, "overlaps"),
    (dict(D=P[4]), EOVERLAP, "overlaps"),
    (dict(D=ENDS, ends=ENDS), EOVERLAP, "overlaps ends"),
])
def test_i8_product(L, fn, kw, code, needle):  # noqa: F811
    assert fn(L, **kw) == code, err(L)
    assert needle in err(L)


def test_i8_gated(L):  # noqa: F811
    assert i8_gated(L, et=1) == EINVAL and "elem_type" in err(L)
    assert i8_gated(L, act=4) == EINVAL and "bmm_act" in err(L)
    assert i8(L, act=1) == EINVAL and "without a gate" in err(L)
    assert i8_gated(L, C=0) == EINVAL and "Wu is null" in err(L)
    assert i8_gated(L, sc=P[6] + 4) == EALIGN and "Wu_scales" in err(L)


def test_i8_empty_is_noop(L):  # noqa: F811
    for fn in (i8, i8_gated):
        for kw in (dict(batch=0), dict(M=0), dict(N=0, ld_d=0)):
            assert fn(L, D=0, A=0, sa=0, B=0, sb=0, **kw) == 0


def i8_quantize(L, codes=P[0], scales=P[1], src=P[2], batch=1, rows=5, K=64, ld=64, et=3):  # noqa: F811
    return L.bmm_i8_quantize(codes, scales, src, batch, rows, K, ld, et, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(et=4), EINVAL, "elem_type"), (dict(rows=-1), EINVAL, "negative"),
    (dict(K=48), EINVAL, "multiple of 32"), (dict(K=1 << 22, ld=1 << 22), EINVAL, "too large"),
    (dict(ld=32), EINVAL, "ld"), (dict(ld=68), EALIGN, "multiple of 8"),
    (dict(rows=1 << 40, batch=1 << 20), EINVAL, "too large"),
    (dict(src=0), EINVAL, "matrix is null"), (dict(codes=0), EINVAL, "codes is null"),
    (dict(scales=0), EINVAL, "scales is null"), (dict(src=P[2] + 8), EALIGN, "16-byte"),
    (dict(codes=P[0] + 8), EALIGN, "16-byte"), (dict(scales=P[1] + 2), EALIGN, "4-byte"),
    (dict(codes=P[2]), EOVERLAP, "overlaps"), (dict(scales=P[2] + 16), EOVERLAP, "overlaps"),
    (dict(scales=P[0] + 64), EOVERLAP, "overlaps"),
])
def test_i8_quantize(L, kw, code, needle):  # noqa: F811
    assert i8_quantize(L, **kw) == code, err(L)
    assert needle in err(L)


def test_i8_quantize_empty(L):  # noqa: F811
    assert i8_quantize(L, codes=0, scales=0, src=0, rows=0) == 0
    assert i8_quantize(L, codes=0, scales=0, src=0, batch=0) == 0


# ---- the binding ----

X, Y, W, E = empty(BF, 6, 32), empty(BF, 6, 24), empty(I32, 3, 3, 2, 8, 8), empty(I32, 3)
I8 = torch.int8


def codes(*shape, scales=None):
    return lambda d: bmm.I8Operand(empty(I8, *shape)(d), empty(torch.float32, *(scales or shape[:-1]))(d))


def weight(batch=3, N=24, K=64):
    return lambda d: bmm.I8Operand(empty(I32, batch, N // 8, K // 32, 8, 8)(d),
                                   empty(torch.float32, batch, N)(d))


@pytest.mark.parametrize("call,needle", [
    (lambda: bmm.grouped_mma(empty(BF, 2, 6, 32)(0), W(0), E(0)), "rows, columns"),
    (lambda: bmm.grouped_mma(empty(torch.float32, 6, 32)(0), W(0), E(0)), "float16 or bfloat16"),
    (lambda: bmm.grouped_mma(X(0), W(0), empty(torch.int64, 3)(0)), "int32"),
    (lambda: bmm.grouped_mma(X(0), W(0), empty(I32, 1, 3)(0)), "one dimension"),
    (lambda: bmm.grouped_mma(X(0), W(0), empty(I32, 6)(0)[::2]), "contiguous"),
    (lambda: bmm.grouped_mma(X(0), W(0), empty(I32, 4)(0)), "4 ends for the weights of 3"),
    (lambda: bmm.grouped_mma(empty(BF, 6, 48)(0), W(0), E(0)), "disagree on K"),
    (lambda: bmm.grouped_mma(X(0), empty(BF, 3, 24, 32)(0), E(0)), "packed words"),
    (lambda: bmm.grouped_mma(X(0), W(0), E(0), out=empty(BF, 6, 32)(0)), "out must be"),
    (lambda: bmm.grouped_mma(X(0).t(), W(0), E(0)), "innermost stride"),
    (lambda: bmm.grouped_gated(X(0), W(0), empty(I32, 3, 4, 2, 8, 8)(0), E(0)), "differ in shape"),
    (lambda: bmm.grouped_gated(X(0), W(0), W(0), E(0), act="tanh"), "unknown activation"),
    (lambda: bmm.grouped_gated(X(0), W(0), W(0), E(0), save=True, out=empty(BF, 6, 32)(0)[:, :24]),
     "must be contiguous"),
    (lambda: bmm.grouped_mma_backward(X(0), X(0), W(0), E(0)), "dY must be"),
    (lambda: bmm.grouped_mma_backward(Y(0), X(0), W(0), E(0), need_dx=False, need_dw=False), "neither"),
    (lambda: bmm.grouped_mma_backward(Y(0), X(0), W(0), E(0), workspace=empty(BF, 8, 8)(0)[:, :4]),
     "workspace must be contiguous"),
    (lambda: bmm.grouped_gated_backward(Y(0), Y(0), empty(BF, 6, 32)(0)[:, :24], X(0), W(0), W(0), E(0)),
     "same row stride"),
    (lambda: bmm.i8_quantize(empty(I8, 5, 64)(0)), "float32, float16 or bfloat16"),
    (lambda: bmm.i8_pack(codes(20, 64)(0)), "multiple of 8"),
    (lambda: bmm.i8_pack(codes(24, 48)(0)), "of 32"),
    (lambda: bmm.i8_pack(codes(24, 64, scales=(16,))(0)), "disagree on the rows"),
    (lambda: bmm.i8_pack(bmm.I8Operand(X(0), empty(torch.float32, 6)(0))), "int8"),
    (lambda: bmm.i8_mma(codes(5, 64)(0), codes(24, 64)(0)), "packed words"),
    (lambda: bmm.i8_mma(codes(5, 64)(0), weight()(0)), "disagree on batch"),
    (lambda: bmm.i8_mma(codes(5, 96)(0), weight(1)(0)), "disagree on K"),
    (lambda: bmm.i8_mma(codes(5, 64, scales=(5, 1))(0), weight(1)(0)), "scales must be"),
    (lambda: bmm.i8_mma(codes(5, 64)(0), weight(1)(0)._replace(scales=empty(torch.float32, 24)(0))),
     "scales must be"),
    (lambda: bmm.i8_mma(codes(5, 64)(0), weight(1)(0), dtype=I8), "dtype must be"),
    (lambda: bmm.i8_mma(codes(1, 5, 64)(0), weight()(0), E(0)), "must be .rows, K"),
    (lambda: bmm.i8_mma(codes(5, 64)(0), weight(2)(0), E(0)), "3 ends for the weights of 2"),
    (lambda: bmm.i8_mma(bmm.I8Operand(X(0), empty(torch.float32, 6)(0)), weight(1)(0)), "must be int8"),
    (lambda: bmm.i8_gated(codes(5, 64)(0), weight(1)(0), weight(1, 32)(0)), "differ in shape"),
    (lambda: bmm.i8_gated(codes(5, 64)(0), weight(1)(0), weight(1)(0), dtype=torch.float32),
     "float16 or bfloat16"),
])
def test_binding(gpus, call, needle):  # noqa: F811
    with pytest.raises(ValueError, match=needle):
        call()
    assert not gpus.launches


def test_binding_refuses_the_cpu():
    x, w = torch.zeros(6, 32, dtype=BF), torch.zeros(3, 3, 2, 8, 8, dtype=I32)
    ends = torch.tensor([1, 2, 3], dtype=I32)
    q = bmm.I8Operand(torch.zeros(5, 64, dtype=I8), torch.zeros(5))
    v = bmm.I8Operand(torch.zeros(1, 3, 2, 8, 8, dtype=I32), torch.zeros(1, 24))
    y = torch.zeros(6, 24, dtype=BF)
    for call in (lambda: bmm.grouped_mma(x, w, ends), lambda: bmm.grouped_gated(x, w, w, ends),
                 lambda: bmm.grouped_mma_backward(y, x, w, ends),
                 lambda: bmm.grouped_gated_backward(y, y, y, x, w, w, ends),
                 lambda: bmm.i8_quantize(x), lambda: bmm.i8_mma(q, v), lambda: bmm.i8_gated(q, v, v)):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()


# ---- which GPU a call runs on ----

CALLS = {
    "grouped_mma": (bmm.grouped_mma, [X, W, E]),
    "grouped_mma_out": (lambda x, w, e, o: bmm.grouped_mma(x, w, e, out=o), [X, W, E, Y]),
    "grouped_gated": (bmm.grouped_gated, [X, W, W, E]),
    "grouped_gated_save": (lambda x, g, u, e: bmm.grouped_gated(x, g, u, e, save=True), [X, W, W, E]),
    "grouped_mma_backward": (bmm.grouped_mma_backward, [Y, X, W, E]),
    "grouped_mma_backward_workspace": (lambda *t: bmm.grouped_mma_backward(*t[:4], workspace=t[4]),
                                       [Y, X, W, E, empty(torch.uint8, 4096)]),
    "grouped_gated_backward": (bmm.grouped_gated_backward, [Y, Y, Y, X, W, W, E]),
    "i8_quantize": (bmm.i8_quantize, [X]),
    "i8_mma": (lambda a, sa, b, sb: bmm.i8_mma(bmm.I8Operand(a, sa), bmm.I8Operand(b, sb)),
               [empty(I8, 5, 64), empty(torch.float32, 5), empty(I32, 1, 3, 2, 8, 8),
                empty(torch.float32, 1, 24)]),
    "i8_mma_ends": (lambda a, sa, b, sb, e: bmm.i8_mma(bmm.I8Operand(a, sa), bmm.I8Operand(b, sb), e),
                    [empty(I8, 5, 64), empty(torch.float32, 5), empty(I32, 3, 3, 2, 8, 8),
                     empty(torch.float32, 3, 24), E]),
    "i8_gated": (lambda a, sa, b, sb, c, sc: bmm.i8_gated(bmm.I8Operand(a, sa), bmm.I8Operand(b, sb),
                                                         bmm.I8Operand(c, sc)),
                 [empty(I8, 5, 64), empty(torch.float32, 5), empty(I32, 1, 3, 2, 8, 8),
                  empty(torch.float32, 1, 24), empty(I32, 1, 3, 2, 8, 8), empty(torch.float32, 1, 24)]),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_runs_where_its_tensors_are(gpus, name, device):  # noqa: F811
    call, tensors = CALLS[name]
    out = call(*(t(device) for t in tensors))
    assert [l[1:] for l in gpus.launches] == [(device, 1000 + device)]
    assert gpus.state.device == 0
    for t in out if isinstance(out, tuple) else (out,):
        assert t.get_device() == device


@pytest.mark.parametrize("name", [n for n, (_, ts) in CALLS.items() if len(ts) > 1])
def test_refuses_tensors_of_two_gpus(gpus, name):  # noqa: F811
    call, tensors = CALLS[name]
    for odd in range(len(tensors)):
        with pytest.raises(ValueError, match="one GPU"):
            call(*(t(int(i == odd)) for i, t in enumerate(tensors)))
    assert not gpus.launches


def test_empty_tail_is_asked_for_with_fresh_outputs_only(gpus, monkeypatch):  # noqa: F811
    """Outputs that the binding makes become zero behind the last group; given ones stay."""
    seen = []

    def note(name, real):
        def call(*args):
            d = next(a for a in args if type(a).__name__ == "CArgObject")._obj
            seen.append((name, d.zero_tail))
            return real(*args)
        return call
    lib = bmm._lib
    for name in ("bmm_grouped_mma", "bmm_i8_mma"):
        monkeypatch.setattr(lib, name, note(name, getattr(lib, name)), raising=False)
    bmm.grouped_mma(X(0), W(0), E(0))
    bmm.grouped_mma(X(0), W(0), E(0), out=Y(0))
    bmm.i8_mma(codes(5, 64)(0), weight()(0), E(0))
    bmm.i8_mma(codes(5, 64)(0), weight()(0), E(0), out=empty(torch.float32, 5, 24)(0))
    assert [s[1] for s in seen] == [1, 0, 1, 0]
