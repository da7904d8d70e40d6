"""Refusals of the feed-forward operators, on the CPU: every invalid argument is
rejected on the host before any HIP call, and empty problems are no-ops."""
import ctypes
import os

import pytest
import torch

import bf16_matrix_multiply_amd as bmm

EINVAL, EALIGN, EOVERLAP = -1, -2, -3
# Fake device addresses: only compared, never dereferenced.
P = [0x7F0000000000 + i * 0x1000000000 for i in range(12)]


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bmm.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return bmm.lib()


def err(L):
    return L.bmm_last_error().decode()


def gated(L, H=P[0], G=0, U=0, X=P[3], Wg=P[4], Wu=P[5], batch=1, M=5, F=24, K=32, ld_x=32,
          ld_h=24, dtype=1, act=0):
    d = bmm.GatedDesc(batch, M, F, K, ld_x, ld_h, dtype, act)
    return L.bmm_gated(H, G, U, X, Wg, Wu, ctypes.byref(d), None)


GATED_DESC = [
    (dict(dtype=2), EINVAL, "dtype"),
    (dict(act=4), EINVAL, "bmm_act"),
    (dict(act=-1), EINVAL, "bmm_act"),
    (dict(batch=-1), EINVAL, "negative"),
    (dict(M=-1), EINVAL, "negative"),
    (dict(F=20, ld_h=24), EINVAL, "multiple of 8"),
    (dict(K=24), EINVAL, "multiple of 16"),
    (dict(F=(1 << 20) + 8, ld_h=1 << 21), EINVAL, "too large"),
    (dict(K=1 << 22, ld_x=1 << 22), EINVAL, "too large"),
    (dict(M=1 << 41), EINVAL, "too large"),
    (dict(M=1 << 40, batch=1 << 20), EINVAL, "too large"),
    (dict(ld_x=16), EINVAL, "ld_x"),
    (dict(ld_h=16), EINVAL, "ld_h"),
    (dict(ld_x=(1 << 21) + 8), EINVAL, "2^21"),
    (dict(ld_x=36), EALIGN, "multiples of 8"),
    (dict(ld_h=28), EALIGN, "multiples of 8"),
]


@pytest.mark.parametrize("kw,code,needle", GATED_DESC + [
    (dict(G=P[1]), EINVAL, "both or neither"),
    (dict(U=P[1]), EINVAL, "both or neither"),
    (dict(H=0), EINVAL, "H is null"),
    (dict(X=0), EINVAL, "X is null"),
    (dict(Wg=0), EINVAL, "Wg is null"),
    (dict(Wu=0), EINVAL, "Wu is null"),
    (dict(H=P[0] + 8), EALIGN, "H must be"),
    (dict(G=P[1] + 2, U=P[2]), EALIGN, "G must be"),
    (dict(X=P[3] + 2), EALIGN, "X must be"),
    (dict(Wu=P[5] + 4), EALIGN, "Wu must be"),
    (dict(H=P[3] + 64), EOVERLAP, "H overlaps X"),
    (dict(H=P[4]), EOVERLAP, "H overlaps Wg"),
    (dict(G=P[0], U=P[2]), EOVERLAP, "H overlaps G"),
    (dict(G=P[1], U=P[1] + 16), EOVERLAP, "G overlaps U"),
    # rows of one buffer side by side, one column group into the other
    (dict(G=P[0] + 32, U=P[0] + 96, ld_h=72), EOVERLAP, "H overlaps G"),
])
def test_gated_rejects(L, kw, code, needle):
    assert gated(L, **kw) == code, err(L)
    assert needle in err(L)


def test_gated_null_descriptor(L):
    assert L.bmm_gated(P[0], 0, 0, P[1], P[2], P[3], None, None) == EINVAL
    assert "descriptor" in err(L)
    assert L.bmm_gated_backward_workspace_bytes(None) == EINVAL


def test_gated_empty_is_noop(L):
    for kw in (dict(batch=0), dict(M=0), dict(F=0, ld_h=0)):
        assert gated(L, H=0, X=0, Wg=0, Wu=0, **kw) == 0


def backward(L, dX=P[0], dWg=P[1], dWu=P[2], dH=P[3], G=P[4], U=P[5], X=P[6], Wg=P[7], Wu=P[8],
             ws=P[9], ws_bytes=1 << 30, batch=1, M=5, F=24, K=32, ld_x=32, ld_h=24, dtype=1, act=0):
    d = bmm.GatedDesc(batch, M, F, K, ld_x, ld_h, dtype, act)
    return L.bmm_gated_backward(dX, dWg, dWu, dH, G, U, X, Wg, Wu, ctypes.byref(d), ws, ws_bytes,
                                None)


@pytest.mark.parametrize("kw,code,needle", GATED_DESC + [
    (dict(dWg=0), EINVAL, "both or neither"),
    (dict(dX=0, dWg=0, dWu=0), EINVAL, "all null"),
    (dict(dH=0), EINVAL, "dH is null"),
    (dict(G=0), EINVAL, "G is null"),
    (dict(U=0), EINVAL, "U is null"),
    (dict(X=0), EINVAL, "X is null"),
    (dict(Wg=0), EINVAL, "Wg is null"),
    (dict(ws=0), EINVAL, "workspace is null"),
    (dict(ws_bytes=639), EINVAL, "workspace_bytes"),
    (dict(ws=P[9] + 4), EALIGN, "workspace must be"),
    (dict(dX=P[0] + 8), EALIGN, "dX must be"),
    (dict(dWu=P[1] + 16), EOVERLAP, "dWg overlaps dWu"),
    (dict(dX=P[3]), EOVERLAP, "dX overlaps dH"),
    (dict(ws=P[6] - 128), EOVERLAP, "workspace overlaps X"),
    (dict(ws=P[0] + 16), EOVERLAP, "dX overlaps workspace"),
])
def test_gated_backward_rejects(L, kw, code, needle):
    assert backward(L, **kw) == code, err(L)
    assert needle in err(L)


def test_gated_backward_workspace(L):
    # 5 rows of [dG | dU], each half padded from 24 to 32 values, to 256 bytes
    assert bmm.gated_backward_workspace_bytes(1, 5, 24, 32) == 5 * 64 * 2 // 256 * 256 + 256
    assert bmm.gated_backward_workspace_bytes(1, 0, 24, 32) == 0
    # many rows into small gradients: partial sums after it
    assert bmm.gated_backward_workspace_bytes(1, 65536, 64, 64) > 65536 * 128 * 2
    with pytest.raises(bmm.BmmError, match="multiple of 8"):
        bmm.gated_backward_workspace_bytes(1, 5, 12, 32)


def test_gated_backward_empty_is_noop(L):
    null = dict(dX=0, dWg=0, dWu=0, dH=0, G=0, U=0, X=0, Wg=0, Wu=0, ws=0, ws_bytes=0)
    for kw in (dict(batch=0), dict(K=0, ld_x=0), dict(M=0, F=0, ld_h=0)):
        assert backward(L, **{**null, **kw}) == 0, err(L)


def convert(L, fn="bmm_mx4_quantize", codes=P[0], scales=P[1], mat=P[2], batch=1, rows=5, K=64,
            ld=64, et=3):
    a = (codes, scales, mat) if fn == "bmm_mx4_quantize" else (mat, codes, scales)
    return getattr(L, fn)(*a, batch, rows, K, ld, et, None)


@pytest.mark.parametrize("fn", ["bmm_mx4_quantize", "bmm_mx4_dequantize"])
@pytest.mark.parametrize("kw,code,needle", [
    (dict(et=0), EINVAL, "elem_type"),
    (dict(et=4), EINVAL, "elem_type"),
    (dict(rows=-1), EINVAL, "negative"),
    (dict(K=48), EINVAL, "multiple of 32"),
    (dict(K=1 << 22, ld=1 << 22), EINVAL, "too large"),
    (dict(rows=1 << 41), EINVAL, "too large"),
    (dict(ld=32), EINVAL, "ld (32) < K (64)"),
    (dict(ld=68), EALIGN, "multiple of 8"),
    (dict(codes=0), EINVAL, "codes is null"),
    (dict(scales=0), EINVAL, "scales is null"),
    (dict(mat=0), EINVAL, "null"),
    (dict(codes=P[0] + 8), EALIGN, "codes must be"),
    (dict(scales=P[1] + 4), EALIGN, "scales must be"),
    (dict(mat=P[2] + 2), EALIGN, "aligned"),
    (dict(mat=P[0] + 512), EOVERLAP, "overlaps codes"),
    (dict(scales=P[0] + 16), EOVERLAP, "codes overlaps scales"),
])
def test_mx4_convert_rejects(L, fn, kw, code, needle):
    assert convert(L, fn, **kw) == code, err(L)
    assert needle in err(L)


def test_mx4_convert_empty_is_noop(L):
    for fn in ("bmm_mx4_quantize", "bmm_mx4_dequantize"):
        for kw in (dict(batch=0), dict(rows=0), dict(K=0, ld=0)):
            assert convert(L, fn, codes=0, scales=0, mat=0, **kw) == 0


def test_mx4_sizes(L):
    assert L.bmm_mx4_codes_bytes(2, 17, 160) == 2 * 2 * 2 * 1024
    assert L.bmm_mx4_scales_bytes(2, 17, 544) == 2 * 2 * 2 * 256
    assert L.bmm_mx4_codes_bytes(1, 0, 32) == 0
    for bad in ((-1, 16, 32), (1, -1, 32), (1, 16, 33), (1, 16, 1 << 22)):
        assert L.bmm_mx4_codes_bytes(*bad) == EINVAL
        assert L.bmm_mx4_scales_bytes(*bad) == EINVAL


def product(L, D=P[0], A=P[1], As=P[2], B=P[3], Bs=P[4], batch=1, M=5, N=24, K=64, ld=24, et=3):
    return L.bmm_mx4_mma(D, A, As, B, Bs, batch, M, N, K, ld, et, None)


def mx4_gated(L, D=P[0], A=P[1], As=P[2], B=P[3], Bs=P[4], C=P[5], Cs=P[6], batch=1, M=5, N=24,
              K=64, ld=24, act=0, et=3):
    return L.bmm_mx4_gated(D, A, As, B, Bs, C, Cs, batch, M, N, K, ld, act, et, None)


@pytest.mark.parametrize("fn", [product, mx4_gated])
@pytest.mark.parametrize("kw,code,needle", [
    (dict(et=4), EINVAL, "elem_type"),
    (dict(M=-1), EINVAL, "negative"),
    (dict(N=20), EINVAL, "multiple of 8"),
    (dict(K=48), EINVAL, "multiple of 32"),
    (dict(K=1 << 22), EINVAL, "too large"),
    (dict(ld=16), EINVAL, "ld (16)"),
    (dict(ld=28), EALIGN, "multiple of 8"),
    (dict(D=0), EINVAL, "is null"),
    (dict(A=0), EINVAL, "codes is null"),
    (dict(As=0), EINVAL, "scales is null"),
    (dict(Bs=0), EINVAL, "scales is null"),
    (dict(D=P[0] + 8), EALIGN, "must be 16-byte"),
    (dict(A=P[1] + 8), EALIGN, "codes must be"),
    (dict(D=P[3] + 512), EOVERLAP, "overlaps"),
    (dict(D=P[4]), EOVERLAP, "overlaps"),
])
def test_mx4_product_rejects(L, fn, kw, code, needle):
    assert fn(L, **kw) == code, err(L)
    assert needle in err(L)


def test_mx4_gated_rejects(L):
    assert mx4_gated(L, et=1) == EINVAL and "elem_type" in err(L)
    assert mx4_gated(L, act=4) == EINVAL and "bmm_act" in err(L)
    assert mx4_gated(L, C=0) == EINVAL and "Wu_codes is null" in err(L)
    assert mx4_gated(L, Cs=P[6] + 4) == EALIGN and "Wu_scales" in err(L)


def test_mx4_product_empty_is_noop(L):
    for fn in (product, mx4_gated):
        for kw in (dict(batch=0), dict(M=0), dict(N=0, ld=0)):
            assert fn(L, D=0, A=0, As=0, B=0, Bs=0, **kw) == 0


def test_binding_rejects_before_the_library():
    """Shapes, types and devices are checked in the binding."""
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    w = torch.zeros(1, 3, 2, 8, 8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensors"):
        bmm.gated(x, w, w)
    with pytest.raises(ValueError, match="unknown activation"):
        bmm.gated(x, w, w, act="tanh")
    with pytest.raises(ValueError, match="neither"):
        bmm.gated_backward(x, x, x, x, w, w, need_dx=False, need_dw=False)
    with pytest.raises(ValueError, match="GPU tensors"):
        bmm.mx4_quantize(x)
    op = bmm.Mx4Operand(torch.zeros(1, 1, 1, 4, 16, 16, dtype=torch.uint8),
                        torch.zeros(1, 1, 1, 4, 16, 4, dtype=torch.uint8), 4, 32)
    with pytest.raises(ValueError, match="GPU tensors"):
        bmm.mx4_dequantize(op)
    with pytest.raises(ValueError, match="uint8 tensor of shape"):
        bmm.mx4_mma(op._replace(K=160), op)
    with pytest.raises(ValueError, match="uint8 tensor of shape"):
        bmm.mx4_gated(op._replace(rows=17), op, op)
