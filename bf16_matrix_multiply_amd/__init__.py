"""Python binding of libbmm.so: the tiled f16/bf16 multiply-accumulate
D = A * B^T + C on MI355X (gfx950).

Argument marshalling only. Each function takes torch tensors on one GPU, reads
their pointers, extents and that GPU's current torch stream, and calls the C
ABI of ``include/bmm.h`` with the same name; every step of the computation runs
in the library's HIP kernels. If the library is not built, every call raises;
there is no other code path.

Layouts (mma.sync page of the TVM tirx tile-op documentation, "Operand
coordinates and ownership"):
    A packed: (batch, M/16, K/16, 16, 8) 32-bit words
    B packed: (batch, N/8,  K/16,  8, 8) 32-bit words
    C, D:     (batch, M/16, N/8,  16, 8) float32
or, with an atom K of 8 (the m16n8k8 form), A (batch, M/16, K/8, 16, 4) and
B (batch, N/8, K/8, 8, 4). Packed words are held in int32 tensors (bit
containers).
"""
from __future__ import annotations

import ctypes
import functools
import os
import typing

import torch

__all__ = ["BmmError", "pack_operand", "pack_operand_kmajor", "box_copy", "box_store",
           "box_reduce_add", "mma_tile", "mma_tile_splitk", "mma_tile_splitk_noalloc",
           "splitk_default", "splitk_suggested", "NOALLOC_SCRATCH_BYTES",
           "splitk_workspace_bytes", "select_kernel", "library_path", "KERNELS", "MmaOpts",
           "ELEM_TYPES", "ACTS", "gated", "gated_backward", "gated_backward_workspace_bytes",
           "ffn_plan", "FFN_PRODUCTS", "FFN_TILES", "Mx4Operand", "mx4_quantize", "mx4_dequantize",
           "mx4_mma", "mx4_gated", "grouped_mma", "grouped_mma_backward",
           "grouped_mma_backward_workspace_bytes", "grouped_gated", "grouped_gated_backward",
           "grouped_gated_backward_workspace_bytes", "I8Operand", "i8_quantize", "i8_pack",
           "i8_mma", "i8_gated", "group_plan", "GROUP_PRODUCTS"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libbmm.so")

BMM_F16, BMM_BF16 = 0, 1
_DTYPES = {"f16": BMM_F16, "float16": BMM_F16, torch.float16: BMM_F16,
           "bf16": BMM_BF16, "bfloat16": BMM_BF16, torch.bfloat16: BMM_BF16}
KERNELS = {"auto": 0, "direct": 1, "tiled": 2, "skinny": 3, "tiled128": 4, "tiled256x128": 5}
NOALLOC_SCRATCH_BYTES = 64 << 20   # BMM_NOALLOC_SCRATCH_BYTES
ELEM_TYPES = {"f32": 1, "f16": 2, "bf16": 3, "i32": 4, "i64": 5}
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
FFN_PRODUCTS = {"gated": 0, "gated_dx": 1, "gated_dx_rest": 2, "gated_dw": 3, "mx4_mma": 4,
                "mx4_gated": 5}
FFN_TILES = {"128x128": 0, "256x128": 1, "256x192": 2, "256x256": 3, "few_rows": 4, "none": 5}
GROUP_PRODUCTS = {"grouped_mma": 0, "grouped_mma_dx": 1, "grouped_mma_dw": 2, "grouped_gated": 3,
                  "grouped_gated_dx": 4, "grouped_gated_dw": 5, "i8_mma": 6, "i8_gated": 7}
_HALF_DTYPES = {torch.float16: BMM_F16, torch.bfloat16: BMM_BF16}
_ELEM_DTYPES = {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
KERNEL_NAMES = {v: k for k, v in KERNELS.items()}
FFN_TILE_NAMES = {v: k for k, v in FFN_TILES.items()}


class BmmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"bmm error {code}: {msg}")
        self.code = code


class BoxDesc(ctypes.Structure):
    _fields_ = [
        ("rank", ctypes.c_int32),
        ("elem_bytes", ctypes.c_int32),
        ("dims", ctypes.c_int64 * 5),
        ("strides", ctypes.c_int64 * 5),
        ("box", ctypes.c_int32 * 5),
        ("coords", ctypes.c_int64 * 5),
        ("n_repeat", ctypes.c_int32),
        ("coord_step", ctypes.c_int64 * 5),
        ("swizzle", ctypes.c_int32),
        ("oob_fill", ctypes.c_int32),
    ]


class MmaOpts(ctypes.Structure):
    _fields_ = [
        ("atom_k", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("scaled", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("beta", ctypes.c_float),
    ]


class GatedDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("M", ctypes.c_int64),
        ("F", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("ld_x", ctypes.c_int64),
        ("ld_h", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
    ]


class GroupedDesc(ctypes.Structure):
    _fields_ = [
        ("groups", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("ld_x", ctypes.c_int64),
        ("ld_y", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("zero_tail", ctypes.c_int32),
    ]


class I8Desc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("M", ctypes.c_int64),
        ("N", ctypes.c_int64),
        ("K", ctypes.c_int64),
        ("ld_a", ctypes.c_int64),
        ("ld_d", ctypes.c_int64),
        ("elem_type", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("zero_tail", ctypes.c_int32),
    ]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded libbmm.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built: run `python -m bf16_matrix_multiply_amd.build` "
                "(or __graft_entry__.build()) first")
        L = ctypes.CDLL(_LIB_PATH)
        p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.bmm_abi_version.restype = ctypes.c_int
        L.bmm_last_error.restype = ctypes.c_char_p
        L.bmm_pack_operand.argtypes = [p, p, i64, i64, i64, i64, i32, p]
        L.bmm_pack_operand_kmajor.argtypes = [p, p, i64, i64, i64, i64, i32, p]
        L.bmm_pack_operand_k8.argtypes = [p, p, i64, i64, i64, i64, i32, p]
        L.bmm_pack_operand_kmajor_k8.argtypes = [p, p, i64, i64, i64, i64, i32, p]
        L.bmm_mma_tile_opts.argtypes = [p, p, p, p, ctypes.c_float, i64, i64, i64, i64,
                                        ctypes.c_int, ctypes.POINTER(MmaOpts), p]
        L.bmm_box_copy.argtypes = [p, p, ctypes.POINTER(BoxDesc), ctypes.POINTER(i64), p]
        L.bmm_mma_tile.argtypes = [p, p, p, p, ctypes.c_float, i64, i64, i64, i64, ctypes.c_int,
                                   p]
        L.bmm_mma_tile_with.argtypes = [p, p, p, p, ctypes.c_float, i64, i64, i64, i64,
                                        ctypes.c_int, i32, p]
        L.bmm_mma_tile_scaled.argtypes = [p, p, p, p, ctypes.c_float, ctypes.c_float,
                                          ctypes.c_float, i64, i64, i64, i64, ctypes.c_int, i32, p]
        L.bmm_select_kernel.argtypes = [i64, i64, i64, i64]
        L.bmm_box_store.argtypes = [p, p, ctypes.POINTER(BoxDesc), ctypes.POINTER(i64), p]
        L.bmm_box_reduce_add.argtypes = [p, p, ctypes.POINTER(BoxDesc), i32,
                                         ctypes.POINTER(i64), p]
        L.bmm_mma_tile_splitk.argtypes = [p, p, p, p, ctypes.c_float, i64, i64, i64, i64,
                                          ctypes.c_int, i32, i32, p, i64, p]
        L.bmm_mma_tile_splitk_noalloc.argtypes = [p, p, p, p, ctypes.c_float, i64, i64, i64,
                                                  i64, ctypes.c_int, i32, i32, p]
        L.bmm_mma_splitk_workspace_bytes.argtypes = [i64, i64, i64, i64, i32, i32]
        L.bmm_mma_splitk_workspace_bytes.restype = i64
        L.bmm_splitk_default.argtypes = [i64, i64, i64, i64, i32]
        L.bmm_splitk_suggested.argtypes = [i64, i64, i64, i64, i32]
        for f in (L.bmm_pack_operand, L.bmm_pack_operand_kmajor, L.bmm_pack_operand_k8,
                  L.bmm_pack_operand_kmajor_k8,
                  L.bmm_box_copy, L.bmm_mma_tile, L.bmm_mma_tile_with, L.bmm_mma_tile_scaled,
                  L.bmm_mma_tile_opts, L.bmm_select_kernel, L.bmm_box_store,
                  L.bmm_box_reduce_add, L.bmm_mma_tile_splitk, L.bmm_mma_tile_splitk_noalloc,
                  L.bmm_splitk_default, L.bmm_splitk_suggested):
            f.restype = ctypes.c_int
        desc = ctypes.POINTER(GatedDesc)
        L.bmm_gated.argtypes = [p] * 6 + [desc, p]
        L.bmm_gated_backward.argtypes = [p] * 9 + [desc, p, i64, p]
        L.bmm_gated_backward_workspace_bytes.argtypes = [desc]
        L.bmm_gated_backward_workspace_bytes.restype = i64
        for f in (L.bmm_mx4_codes_bytes, L.bmm_mx4_scales_bytes):
            f.argtypes = [i64, i64, i64]
            f.restype = i64
        L.bmm_mx4_quantize.argtypes = [p, p, p, i64, i64, i64, i64, i32, p]
        L.bmm_mx4_dequantize.argtypes = [p, p, p, i64, i64, i64, i64, i32, p]
        L.bmm_mx4_mma.argtypes = [p] * 5 + [i64] * 5 + [i32, p]
        L.bmm_mx4_gated.argtypes = [p] * 7 + [i64] * 5 + [i32, i32, p]
        L.bmm_ffn_plan.argtypes = [i32, i64, i64, i64, i64, ctypes.POINTER(i32)]
        for f in (L.bmm_ffn_plan, L.bmm_gated, L.bmm_gated_backward, L.bmm_mx4_quantize,
                  L.bmm_mx4_dequantize, L.bmm_mx4_mma, L.bmm_mx4_gated):
            f.restype = ctypes.c_int
        desc, i8 = ctypes.POINTER(GroupedDesc), ctypes.POINTER(I8Desc)
        L.bmm_grouped_mma.argtypes = [p] * 4 + [desc, p]
        L.bmm_grouped_mma_backward.argtypes = [p] * 6 + [desc, p, i64, p]
        L.bmm_grouped_gated.argtypes = [p] * 7 + [desc, p]
        L.bmm_grouped_gated_backward.argtypes = [p] * 10 + [desc, p, i64, p]
        for f in (L.bmm_grouped_mma_backward_workspace_bytes,
                  L.bmm_grouped_gated_backward_workspace_bytes):
            f.argtypes = [desc]
            f.restype = i64
        L.bmm_i8_quantize.argtypes = [p, p, p, i64, i64, i64, i64, i32, p]
        L.bmm_i8_mma.argtypes = [p] * 6 + [i8, p]
        L.bmm_i8_gated.argtypes = [p] * 8 + [i8, p]
        L.bmm_group_plan.argtypes = [i32, i64, i64, i64, i64, ctypes.POINTER(i32)]
        for f in (L.bmm_grouped_mma, L.bmm_grouped_mma_backward, L.bmm_grouped_gated,
                  L.bmm_grouped_gated_backward, L.bmm_i8_quantize, L.bmm_i8_mma, L.bmm_i8_gated,
                  L.bmm_group_plan):
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def _dtype_code(dtype, fn: str) -> int:
    """The C ABI's element type for ``dtype``. Packed words carry no type, so the
    caller must name it: a missing or unknown dtype is an error, never a default
    (the tile operation changes no input type)."""
    if dtype is None:
        raise ValueError(f"{fn}: dtype is required ('f16' or 'bf16'): packed words carry no type")
    try:
        return _DTYPES[dtype]
    except (KeyError, TypeError):
        raise ValueError(f"{fn}: unknown dtype {dtype!r}; expected 'f16' or 'bf16'") from None


def _check(rc: int):
    if rc < 0:
        raise BmmError(rc, lib().bmm_last_error().decode())
    return rc


def _stream(t: torch.Tensor | None = None):
    if t is not None and not t.is_cuda:
        raise ValueError("bmm operates on GPU tensors only")
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require_cuda(*ts):
    """Every given tensor is on a GPU, and all on the same one."""
    device = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("bmm operates on GPU tensors only")
        if device is not None and t.device != device:
            raise ValueError(f"bmm operates on tensors of one GPU, got {device} and {t.device}")
        device = t.device


_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_gpu(device, fn, *args):
    """fn with that GPU as the current one: what it enqueues goes to its current
    stream."""
    with torch.cuda.device(device):
        return fn(*args)


def _on_its_gpu(fn):
    """fn, run on the GPU of its first tensor."""
    @functools.wraps(fn)
    def call(*args, **kw):
        t = args[0] if args else next((v for v in kw.values() if isinstance(v, torch.Tensor)), None)
        device = t.get_device() if isinstance(t, torch.Tensor) else -1
        if device < 0 or device == _current_device():   # (the CPU: fn refuses it)
            return fn(*args, **kw)
        return _on_gpu(device, functools.partial(fn, **kw), *args)
    return call


@_on_its_gpu
def pack_operand(x: torch.Tensor, atom_rows: int, K: int | None = None,
                 out: torch.Tensor | None = None, atom_k: int = 16) -> torch.Tensor:
    """Row-major (batch, rows, ld) or (rows, ld) 16-bit tensor -> packed words
    (batch, rows/R, K/atom_k, R, atom_k/2) int32 (R = atom_rows: 16 for A, 8
    for B; atom_k 16, or 8 for bmm_pack_operand_k8).

    The source must have unit innermost stride and rows ``ld`` elements apart,
    with batches ``rows * ld`` apart; K (default ld) may be smaller than ld."""
    if atom_k not in (16, 8):
        raise ValueError("pack_operand: atom_k must be 16 or 8")
    _require_cuda(x, out)
    if x.element_size() != 2:
        raise ValueError("pack_operand takes 16-bit (f16/bf16 bit) tensors")
    if x.dim() == 2:
        x = x.unsqueeze(0)
    batch, rows, ld = x.shape
    # (an empty source has nothing to pack; torch gives it arbitrary strides)
    if x.numel() and (x.stride(2) != 1 or (rows > 1 and x.stride(1) != ld) or
                      (batch > 1 and x.stride(0) != rows * ld)):
        raise ValueError("pack_operand: source must be (batch, rows, ld) with dense strides")
    K = ld if K is None else K
    shape = (batch, rows // atom_rows, K // atom_k, atom_rows, atom_k // 2)
    if out is None:
        out = torch.empty(shape, dtype=torch.int32, device=x.device)
    elif tuple(out.shape) != shape or not out.is_contiguous() or out.element_size() != 4:
        raise ValueError(f"pack_operand: out must be a contiguous 32-bit tensor of shape {shape}")
    fn = lib().bmm_pack_operand if atom_k == 16 else lib().bmm_pack_operand_k8
    _check(fn(_ptr(out), _ptr(x), batch, rows, K, ld, atom_rows, _stream(x)))
    return out


@_on_its_gpu
def pack_operand_kmajor(xt: torch.Tensor, atom_rows: int, rows: int | None = None,
                        out: torch.Tensor | None = None, atom_k: int = 16) -> torch.Tensor:
    """K-major (batch, K, ld) or (K, ld) 16-bit tensor holding element (row, k)
    at [b, k, row] -> packed words (batch, rows/R, K/atom_k, R, atom_k/2) int32,
    the same words pack_operand gives for the row-major matrix (atom_k 16, or 8
    for bmm_pack_operand_kmajor_k8). rows defaults to ld."""
    if atom_k not in (16, 8):
        raise ValueError("pack_operand_kmajor: atom_k must be 16 or 8")
    _require_cuda(xt, out)
    if xt.element_size() != 2:
        raise ValueError("pack_operand_kmajor takes 16-bit (f16/bf16 bit) tensors")
    if xt.dim() == 2:
        xt = xt.unsqueeze(0)
    batch, K, ld = xt.shape
    if xt.numel() and (xt.stride(2) != 1 or (K > 1 and xt.stride(1) != ld) or
                       (batch > 1 and xt.stride(0) != K * ld)):
        raise ValueError("pack_operand_kmajor: source must be (batch, K, ld) with dense strides")
    rows = ld if rows is None else rows
    shape = (batch, rows // atom_rows, K // atom_k, atom_rows, atom_k // 2)
    if out is None:
        out = torch.empty(shape, dtype=torch.int32, device=xt.device)
    elif tuple(out.shape) != shape or not out.is_contiguous() or out.element_size() != 4:
        raise ValueError(f"pack_operand_kmajor: out must be a contiguous 32-bit tensor of shape {shape}")
    fn = lib().bmm_pack_operand_kmajor if atom_k == 16 else lib().bmm_pack_operand_kmajor_k8
    _check(fn(_ptr(out), _ptr(xt), batch, rows, K, ld, atom_rows, _stream(xt)))
    return out


@_on_its_gpu
def box_copy(src: torch.Tensor, box, coords, n_repeat: int = 1, coord_step=None,
             swizzle: int = 0, dims=None, strides=None, oob_fill: int = 0,
             out: torch.Tensor | None = None):
    """Stage boxes of ``src`` through LDS; return ((n_repeat, *box) image, bytes).

    dims/strides default to ``src``'s own extents and byte strides (outer to
    inner); strides are in bytes."""
    _require_cuda(src, out)
    d = _box_desc(src, box, coords, n_repeat, coord_step, swizzle, dims, strides, oob_fill)
    shape = (n_repeat, *box)
    if out is None:
        out = torch.empty(shape, dtype=src.dtype, device=src.device)
    nbytes = ctypes.c_int64(-1)
    _check(lib().bmm_box_copy(_ptr(out), _ptr(src), ctypes.byref(d), ctypes.byref(nbytes),
                              _stream(src)))
    return out, nbytes.value


def _box_desc(t: torch.Tensor, box, coords, n_repeat, coord_step, swizzle, dims, strides,
              oob_fill=0) -> BoxDesc:
    rank = len(box)
    dims = list(t.shape) if dims is None else list(dims)
    strides = [s * t.element_size() for s in t.stride()] if strides is None else list(strides)
    coord_step = [0] * rank if coord_step is None else list(coord_step)
    if not (len(dims) == len(strides) == len(coords) == len(coord_step) == rank):
        raise ValueError("box: box, coords, coord_step, dims and strides need one entry "
                         "per dimension")
    d = BoxDesc()
    d.rank, d.elem_bytes = rank, t.element_size()
    for i in range(rank):
        d.dims[i], d.strides[i], d.box[i] = dims[i], strides[i], box[i]
        d.coords[i], d.coord_step[i] = coords[i], coord_step[i]
    d.n_repeat, d.swizzle, d.oob_fill = n_repeat, swizzle, oob_fill
    return d


@_on_its_gpu
def box_store(dst: torch.Tensor, image: torch.Tensor, box, coords, n_repeat: int = 1,
              coord_step=None, swizzle: int = 0, dims=None, strides=None) -> int:
    """Write the compact (n_repeat, *box) ``image`` into ``dst``'s boxes (in place;
    elements outside the tensor are skipped). Returns the image bytes read."""
    _require_cuda(dst, image)
    if image.element_size() != dst.element_size() or not image.is_contiguous():
        raise ValueError("box_store: image must be contiguous with dst's element size")
    d = _box_desc(dst, box, coords, n_repeat, coord_step, swizzle, dims, strides)
    nbytes = ctypes.c_int64(-1)
    _check(lib().bmm_box_store(_ptr(dst), _ptr(image), ctypes.byref(d), ctypes.byref(nbytes),
                               _stream(dst)))
    return nbytes.value


@_on_its_gpu
def box_reduce_add(dst: torch.Tensor, image: torch.Tensor, box, coords, elem_type: str,
                   n_repeat: int = 1, coord_step=None, swizzle: int = 0, dims=None,
                   strides=None) -> int:
    """Add the compact (n_repeat, *box) ``image`` into ``dst``'s boxes (in place),
    one rounding per add in ``elem_type`` ("f32", "f16", "bf16", "i32", "i64")."""
    _require_cuda(dst, image)
    if image.element_size() != dst.element_size() or not image.is_contiguous():
        raise ValueError("box_reduce_add: image must be contiguous with dst's element size")
    d = _box_desc(dst, box, coords, n_repeat, coord_step, swizzle, dims, strides)
    nbytes = ctypes.c_int64(-1)
    _check(lib().bmm_box_reduce_add(_ptr(dst), _ptr(image), ctypes.byref(d), ELEM_TYPES[elem_type],
                                    ctypes.byref(nbytes), _stream(dst)))
    return nbytes.value


def splitk_workspace_bytes(batch, M_rep, N_rep, K_rep, atom_k, splits) -> int:
    return _check(lib().bmm_mma_splitk_workspace_bytes(batch, M_rep, N_rep, K_rep, atom_k,
                                                       splits))


def splitk_default(batch, M_rep, N_rep, K_rep, atom_k=16) -> int:
    return _check(lib().bmm_splitk_default(batch, M_rep, N_rep, K_rep, atom_k))


def splitk_suggested(batch, M_rep, N_rep, K_rep, atom_k=16) -> int:
    """bmm_splitk_suggested: the split count when mma_tile_splitk is expected
    to beat mma_tile for this shape, else 1."""
    return _check(lib().bmm_splitk_suggested(batch, M_rep, N_rep, K_rep, atom_k))


@_on_its_gpu
def mma_tile_splitk(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None,
                    c: float = 0.0, dtype=None, splits: int | None = None,
                    out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Split-K form: D = (((C + P_0) + P_1) + ...), P_s the partial sums of
    balanced ranges of 32-value K steps (bmm_mma_tile_splitk). ``splits``
    defaults to bmm_splitk_default; ``workspace`` (float32, at least
    bmm_mma_splitk_workspace_bytes) is allocated here when not given. ``dtype``
    ('f16' or 'bf16') is required."""
    dt = _dtype_code(dtype, "mma_tile_splitk")
    _require_cuda(A, B, C, out, workspace)
    if A.dim() != 5 or B.dim() != 5 or A.shape[3] != 16 or B.shape[3] != 8 or \
            A.shape[4] not in (8, 4) or B.shape[4] != A.shape[4]:
        raise ValueError("mma_tile_splitk: A must be (batch, M_rep, K_rep, 16, w) and B "
                         "(batch, N_rep, K_rep, 8, w) packed words, w = 8 or 4")
    atom_k = 2 * A.shape[4]
    batch, M_rep, K_rep = A.shape[:3]
    N_rep = B.shape[1]
    if B.shape[0] != batch or B.shape[2] != K_rep:
        raise ValueError("mma_tile_splitk: A and B disagree on batch or K_rep")
    for t, name in ((A, "A"), (B, "B")):
        if not t.is_contiguous() or t.element_size() != 4:
            raise ValueError(f"mma_tile_splitk: {name} must be a contiguous 32-bit tensor")
    shape = (batch, M_rep, N_rep, 16, 8)
    if C is not None and (tuple(C.shape) != shape or C.dtype != torch.float32
                          or not C.is_contiguous()):
        raise ValueError(f"mma_tile_splitk: C must be a contiguous float32 tensor of shape {shape}")
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=A.device)
    elif tuple(out.shape) != shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError(f"mma_tile_splitk: out must be a contiguous float32 tensor of shape {shape}")
    if splits is None:
        splits = splitk_default(batch, M_rep, N_rep, K_rep, atom_k)
    need = splitk_workspace_bytes(batch, M_rep, N_rep, K_rep, atom_k, splits)
    if workspace is None:
        workspace = torch.empty(max(need // 4, 1), dtype=torch.float32, device=A.device)
    elif not workspace.is_contiguous():
        raise ValueError("mma_tile_splitk: workspace must be contiguous")
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().bmm_mma_tile_splitk(_ptr(out), _ptr(A), _ptr(B), _ptr(C), float(c), batch, M_rep,
                                     N_rep, K_rep, dt, atom_k, splits,
                                     _ptr(workspace), ws_bytes, _stream(A)))
    return out


@_on_its_gpu
def mma_tile_splitk_noalloc(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None,
                            c: float = 0.0, dtype=None, splits: int | None = None,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """bmm_mma_tile_splitk_noalloc: the split-K form with its partial sums in
    the library's static per-device scratch (NOALLOC_SCRATCH_BYTES) instead of
    a workspace. ``out`` must be given: this call allocates nothing. Calls
    that overlap on one device race on the scratch."""
    dt = _dtype_code(dtype, "mma_tile_splitk_noalloc")
    if out is None:
        raise ValueError("mma_tile_splitk_noalloc: out is required (this form allocates nothing)")
    _require_cuda(A, B, C, out)
    if A.dim() != 5 or B.dim() != 5 or A.shape[3] != 16 or B.shape[3] != 8 or \
            A.shape[4] not in (8, 4) or B.shape[4] != A.shape[4]:
        raise ValueError("mma_tile_splitk_noalloc: A must be (batch, M_rep, K_rep, 16, w) and B "
                         "(batch, N_rep, K_rep, 8, w) packed words, w = 8 or 4")
    atom_k = 2 * A.shape[4]
    batch, M_rep, K_rep = A.shape[:3]
    N_rep = B.shape[1]
    if B.shape[0] != batch or B.shape[2] != K_rep:
        raise ValueError("mma_tile_splitk_noalloc: A and B disagree on batch or K_rep")
    for t, name in ((A, "A"), (B, "B")):
        if not t.is_contiguous() or t.element_size() != 4:
            raise ValueError(f"mma_tile_splitk_noalloc: {name} must be a contiguous 32-bit tensor")
    shape = (batch, M_rep, N_rep, 16, 8)
    for t, name in ((C, "C"), (out, "out")):
        if t is not None and (tuple(t.shape) != shape or t.dtype != torch.float32
                              or not t.is_contiguous()):
            raise ValueError(f"mma_tile_splitk_noalloc: {name} must be a contiguous float32 "
                             f"tensor of shape {shape}")
    if splits is None:
        splits = splitk_default(batch, M_rep, N_rep, K_rep, atom_k)
    _check(lib().bmm_mma_tile_splitk_noalloc(_ptr(out), _ptr(A), _ptr(B), _ptr(C), float(c),
                                             batch, M_rep, N_rep, K_rep, dt, atom_k, splits,
                                             _stream(A)))
    return out


@_on_its_gpu
def mma_tile(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor | None = None,
             c: float = 0.0, dtype=None, out: torch.Tensor | None = None,
             kernel: str = "auto", alpha: float | None = None,
             beta: float | None = None) -> torch.Tensor:
    """D = A * B^T + C over packed operands; returns D (batch, M/16, N/8, 16, 8).

    C is a float32 tensor in D's layout or None (then every element starts
    from the scalar ``c``). ``out`` may be C itself (in place). With alpha or
    beta given, the alpha/beta form runs instead (bmm_mma_tile_scaled):
    D = fma(alpha, A * B^T, beta * C), the product accumulated from zero.
    Operands packed with an atom K of 8 ((..., 16, 4) and (..., 8, 4) words)
    go through bmm_mma_tile_opts with atom_k = 8. ``dtype`` ('f16' or 'bf16',
    the type both operands were packed from) is required."""
    dt = _dtype_code(dtype, "mma_tile")
    _require_cuda(A, B, C, out)
    if A.dim() != 5 or B.dim() != 5 or A.shape[3] != 16 or B.shape[3] != 8 or \
            A.shape[4] not in (8, 4) or B.shape[4] != A.shape[4]:
        raise ValueError("mma_tile: A must be (batch, M_rep, K_rep, 16, w) and B "
                         "(batch, N_rep, K_rep, 8, w) packed words, w = 8 (k = 16) or 4 (k = 8)")
    atom_k = 2 * A.shape[4]
    batch, M_rep, K_rep = A.shape[:3]
    if B.shape[0] != batch or B.shape[2] != K_rep:
        raise ValueError("mma_tile: A and B disagree on batch or K_rep")
    N_rep = B.shape[1]
    shape = (batch, M_rep, N_rep, 16, 8)
    for t, name in ((A, "A"), (B, "B")):
        if not t.is_contiguous() or t.element_size() != 4:
            raise ValueError(f"mma_tile: {name} must be a contiguous 32-bit tensor")
    if C is not None and (tuple(C.shape) != shape or C.dtype != torch.float32
                          or not C.is_contiguous()):
        raise ValueError(f"mma_tile: C must be a contiguous float32 tensor of shape {shape}")
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=A.device)
    elif tuple(out.shape) != shape or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError(f"mma_tile: out must be a contiguous float32 tensor of shape {shape}")
    if atom_k == 8:
        scaled = not (alpha is None and beta is None)
        opts = MmaOpts(8, KERNELS[kernel], int(scaled), 1.0 if alpha is None else float(alpha),
                       1.0 if beta is None else float(beta))
        _check(lib().bmm_mma_tile_opts(_ptr(out), _ptr(A), _ptr(B), _ptr(C), float(c), batch,
                                       M_rep, N_rep, K_rep, dt, ctypes.byref(opts),
                                       _stream(A)))
    elif alpha is None and beta is None:
        _check(lib().bmm_mma_tile_with(_ptr(out), _ptr(A), _ptr(B), _ptr(C), float(c), batch,
                                       M_rep, N_rep, K_rep, dt, KERNELS[kernel],
                                       _stream(A)))
    else:
        _check(lib().bmm_mma_tile_scaled(
            _ptr(out), _ptr(A), _ptr(B), _ptr(C), float(c), 1.0 if alpha is None else float(alpha),
            1.0 if beta is None else float(beta), batch, M_rep, N_rep, K_rep, dt,
            KERNELS[kernel], _stream(A)))
    return out


def select_kernel(batch: int, M_rep: int, N_rep: int, K_rep: int) -> str:
    return KERNEL_NAMES[_check(lib().bmm_select_kernel(batch, M_rep, N_rep, K_rep))]


# ---- feed-forward operators ----

def _act_code(act: str, fn: str) -> int:
    try:
        return ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"{fn}: unknown activation {act!r}; expected one of {sorted(ACTS)}") from None


# One token's calls last about as long on the GPU as their marshalling does, so
# the common case of each check below comes first and costs a few attribute
# reads; the slow path names the fault.

def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _rows_ld(t: torch.Tensor, name: str, fn: str) -> int:
    """Elements between the rows of a (rows, cols) or (batch, rows, cols) matrix
    with unit innermost stride and batches rows * ld apart."""
    stride = t.stride()
    if len(stride) == 2 and stride[1] == 1:
        rows, cols = t.shape
        if rows <= 1:
            return (cols + 7) >> 3 << 3
        if cols > 1:
            return stride[0]
    if t.dim() not in (2, 3):
        raise ValueError(f"{fn}: {name} must be (rows, cols) or (batch, rows, cols)")
    rows, cols = t.shape[-2:]
    if t.numel() == 0:
        return -(-cols // 8) * 8
    ld = t.stride(-2) if rows > 1 else \
        (t.stride(0) if t.dim() == 3 and t.shape[0] > 1 else -(-cols // 8) * 8)
    if (t.stride(-1) != 1 and cols > 1) or \
            (t.dim() == 3 and t.shape[0] > 1 and t.stride(0) != rows * ld):
        raise ValueError(f"{fn}: {name} must have unit innermost stride and dense batches")
    return ld


def _out(t, shape, dtype, like, fn):
    """The output and the elements between its rows."""
    if t is None:
        return like.new_empty(shape, dtype=dtype), shape[-1]
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{fn}: out must be a {dtype} tensor of shape {tuple(shape)}")
    return t, _rows_ld(t, "out", fn)


def _gated_weights(Wg, Wu, batch, K, fn) -> int:
    """F of two packed weights (batch, F/8, K/16, 8, 8)."""
    shape = Wg.shape
    if len(shape) == 5 and shape == (batch, shape[1], K >> 4, 8, 8) and Wu.shape == shape \
            and K & 15 == 0 and Wg.element_size() == 4 and Wu.element_size() == 4 \
            and Wg.is_contiguous() and Wu.is_contiguous():
        return 8 * shape[1]
    for w, name in ((Wg, "Wg"), (Wu, "Wu")):
        if w.dim() != 5 or w.shape[3:] != (8, 8) or w.element_size() != 4 or not w.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous packed words (batch, F/8, K/16, 8, 8) "
                             "(pack_operand with atom_rows 8)")
    if Wg.shape != Wu.shape:
        raise ValueError(f"{fn}: Wg and Wu differ in shape")
    raise ValueError(f"{fn}: X and the weights disagree on batch or K")


def _half_matrix(t, name, fn):
    try:
        return _HALF_DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{fn}: {name} must be float16 or bfloat16, got {t.dtype}") from None


def gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu",
          save: bool = False, out: torch.Tensor | None = None):
    """H = act(X Wg^T) * (X Wu^T) (bmm_gated): the gated half of a feed-forward
    block in one kernel.

    X is (M, K) or (batch, M, K) float16 or bfloat16, rows any multiple of 8
    elements apart; Wg and Wu are packed B operands (pack_operand(w, 8)) of
    the same type. Returns H (..., M, F) in X's type, and with ``save`` (H, G,
    U), the projections that gated_backward takes. ``act`` is one of ACTS."""
    code = _act_code(act, "gated")
    device = X.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, gated, X, Wg, Wu, act, save, out)
    if not (out is None and 0 <= device == Wg.get_device() == Wu.get_device()):
        _require_cuda(X, Wg, Wu, out)
    dt = _half_matrix(X, "X", "gated")
    ld_x = _rows_ld(X, "X", "gated")
    *lead, M, K = X.shape
    batch = lead[0] if lead else 1
    F = _gated_weights(Wg, Wu, batch, K, "gated")
    H, ld_h = _out(out, (*lead, M, F), X.dtype, X, "gated")
    G = U = None
    if save:
        if ld_h != F and H.numel():
            raise ValueError("gated: with save, out must be contiguous")
        G, U = X.new_empty((*lead, M, F)), X.new_empty((*lead, M, F))
    d = GatedDesc(batch, M, F, K, ld_x, ld_h, dt, code)
    rc = (_lib or lib()).bmm_gated(H.data_ptr(), _addr(G), _addr(U), X.data_ptr(), Wg.data_ptr(),
                                   Wu.data_ptr(), ctypes.byref(d),
                                   _current_stream(device))
    if rc < 0:
        _check(rc)
    return (H, G, U) if save else H


def gated_backward_workspace_bytes(batch: int, M: int, F: int, K: int) -> int:
    """bmm_gated_backward_workspace_bytes for these extents."""
    d = GatedDesc(batch, M, F, K, K, F, BMM_BF16, 0)
    return _check(lib().bmm_gated_backward_workspace_bytes(ctypes.byref(d)))


@_on_its_gpu
def gated_backward(dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor, X: torch.Tensor,
                   Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu", need_dx: bool = True,
                   need_dw: bool = True, workspace: torch.Tensor | None = None):
    """Gradients of gated (bmm_gated_backward): (dX, dWg, dWu) for dH = dL/dH and
    the projections G and U that gated(..., save=True) returned.

    dX is (..., M, K); dWg and dWu are row-major (F, K) ((batch, F, K) for a
    batched X), all in X's type; None stands for what need_dx or need_dw leaves
    out. dH, G and U share one row stride. ``workspace`` (any contiguous
    tensor of at least gated_backward_workspace_bytes) is allocated here when
    not given."""
    fn = "gated_backward"
    code = _act_code(act, fn)
    if not (need_dx or need_dw):
        raise ValueError(f"{fn}: neither need_dx nor need_dw")
    _require_cuda(dH, G, U, X, Wg, Wu, workspace)
    dt = _half_matrix(X, "X", fn)
    ld_x = _rows_ld(X, "X", fn)
    *lead, M, K = X.shape
    batch = lead[0] if lead else 1
    F = _gated_weights(Wg, Wu, batch, K, fn)
    ld_h = _rows_ld(dH, "dH", fn)
    shape, stride, dtype = (*lead, M, F), dH.stride(), X.dtype
    for t, name in ((dH, "dH"), (G, "G"), (U, "U")):
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{fn}: {name} must be a {dtype} tensor of shape {shape}")
        if t.stride() != stride and _rows_ld(t, name, fn) != ld_h:
            raise ValueError(f"{fn}: dH, G and U must have the same row stride")
    d = GatedDesc(batch, M, F, K, ld_x, ld_h, dt, code)
    need = _check(lib().bmm_gated_backward_workspace_bytes(ctypes.byref(d)))
    if workspace is None:
        workspace = X.new_empty(need, dtype=torch.uint8)
    elif not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous")
    dX = X.new_empty((*lead, M, K)) if need_dx else None
    dWg = dWu = None
    if need_dw:
        dWg = X.new_empty((*lead, F, K))
        dWu = X.new_empty((*lead, F, K))
    _check(lib().bmm_gated_backward(_addr(dX), _addr(dWg), _addr(dWu), _addr(dH), _addr(G), _addr(U),
                                    _addr(X), _addr(Wg), _addr(Wu), ctypes.byref(d), _addr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _current_stream(_current_device())))
    return dX, dWg, dWu


def ffn_plan(product: str, batch: int, M: int, F: int, K: int) -> tuple[str, int]:
    """How a feed-forward product of these extents is made (bmm_ffn_plan): its tile, one
    of FFN_TILES, and the number of parts that its sum is cut into. ``product`` is one
    of FFN_PRODUCTS; F is N for "mx4_mma"."""
    splits = ctypes.c_int32()
    tile = _check(lib().bmm_ffn_plan(FFN_PRODUCTS[product], batch, M, F, K, ctypes.byref(splits)))
    return FFN_TILE_NAMES[tile], splits.value


class Mx4Operand(typing.NamedTuple):
    """A 4-bit operand: codes (batch, ceil(rows/16), ceil(K/128), 4, 16, 16) and
    scales (batch, ceil(rows/16), ceil(K/512), 4, 16, 4) uint8, of a (rows, K)
    matrix, or with ``batched`` a (batch, rows, K) one (include/bmm.h gives
    the layout)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    K: int
    batched: bool = False

    @property
    def batch(self) -> int:
        return self.codes.shape[0]


def _mx4_shapes(batch, rows, K):
    r16 = (rows + 15) >> 4
    return (batch, r16, (K + 127) >> 7, 4, 16, 16), (batch, r16, (K + 511) >> 9, 4, 16, 4)


def _mx4_check(op: Mx4Operand, name, fn) -> int:
    """The operand's batch count."""
    codes, scales, rows, K, batched = op
    batch = codes.shape[0]
    want = _mx4_shapes(batch, rows, K)
    if codes.shape == want[0] and scales.shape == want[1] and codes.dtype == scales.dtype == \
            torch.uint8 and codes.is_contiguous() and scales.is_contiguous() and \
            0 <= codes.get_device() == scales.get_device() and (batched or batch == 1):
        return batch
    for t, shape, part in ((codes, want[0], "codes"), (scales, want[1], "scales")):
        if t.shape != shape or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError(f"{fn}: {name}.{part} must be a contiguous uint8 tensor of shape {shape}")
    if batch != 1 and not batched:
        raise ValueError(f"{fn}: {name} has {batch} batches but is not batched")
    _require_cuda(codes, scales)


def mx4_quantize(X: torch.Tensor) -> Mx4Operand:
    """(rows, K) or (batch, rows, K) float32, float16 or bfloat16 to a 4-bit
    operand (bmm_mx4_quantize): blocks of 32 along K, one power-of-two scale
    each. K is a multiple of 32; rows may be any multiple of 8 elements apart."""
    fn = "mx4_quantize"
    device = X.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, mx4_quantize, X)
    if not X.is_cuda:
        _require_cuda(X)
    elem = _ELEM_DTYPES.get(X.dtype)
    if elem is None:
        raise ValueError(f"{fn}: X must be float32, float16 or bfloat16, got {X.dtype}")
    ld = _rows_ld(X, "X", fn)
    *lead, rows, K = X.shape
    batch = lead[0] if lead else 1
    cs, ss = _mx4_shapes(batch, rows, K)
    codes = X.new_empty(cs, dtype=torch.uint8)
    scales = codes.new_empty(ss)
    rc = (_lib or lib()).bmm_mx4_quantize(codes.data_ptr(), scales.data_ptr(), X.data_ptr(), batch,
                                          rows, K, ld, elem, _current_stream(device))
    if rc < 0:
        _check(rc)
    return Mx4Operand(codes, scales, rows, K, bool(lead))


def mx4_dequantize(A: Mx4Operand, dtype: torch.dtype = torch.float32,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The (rows, K) or (batch, rows, K) values of a 4-bit operand in ``dtype``
    (bmm_mx4_dequantize)."""
    fn = "mx4_dequantize"
    batch = _mx4_check(A, "A", fn)
    device = A.codes.get_device()
    if device != _current_device():
        return _on_gpu(device, mx4_dequantize, A, dtype, out)
    if out is not None:
        _require_cuda(A.codes, out)
    elem = _ELEM_DTYPES.get(dtype)
    if elem is None:
        raise ValueError(f"{fn}: dtype must be float32, float16 or bfloat16, got {dtype}")
    codes, scales, rows, K, batched = A
    out, ld = _out(out, (batch, rows, K) if batched else (rows, K), dtype, codes, fn)
    rc = (_lib or lib()).bmm_mx4_dequantize(out.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                            batch, rows, K, ld, elem,
                                            _current_stream(device))
    if rc < 0:
        _check(rc)
    return out


def mx4_mma(A: Mx4Operand, B: Mx4Operand, dtype: torch.dtype = torch.float32,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """D = A * B^T over 4-bit operands (bmm_mx4_mma): row-major (M, N) or (batch,
    M, N) in ``dtype`` (float32, float16 or bfloat16). B's rows are a multiple
    of 8."""
    fn = "mx4_mma"
    batch = _mx4_check(A, "A", fn)
    batch_b = _mx4_check(B, "B", fn)
    device = A.codes.get_device()
    if device != _current_device():
        return _on_gpu(device, mx4_mma, A, B, dtype, out)
    if out is not None or B.codes.get_device() != device:
        _require_cuda(A.codes, B.codes, out)
    elem = _ELEM_DTYPES.get(dtype)
    if elem is None:
        raise ValueError(f"{fn}: dtype must be float32, float16 or bfloat16, got {dtype}")
    a, a_scales, M, K, batched = A
    b, b_scales, N, K_b, _ = B
    if batch != batch_b or K != K_b:
        raise ValueError(f"{fn}: A and B disagree on batch or K")
    out, ld = _out(out, (batch, M, N) if batched else (M, N), dtype, a, fn)
    rc = (_lib or lib()).bmm_mx4_mma(out.data_ptr(), a.data_ptr(), a_scales.data_ptr(), b.data_ptr(),
                                     b_scales.data_ptr(), batch, M, N, K, ld, elem,
                                     _current_stream(device))
    if rc < 0:
        _check(rc)
    return out


def mx4_gated(X: Mx4Operand, Wg: Mx4Operand, Wu: Mx4Operand, act: str = "silu",
              dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """H = act(X Wg^T) * (X Wu^T) over 4-bit operands (bmm_mx4_gated): row-major
    (M, F) or (batch, M, F) in ``dtype`` (float16 or bfloat16). The weights' F
    rows are a multiple of 8."""
    fn = "mx4_gated"
    code = _act_code(act, fn)
    batch = _mx4_check(X, "X", fn)
    batch_g, batch_u = _mx4_check(Wg, "Wg", fn), _mx4_check(Wu, "Wu", fn)
    device = X.codes.get_device()
    if device != _current_device():
        return _on_gpu(device, mx4_gated, X, Wg, Wu, act, dtype, out)
    if not (out is None and device == Wg.codes.get_device() == Wu.codes.get_device()):
        _require_cuda(X.codes, Wg.codes, Wu.codes, out)
    if dtype not in _HALF_DTYPES:
        raise ValueError(f"{fn}: dtype must be float16 or bfloat16, got {dtype}")
    x, x_scales, M, K, batched = X
    g, g_scales, F, K_g, _ = Wg
    u, u_scales, F_u, K_u, _ = Wu
    if F != F_u or K_g != K_u or batch_g != batch_u:
        raise ValueError(f"{fn}: Wg and Wu differ in shape")
    if batch != batch_g or K != K_g:
        raise ValueError(f"{fn}: X and the weights disagree on batch or K")
    out, ld = _out(out, (batch, M, F) if batched else (M, F), dtype, x, fn)
    rc = (_lib or lib()).bmm_mx4_gated(out.data_ptr(), x.data_ptr(), x_scales.data_ptr(),
                                       g.data_ptr(), g_scales.data_ptr(), u.data_ptr(),
                                       u_scales.data_ptr(), batch, M, F, K, ld, code,
                                       _ELEM_DTYPES[dtype], _current_stream(device))
    if rc < 0:
        _check(rc)
    return out


# ---- products by groups of rows (the experts of a mixture) ----

def _group_weights(ws, names, ends, K, fn):
    """(groups, N) of packed weights (groups, N/8, K/16, 8, 8) and their row ends."""
    shape = ws[0].shape
    if ends.dtype != torch.int32 or ends.dim() != 1 or not ends.is_contiguous():
        raise ValueError(f"{fn}: ends must be a contiguous int32 tensor of one dimension")
    for w, name in zip(ws, names):
        if w.dim() != 5 or w.shape[3:] != (8, 8) or w.element_size() != 4 or not w.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous packed words (groups, N/8, K/16, 8, 8) "
                             "(pack_operand with atom_rows 8)")
        if w.shape != shape:
            raise ValueError(f"{fn}: {names[0]} and {name} differ in shape")
    if shape[0] != ends.shape[0]:
        raise ValueError(f"{fn}: {ends.shape[0]} ends for the weights of {shape[0]} groups")
    if K != 16 * shape[2]:
        raise ValueError(f"{fn}: X and the weights disagree on K")
    return shape[0], 8 * shape[1]


def _group_rows(X, name, fn):
    """(element type, row stride) of a (T, K) matrix."""
    if X.dim() != 2:
        raise ValueError(f"{fn}: {name} must be (rows, columns), all groups' rows one after another")
    return _half_matrix(X, name, fn), _rows_ld(X, name, fn)


def grouped_mma(X: torch.Tensor, W: torch.Tensor, ends: torch.Tensor,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W_e^T for the rows of each group e (bmm_grouped_mma): the rows of each
    expert of a mixture with its own weight, in one kernel.

    X is (T, K) float16 or bfloat16, its rows sorted by group, any multiple of 8
    elements apart; W is (E, N/8, K/16, 8, 8) packed words (pack_operand(w, 8) of
    (E, N, K)) of the same type. ``ends`` is (E,) int32 on the same GPU: group e has
    the rows from ends[e - 1] (the first from 0) up to ends[e], the running sum of
    the groups' sizes; the host does not read it. Rows behind the last group are
    not read; their outputs are zero, or with ``out`` given left as they were.
    Returns Y (T, N) in X's type."""
    fn = "grouped_mma"
    device = X.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, grouped_mma, X, W, ends, out)
    if not (out is None and 0 <= device == W.get_device() == ends.get_device()):
        _require_cuda(X, W, ends, out)
    dt, ld_x = _group_rows(X, "X", fn)
    T, K = X.shape
    E, N = _group_weights((W,), ("W",), ends, K, fn)
    Y, ld_y = _out(out, (T, N), X.dtype, X, fn)
    d = GroupedDesc(E, T, N, K, ld_x, ld_y, dt, 0, out is None)
    rc = (_lib or lib()).bmm_grouped_mma(Y.data_ptr(), X.data_ptr(), W.data_ptr(), ends.data_ptr(),
                                         ctypes.byref(d), _current_stream(device))
    if rc < 0:
        _check(rc)
    return Y


def grouped_gated(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, ends: torch.Tensor,
                  act: str = "silu", save: bool = False, out: torch.Tensor | None = None):
    """H = act(X Wg_e^T) * (X Wu_e^T) for the rows of each group e (bmm_grouped_gated).

    X, the weights and ``ends`` as in grouped_mma. Returns H (T, F) in X's type, and
    with ``save`` (H, G, U), the projections that grouped_gated_backward takes."""
    fn = "grouped_gated"
    code = _act_code(act, fn)
    device = X.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, grouped_gated, X, Wg, Wu, ends, act, save, out)
    if not (out is None and 0 <= device == Wg.get_device() == Wu.get_device() == ends.get_device()):
        _require_cuda(X, Wg, Wu, ends, out)
    dt, ld_x = _group_rows(X, "X", fn)
    T, K = X.shape
    E, F = _group_weights((Wg, Wu), ("Wg", "Wu"), ends, K, fn)
    H, ld_h = _out(out, (T, F), X.dtype, X, fn)
    G = U = None
    if save:
        if ld_h != F and H.numel():
            raise ValueError(f"{fn}: with save, out must be contiguous")
        # (with out given its rows behind the last group stay, and G and U have no old ones)
        new = X.new_empty if out is None else X.new_zeros
        G, U = new((T, F)), new((T, F))
    d = GroupedDesc(E, T, F, K, ld_x, ld_h, dt, code, out is None)
    rc = (_lib or lib()).bmm_grouped_gated(H.data_ptr(), _addr(G), _addr(U), X.data_ptr(),
                                           Wg.data_ptr(), Wu.data_ptr(), ends.data_ptr(),
                                           ctypes.byref(d), _current_stream(device))
    if rc < 0:
        _check(rc)
    return (H, G, U) if save else H


def grouped_mma_backward_workspace_bytes(groups: int, T: int, N: int, K: int) -> int:
    """bmm_grouped_mma_backward_workspace_bytes for these extents."""
    d = GroupedDesc(groups, T, N, K, K, N, BMM_BF16, 0, 1)
    return _check(lib().bmm_grouped_mma_backward_workspace_bytes(ctypes.byref(d)))


def grouped_gated_backward_workspace_bytes(groups: int, T: int, F: int, K: int) -> int:
    """bmm_grouped_gated_backward_workspace_bytes for these extents."""
    d = GroupedDesc(groups, T, F, K, K, F, BMM_BF16, 0, 1)
    return _check(lib().bmm_grouped_gated_backward_workspace_bytes(ctypes.byref(d)))


def _grad_workspace(need, workspace, X, fn):
    if workspace is None:
        return X.new_empty(need, dtype=torch.uint8)
    if not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous")
    return workspace


def _same_rows(ts, names, shape, dtype, fn) -> int:
    """The common row stride of matrices of one shape and type."""
    ld = None
    for t, name in zip(ts, names):
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{fn}: {name} must be a {dtype} tensor of shape {shape}")
        own = _rows_ld(t, name, fn)
        if ld is not None and own != ld:
            raise ValueError(f"{fn}: {', '.join(names)} must have the same row stride")
        ld = own
    return ld


@_on_its_gpu
def grouped_mma_backward(dY: torch.Tensor, X: torch.Tensor, W: torch.Tensor, ends: torch.Tensor,
                         need_dx: bool = True, need_dw: bool = True,
                         workspace: torch.Tensor | None = None):
    """Gradients of grouped_mma (bmm_grouped_mma_backward): (dX, dW) for dY = dL/dY.

    dX is (T, K), zero behind the last group; dW is row-major (E, N, K), zero for a
    group without rows; both in X's type, None for what need_dx or need_dw leaves
    out. ``workspace`` (any contiguous tensor of at least
    grouped_mma_backward_workspace_bytes) is allocated here when not given."""
    fn = "grouped_mma_backward"
    if not (need_dx or need_dw):
        raise ValueError(f"{fn}: neither need_dx nor need_dw")
    _require_cuda(dY, X, W, ends, workspace)
    dt, ld_x = _group_rows(X, "X", fn)
    T, K = X.shape
    E, N = _group_weights((W,), ("W",), ends, K, fn)
    ld_y = _same_rows((dY,), ("dY",), (T, N), X.dtype, fn)
    d = GroupedDesc(E, T, N, K, ld_x, ld_y, dt, 0, 1)
    need = _check(lib().bmm_grouped_mma_backward_workspace_bytes(ctypes.byref(d)))
    workspace = _grad_workspace(need, workspace, X, fn)
    dX = X.new_empty((T, K)) if need_dx else None
    dW = X.new_empty((E, N, K)) if need_dw else None
    _check(lib().bmm_grouped_mma_backward(
        _addr(dX), _addr(dW), _addr(dY), _addr(X), _addr(W), _addr(ends), ctypes.byref(d),
        _addr(workspace), workspace.numel() * workspace.element_size(),
        _current_stream(_current_device())))
    return dX, dW


@_on_its_gpu
def grouped_gated_backward(dH: torch.Tensor, G: torch.Tensor, U: torch.Tensor, X: torch.Tensor,
                           Wg: torch.Tensor, Wu: torch.Tensor, ends: torch.Tensor,
                           act: str = "silu", need_dx: bool = True, need_dw: bool = True,
                           workspace: torch.Tensor | None = None):
    """Gradients of grouped_gated (bmm_grouped_gated_backward): (dX, dWg, dWu) for dH
    = dL/dH and the projections that grouped_gated(..., save=True) returned.

    As grouped_mma_backward, with dWg and dWu (E, F, K) in dW's place. dH, G and U
    share one row stride."""
    fn = "grouped_gated_backward"
    code = _act_code(act, fn)
    if not (need_dx or need_dw):
        raise ValueError(f"{fn}: neither need_dx nor need_dw")
    _require_cuda(dH, G, U, X, Wg, Wu, ends, workspace)
    dt, ld_x = _group_rows(X, "X", fn)
    T, K = X.shape
    E, F = _group_weights((Wg, Wu), ("Wg", "Wu"), ends, K, fn)
    ld_h = _same_rows((dH, G, U), ("dH", "G", "U"), (T, F), X.dtype, fn)
    d = GroupedDesc(E, T, F, K, ld_x, ld_h, dt, code, 1)
    need = _check(lib().bmm_grouped_gated_backward_workspace_bytes(ctypes.byref(d)))
    workspace = _grad_workspace(need, workspace, X, fn)
    dX = X.new_empty((T, K)) if need_dx else None
    dWg = dWu = None
    if need_dw:
        dWg, dWu = X.new_empty((E, F, K)), X.new_empty((E, F, K))
    _check(lib().bmm_grouped_gated_backward(
        _addr(dX), _addr(dWg), _addr(dWu), _addr(dH), _addr(G), _addr(U), _addr(X), _addr(Wg),
        _addr(Wu), _addr(ends), ctypes.byref(d), _addr(workspace),
        workspace.numel() * workspace.element_size(), _current_stream(_current_device())))
    return dX, dWg, dWu


def group_plan(product: str, groups: int, T: int, N: int, K: int) -> tuple[str, int]:
    """How a product by groups or of 8-bit integers is made (bmm_group_plan): its tile,
    one of FFN_TILES, and the number of parts that its sum is cut into. ``product`` is
    one of GROUP_PRODUCTS; N is the width F of a gated block; groups 0: one 8-bit
    weight."""
    splits = ctypes.c_int32()
    tile = _check(lib().bmm_group_plan(GROUP_PRODUCTS[product], groups, T, N, K,
                                       ctypes.byref(splits)))
    return FFN_TILE_NAMES[tile], splits.value


# ---- 8-bit integers ----

class I8Operand(typing.NamedTuple):
    """8-bit codes with a float32 scale for each row. As i8_quantize makes them:
    codes (rows, K) or (batch, rows, K) int8, scales (rows,) or (batch, rows). As a
    weight (i8_pack): codes (batch, rows/8, K/32, 8, 8) packed 32-bit words, scales
    (batch, rows); by groups the batch is the groups."""
    codes: torch.Tensor
    scales: torch.Tensor


def i8_quantize(X: torch.Tensor) -> I8Operand:
    """(rows, K) or (batch, rows, K) float32, float16 or bfloat16 to codes -127 .. 127
    and a scale for each row, max |x| / 127 (bmm_i8_quantize). K is a multiple of 32;
    rows may be any multiple of 8 elements apart."""
    fn = "i8_quantize"
    device = X.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, i8_quantize, X)
    if not X.is_cuda:
        _require_cuda(X)
    elem = _ELEM_DTYPES.get(X.dtype)
    if elem is None:
        raise ValueError(f"{fn}: X must be float32, float16 or bfloat16, got {X.dtype}")
    ld = _rows_ld(X, "X", fn)
    *lead, rows, K = X.shape
    codes = X.new_empty(X.shape, dtype=torch.int8)
    scales = X.new_empty((*lead, rows), dtype=torch.float32)
    rc = (_lib or lib()).bmm_i8_quantize(codes.data_ptr(), scales.data_ptr(), X.data_ptr(),
                                         lead[0] if lead else 1, rows, K, ld, elem,
                                         _current_stream(device))
    if rc < 0:
        _check(rc)
    return I8Operand(codes, scales)


def i8_pack(A: I8Operand) -> I8Operand:
    """Row-major codes (rows, K) or (batch, rows, K) as a weight of i8_mma and
    i8_gated (pack_operand of the codes, two as a 16-bit value). Rows are a multiple
    of 8, K of 32."""
    codes, scales = A
    if codes.dtype != torch.int8 or codes.dim() not in (2, 3) or not codes.is_contiguous():
        raise ValueError("i8_pack: codes must be contiguous int8 (rows, K) or (batch, rows, K)")
    if codes.shape[:-1] != scales.shape:
        raise ValueError("i8_pack: codes and scales disagree on the rows")
    if codes.shape[-2] % 8 or codes.shape[-1] % 32:
        raise ValueError("i8_pack: rows must be a multiple of 8 and K of 32")
    return I8Operand(pack_operand(codes.view(torch.int16), 8),
                     scales if scales.dim() == 2 else scales[None])


def _i8_rows(A, name, fn):
    """(row stride, batch) of a row-major operand."""
    codes, scales = A
    if codes.dtype != torch.int8:
        raise ValueError(f"{fn}: {name}.codes must be int8, got {codes.dtype}")
    shape, stride = codes.shape, codes.stride()
    if scales.shape != shape[:-1] or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"{fn}: {name}.scales must be contiguous float32 of shape {tuple(shape[:-1])}")
    if len(shape) == 2 and stride[1] == 1 and shape[0] > 1 and shape[1] > 1:
        return stride[0], 1
    return _rows_ld(codes, f"{name}.codes", fn), shape[0] if len(shape) == 3 else 1


def _i8_weight(B, name, K, fn):
    """(batch, N) of a packed operand."""
    codes, scales = B
    shape = codes.shape
    if codes.dim() != 5 or shape[3:] != (8, 8) or codes.element_size() != 4 \
            or not codes.is_contiguous():
        raise ValueError(f"{fn}: {name}.codes must be contiguous packed words (batch, N/8, K/32, 8, 8) "
                         "(i8_pack)")
    batch, N = shape[0], 8 * shape[1]
    if scales.shape != (batch, N) or scales.dtype != torch.float32 or not scales.is_contiguous():
        raise ValueError(f"{fn}: {name}.scales must be contiguous float32 of shape {(batch, N)}")
    if K != 32 * shape[2]:
        raise ValueError(f"{fn}: the operands disagree on K")
    return batch, N


def _i8_desc(A, ws, names, ends, dtype, act, out, fn):
    """(output, descriptor) of a product of a row-major operand and packed weights."""
    ld_a, batch = _i8_rows(A, names[0], fn)
    shape = A.codes.shape
    M, K = shape[-2:]
    batch_w, N = _i8_weight(ws[0], names[1], K, fn)
    if len(ws) == 2 and _i8_weight(ws[1], names[2], K, fn) != (batch_w, N):
        raise ValueError(f"{fn}: {names[1]} and {names[2]} differ in shape")
    if ends is None:
        if batch != batch_w:
            raise ValueError(f"{fn}: {names[0]} and {names[1]} disagree on batch")
    else:
        if len(shape) != 2:
            raise ValueError(f"{fn}: with ends, {names[0]} must be (rows, K)")
        if ends.dtype != torch.int32 or ends.dim() != 1 or not ends.is_contiguous():
            raise ValueError(f"{fn}: ends must be a contiguous int32 tensor of one dimension")
        if ends.shape[0] != batch_w:
            raise ValueError(f"{fn}: {ends.shape[0]} ends for the weights of {batch_w} groups")
    D, ld_d = _out(out, (*shape[:-1], N), dtype, A.codes, fn)
    return D, I8Desc(batch_w, M, N, K, ld_a, ld_d, _ELEM_DTYPES[dtype], act, out is None)


def i8_mma(A: I8Operand, B: I8Operand, ends: torch.Tensor | None = None,
           dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """D = A B^T of 8-bit integers with a scale for each row of both (bmm_i8_mma):
    (M, N) or (batch, M, N) in ``dtype`` (float32, float16 or bfloat16).

    A is row-major (i8_quantize), B packed (i8_pack of an i8_quantize, or a
    checkpoint's codes). With ``ends`` the rows of A are sorted by group and B holds
    a weight for each, as in grouped_mma."""
    fn = "i8_mma"
    a, sa = A
    b, sb = B
    device = a.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, i8_mma, A, B, ends, dtype, out)
    _require_cuda(a, sa, b, sb, ends, out)
    if dtype not in _ELEM_DTYPES:
        raise ValueError(f"{fn}: dtype must be float32, float16 or bfloat16, got {dtype}")
    D, d = _i8_desc(A, (B,), ("A", "B"), ends, dtype, 0, out, fn)
    rc = (_lib or lib()).bmm_i8_mma(D.data_ptr(), a.data_ptr(), sa.data_ptr(), b.data_ptr(),
                                    sb.data_ptr(), _addr(ends), ctypes.byref(d),
                                    _current_stream(device))
    if rc < 0:
        _check(rc)
    return D


def i8_gated(X: I8Operand, Wg: I8Operand, Wu: I8Operand, ends: torch.Tensor | None = None,
             act: str = "silu", dtype: torch.dtype = torch.bfloat16,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """H = act(X Wg^T) * (X Wu^T) over 8-bit integers (bmm_i8_gated): (M, F) or (batch,
    M, F) in ``dtype`` (float16 or bfloat16). Operands and ``ends`` as in i8_mma."""
    fn = "i8_gated"
    code = _act_code(act, fn)
    x, sx = X
    device = x.get_device()
    if device >= 0 and device != _current_device():
        return _on_gpu(device, i8_gated, X, Wg, Wu, ends, act, dtype, out)
    _require_cuda(x, sx, *Wg, *Wu, ends, out)
    if dtype not in _HALF_DTYPES:
        raise ValueError(f"{fn}: dtype must be float16 or bfloat16, got {dtype}")
    H, d = _i8_desc(X, (Wg, Wu), ("X", "Wg", "Wu"), ends, dtype, code, out, fn)
    rc = (_lib or lib()).bmm_i8_gated(H.data_ptr(), x.data_ptr(), sx.data_ptr(),
                                      Wg.codes.data_ptr(), Wg.scales.data_ptr(),
                                      Wu.codes.data_ptr(), Wu.scales.data_ptr(), _addr(ends),
                                      ctypes.byref(d), _current_stream(device))
    if rc < 0:
        _check(rc)
    return H
