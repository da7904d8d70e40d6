/*
 * bmm.h — C ABI of the MI355X (gfx950) tiled f16/bf16 multiply-accumulate
 * D = A * B^T + C with float32 accumulation, over the packed operand layouts
 * of the Apache TVM "tirx" mma.sync tile-op page.
 *
 * Conventions shared by every entry point:
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; the
 *     library keeps no reference to it after the call returns.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the null
 *     stream) and return once the kernels are enqueued.
 *   - Arguments are validated on the host, once per call, before any HIP
 *     call (the cp.async.bulk.tensor page, "Example: two explicit 8x16
 *     boxes": descriptor set-up is host work, not repeated per box). On a
 *     failed check nothing is launched and nothing is written.
 *   - Invalid fields are rejected, never promoted, folded, transposed or
 *     reinterpreted (cp.async.bulk.tensor page, "Operands and descriptor
 *     fields"; mma.sync page introduction: no implicit type change, K-atom
 *     choice or transpose).
 *   - Return value: BMM_OK (0) or a negative status; bmm_last_error()
 *     returns a message for the last failure on the calling thread.
 *   - The library allocates no device memory. Scratch space (the split-K
 *     partial sums) is a caller-owned workspace, except in
 *     bmm_mma_tile_splitk_noalloc, which uses a fixed static array per device.
 *   - Destination first (mma.sync page, "Operand coordinates and
 *     ownership": the call takes D, A, B, C).
 */
#ifndef BMM_H
#define BMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BMM_F16 = 0, BMM_BF16 = 1 } bmm_dtype;

enum {
  BMM_OK = 0,
  BMM_EINVAL = -1,   /* bad extent, dtype, field value or null pointer */
  BMM_EALIGN = -2,   /* pointer or stride not aligned as required */
  BMM_EOVERLAP = -3, /* destination overlaps a source (other than D == C) */
  BMM_ERANGE = -4,   /* a box image larger than the staging limit */
  BMM_EHIP = -5      /* the HIP runtime reported an error at launch */
};

/* Kernel selection for bmm_mma_tile_with. AUTO picks by shape (TILED with
 * more than 128 256 x 256 tiles, ragged ones counted, else TILED_256x128 with
 * more than 128 256 x 128 tiles, else TILED_128 with at least 128 128 x 128
 * tiles, else SKINNY, else DIRECT if a grid limit rules the others out); the
 * others force one kernel (every kernel accepts every valid shape within its
 * launch-grid limits). All three tiled kernels give identical results. */
typedef enum {
  BMM_KERNEL_AUTO = 0,
  BMM_KERNEL_DIRECT = 1, /* one wave per 16x16 output block, operands straight from HBM */
  BMM_KERNEL_TILED = 2,  /* LDS-staged 256x256 macro tiles for large M and N */
  BMM_KERNEL_SKINNY = 3, /* few output tiles: K split across the waves of a workgroup, B streamed */
  BMM_KERNEL_TILED_128 = 4, /* LDS-staged 128x128 macro tiles, two workgroups per CU */
  BMM_KERNEL_TILED_256x128 = 5 /* LDS-staged 256 (M) x 128 (N) macro tiles, one per CU */
} bmm_kernel;

/*
 * bmm_pack_operand — row-major halves to packed b32 atoms.
 *
 * Defined by the mma.sync page, "Operand coordinates and ownership" (A is
 * (M_repeat, K_repeat, 16, k/2) and B is (N_repeat, K_repeat, 8, k/2) b32
 * words, each word two adjacent K values) and the worked example's host
 * code (row-major halves reshaped, transposed and viewed as uint32, so the
 * even K value is the low 16 bits). Atom K is k = 16.
 *
 *   dst[b, r, kr, i, w] = src[b, R*r+i, 16*kr+2*w] | src[b, R*r+i, 16*kr+2*w+1] << 16
 *
 * dst       (batch, rows/R, K/16, R, 8) uint32, contiguous, 16-byte aligned.
 * src       (batch, rows, ld_src) 16-bit values (f16 or bf16 bits; the bits are
 *           moved, never converted), batch stride rows*ld_src elements,
 *           16-byte aligned.
 * rows      multiple of atom_rows; K multiple of 16; ld_src >= K and a
 *           multiple of 8 (16-byte row starts). Zero batch, rows or K is a
 *           no-op.
 * atom_rows R: 16 for an A operand, 8 for a B operand.
 * Errors: BMM_EINVAL (extents, atom_rows), BMM_EALIGN, BMM_EOVERLAP (dst and
 * src overlap), BMM_EHIP.
 */
int bmm_pack_operand(uint32_t* dst, const uint16_t* src, int64_t batch, int64_t rows,
                     int64_t K, int64_t ld_src, int32_t atom_rows, void* stream);

/*
 * bmm_pack_operand_k8 — row-major halves to packed atoms with an atom K of 8.
 *
 * The mma.sync page's introduction names the m16n8k8 form beside m16n8k16,
 * and its table of shapes gives k = 8 for f16/bf16 inputs. With k = 8 the
 * layouts of "Operand coordinates and ownership" hold k/2 = 4 words per atom
 * row: A is (M_repeat, K_repeat, 16, 4) and B is (N_repeat, K_repeat, 8, 4)
 * words, K_repeat = K/8:
 *
 *   dst[b, r, kr, i, w] = src[b, R*r+i, 8*kr+2*w] | src[b, R*r+i, 8*kr+2*w+1] << 16
 *
 * dst  (batch, rows/R, K/8, R, 4) uint32, contiguous, 16-byte aligned.
 * K    a multiple of 8. Every other argument, and the errors, as
 *      bmm_pack_operand.
 * The result feeds bmm_mma_tile_opts with atom_k = 8.
 */
int bmm_pack_operand_k8(uint32_t* dst, const uint16_t* src, int64_t batch, int64_t rows,
                        int64_t K, int64_t ld_src, int32_t atom_rows, void* stream);

/*
 * bmm_pack_operand_kmajor — packing from a K-major (transposed) source.
 *
 * The mma.sync page ("Accumulation, transpose and alpha/beta") leaves a
 * logical transpose to explicit preparation: a view cannot move values
 * between lanes, so an operand whose K values are not contiguous must be
 * rewritten. This is that preparation for the packed layouts: the source
 * holds element (row, k) of the logical operand at src[b, k, row] (rows
 * contiguous), and the result is exactly what bmm_pack_operand gives for the
 * row-major matrix:
 *
 *   dst[b, r, kr, i, w] = src[b, 16*kr+2*w, R*r+i] | src[b, 16*kr+2*w+1, R*r+i] << 16
 *
 * dst       (batch, rows/R, K/16, R, 8) uint32, contiguous, 16-byte aligned.
 * src       (batch, K, ld_src) 16-bit values, batch stride K*ld_src, 16-byte aligned.
 * rows      multiple of atom_rows; K multiple of 16 and below 2^22; ld_src >= rows and
 *           a multiple of 8; batch at most 65535; rows below 2^36. Zero batch, rows or K is a
 *           no-op.
 * Errors: as bmm_pack_operand.
 */
int bmm_pack_operand_kmajor(uint32_t* dst, const uint16_t* src, int64_t batch, int64_t rows,
                            int64_t K, int64_t ld_src, int32_t atom_rows, void* stream);

/*
 * bmm_pack_operand_kmajor_k8 — K-major source to the m16n8k8 layout.
 *
 * The two preparations above together: a K-major (transposed) source, as for
 * bmm_pack_operand_kmajor, packed into atoms with an atom K of 8, as for
 * bmm_pack_operand_k8 (mma.sync page: "Accumulation, transpose and
 * alpha/beta"; the m16n8k8 form of the introduction and the table of shapes).
 * The result is exactly what bmm_pack_operand_k8 gives for the row-major
 * matrix:
 *
 *   dst[b, r, kr, i, w] = src[b, 8*kr+2*w, R*r+i] | src[b, 8*kr+2*w+1, R*r+i] << 16
 *
 * dst  (batch, rows/R, K/8, R, 4) uint32, contiguous, 16-byte aligned.
 * K    a multiple of 8 and below 2^22. Every other argument, and the errors, as
 *      bmm_pack_operand_kmajor.
 */
int bmm_pack_operand_kmajor_k8(uint32_t* dst, const uint16_t* src, int64_t batch, int64_t rows,
                               int64_t K, int64_t ld_src, int32_t atom_rows, void* stream);

/*
 * bmm_box_copy — a rectangular global box through an LDS image.
 *
 * The role of the TMA tile-mode box load on the cp.async.bulk.tensor page
 * ("Operands and descriptor fields", "Example: two explicit 8x16 boxes"):
 * for each repeat t the box at coords + t*coord_step is staged into a
 * shared-memory (LDS) image, laid out with the requested swizzle, and the
 * image is written out compact and unswizzled:
 *
 *   dst_image[t, j_0..j_{rank-1}] = src[coords + t*coord_step + j] if every
 *                                   coordinate is inside dims, else 0.
 *
 * desc fields (outer-to-inner order, as on the page):
 *   rank        1..5
 *   elem_bytes  1, 2, 4 or 8 (the storage type; never reinterpreted)
 *   dims        global extents, each >= 1
 *   strides     byte strides; strides[rank-1] == elem_bytes; outer strides
 *               multiples of 16 ("suitably aligned outer byte strides")
 *   box         1..256 per dimension
 *   coords      start coordinates; may lie partly or wholly outside dims
 *   n_repeat    >= 1 repeats (the leading image axis)
 *   coord_step  per-repeat coordinate increment
 *   swizzle     0..3: none / 32-byte / 64-byte / 128-byte XOR swizzle of
 *               the LDS image (internal; the exported image is unswizzled)
 *   oob_fill    0 (zero fill, the page's default) is the only value accepted
 * dst_image    (n_repeat, box...) compact, 16-byte aligned; must not overlap src.
 * src          16-byte aligned base of the global tensor.
 * bytes_moved  nullable host pointer; receives n_repeat * prod(box) * elem_bytes.
 * One repeat's image may hold at most 65536 bytes (else BMM_ERANGE).
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP, BMM_ERANGE, BMM_EHIP.
 */
typedef struct {
  int32_t rank;
  int32_t elem_bytes;
  int64_t dims[5];
  int64_t strides[5];
  int32_t box[5];
  int64_t coords[5];
  int32_t n_repeat;
  int64_t coord_step[5];
  int32_t swizzle;
  int32_t oob_fill;
} bmm_box_desc;

int bmm_box_copy(void* dst_image, const void* src, const bmm_box_desc* desc,
                 int64_t* bytes_moved, void* stream);

/*
 * bmm_box_store — a compact image written into a rectangular global box.
 *
 * The store direction of the cp.async.bulk.tensor page ("Stores, reductions,
 * and completion": the load's coordinate/box contract, global destination
 * first). Each repeat's image is staged through an LDS image (with the
 * requested swizzle) and written out:
 *
 *   dst[coords + t*coord_step + j] = src_image[t, j_0..j_{rank-1}]
 *                                    for every coordinate inside dims;
 *   elements outside dims are not written.
 *
 * Repeats are applied in ascending t: where the boxes of two repeats
 * overlap, the later repeat's values stand.
 * desc         as bmm_box_copy; additionally the destination view must not
 *              overlap itself (each outer stride at least the byte extent of
 *              the dimensions inside it), else BMM_EINVAL.
 * src_image    (n_repeat, box...) compact, 16-byte aligned, not overlapping dst.
 * bytes_moved  nullable; receives n_repeat * prod(box) * elem_bytes (image bytes read).
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP, BMM_ERANGE, BMM_EHIP.
 */
int bmm_box_store(void* dst, const void* src_image, const bmm_box_desc* desc,
                  int64_t* bytes_moved, void* stream);

/* Element types of bmm_box_reduce_add; each must match desc->elem_bytes. */
typedef enum {
  BMM_ELEM_F32 = 1,  /* 4 bytes */
  BMM_ELEM_F16 = 2,  /* 2 bytes, IEEE binary16 */
  BMM_ELEM_BF16 = 3, /* 2 bytes, bfloat16 */
  BMM_ELEM_I32 = 4,  /* 4 bytes, wraps modulo 2^32 (signed or unsigned alike) */
  BMM_ELEM_I64 = 5   /* 8 bytes, wraps modulo 2^64 */
} bmm_elem_type;

/*
 * bmm_box_reduce_add — add a compact image into a rectangular global box.
 *
 * The add reduction of the cp.async.bulk.tensor page ("Stores, reductions,
 * and completion"); the destination holds its starting value beforehand.
 *
 *   dst[coords + t*coord_step + j] = dst[...] + src_image[t, j]
 *
 * for every coordinate inside dims, repeats in ascending t, one rounding per
 * add in the element type (round to nearest even; f16 and bf16 sums are
 * correctly rounded). Arguments, ordering and errors as bmm_box_store, plus
 * BMM_EINVAL for an elem_type that is not a bmm_elem_type or does not match
 * elem_bytes. NaN payloads of float results are unspecified.
 */
int bmm_box_reduce_add(void* dst, const void* src_image, const bmm_box_desc* desc,
                       int32_t elem_type, int64_t* bytes_moved, void* stream);

/*
 * bmm_mma_tile — D = A * B^T + C over packed operands.
 *
 * Defined by the mma.sync page: "Operand coordinates and ownership" (the
 * layouts below; A and B share one input dtype, the accumulator is float32)
 * and "Accumulation, transpose and alpha/beta" (repeat order batch, M, N,
 * then K; C is a matching tensor or a scalar broadcast; only the first K
 * step reads C, later steps read D).
 *
 * D  (batch, M_rep, N_rep, 16, 8) float32, written.
 * A  (batch, M_rep, K_rep, 16, 8) uint32 words (two halves per word, even K low).
 * B  (batch, N_rep, K_rep, 8, 8)  uint32 words; B's logical axes are (N, K).
 * C  (batch, M_rep, N_rep, 16, 8) float32, or NULL to use c_scalar for every
 *    element. C == D (in place) is allowed: each output is read before it is
 *    written by the same thread. Any other overlap of D with A, B or C is
 *    rejected.
 * Every pointer is 16-byte aligned. Extents are >= 0; a zero batch, M_rep or
 * N_rep is a no-op; K_rep = 0 gives D = C (the empty sum).
 * Summation order inside the hardware's 32-deep MFMA step is the hardware's;
 * between steps K is taken in ascending order from C.
 * This entry point takes no workspace and so never splits K: for shapes with
 * few output tiles and a long K, bmm_splitk_suggested says when
 * bmm_mma_tile_splitk is faster, and with how many splits.
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP, BMM_EHIP.
 */
int bmm_mma_tile(float* D, const uint32_t* A, const uint32_t* B, const float* C,
                 float c_scalar, int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep,
                 bmm_dtype dtype, void* stream);

/* bmm_mma_tile with an explicit kernel choice (bmm_kernel); same contract. */
int bmm_mma_tile_with(float* D, const uint32_t* A, const uint32_t* B, const float* C,
                      float c_scalar, int64_t batch, int64_t M_rep, int64_t N_rep,
                      int64_t K_rep, bmm_dtype dtype, int32_t kernel, void* stream);

/*
 * bmm_mma_tile_scaled — D = alpha * (A * B^T) + beta * C, scaling at the call site.
 *
 * The mma.sync page ("Accumulation, transpose and alpha/beta") puts alpha/beta
 * scaling before or after the MMA at the call site, with the intended
 * rounding order; this entry point fixes that order: the product is
 * accumulated from zero (K ascending between 32-deep hardware steps), then
 *   D = fma(alpha, acc, fl(beta * C))
 * with one rounding for the final multiply-add (the fma page: a*b+c is one
 * fused operation). C (or c_scalar when C is NULL) is read once, in the
 * epilogue; D == C in place is allowed. Operands, layouts, kernel choice and
 * errors as bmm_mma_tile_with. alpha = beta = 1 differs from bmm_mma_tile
 * only in where C enters the sum (it is added last here, first there).
 */
int bmm_mma_tile_scaled(float* D, const uint32_t* A, const uint32_t* B, const float* C,
                        float c_scalar, float alpha, float beta, int64_t batch, int64_t M_rep,
                        int64_t N_rep, int64_t K_rep, bmm_dtype dtype, int32_t kernel,
                        void* stream);

/*
 * bmm_mma_tile_opts — every form of the multiply-accumulate behind one call.
 *
 * The options select what the other mma entry points fix:
 *   atom_k  16: operands in the k = 16 layout (bmm_pack_operand), K_rep
 *           counts 16-deep atoms; 8: the m16n8k8 layout (bmm_pack_operand_k8,
 *           the mma.sync page's introduction and table of shapes), A is
 *           (batch, M_rep, K_rep, 16, 4) and B (batch, N_rep, K_rep, 8, 4)
 *           words and K_rep counts 8-deep atoms. The sum is the same
 *           function of the logical operands in both layouts; the hardware
 *           step stays 32 K values deep.
 *   kernel  a bmm_kernel value.
 *   scaled  0: the C-then-D recurrence of bmm_mma_tile; 1: the alpha/beta
 *           form of bmm_mma_tile_scaled with these alpha and beta (ignored
 *           when scaled = 0).
 * opts = NULL means {16, BMM_KERNEL_AUTO, 0, 1, 1}, i.e. bmm_mma_tile.
 * D, A, B, C, c_scalar, extents, dtype: as bmm_mma_tile.
 * Errors: as bmm_mma_tile_with; BMM_EINVAL also for atom_k not 16 or 8 and
 * scaled not 0 or 1.
 */
typedef struct {
  int32_t atom_k;
  int32_t kernel;
  int32_t scaled;
  float alpha;
  float beta;
} bmm_mma_opts;

int bmm_mma_tile_opts(float* D, const uint32_t* A, const uint32_t* B, const float* C,
                      float c_scalar, int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep,
                      bmm_dtype dtype, const bmm_mma_opts* opts, void* stream);

/*
 * bmm_mma_tile_splitk — the multiply-accumulate with K split across workgroups.
 *
 * For shapes with few output tiles and a long K. The K axis is cut at
 * multiples of 32 values into S = min(splits, ceil(K / 32)) balanced ranges
 * of whole 32-value steps: split s takes steps [s*n/S, (s+1)*n/S) of the
 * n = ceil(K / 32). Each split's partial sum P_s starts from zero; then the
 * partial sums are add-reduced into a destination that starts at C (the
 * cp.async.bulk.tensor page, "Stores, reductions, and completion": the
 * reduction destination is initialised to the intended starting value):
 *
 *   D = (((C + P_0) + P_1) + ...) + P_{S-1}      (fp32, in this order)
 *
 * so the result is the same on every run and for every schedule. K = 0
 * gives D = C.
 * D, A, B, C, c_scalar, extents, dtype: as bmm_mma_tile (in place D == C
 * allowed); atom_k 16 or 8 as in bmm_mma_tile_opts; K < 2^22 values.
 * splits     1..65535 (bmm_splitk_default suggests one).
 * workspace  device memory of at least bmm_mma_splitk_workspace_bytes(...)
 *            bytes (S * batch * M_rep * N_rep * 512), 16-byte aligned, not
 *            overlapping D, A, B or C; owned by the caller, clobbered.
 * Errors: as bmm_mma_tile_with; BMM_EINVAL also for splits, K and a missing
 * or short workspace, BMM_EOVERLAP for an overlapping workspace.
 */
int bmm_mma_tile_splitk(float* D, const uint32_t* A, const uint32_t* B, const float* C,
                        float c_scalar, int64_t batch, int64_t M_rep, int64_t N_rep,
                        int64_t K_rep, bmm_dtype dtype, int32_t atom_k, int32_t splits,
                        float* workspace, int64_t workspace_bytes, void* stream);

/*
 * bmm_mma_tile_splitk_noalloc — bmm_mma_tile_splitk without a workspace, for
 * callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc. It calls no
 * allocating routine.
 *
 * The partial sums go to a static device array of BMM_NOALLOC_SCRATCH_BYTES
 * (64 MiB) per device, set up on the first call on that device (the device
 * of `stream`; the current device for the null stream) and held until the
 * process ends. Same arguments, arithmetic, bits and errors as bmm_mma_tile_splitk,
 * minus the workspace; a request whose partial sums
 * (bmm_mma_splitk_workspace_bytes) exceed the array returns BMM_ERANGE and
 * launches nothing. Every call on one device shares that device's array, so
 * calls that overlap on one device (other streams, other threads) race and
 * must be serialised by the caller. Nothing in the array needs clearing: each
 * split writes its whole partial sum before the reduce reads it.
 */
#define BMM_NOALLOC_SCRATCH_BYTES (64LL << 20)
int bmm_mma_tile_splitk_noalloc(float* D, const uint32_t* A, const uint32_t* B, const float* C,
                                float c_scalar, int64_t batch, int64_t M_rep, int64_t N_rep,
                                int64_t K_rep, bmm_dtype dtype, int32_t atom_k, int32_t splits,
                                void* stream);

/* Workspace bytes bmm_mma_tile_splitk needs (0 when K = 0), or < 0. */
int64_t bmm_mma_splitk_workspace_bytes(int64_t batch, int64_t M_rep, int64_t N_rep,
                                       int64_t K_rep, int32_t atom_k, int32_t splits);

/* A split count for bmm_mma_tile_splitk: enough tiles x splits for every CU,
 * each split at least 1024 K values deep, at most 32; 1 when splitting does
 * not pay. (The split-K form uses 256 x 256 tiles when there are at least
 * 128 of them, or from K = 16384 values when there are at least 8 of them,
 * and 128 x 128 tiles otherwise.) */
int bmm_splitk_default(int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep,
                       int32_t atom_k);

/* Whether to call bmm_mma_tile_splitk instead of bmm_mma_tile for this
 * shape: the split count to use when the split-K form is expected to be the
 * faster of the two (shapes with few output tiles and a long K, e.g.
 * 1024 x 1024 x 65536: 123 against 335 us on MI355X), 1 when the plain entry
 * point is expected to be at least as fast, or < 0 for invalid extents. The
 * plain entry point never splits K itself, since it takes no workspace. */
int bmm_splitk_suggested(int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep,
                         int32_t atom_k);

/* Which kernel AUTO would run for this shape (K_rep in 16-deep atoms; a
 * bmm_kernel value), or < 0. */
int bmm_select_kernel(int64_t batch, int64_t M_rep, int64_t N_rep, int64_t K_rep);

/*
 * ---- Feed-forward operators ----
 *
 * Activations and gradients are row-major matrices of 16-bit values (f16 or
 * bf16 bits, named by dtype): (batch, rows, ld) with `ld` elements between
 * rows and rows * ld between batches, ld a multiple of 8, base 16-byte
 * aligned. Any number of rows is taken. Weights are packed B operands as
 * bmm_pack_operand (atom_rows 8) lays them out, or 4-bit operands.
 */

/* Activations. GELU is x Phi(x); GELU_TANH is 0.5 x (1 + tanh(sqrt(2 / pi)
 * (x + 0.044715 x^3))). */
typedef enum {
  BMM_ACT_SILU = 0,
  BMM_ACT_GELU = 1,
  BMM_ACT_GELU_TANH = 2,
  BMM_ACT_RELU = 3
} bmm_act;

/*
 * Extents of a gated feed-forward block.
 *   batch  independent blocks (each with its own weights)
 *   M      rows of X (tokens); any
 *   F      width of the block, a multiple of 8, at most 2^20
 *   K      width of X, a multiple of 16, at most 2^21
 *   ld_x   elements between rows of X: >= K, a multiple of 8, at most 2^21
 *   ld_h   elements between rows of H, G, U and dH: >= F, a multiple of 8, at
 *          most 2^21
 *   dtype  bmm_dtype of every 16-bit value
 *   act    bmm_act
 */
typedef struct {
  int64_t batch;
  int64_t M;
  int64_t F;
  int64_t K;
  int64_t ld_x;
  int64_t ld_h;
  int32_t dtype;
  int32_t act;
} bmm_gated_desc;

/*
 * bmm_gated — H = act(G) * U with G = X Wg^T and U = X Wu^T, in one kernel.
 *
 * H      (batch, M, ld_h) written in the first F columns of each row.
 * G, U   as H, or both NULL. When given they receive the projections, rounded
 *        to dtype, which bmm_gated_backward takes; H is made from the
 *        unrounded float32 projections either way.
 * X      (batch, M, ld_x), the first K columns of each row are read.
 * Wg, Wu (batch, F/8, K/16, 8, 8) packed words (bmm_pack_operand, atom_rows 8).
 * The sums are float32; H, G and U are rounded once (nearest even). K = 0
 * gives H = act(0) * 0 = 0. Zero batch, M or F is a no-op.
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP (outputs with each other or
 * with an input; interleaved rows of one buffer are no overlap), BMM_EHIP.
 */
int bmm_gated(uint16_t* H, uint16_t* G, uint16_t* U, const uint16_t* X, const uint32_t* Wg,
              const uint32_t* Wu, const bmm_gated_desc* desc, void* stream);

/*
 * bmm_gated_backward — gradients of bmm_gated from dH and the kept projections.
 *
 *   dG = dH * U * act'(G), dU = dH * act(G)   (relu'(x) = 1 for x > 0, else 0)
 *   dX = dG Wg + dU Wu;  dWg = dG^T X;  dWu = dU^T X
 *
 * dX         (batch, M, K) contiguous, or NULL when it is not wanted.
 * dWg, dWu   (batch, F, K) contiguous and row-major, or both NULL. (M = 0
 *            writes zeros, the empty sum; F = 0 does so for dX.)
 * dH, G, U   (batch, M, ld_h); X (batch, M, ld_x); Wg, Wu as bmm_gated (may be
 *            NULL when dX is).
 * dG and dU are rounded to dtype before they are multiplied; sums are
 * float32, each gradient is rounded once. For f16, dG and dU are held times a
 * power of two that brings the largest finite magnitude of the call to [2^14,
 * 2^15), and the sums are divided by it: values down to 2^-28 of the largest
 * keep f16's 11 digits, those below 2^-39 of it count as zero, and no finite
 * value overflows before a gradient's own rounding does. The result is the
 * same on every run.
 * workspace  device memory of at least bmm_gated_backward_workspace_bytes(desc)
 *            bytes, 16-byte aligned, overlapping nothing else; owned by the
 *            caller, clobbered.
 * Errors: as bmm_gated; BMM_EINVAL also for a missing or short workspace and
 * when nothing is wanted.
 */
int bmm_gated_backward(uint16_t* dX, uint16_t* dWg, uint16_t* dWu, const uint16_t* dH,
                       const uint16_t* G, const uint16_t* U, const uint16_t* X,
                       const uint32_t* Wg, const uint32_t* Wu, const bmm_gated_desc* desc,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes bmm_gated_backward needs for these extents, or < 0. */
int64_t bmm_gated_backward_workspace_bytes(const bmm_gated_desc* desc);

/*
 * 4-bit operands: microscaled floats (OCP Microscaling Formats v1.0, MXFP4).
 *
 * 32 neighbouring K values of a row share a scale 2^(byte - 127) (byte 255:
 * NaN, the whole block stands for NaN); a value's code is a sign bit and an
 * index into {0, 0.5, 1, 1.5, 2, 3, 4, 6}.
 *
 * codes   (batch, ceil(rows/16), ceil(K/128), 4, 16, 16) bytes:
 *         [b, r, s, g, i, j] holds row 16 r + i, K values 128 s + 32 g + 2 j
 *         (low half) and 128 s + 32 g + 2 j + 1 (high half).
 * scales  (batch, ceil(rows/16), ceil(K/512), 4, 16, 4) bytes:
 *         [b, r, q, g, i, t] scales row 16 r + i, K values
 *         512 q + 128 t + 32 g .. + 31.
 * Both contiguous, codes and scales 16-byte aligned. Codes and scales of rows
 * and K values outside the matrix are zero. The same layout serves as A and
 * as B. K is a multiple of 32, below 2^22.
 */
int64_t bmm_mx4_codes_bytes(int64_t batch, int64_t rows, int64_t K);
int64_t bmm_mx4_scales_bytes(int64_t batch, int64_t rows, int64_t K);

/*
 * bmm_mx4_quantize — a row-major matrix to a 4-bit operand.
 *
 * Per block: e = floor(log2(largest magnitude)) - 2, at least -127; the scale
 * byte is e + 127 and each code is x / 2^e rounded to the nearest value, ties
 * to the even code, at most 6 in magnitude. A block with a NaN or an infinity
 * gets scale byte 255; a block of zeros gets scale byte 0.
 * src  (batch, rows, ld_src) values of elem_type (BMM_ELEM_F32, _F16 or
 *      _BF16), batch stride rows * ld_src, 16-byte aligned; ld_src >= K and a
 *      multiple of 8. Padding of codes and scales is written too.
 * Zero batch, rows or K is a no-op.
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP, BMM_EHIP.
 */
int bmm_mx4_quantize(uint8_t* codes, uint8_t* scales, const void* src, int64_t batch, int64_t rows,
                     int64_t K, int64_t ld_src, int32_t elem_type, void* stream);

/* bmm_mx4_dequantize — the values of a 4-bit operand, rounded to elem_type
 * (exact but for f16's range and values below the type's smallest). dst as
 * src above; columns from K on are not written. */
int bmm_mx4_dequantize(void* dst, const uint8_t* codes, const uint8_t* scales, int64_t batch,
                       int64_t rows, int64_t K, int64_t ld_dst, int32_t elem_type, void* stream);

/*
 * bmm_mx4_mma — D = A * B^T over 4-bit operands.
 *
 * D  (batch, M, ld_d) of elem_type (BMM_ELEM_F32, _F16 or _BF16), written in
 *    the first N columns; ld_d >= N, a multiple of 8, at most 2^21; 16-byte
 *    aligned.
 * A  4-bit operand of M rows, B of N rows, both of K values; N a multiple of 8.
 * Sums are float32, rounded once. K = 0 gives zeros; zero batch, M or N is a
 * no-op.
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP, BMM_EHIP.
 */
int bmm_mx4_mma(void* D, const uint8_t* A_codes, const uint8_t* A_scales, const uint8_t* B_codes,
                const uint8_t* B_scales, int64_t batch, int64_t M, int64_t N, int64_t K,
                int64_t ld_d, int32_t elem_type, void* stream);

/*
 * bmm_mx4_gated — H = act(X Wg^T) * (X Wu^T) over 4-bit operands.
 *
 * H  (batch, M, ld_h) of elem_type BMM_ELEM_F16 or BMM_ELEM_BF16, written in
 *    the first F columns; X of M rows, Wg and Wu of F rows, all of K values; F
 *    a multiple of 8. Otherwise as bmm_mx4_mma.
 */
int bmm_mx4_gated(void* H, const uint8_t* X_codes, const uint8_t* X_scales,
                  const uint8_t* Wg_codes, const uint8_t* Wg_scales, const uint8_t* Wu_codes,
                  const uint8_t* Wu_scales, int64_t batch, int64_t M, int64_t F, int64_t K,
                  int64_t ld_h, int32_t act, int32_t elem_type, void* stream);

/*
 * bmm_ffn_plan — how the product of these extents is made (diagnostics and
 * tests): a bmm_ffn_tile, or < 0. *splits (may be NULL) receives the number of
 * parts that its sum is cut into. F is the columns of D for BMM_FFN_MX4_MMA.
 * The rows of dX may be made in two launches; BMM_FFN_GATED_DX is the first.
 * BMM_TILE_NONE: there is nothing to make, or no second launch.
 */
typedef enum {
  BMM_FFN_GATED = 0,
  BMM_FFN_GATED_DX = 1,
  BMM_FFN_GATED_DX_REST = 2,
  BMM_FFN_GATED_DW = 3,
  BMM_FFN_MX4_MMA = 4,
  BMM_FFN_MX4_GATED = 5
} bmm_ffn_product;

/* Rows x columns of a tile (gated: columns of both weights together). */
typedef enum {
  BMM_TILE_128X128 = 0,
  BMM_TILE_256X128 = 1,
  BMM_TILE_256X192 = 2,
  BMM_TILE_256X256 = 3,
  BMM_TILE_FEW_ROWS = 4, /* up to 64 rows: the weights are read once */
  BMM_TILE_NONE = 5
} bmm_ffn_tile;

int bmm_ffn_plan(int32_t product, int64_t batch, int64_t M, int64_t F, int64_t K,
                 int32_t* splits);

/*
 * ---- Products by groups of rows (the experts of a mixture) ----
 *
 * T rows lie sorted by group (by expert): group e of `groups` has the rows from
 * ends[e - 1] up to ends[e], group 0 from 0, any number of them, also none. Rows
 * from ends[groups - 1] on belong to no group (a batch padded to a fixed size):
 * they are not read, and their outputs become zero with zero_tail and stay as
 * they are without. ends is device memory and is read by the kernels only, so a
 * captured graph takes other groups on every replay. Ends are held to 0 .. T and
 * to be no smaller than the ones before: other values count as the nearest such
 * ones, and nothing outside of the matrices is touched.
 *
 * Extents of a product by groups.
 *   groups     1 .. 4096
 *   T          rows in all, below 2^31
 *   N          width of the outputs (of the gated block), a multiple of 8, at
 *              most 2^20
 *   K          width of X, a multiple of 16, at most 2^21
 *   ld_x       elements between rows of X: >= K, a multiple of 8, at most 2^21
 *   ld_y       elements between rows of Y and dY (H, G, U and dH): >= N, a
 *              multiple of 8, at most 2^21
 *   dtype      bmm_dtype of every 16-bit value
 *   act        bmm_act of the gated block (0 otherwise)
 *   zero_tail  1: outputs of rows behind the last group become zero; 0: stay
 */
typedef struct {
  int64_t groups;
  int64_t T;
  int64_t N;
  int64_t K;
  int64_t ld_x;
  int64_t ld_y;
  int32_t dtype;
  int32_t act;
  int32_t zero_tail;
} bmm_grouped_desc;

/*
 * bmm_grouped_mma — Y = X W_e^T for the rows of each group e, in one kernel.
 *
 * Y    (T, ld_y), written in the first N columns of each row.
 * X    (T, ld_x), the first K columns of each row are read.
 * W    (groups, N/8, K/16, 8, 8) packed words (bmm_pack_operand, atom_rows 8).
 * ends (groups) int32, as above.
 * The sums are float32, rounded once. K = 0 gives zeros; T = 0 or N = 0 is a
 * no-op.
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP (an output with an input or with
 * another output; interleaved rows of one buffer are no overlap), BMM_EHIP.
 */
int bmm_grouped_mma(uint16_t* Y, const uint16_t* X, const uint32_t* W, const int32_t* ends,
                    const bmm_grouped_desc* desc, void* stream);

/*
 * bmm_grouped_mma_backward — gradients of bmm_grouped_mma from dY.
 *
 *   dX = dY W_e for the rows of each group;  dW_e = dY^T X over group e's rows
 *
 * dX   (T, K) contiguous, or NULL when it is not wanted.
 * dW   (groups, N, K) contiguous and row-major, or NULL. A group without rows
 *      gets zeros. (One that is empty, dX for T = 0 or dW for N = 0, is NULL also
 *      where it is wanted.)
 * dY   (T, ld_y); X (T, ld_x); W may be NULL when dX is, X when dW is.
 * Sums are float32, rounded once; the result is the same on every run.
 * workspace  device memory of at least bmm_grouped_mma_backward_workspace_bytes
 *            bytes, 16-byte aligned, overlapping nothing else; owned by the
 *            caller, clobbered.
 * Errors: as bmm_grouped_mma; BMM_EINVAL also for a missing or short workspace
 * and when nothing is wanted.
 */
int bmm_grouped_mma_backward(uint16_t* dX, uint16_t* dW, const uint16_t* dY, const uint16_t* X,
                             const uint32_t* W, const int32_t* ends, const bmm_grouped_desc* desc,
                             void* workspace, int64_t workspace_bytes, void* stream);
int64_t bmm_grouped_mma_backward_workspace_bytes(const bmm_grouped_desc* desc);

/*
 * bmm_grouped_gated — H = act(X Wg_e^T) * (X Wu_e^T) for the rows of each group
 * e, in one kernel: bmm_gated with weights of each group.
 *
 * H, G, U as Y of bmm_grouped_mma; G and U both or neither. Wg, Wu as its W.
 */
int bmm_grouped_gated(uint16_t* H, uint16_t* G, uint16_t* U, const uint16_t* X, const uint32_t* Wg,
                      const uint32_t* Wu, const int32_t* ends, const bmm_grouped_desc* desc,
                      void* stream);

/*
 * bmm_grouped_gated_backward — gradients of bmm_grouped_gated from dH and the
 * kept projections: bmm_gated_backward with the weights and weight gradients of
 * each group (dWg, dWu: (groups, N, K), zeros for a group without rows). For f16
 * the largest magnitude that scales dG and dU is that of the call, of all groups.
 */
int bmm_grouped_gated_backward(uint16_t* dX, uint16_t* dWg, uint16_t* dWu, const uint16_t* dH,
                               const uint16_t* G, const uint16_t* U, const uint16_t* X,
                               const uint32_t* Wg, const uint32_t* Wu, const int32_t* ends,
                               const bmm_grouped_desc* desc, void* workspace,
                               int64_t workspace_bytes, void* stream);
int64_t bmm_grouped_gated_backward_workspace_bytes(const bmm_grouped_desc* desc);

/*
 * ---- 8-bit integers ----
 *
 * A row is K codes from -127 to 127 and a float32 scale; code times scale is the
 * value. Activations are row-major codes. Weights are packed B operands of their
 * codes, two neighbouring ones taken as a 16-bit value: bmm_pack_operand of the
 * (rows, K/2) 16-bit matrix that the codes are, atom_rows 8, so (batch, N/8, K/32,
 * 8, 8) words.
 *
 * bmm_i8_quantize — a row-major matrix to codes (batch, rows, K), contiguous, and
 * scales (batch, rows).
 *
 * scale = max |x| / 127 over the row, in float32; code = 127 x / max |x|, the real
 * quotient rounded to nearest, ties to even. A row of zeros gets scale 0 and codes
 * 0; one with a NaN or an infinity scale NaN and codes 0.
 * src  (batch, rows, ld_src) values of elem_type (BMM_ELEM_F32, _F16 or _BF16),
 *      batch stride rows * ld_src, 16-byte aligned; ld_src >= K and a multiple of
 *      8; K a multiple of 32, below 2^22. Zero batch or rows is a no-op; K = 0
 *      writes zero scales.
 * Errors: BMM_EINVAL, BMM_EALIGN, BMM_EOVERLAP, BMM_EHIP.
 */
int bmm_i8_quantize(int8_t* codes, float* scales, const void* src, int64_t batch, int64_t rows,
                    int64_t K, int64_t ld_src, int32_t elem_type, void* stream);

/*
 * Extents of a product of 8-bit integers.
 *   batch      independent products; with ends: the groups, 1 .. 4096
 *   M          rows of A (with ends: in all, below 2^31)
 *   N          columns of D, a multiple of 8, at most 2^20
 *   K          codes of a row, a multiple of 32, below 2^17 (sums of 128 * 128 K
 *              stay below 2^31)
 *   ld_a       codes between rows of A: >= K, a multiple of 16, at most 2^22
 *   ld_d       elements between rows of D: >= N, a multiple of 8, at most 2^21
 *   elem_type  of D: BMM_ELEM_F32, _F16 or _BF16 (gated: _F16 or _BF16)
 *   act        bmm_act of the gated block (0 otherwise)
 *   zero_tail  with ends, as in bmm_grouped_desc
 * More tiles than one launch may have (2^24 workgroups: without ends, batch * M from
 * about 2^32 on) are refused with BMM_EHIP.
 */
typedef struct {
  int64_t batch;
  int64_t M;
  int64_t N;
  int64_t K;
  int64_t ld_a;
  int64_t ld_d;
  int32_t elem_type;
  int32_t act;
  int32_t zero_tail;
} bmm_i8_desc;

/*
 * bmm_i8_mma — D[m][n] = A_scales[m] B_scales[n] (sum over k of A[m][k] B[n][k]).
 *
 * D         (batch, M, ld_d), with ends (M, ld_d), of elem_type.
 * A         (batch, M, ld_a) codes, batch stride M * ld_a; A_scales (batch, M).
 * B         (batch, N/8, K/32, 8, 8) packed words; B_scales (batch, N).
 * ends      NULL, or (batch) int32: the groups of A's rows, as bmm_grouped_mma;
 *           A is then (M, ld_a) and A_scales (M).
 * The sums are exact; they are rounded to float32, multiplied by the row's scale
 * and then by the column's, and rounded to elem_type. K = 0 gives zeros (NaN where
 * a scale is no finite number); zero batch (without ends), M or N is a no-op.
 * Errors: BMM_EINVAL, BMM_EALIGN (16 bytes; A_scales 4), BMM_EOVERLAP, BMM_EHIP.
 */
int bmm_i8_mma(void* D, const int8_t* A, const float* A_scales, const uint32_t* B,
               const float* B_scales, const int32_t* ends, const bmm_i8_desc* desc, void* stream);

/* bmm_i8_gated — H = act(X Wg^T) * (X Wu^T) over 8-bit integers, the projections
 * as bmm_i8_mma gives them in float32. */
int bmm_i8_gated(void* H, const int8_t* X, const float* X_scales, const uint32_t* Wg,
                 const float* Wg_scales, const uint32_t* Wu, const float* Wu_scales,
                 const int32_t* ends, const bmm_i8_desc* desc, void* stream);

/*
 * bmm_group_plan — as bmm_ffn_plan, for the products by groups (T rows in all) and
 * of 8-bit integers (groups 0: one weight, no groups). N is the width F of a gated
 * block.
 */
typedef enum {
  BMM_GROUPED_MMA = 0,
  BMM_GROUPED_MMA_DX = 1,
  BMM_GROUPED_MMA_DW = 2,
  BMM_GROUPED_GATED = 3,
  BMM_GROUPED_GATED_DX = 4,
  BMM_GROUPED_GATED_DW = 5,
  BMM_I8_MMA = 6,
  BMM_I8_GATED = 7
} bmm_group_product;

int bmm_group_plan(int32_t product, int64_t groups, int64_t T, int64_t N, int64_t K,
                   int32_t* splits);

/* Message for the last failed call on this thread ("" if none). */
const char* bmm_last_error(void);

/* ABI version: 1. */
int bmm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BMM_H */
