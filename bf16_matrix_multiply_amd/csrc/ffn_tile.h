// The MFMA tile kernel of the feed-forward operators: D = A * B^T with the
// operands read where they lie, and the operator's own epilogue.
//
// A product here is one of
//   H  = act(X Wg^T) * (X Wu^T)      A rows,       B packed, two sources   gated
//   dX = [dG | dU] [Wg ; Wu]         A rows,       B packed, transposed    store
//   dW = [dG | dU]^T X               A transposed, B transposed            store
//   D  = A B^T, 4-bit                A, B 4-bit                            store
//   H  = act(..) * (..), 4-bit       A, B 4-bit, two sources               gated
//   Y  = X W^T                       A rows,       B packed                store
// The first, the last and the two sums of the second and third also by groups
// (ffn_groups.h): tiles of a group's rows with the group's own B, or for dW sums
// over a group's rows. The first and the last also with 8-bit integers, two of
// which take the place of a 16-bit value everywhere but in the MFMA (16x16x64).
//
// "rows": row-major, the summed axis contiguous. "transposed": row-major with
// the summed axis across rows (the matrix enters as its transpose). "packed":
// atoms of 8 rows x 16 summed values (bmm_pack_operand, atom_rows 8).
//
// A workgroup of 4 waves in a 2 x 2 grid makes a TM x TN tile. The sum advances
// in slabs of 64 bytes a row: 32 16-bit values, or 128 4-bit values. One MFMA
// (16x16x32, or the scaled 16x16x128 for 4 bits) multiplies a 16-row fragment
// of B (first operand) and one of A (second) over a slab, so lane l holds
// D[m = l % 16][n = 4 (l / 16) .. + 3] of the 16 x 16 block: four neighbouring
// columns. Lane l supplies row l % 16 and the 16 bytes of summed chunk l / 16.
//
// Staging: every wave moves 1 KB pieces from memory to LDS with direct loads
// (lane l's 16 bytes land at 16 l). The lanes' source addresses arrange the
// piece, so that 16 neighbouring lanes ask for whole 128-byte lines (a line
// asked for by halves costs the cache two requests: with 64 bytes of a row in
// a piece the gated block took 800 us for 8192 x 4096 -> 8192, and a half more
// line requests), and so that the reads that follow are spread over all banks.
// A ds_read_b128 serves 16 lanes a cycle, of lanes 0-31 first 0-3, 12-15 and
// 20-27, then the others; a ds_read_b64 lanes 0-31, then 32-63. No conflicts
// are counted for any of these:
// - 4-bit: the piece is a fragment in lane order;
// - packed: the piece is two atom rows of 512 bytes as they are;
// - rows: 8 rows x 128 bytes, two slabs at once; the 16-byte chunk c of row r
//   lies at chunk c ^ rows_swizzle(r);
// - transposed: [64-column block][32 summed rows][128 bytes], read with the
//   hardware's transposing LDS read (ds_read_b64_tr_b16: of 16 lanes, lane
//   4 k + a reads four columns 4a .. 4a + 3 of summed row k, and lane i
//   receives column i of the four rows). Pairs of 16-byte chunks of summed row
//   k are exchanged by k's bits 1 and 3;
// - transposed packed: the piece is four atoms (8 summed rows x 64 columns) as
//   they are, with the two 128-byte halves of an atom exchanged for every other
//   8 summed rows; read as above.
// What lies outside the matrices is read as zero: such lanes are given an
// address past the buffer's end, so no memory is touched.
//
// Schedule: a ring of four stages. Slab s is multiplied from registers while
// the wave reads the fragments of slab s + 1 from LDS into its second register
// set and sends the loads of slab s + 4 into the stage whose fragments it holds;
// reads and loads are placed between the MFMAs, and one barrier a slab, after
// its first two MFMAs, publishes the loads that every wave waited for at the end
// of the slab before. The loop runs whole turns of the ring: slabs past the end
// read as zeros.
//
// Measured on MI355X, 8192 x 4096 -> 8192 bf16: gated 746-781 us = 1408-1474 TFLOP/s
// from box to box (the library's plain 8192^3 product, as many operations, 663-707
// us), of which 680 us are the slab loops; dX and dW of its backward pass 760-790 us
// each; 8192^3 with 4-bit operands 237 us = 4.6 PFLOP/s. Bound by the matrix cores
// at the clock that the power limit leaves (bf16, 1.7-1.8 GHz), and by the LDS, whose
// reads and loads leave bubbles between the MFMAs of the one wave that a SIMD has
// room for (4 bits: without them 169 us). Tried and slower or no faster: reads and loads in bursts
// (820 -> 1000-1500 us), workgroups that go on to the next tile, a copy of the loop
// for each wave with its reads and loads shifted, one barrier for two slabs, and
// for 4 bits 32 x 32 x 64 MFMAs.
//
// By groups: 16384 rows of 8 groups, 8192 -> 4096 bf16, 847-895 us (as many operations
// as the product of 8192^3; MFMA utilisation 0.66 at 1.5-1.6 GHz), of which a last
// round of a few small tiles, with the whole sum each, takes 67 (groups of whole tiles:
// 826); dX of 16384 rows of 16 groups, 2048 -> 4096 gated, 500-527 us, of which that
// round 85 (440); its weight gradients 535-580 us (0.47 at 2.0 GHz: results of 537 MB
// from sums of 32 slabs); 24576 rows of 64 groups, 2048 -> 1408 gated with projections
// kept, f16, 350 us (0.44 at 1.9 GHz: each group's weight comes from memory for the few
// tiles that share it; with one weight for all of them 296). 8192^3 with 8-bit integers
// 375-385 us = 2.9 PTOP/s (0.70 at 1.9 GHz).
// What writes the results faster in a probe, four lanes side by side on 64 bytes of a row,
// did not pay by groups: with the lanes' results turned in registers for it, the weight
// gradients of 24576 rows of 64 groups, 2048 x 1408, took 213 us instead of 219, those with
// fewer rows 2% longer.
#pragma once

#include <type_traits>

#include "ffn.h"
#include "ffn_groups.h"

namespace bmm {
namespace ffn {

enum Src : int { kRows, kTrans, kPacked, kPacked2, kPackedT2, kCodes, kCodes2 };
enum Epi : int { kStore, kGated };
// By groups: of the rows of A and D, or of the summed rows of A and B.
enum Grouped : int { kWhole, kGroupRows, kGroupSums };

constexpr uint32_t kXcds = 8;
// M tiles in a band: an XCD works on 4 x 8 tiles at a time, whose 12 panels share
// its L2. Gated 8192 x 4096 -> 8192: 4 746 us, 8 756, 16 763, 32 799.
constexpr uint32_t kGroupM = 4;
constexpr int kTileWaves = 4;
constexpr int kBufferFlags = 0x00020000;           // raw, untyped buffer
constexpr uint32_t kOutOfRange = 0x7fffffffu;      // an offset past every buffer's end

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) void lds_void;

constexpr bool two_sources(int src) { return src == kPacked2 || src == kCodes2; }
constexpr bool four_bit(int src) { return src == kCodes || src == kCodes2; }
// Summed values a slab.
constexpr int slab_values(int src) { return four_bit(src) ? 128 : 32; }

// s_waitcnt immediate: vmcnt in bits [3:0] and [15:14], expcnt [6:4], lgkmcnt [11:8].
constexpr int waitcnt_imm(int vm, int lgkm) {
  return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}

// f(integral_constant i) for i in [A, B).
template <int A, int B, class Fn>
__device__ __forceinline__ void static_for(Fn fn) {
  if constexpr (A < B) {
    fn(std::integral_constant<int, A>{});
    static_for<A + 1, B>(fn);
  }
}

// Which of n items that are spread over `span` places (at the start of their
// shares, or with `middle` in the middle) falls on this place; -1: none.
constexpr int item_at(int place, int n, int middle, int span) {
  for (int i = 0; i < n; ++i)
    if ((2 * i + middle) * span / (2 * n) == place) return i;
  return -1;
}

struct TileAt {
  int64_t b, mt, nt;
};

// Linear workgroup id -> work index, each XCD taking a contiguous run. (All of
// these fit 32 bits; 64-bit divisions took about 1 us of every workgroup.)
__device__ __forceinline__ uint32_t xcd_run(uint32_t w, uint32_t n) {
  const uint32_t q = n / kXcds, r = n % kXcds;
  const uint32_t xcd = w % kXcds, k = w / kXcds;
  return xcd * q + (xcd < r ? xcd : r) + k;
}

// Linear tile index -> (batch, M tile, N tile), in bands of kGroupM M tiles.
__device__ __forceinline__ TileAt tile_at(uint32_t t, uint32_t MT, uint32_t NT, bool batched) {
  uint32_t b = 0;
  if (batched) {
    b = t / (MT * NT);
    t -= b * (MT * NT);
  }
  const uint32_t group = kGroupM * NT, first = t / group, first_m = first * kGroupM;
  const uint32_t gm = MT - first_m < kGroupM ? MT - first_m : kGroupM;
  const uint32_t v = t - first * group;
  return {b, first_m + v % gm, v / gm};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t bytes = kOutOfRange) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(bytes), kBufferFlags);
}

// The exchange of 16-byte chunks in the row-major image: by r / 2: 0, 2, 0, 2, 4, 6, 4, 6.
__device__ __forceinline__ int rows_swizzle(int r) { return (r & 2) | ((r >> 1) & 4); }

// Bits 1 and 3 of a summed row's index within its slab: the exchange of chunk
// pairs of the transposed image.
__device__ __forceinline__ int trans_swizzle(int k) { return ((k >> 1) & 1) | ((k >> 2) & 2); }

// Slabs that one round of an operand's loads brings.
constexpr int slabs_a_load(int src) { return src == kRows ? 2 : 1; }

// The loads of one operand: 1 KB piece 4 r + wave of T / 16 (rows: of T / 8).
template <int SRC, int T>
struct Loader {
  static constexpr int kSlabs = slabs_a_load(SRC), kLoads = T / 64 * kSlabs;
  const char* base0;       // slab 0, source 0 (or this wave's source)
  const char* base1;       // kPackedT2: slab 0 of source 1
  int64_t step;            // bytes from one round to the next
  int64_t end;             // summed values to take (kPackedT2: slabs)
  int64_t per;             // kPackedT2: slabs of one source
  int64_t n_rows;          // kPackedT2: summed values that exist in one source
  int k_lane;              // this lane's first summed value within a round
  uint32_t off[4];         // fixed size: T / 64 are used (rows: one)
  uint32_t bytes;          // rows: size of the buffer, past which no row exists
  uint32_t piece;          // rows: bytes from a piece to this wave's next one

  // r0: first row (column of D for B) of the tile; n: rows that exist; slab_end:
  // slabs from there on read as zeros.
  __device__ __forceinline__ void init(const TileArgs& p, const void* s0, const void* s1,
                                       int64_t batch_off, int64_t ld, int64_t r0, int64_t n,
                                       int64_t slab_end, int lane, int wave) {
    end = slab_end * slab_values(SRC) < p.K ? slab_end * slab_values(SRC) : p.K;
    per = n_rows = 0;
    base1 = nullptr;
    bytes = kOutOfRange;
    piece = 0;
    if constexpr (SRC == kRows) {
      const int row = 8 * wave + (lane >> 3), c = (lane & 7) ^ rows_swizzle(row & 15);
      k_lane = 8 * c;
      step = 128;
      base0 = static_cast<const char*>(s0) + 2 * (batch_off + r0 * ld);
      off[0] = uint32_t(row * ld * 2 + 16 * c);
      piece = uint32_t(64 * ld);
      bytes = uint32_t((n - r0 < T ? n - r0 : T) * ld * 2);   // ld <= 2^21: at most 2^30
    } else if constexpr (SRC == kTrans) {
      k_lane = 8 * wave + (lane >> 3);
      const int e = (lane & 7) ^ (2 * trans_swizzle(k_lane));
      step = 64 * ld;
      base0 = static_cast<const char*>(s0) + 2 * (batch_off + r0);
#pragma unroll
      for (int r = 0; r < T / 64; ++r)
        off[r] = r0 + 64 * r + 8 * e < n ? uint32_t(k_lane * ld * 2 + 128 * r + 16 * e)
                                         : kOutOfRange;
    } else if constexpr (SRC == kPackedT2) {
      // one atom row of 8 summed values a wave; n columns make n / 16 atoms in it
      const int x = lane ^ (8 * (wave & 1));
      k_lane = 8 * wave + ((x & 15) >> 1);
      step = 64 * n;
      end = slab_end;
      per = p.b_sum / 32;
      n_rows = p.b_rows;
      base0 = static_cast<const char*>(s0) + 2 * batch_off + 16 * r0;
      base1 = static_cast<const char*>(s1) + 2 * batch_off + 16 * r0;
#pragma unroll
      for (int r = 0; r < T / 64; ++r)
        off[r] = r0 + 64 * r + 16 * (lane >> 4) < n ? uint32_t(wave * n * 16 + 1024 * r + 16 * x)
                                                    : kOutOfRange;
    } else if constexpr (SRC == kPacked || SRC == kPacked2) {
      k_lane = (lane & 16) + 8 * (lane & 1);
      step = 512;
      base0 = static_cast<const char*>(SRC == kPacked2 && (wave & 1) ? s1 : s0) +
              2 * (batch_off + r0 * p.K);
#pragma unroll
      for (int r = 0; r < T / 64; ++r) {
        const int piece = SRC == kPacked2 ? 2 * r + (wave >> 1) : 4 * r + wave;
        const int half = 2 * piece + (lane >> 5);   // 8-column atom row
        off[r] = r0 + 8 * half < n ? uint32_t(half * p.K * 16 + 16 * (lane & 31)) : kOutOfRange;
      }
    } else {
      const int64_t row_bytes = (p.K + 127) / 128 * 1024;   // a group of 16 rows
      k_lane = 32 * (lane >> 4);
      step = 1024;
      base0 = static_cast<const char*>(SRC == kCodes2 && (wave & 1) ? s1 : s0) + batch_off +
              r0 / 16 * row_bytes;
#pragma unroll
      for (int r = 0; r < T / 64; ++r) {
        const int cb = SRC == kCodes2 ? 2 * r + (wave >> 1) : 4 * r + wave;
        off[r] = r0 + 16 * cb < n ? uint32_t(cb * row_bytes + 16 * lane) : kOutOfRange;
      }
    }
  }

  // Where round k starts, and whether this lane's summed values exist.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t round(int64_t k, bool& ok) const {
    constexpr int kValues = kSlabs * slab_values(SRC);
    int64_t left;        // summed values from this round on
    const char* at;
    if constexpr (SRC == kPackedT2) {
      const int64_t j = k < per ? k : k - per;
      at = (k < per ? base0 : base1) + j * step;
      left = k < end ? n_rows - 32 * j : 0;
    } else {
      at = base0 + k * step;
      left = end - kValues * k;
    }
    ok = k_lane < int(left < kValues ? left : kValues);
    return buffer(at, bytes);
  }
  // This wave's r-th piece.
  __device__ __forceinline__ void load(char* stage, __amdgpu_buffer_rsrc_t rsrc, bool ok, int r,
                                       int wave) const {
    const uint32_t o = SRC == kRows ? (ok ? off[0] : 1u << 30) + r * piece
                                    : ok ? off[r] : kOutOfRange;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(stage + 1024 * (4 * r + wave)), 16,
                                             o, 0, 0, 0);
  }
};

// This lane's 16 bytes of the wave's fragment f (16 rows of the tile) in a stage;
// rows: of slab h of the stage's two.
template <int SRC>
struct Reader {
  int at[4];      // byte offset of the lane in the wave's first fragment; rows: by h;
                  // transposed: in the first four
  int at4[4];     // transposed: four summed rows on

  // first: the wave's first fragment.
  __device__ __forceinline__ void init(int lane, int first) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (SRC == kRows) {
      at[0] = 2048 * first + 128 * i + 16 * (g ^ rows_swizzle(i));
      at[1] = at[0] ^ 64;
    } else if constexpr (SRC == kTrans || SRC == kPackedT2) {
      const int k = 8 * g + (i >> 2);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int f = first + b;
        if constexpr (SRC == kTrans) {
          at[b] = 4096 * (f >> 2) + 128 * k + 8 * (i & 3) + 32 * ((f & 3) ^ trans_swizzle(k));
          at4[b] = at[b] + 512;
        } else {
          at[b] = 4096 * (f >> 2) + 256 * (f & 3) + 1024 * g + ((8 * i) ^ (128 * (g & 1)));
          at4[b] = at[b] ^ 128;
        }
        // kept apart: the compiler follows an address only a few steps back to
        // its stage, and waits for every load in flight where it cannot
        asm volatile("" : "+v"(at4[b]));
      }
    } else if constexpr (SRC == kPacked || SRC == kPacked2) {
      at[0] = 1024 * first + 512 * (i >> 3) + 256 * (g >> 1) + 32 * (i & 7) + 16 * (g & 1);
    } else {
      at[0] = 1024 * first + 16 * lane;
    }
  }

  // Keeps the compiler from making the stages' addresses ahead, outside of a loop over
  // tiles: it would not know what they point to any more, and wait as above.
  __device__ __forceinline__ void renew() {
    constexpr int n = SRC == kTrans || SRC == kPackedT2 ? 4 : SRC == kRows ? 2 : 1;
#pragma unroll
    for (int b = 0; b < n; ++b) {
      asm volatile("" : "+v"(at[b]));
      if constexpr (n == 4) asm volatile("" : "+v"(at4[b]));
    }
  }

  __device__ __forceinline__ u32x4 read(const char* stage, int f, int h) const {
    if constexpr (SRC == kTrans || SRC == kPackedT2) {
      const int block = 4096 * (f >> 2), b = f & 3;
      const u32x2 lo = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(stage + (block + at[b]))));
      const u32x2 hi = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(stage + (block + at4[b]))));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else if constexpr (SRC == kRows) {
      return *(const volatile lds_u32x4*)(stage + (2048 * f + at[h]));
    } else {
      return *(const volatile lds_u32x4*)(stage + (1024 * f + at[0]));
    }
  }
};

// Scale words of a tile's 16-row groups (a word a lane holds four slabs' scales).
struct Scales {
  __amdgpu_buffer_rsrc_t at;   // the tile's first group
  int64_t row_bytes;           // a group
  int64_t end;                 // words of a lane in a group
  int last;                    // last group that exists, counted from the tile's first one
  __device__ __forceinline__ void init(const uint8_t* s, int64_t batch_off, int64_t K, int64_t r0,
                                       int64_t n) {
    end = (K + 511) / 512;
    row_bytes = end * 256;
    at = buffer(s + batch_off + r0 / 16 * row_bytes, end ? kOutOfRange : 0);
    const int64_t l = (n + 15) / 16 - 1 - r0 / 16;
    last = l < 255 ? int(l) : 255;
  }
  // Group i (one past the matrix reads its last one; its outputs are not
  // stored), slabs 4 q .. 4 q + 3 (past the end: the last word, not used).
  __device__ __forceinline__ uint32_t word(int i, int64_t q, int lane) const {
    const int64_t w = q < end ? q : end - 1;
    return __builtin_amdgcn_raw_buffer_load_b32(at, 4 * lane,
                                                int((i < last ? i : last) * row_bytes + 256 * w), 0);
  }
};

// A sum from the accumulator registers, here and not earlier: with a branch for
// each output type the compiler reads all 64 before it, more than fit.
__device__ __forceinline__ f32x4 sum(f32x4 acc) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(x) : "a"(acc[e]));
    v[e] = x;
  }
  return v;
}

// acc += b a^T over 32 values, in place. Written out, since the compiler gives
// the result of its own form other registers than the sum it starts from; with
// all 256 accumulator registers in use it then moved a third of them about in
// every slab. Nothing but these instructions may touch the accumulators between
// settle() and settle(): the compiler does not know that the results take time.
template <int DT>
__device__ __forceinline__ void mfma(u32x4 b, u32x4 a, f32x4& acc) {
  if constexpr (DT == kBF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else if constexpr (DT == kI8)   // (the accumulators hold whole numbers)
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
// Enough wait states for any MFMA's result to be read, or for accumulators that
// were just written to be used (18 are needed at most).
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 7"); }
// 16 x 16 x 128 with 4-bit operands; byte SEL of each lane's scale word scales
// its 32 values.
template <int SEL>
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 b, u32x4 a, uint32_t sb, uint32_t sa, f32x4 acc) {
  const i32x8 x = {int(b[0]), int(b[1]), int(b[2]), int(b[3]), 0, 0, 0, 0};
  const i32x8 y = {int(a[0]), int(a[1]), int(a[2]), int(a[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, SEL, int(sb), SEL,
                                                          int(sa));
}

// ---- epilogue ----

// Two neighbouring 16-column blocks (v0: columns 0-15, v1: 16-31; lane group g
// holds columns 4g .. 4g + 3 of each) to one 16-byte store a lane: groups
// exchange halves, so that group g holds columns 16 (g % 2) + 8 (g / 2) .. + 7.
template <int DT>
__device__ __forceinline__ u32x4 join16(f32x4 v0, f32x4 v1) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = pack2<DT>(v0[2 * i], v0[2 * i + 1]);
    const uint32_t y = pack2<DT>(v1[2 * i], v1[2 * i + 1]);
    const auto s = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    o[i] = s[0];
    o[2 + i] = s[1];
  }
  return o;
}

template <int DT>
__device__ __forceinline__ u32x2 pack4(f32x4 v) {
  return u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

template <int ACT>
__device__ __forceinline__ f32x4 gate(f32x4 g, f32x4 u) {
  f32x4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = act<ACT>(g[i]) * u[i];
  return h;
}

// The output rows of a wave from d on, `left` of at most n: what lies past them
// is not written.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t out_rows(const void* d, int64_t row_bytes,
                                                           int64_t left, int n) {
  const int64_t rows = left < 0 ? 0 : left < n ? left : n;
  return buffer(d, uint32_t(rows * row_bytes));   // ld <= 2^21: at most 2^30
}

// Outputs are touched once: non-temporal, so that they do not push the operands
// out of the caches (gated with projections kept, 8192 x 4096 -> 8192: 819
// against 843 us). Partial sums stay: the join reads them right after. By groups,
// where the sums are short, the caches take the results faster: 24576 rows of 64
// groups gated 2048 -> 1408, projections kept, 358 us against 370.
constexpr int kNonTemporal = 2;

// The kernel's I-th argument (it and those before are TileArgs), read again: what is
// needed of it only after a sum would otherwise be kept in (spilled) scalar registers.
template <int I>
__device__ __forceinline__ const TileArgs& args_again() {
  uint64_t at = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr()) +
                I * sizeof(TileArgs);
  asm volatile("" : "+s"(at));
  return *(const TileArgs*)reinterpret_cast<const __attribute__((address_space(4))) TileArgs*>(at);
}

// Where a tile lies and what it sums. By groups rows, values and columns are below
// 2^31.
template <int GRP>
struct Place {
  using Int = std::conditional_t<GRP == kWhole, int64_t, int32_t>;
  Int b;                 // batch or group
  Int m0, n0;            // first row within the group, first column
  Int M, K;              // rows of the group, values to sum
  Int d_row;             // first row of D of the group
  Int s0, s1;            // the slabs to sum
  int64_t a_off, b_off;  // elements (4-bit codes: bytes) to the batch's or group's operands
  uint32_t split;
  bool empty;            // the rows behind the last group
};

// The slabs of split `at.split`.
template <int GRP>
__device__ __forceinline__ void slabs_of(Place<GRP>& at, int values, uint32_t splits) {
  const auto r = slab_range(at.K, values, at.split, splits);
  at.s0 = r.first;
  at.s1 = r.end;
}

// Which tile of a product by groups of rows workgroup w makes; false: none. The host
// knows a bound of the tiles only. `small`: by the body for 128 rows, where a tile of 256
// holds no more of its group. How they lie: row_layout (group_counts.h); then, in
// workgroups of their own behind those of the groups, the tiles of the rows behind the
// last group, which only store zeros. (Among the groups' tiles they would fill one XCD's
// run and leave the others more than a round: 64 rows of 8 groups and a tail of 24 in tiles
// of 128 x 128, gated 4096 -> 8192, 206 us, now 179, without a tail 177; 4096 -> 8192 of
// the same rows 129, now 96.)
template <int TM, int COLS>
__device__ __forceinline__ bool locate_rows(const TileArgs& p, uint32_t w, uint32_t NT, int values,
                                            int lane, Place<kGroupRows>& at, bool& small) {
  Groups groups;
  groups.init(p.ends, int(p.batch), int(p.M), lane);
  const auto rows = groups.tiles<TM>(p.zero_tail);
  const uint32_t splits = p.splits > 1 ? p.splits : 1;
  const RowLayout lay = row_layout<TM>(rows.grouped, rows.grouped_small, NT, splits);
  const bool mixed = lay.mixed;
  const uint32_t n_full = lay.full * NT * splits, n_last = lay.last * NT * splits, cut = lay.cut;
  uint32_t MT = lay.full, half = 0;
  const bool tail = w >= n_full + cut + n_last, halves = !tail && w >= n_full - cut + n_last,
             lasts = !tail && !halves && w >= n_full - cut;
  if (tail) {
    w -= n_full + cut + n_last;
    MT = uint32_t(rows.total + rows.total_small - rows.grouped - rows.grouped_small);
    if (w >= MT * NT * splits) return false;
  } else if (halves) {
    w -= n_full - cut + n_last;
    half = w % 2;
    w = n_full - cut + w / 2;
  } else if (lasts) {
    w = xcd_run(w - (n_full - cut), n_last);
    MT = lay.last;
  } else {
    w = xcd_run(w, n_full - cut);
  }
  at.split = w / (MT * NT);
  w -= at.split * (MT * NT);
  const int r = int(w / NT);
  const Group g = tail ? groups.behind(rows, r)
                  : lasts ? groups.find_small<TM>(rows, r)
                  : mixed ? groups.find_any<TM>(rows, r) : groups.find<TM>(rows, r);
  const int k = tail ? int(MT) : lasts ? 1
                : full_tiles<TM>(g.rows) + (mixed ? small_tiles<TM>(g.rows) : 0);
  const BandTile t = band_tile(w - uint32_t(r - g.tile) * NT, uint32_t(k), NT);
  at.empty = tail;
  at.b = tail ? 0 : g.e;
  at.m0 = lasts ? g.rows / 256 * 256 : int(t.row * TM + 128 * half);
  at.n0 = int(t.col * COLS);
  at.M = g.rows;
  at.K = tail ? 0 : int(p.K);
  at.d_row = g.start;
  at.a_off = g.start * p.lda;
  at.b_off = at.b * p.b_bs;
  slabs_of(at, values, splits);
  small = TM == 256 && (halves || at.M - at.m0 <= 128);
  return at.m0 < at.M;
}

// The tiles of sums by groups that one workgroup makes one after another. A sum is as
// long as its group has rows, so an XCD that took whole groups would have too much or
// too little to do (16 groups: 2841 rows in two of them, 2048 in the mean); the groups'
// units (tiles, times splits) are taken in rounds instead, the largest groups first,
// and in each round an XCD takes neighbouring units. Groups without rows are not in it
// (fill_empty), but for split sums, of which the join takes every part.
struct SumList {
  Groups groups;
  int taken;                // groups whose units are in the list
  uint32_t MT, NT, units;   // units: of one group
  uint32_t wg, n_wg;        // this workgroup, of so many (a multiple of the XCDs)

  __device__ __forceinline__ void init(const TileArgs& p, uint32_t wg_, uint32_t n_wg_, uint32_t MT_,
                                       uint32_t NT_, int lane) {
    wg = wg_;
    n_wg = n_wg_;
    groups.init(p.ends, int(p.batch), int(p.K), lane);
    groups.sort();
    taken = p.splits > 1 ? groups.E : groups.filled;
    MT = MT_;
    NT = NT_;
    units = MT * NT * (p.splits > 1 ? p.splits : 1);
  }
  // This workgroup's among the units of a round.
  __device__ __forceinline__ uint32_t place() const {
    return wg % kXcds * (n_wg / kXcds) + wg / kXcds;
  }
  // The tile of round k; false: none.
  template <int TM, int COLS>
  __device__ __forceinline__ bool locate(const TileArgs& p, uint32_t k, int values,
                                         Place<kGroupSums>& at) const {
    const uint32_t w = k * n_wg + place();
    const uint32_t slot = w / units, u = w - slot * units;
    if (slot >= uint32_t(taken)) return false;
    at.split = u / (MT * NT);
    const TileAt t = tile_at(u - at.split * (MT * NT), MT, NT, false);
    const Group g = groups.sorted(int(slot));
    at.empty = false;
    at.b = g.e;
    at.m0 = int(t.mt * TM);
    at.n0 = int(t.nt * COLS);
    at.M = int(p.M);
    at.K = g.rows;
    at.d_row = 0;
    at.a_off = g.start * p.lda;
    at.b_off = g.start * p.ldb;
    slabs_of(at, values, p.splits > 1 ? p.splits : 1);
    return true;
  }
};

// The ring's stages in LDS.
struct Ring {
  char *b0, *b1, *b2, *b3, *a0, *a1, *a2, *a3;
};

// 256 rows: one workgroup a CU (a wave's 64 accumulators of 4 floats fill the
// accumulator registers, so 128 x 128 of D come from 16 fragment reads);
// 128 x 128: two workgroups a CU.
//
// Sums by groups: a workgroup a place of the chip makes one tile after another (`list`).
// It sends the first loads of its next tile before it stores the results of the one
// just summed, and does not wait for the stores: with sums as short as a group has rows
// the stores and the ring's first round trip cost as much as the sum (weight gradients
// of 24576 rows of 64 groups, 2048 x 1408: 242 -> 220 us). The other products gain
// nothing by it.
//
// p is the kernel's ARG-th argument.
template <int DT, int SRCA, int SRCB, int EPI, int GRP, int TM, int TN, int ARG = 0>
__device__ __forceinline__ void make_tile(const TileArgs& p, Place<GRP> at, const SumList& list,
                                          const Ring& ring, int lane, int wave) {
  constexpr int kBM = TM / 32, kBN = TN / 32;   // 16-row and 16-column blocks a wave
  constexpr int kCols = EPI == kGated ? TN / 2 : TN;   // columns of D a tile
  static_assert((EPI == kGated) == two_sources(SRCB), "gated: two sources of B");
  constexpr bool kPairs = Loader<SRCA, TM>::kSlabs == 2;
  constexpr int kValues = slab_values(SRCA);
  constexpr bool kLoop = GRP == kGroupSums;   // one tile after another
  using Int = typename Place<GRP>::Int;
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4;
  const uint32_t splits = p.splits > 1 ? p.splits : 1;
  char *const b0 = ring.b0, *const b1 = ring.b1, *const b2 = ring.b2, *const b3 = ring.b3;
  char *const a0 = ring.a0, *const a1 = ring.a1, *const a2 = ring.a2, *const a3 = ring.a3;

  Loader<SRCA, TM> la;
  Loader<SRCB, TN> lb;
  Scales ca, cb0, cb1;
  if constexpr (DT == kMX4) {
    ca.init(p.as, at.b * p.as_bs, p.K, at.m0, p.M);
    cb0.init(p.bs0, at.b * p.bs_bs, p.K, at.n0, p.N);
    if constexpr (EPI == kGated) cb1.init(p.bs1, at.b * p.bs_bs, p.K, at.n0, p.N);
  }
  Reader<SRCA> ra;
  Reader<SRCB> rb;
  ra.init(lane, kBM * wm);
  rb.init(lane, kBN * wn);
  constexpr int kLoadsA = Loader<SRCA, TM>::kLoads, kLoadsB = Loader<SRCB, TN>::kLoads;
  auto issue_a = [&](char* stage, int64_t k) {
    bool ok;
    const auto at = la.round(k, ok);
#pragma unroll
    for (int r = 0; r < kLoadsA; ++r) la.load(stage, at, ok, r, wave);
    __builtin_amdgcn_sched_barrier(0);   // the waits below count the loads in this order
  };
  auto issue_b = [&](char* stage, int64_t k) {
    bool ok;
    const auto at = lb.round(k, ok);
#pragma unroll
    for (int r = 0; r < kLoadsB; ++r) lb.load(stage, at, ok, r, wave);
    __builtin_amdgcn_sched_barrier(0);
  };

  // 4-bit: this wave's scale words of four slabs, and of the next four
  uint32_t xa[8], xb[8], ya[8], yb[8];
  constexpr int kWords = DT == kMX4 ? kBM + kBN : 0;
  auto load_scale = [&](auto word, int64_t q) {   // one of kWords
    constexpr int i = decltype(word)::value, j = i - kBM;
    if constexpr (i < kBM) ya[i] = ca.word(kBM * wm + i, q, lane);
    else if constexpr (EPI == kGated)
      yb[j] = (j & 1 ? cb1 : cb0).word((kBN * wn + j) >> 1, q, lane);
    else yb[j] = cb0.word(kBN * wn + j, q, lane);
  };
  auto take_scales = [&]() {
    if constexpr (DT == kMX4) {
#pragma unroll
      for (int i = 0; i < kBM; ++i) xa[i] = ya[i];
#pragma unroll
      for (int j = 0; j < kBN; ++j) xb[j] = yb[j];
    }
  };
  f32x4 acc[8][8];   // [16-row block][16-column block], kBM x kBN used
  u32x4 F0[16], F1[16];   // one slab's fragments: B's kBN, then A's kBM
  auto read = [&](const char* sa, int h, const char* sb, u32x4 (&F)[16], int i) {
    F[i] = i < kBN ? rb.read(sb, i, 0) : ra.read(sa, i - kBN, h);
  };
  // Slab s, the ring's turn-th: fragments Fc; reads slab s + 1 from (na, nb) to
  // Fn; loads slab s + 4 to this slab's own stage (ta, tb), whose fragments every
  // wave has read (rows: slabs s + 3 and s + 4 to the stage of s - 1 and s, in
  // odd turns).
  // Stores of the tile before that this wave has sent at least, after this tile's
  // first loads. The first two slabs (`first`) wait for loads that were sent before
  // them and leave the stores in flight.
  constexpr int kStores = !kLoop ? 0 : EPI == kGated ? kBM * (kBN / 4) : kBM * (kBN / 2);
  auto slab = [&](auto turn, auto first, Int s, const char* na, const char* nb, char* ta, char* tb,
                  const u32x4 (&Fc)[16], u32x4 (&Fn)[16]) __attribute__((always_inline)) {
    constexpr int SEL = decltype(turn)::value;
    auto mma = [&](int i) {
      // in blocks of 2 x 2, each MFMA sharing a fragment with the one before: at the
      // power limit up to 1% faster than row by row (backward pass of 8192 x 4096
      // -> 8192 1651 against 1681 us)
      const int q = i / 4, u = i % 4;
      const int r = 2 * (q / (kBN / 2)) + (u >> 1), c = 2 * (q % (kBN / 2)) + ((u & 1) ^ (u >> 1));
      if constexpr (DT == kMX4)
        acc[r][c] = mfma_mx4<SEL>(Fc[c], Fc[kBN + r], xb[c], xa[r], acc[r][c]);
      else
        mfma<DT>(Fc[c], Fc[kBN + r], acc[r][c]);
      __builtin_amdgcn_sched_barrier(0);
    };
    __builtin_amdgcn_sched_barrier(0);
    mma(0);
    mma(1);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    // After the barrier the reads are spread over the first part of the MFMAs
    // (they have to be back at the end of the slab), the loads over all of them:
    // sent in a burst they would wait for each other, and the MFMAs behind them.
    constexpr int kNowA = !kPairs || SEL % 2 == 1 ? kLoadsA : 0, kNow = kNowA + kLoadsB;
    bool oka, okb;
    const auto la_at = la.round(kPairs ? (s + 3) / 2 : s + 4, oka);   // (s0 is even)
    const auto lb_at = lb.round(s + 4, okb);
    constexpr int kMfmas = kBM * kBN, kFrags = kBM + kBN;
    constexpr int kVmem = kNow + (SEL == 0 ? kWords : 0);
    static_for<2, kMfmas>([&](auto at) {
      constexpr int i = decltype(at)::value;
      mma(i);
      constexpr int f = item_at(i - 2, kFrags, 0, kMfmas * 3 / 4), v = item_at(i - 2, kVmem, 1, kMfmas - 2);
      if constexpr (f >= 0) read(na, (SEL + 1) % 2, nb, Fn, f);
      if constexpr (v >= kNow)
        load_scale(std::integral_constant<int, v - kNow>{}, (s >> 2) + 1);
      else if constexpr (v >= kNowA)
        lb.load(tb, lb_at, okb, v - kNowA, wave);
      else if constexpr (v >= 0)
        la.load(ta, la_at, oka, v, wave);
      __builtin_amdgcn_sched_barrier(0);
    });
    // Fn read; own loads of slab s + 2 landed, which were sent in slab s - 2 (rows:
    // an odd slab's, before that slab's loads of B, two or one slab ago)
    constexpr int kBefore = kPairs ? kLoadsB : kLoadsA + kLoadsB;
    constexpr int kOpen = kVmem + kBefore + (SEL == 1 && !kPairs ? kWords : 0);
    constexpr int kWith = kOpen + (decltype(first)::value && SEL < 2 ? kStores : 0);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(kWith < 63 ? kWith : 63, 0));
  };

  char* const r1 = kPairs ? a0 : a1;
  char* const r3 = kPairs ? a2 : a3;
  // The loads of a tile's first four slabs.
  auto begin = [&](const TileArgs& p, const Place<GRP>& q) {
    TileArgs of = p;
    of.K = q.K;
    if (GRP == kGroupRows && q.empty) of.b_sum = of.b_rows = 0;
    la.init(of, p.a, nullptr, q.a_off, p.lda, q.m0, q.M, q.s1, lane, wave);
    lb.init(of, p.b0, p.b1, q.b_off, p.ldb, q.n0, p.N, q.s1, lane, wave);
    issue_a(a0, kPairs ? q.s0 / 2 : q.s0);
    issue_b(b0, q.s0);
    if constexpr (!kPairs) issue_a(r1, q.s0 + 1);
    issue_b(b1, q.s0 + 1);
    issue_a(a2, kPairs ? q.s0 / 2 + 1 : q.s0 + 2);
    issue_b(b2, q.s0 + 2);
    if constexpr (!kPairs) issue_a(r3, q.s0 + 3);
    issue_b(b3, q.s0 + 3);
  };
  static_for<0, kWords>([&](auto i) { load_scale(i, 0); });
  __builtin_amdgcn_sched_barrier(0);
  begin(p, at);
  take_scales();
  if constexpr (kLoop) {
    // As many stores to nowhere as a tile before would have sent at least: the waits of
    // every tile count the same.
    const auto nowhere = buffer(nullptr, 0);
#pragma unroll
    for (int i = 0; i < kStores; ++i)   // (at different places, so that none is left out)
      __builtin_amdgcn_raw_buffer_store_b32(0u, nowhere, kOutOfRange - 16 * i, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (uint32_t tile = 0;; ++tile) {
  // Pinned to accumulator registers one by one: equal starting values would be
  // merged, and the loop would then copy them.
#pragma unroll
  for (int i = 0; i < kBM; ++i)
#pragma unroll
    for (int j = 0; j < kBN; ++j) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      asm volatile("" : "+a"(v));
      acc[i][j] = v;
    }
  settle();
  // slabs 0 and 1 landed (after them: rows, one round of A and two of B)
  constexpr int kFirst = (kPairs ? 1 : 2) * kLoadsA + 2 * kLoadsB + kStores;
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(kFirst < 63 ? kFirst : 63, 15));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  if constexpr (kLoop) {
    ra.renew();
    rb.renew();
  }
#pragma unroll
  for (int i = 0; i < kBM + kBN; ++i) read(a0, 0, b0, F0, i);
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
  // One turn of the ring, or its first half.
  auto turn = [&](auto first, auto half, Int s) __attribute__((always_inline)) {
    if constexpr (kLoop) {
      ra.renew();
      rb.renew();
    }
    slab(std::integral_constant<int, 0>{}, first, s + 0, r1, b1, a0, b0, F0, F1);
    slab(std::integral_constant<int, 1>{}, first, s + 1, a2, b2, r1, b1, F1, F0);
    if constexpr (!decltype(half)::value) {
      slab(std::integral_constant<int, 2>{}, first, s + 2, r3, b3, a2, b2, F0, F1);
      slab(std::integral_constant<int, 3>{}, first, s + 3, a0, b0, r3, b3, F1, F0);
    }
    take_scales();
  };
  const std::true_type yes;
  const std::false_type no;
  if constexpr (kLoop) {
    // (after the first turn: where two slabs are left or one, no two of zeros besides)
    Int s = at.s0;
    turn(yes, no, s);
    for (s += 4; s + 2 < at.s1; s += 4) turn(no, no, s);
    if (s < at.s1) turn(no, yes, s);
  } else {
    for (Int s = at.s0; s < at.s1; s += 4) turn(no, no, s);
  }
  Place<GRP> next;
  bool more = false;
  auto finish = [&](const TileArgs& p) {
  const int64_t row = at.m0 + 16 * kBM * wm, col = at.n0 + (EPI == kGated ? 8 : 16) * kBN * wn;
  // 8-bit integers: the scales of this lane's rows, and of its columns of each block
  float scale_a[8];
  f32x4 scale_b[8];
  if constexpr (DT == kI8) {
    const int64_t left = at.empty || at.M < row ? 0 : at.M - row;
    const int64_t cols = at.empty || p.N < col ? 0 : p.N - col;
    const auto sa = buffer(p.sa + (GRP == kGroupRows ? at.d_row : at.b * p.M) + row,
                           uint32_t(left < 16 * kBM ? left : 16 * kBM) * 4);
    const uint32_t bytes = uint32_t(cols < 16 * kBN ? cols : 16 * kBN) * 4;
    const auto sb0 = buffer(p.sb0 + at.b * p.N + col, bytes);
    const auto sb1 = buffer((EPI == kGated ? p.sb1 : p.sb0) + at.b * p.N + col, bytes);
#pragma unroll
    for (int i = 0; i < kBM; ++i)
      scale_a[i] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(sa, 64 * i + 4 * (lane & 15), 0, 0));
#pragma unroll
    for (int j = 0; j < kBN; ++j) {
      const int c = EPI == kGated ? 64 * (j >> 1) + 16 * g : 64 * j + 16 * g;
      scale_b[j] = __builtin_bit_cast(
          f32x4, __builtin_amdgcn_raw_buffer_load_b128(EPI == kGated && (j & 1) ? sb1 : sb0, c, 0, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kLoop) {
    // The ring is free when every wave has read its last fragments; the zeros loaded past
    // the sum's end have long landed. (The compiler counts loads and stores along every
    // path it sees: no load may be open on one that skips the next ones, and every path
    // has to store as often.)
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
    more = list.template locate<TM, kCols>(p, tile + 1, kValues, next);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (more) begin(p, next);
    __builtin_amdgcn_sched_barrier(0);
  } else {
    // No load may still be writing LDS when the workgroup ends.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
  }
  settle();
#pragma unroll
  for (int i = 0; i < kBM; ++i)
#pragma unroll
    for (int j = 0; j < kBN; ++j) asm volatile("" : "+a"(acc[i][j]));   // read from here on only
  // The sums of block (i, j); 8-bit integers: those values times the scales.
  auto sums = [&](int i, int j) {
    if constexpr (DT == kI8) {
      const f32x4 v = sum(acc[i][j]);
      f32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = v[e];   // (a cast of the element itself takes element 0)
        r[e] = float(__builtin_bit_cast(int, x)) * scale_a[i] * scale_b[j][e];
      }
      return r;
    } else if constexpr (GRP != kWhole) {
      return sum(acc[i][j]);
    } else {
      return acc[i][j];
    }
  };
  constexpr int kPairsN = EPI == kGated ? kBN / 4 : kBN / 2;   // 32-column pieces
  // float32 results: partial sums, and the 4-bit product's where it is asked for
  const bool wide = EPI == kStore && (any_output(DT) ? p.out_type == BMM_ELEM_F32 : splits > 1);
  // (192 columns: 48 of H a wave, the last 16 by themselves)
  constexpr bool kLast = EPI == kGated && kBN % 4 != 0;
  constexpr int kAux = GRP == kWhole ? kNonTemporal : 0;
  // Offsets of this lane's columns in the first 16 rows; those outside are past
  // every buffer's end.
  const int64_t ld = EPI == kStore && splits > 1 ? p.N : p.ldd;
  const uint32_t row_bytes = uint32_t(ld) * (wide ? 4 : 2), step = 16 * row_bytes;
  uint32_t off[8];
  auto offsets = [&]() {
#pragma unroll
    for (int j = 0; j < (wide ? kBN : kPairsN); ++j) {
      const int c = wide ? 16 * j + 4 * g : 32 * j + 16 * (g & 1) + 8 * (g >> 1);
      off[j] = col + c < p.N ? (lane & 15) * row_bytes + (wide ? 4 : 2) * c : kOutOfRange;
    }
  };
  u32x4 out[8][2];
  u32x2 last[8];
  if constexpr (EPI == kGated) {
    auto gate_all = [&](auto type, auto a) {
      constexpr int T = decltype(type)::value, A = decltype(a)::value;
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j)
          out[i][j] = join16<T>(gate<A>(sums(i, 4 * j), sums(i, 4 * j + 1)),
                                gate<A>(sums(i, 4 * j + 2), sums(i, 4 * j + 3)));
      if constexpr (kLast) {
#pragma unroll
        for (int i = 0; i < kBM; ++i) last[i] = pack4<T>(gate<A>(sums(i, kBN - 2), sums(i, kBN - 1)));
      }
    };
    auto gate_type = [&](auto a) {
      if constexpr (!any_output(DT)) gate_all(std::integral_constant<int, DT>{}, a);
      else if (p.out_type == BMM_ELEM_BF16) gate_all(std::integral_constant<int, kBF16>{}, a);
      else gate_all(std::integral_constant<int, kF16>{}, a);
    };
    switch (p.act) {
      case BMM_ACT_SILU: gate_type(std::integral_constant<int, BMM_ACT_SILU>{}); break;
      case BMM_ACT_GELU: gate_type(std::integral_constant<int, BMM_ACT_GELU>{}); break;
      case BMM_ACT_GELU_TANH: gate_type(std::integral_constant<int, BMM_ACT_GELU_TANH>{}); break;
      default: gate_type(std::integral_constant<int, BMM_ACT_RELU>{});
    }
  }

  if constexpr (EPI == kGated) {
    auto store = [&](void* d, auto value, auto last_value) {
      const auto to = out_rows(static_cast<uint16_t*>(d) +
                                   ((GRP == kGroupRows ? at.d_row : at.b * p.M) + row) * ld + col,
                               row_bytes, at.M - row, 16 * kBM);
      offsets();
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(value(i, j), to, off[j] + i * step, 0, kAux);
      if constexpr (kLast) {
        const int c = 32 * kPairsN + 4 * g;
        const uint32_t off_last = col + c < p.N ? (lane & 15) * row_bytes + 2 * c : kOutOfRange;
#pragma unroll
        for (int i = 0; i < kBM; ++i)
          __builtin_amdgcn_raw_buffer_store_b64(last_value(i), to, off_last + i * step, 0, kAux);
      }
    };
    store(p.d, [&](int i, int j) { return out[i][j]; }, [&](int i) { return last[i]; });
    if constexpr (!any_output(DT)) {
      if (p.d1) {
        store(p.d1, [&](int i, int j) { return join16<DT>(sums(i, 4 * j), sums(i, 4 * j + 2)); },
              [&](int i) { return pack4<DT>(sums(i, kBN - 2)); });
        store(p.d2, [&](int i, int j) { return join16<DT>(sums(i, 4 * j + 1), sums(i, 4 * j + 3)); },
              [&](int i) { return pack4<DT>(sums(i, kBN - 1)); });
      }
    }
  } else {
    // Rows below rows0 go to d, those from row1 (a multiple of 16) on to d1.
    const int size = wide ? 4 : 2;
    const bool parts = splits > 1;
    const char* d = parts ? reinterpret_cast<char*>(p.part + at.split * p.part_floats)
                          : static_cast<char*>(p.d);
    const int64_t rows = GRP == kGroupRows || parts ? at.M : p.rows0;
    const auto to = out_rows(d + (((GRP == kGroupRows ? at.d_row : at.b * rows) + row) * ld + col) * size,
                             row_bytes, rows - row, 16 * kBM);
    auto to1 = to;
    int second = kBM;   // first block of 16 rows that goes to d1
    if constexpr (SRCA == kTrans) {
      if (!parts && row + 16 * kBM > p.row1) {
        second = row < p.row1 ? int(p.row1 - row) / 16 : 0;
        to1 = out_rows(static_cast<char*>(p.d1) +
                           ((at.b * rows + row - p.row1) * ld + col) * size,
                       row_bytes, p.row1 + rows - row, 16 * kBM);
      }
    }
    offsets();
    auto store = [&](int i, int j, u32x4 v, auto nt) {
      __builtin_amdgcn_raw_buffer_store_b128(v, SRCA == kTrans && i >= second ? to1 : to,
                                             off[j] + i * step, 0, decltype(nt)::value);
    };
    float rescale = 1.f;
    if constexpr (DT == kF16) rescale = p.rescale ? *p.rescale : 1.f;
    auto result = [&](int i, int j) {
      if constexpr (DT == kI8) return sums(i, j);
      const f32x4 v = sum(acc[i][j]);
      return DT == kF16 ? v * rescale : v;
    };
    auto store16 = [&](auto type) {
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j)
          store(i, j, join16<decltype(type)::value>(result(i, 2 * j), result(i, 2 * j + 1)),
                std::integral_constant<int, kAux>{});
    };
    auto store32 = [&](auto nt) {
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kBN; ++j) store(i, j, __builtin_bit_cast(u32x4, sums(i, j)), nt);
    };
    if constexpr (kLoop) {
      // Two neighbouring blocks in one store of 16 bits a value, or the first of them in
      // float32 and the second later.
      if (wide) rescale = 1.f;   // (the join applies it)
      uint32_t later[4];
#pragma unroll
      for (int j = 0; j < kPairsN; ++j) {
        const int c = 32 * j + 4 * g;
        later[j] = col + c + 16 < p.N ? (lane & 15) * row_bytes + 4 * (c + 16) : kOutOfRange;
        if (wide) off[j] = col + c < p.N ? (lane & 15) * row_bytes + 4 * c : kOutOfRange;
      }
      static_assert(!any_output(DT), "sums by groups are of 16-bit values");
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j) {
          const f32x4 x = result(i, 2 * j);
          const u32x4 v = join16<DT>(x, result(i, 2 * j + 1));
          store(i, j, wide ? __builtin_bit_cast(u32x4, x) : v, std::integral_constant<int, kAux>{});
        }
      if (wide) {
#pragma unroll
        for (int j = 0; j < kPairsN; ++j) off[j] = later[j];
#pragma unroll
        for (int i = 0; i < kBM; ++i)
#pragma unroll
          for (int j = 0; j < kPairsN; ++j)
            store(i, j, __builtin_bit_cast(u32x4, result(i, 2 * j + 1)),
                  std::integral_constant<int, kAux>{});
      }
    } else if constexpr (!any_output(DT)) {
      if (wide) store32(std::integral_constant<int, 0>{});
      else store16(std::integral_constant<int, DT>{});
    } else {
      if (wide) store32(std::integral_constant<int, kAux>{});
      else if (p.out_type == BMM_ELEM_BF16) store16(std::integral_constant<int, kBF16>{});
      else store16(std::integral_constant<int, kF16>{});
    }
  }
  };
  if constexpr (GRP != kWhole) finish(args_again<ARG>());
  else finish(p);
  if (!more) break;
  at = next;
  }
}

// Zeros for the groups whose sums are empty, after the workgroup's tiles: pieces of
// 64 KB, lane after lane, as fast as memory takes them. The workgroups that had one tile
// less come first. As tiles they waited for loads of nothing and for each other's stores:
// backward pass of 41 rows in 41 of 120 groups, 1568 -> 488, 85 -> 67 us; of the gated
// block, 80 rows in 7 of 21, 2256 -> 2832, 225 -> 186. ARG as above.
template <int ARG>
__device__ __forceinline__ void fill_empty(const SumList& list) {
  if (list.taken == list.groups.E) return;
  const TileArgs& p = args_again<ARG>();
  const Groups& groups = list.groups;
  constexpr uint32_t kPiece = 4096;   // in 16 bytes
  const uint32_t sources = p.row1 < p.M ? 2 : 1;
  const int64_t size = p.rows0 * p.ldd / 8;   // of a group's sums
  const uint32_t pieces = uint32_t((size + kPiece - 1) / kPiece);
  const uint32_t all = uint32_t(groups.E - groups.filled) * sources * pieces;
  const uint32_t over = uint32_t(groups.filled) * list.units % list.n_wg, at = list.place();
  for (uint32_t k = at < over ? at + list.n_wg - over : at - over; k < all; k += list.n_wg) {
    const uint32_t item = k / pieces, slot = item / sources;
    const int64_t first = int64_t(k - item * pieces) * kPiece;
    u32x4* to = static_cast<u32x4*>(item % sources ? p.d1 : p.d) +
                groups.sorted(groups.filled + int(slot)).e * size + first;
    const int64_t left = size - first;
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < kPiece; i += kTileWaves * kWave)
      if (i < left) to[i] = u32x4{0, 0, 0, 0};
  }
}

// A workgroup a tile, or by groups of the summed rows a workgroup a place of the chip.
template <int DT, int SRCA, int SRCB, int EPI, int GRP, int TM, int TN>
__global__ __launch_bounds__(kTileWaves* kWave)
__attribute__((amdgpu_waves_per_eu(TM == 256 ? 1 : 2, TM == 256 ? 1 : 2)))
void ffn_tile_kernel(TileArgs p, uint32_t n_tiles, uint32_t MT, uint32_t NT) {
  constexpr int kCols = EPI == kGated ? TN / 2 : TN;
  // The ring. Separate objects, so that the compiler can tell the stages apart;
  // with rows, which come two slabs at a time, A's stages 0 and 1 are one, and 2
  // and 3.
  constexpr bool kPairs = Loader<SRCA, TM>::kSlabs == 2;
  __shared__ __attribute__((aligned(1024))) char b0[TN * 64], b1[TN * 64], b2[TN * 64], b3[TN * 64];
  __shared__ __attribute__((aligned(1024))) char a0[TM * (kPairs ? 128 : 64)],
      a2[TM * (kPairs ? 128 : 64)], a1[kPairs ? 16 : TM * 64], a3[kPairs ? 16 : TM * 64];
  const Ring ring{b0, b1, b2, b3, a0, a1, a2, a3};

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  constexpr int kValues = slab_values(SRCA);
  Place<GRP> at;
  SumList list;
  if constexpr (GRP == kGroupSums) {
    list.init(p, blockIdx.x, gridDim.x, MT, NT, lane);
    if (list.template locate<TM, kCols>(p, 0, kValues, at))
      make_tile<DT, SRCA, SRCB, EPI, GRP, TM, TN>(p, at, list, ring, lane, wave);
    fill_empty<0>(list);
    return;
  } else if constexpr (GRP == kGroupRows) {
    bool small;
    if (!locate_rows<TM, kCols>(p, blockIdx.x, NT, kValues, lane, at, small)) return;
    if constexpr (TM == 256) {
      if (small) {
        make_tile<DT, SRCA, SRCB, EPI, GRP, 128, TN>(p, at, list, ring, lane, wave);
        return;
      }
    }
  } else {
    const uint32_t splits = p.splits > 1 ? p.splits : 1;
    uint32_t work = xcd_run(blockIdx.x, n_tiles * splits);
    at.split = 0;
    if (splits > 1) {
      at.split = work / n_tiles;
      work -= at.split * n_tiles;
    }
    const TileAt t = tile_at(work, MT, NT, p.batch > 1);
    at.b = t.b;
    at.m0 = t.mt * TM;
    at.n0 = t.nt * kCols;
    at.M = p.M;
    at.K = p.K;
    at.a_off = t.b * p.a_bs;
    at.b_off = t.b * p.b_bs;
    at.d_row = 0;
    at.empty = false;
    slabs_of(at, kValues, splits);
  }
  make_tile<DT, SRCA, SRCB, EPI, GRP, TM, TN>(p, at, list, ring, lane, wave);
}

// Workgroups of a product in tiles of TM x TN, NT tiles across D; negative: too many.
template <int GRP, int TM>
int64_t tile_grid(const TileArgs& p, int64_t MT, int64_t NT) {
  const int64_t splits = p.splits > 1 ? p.splits : 1;
  const int64_t n = (GRP == kGroupRows ? 1 : p.batch) * MT * NT;
  // (sums: their units are counted in 32 bits)
  if (n * splits > (GRP == kGroupSums ? 0x7fffffff : kMaxWorkgroups) || NT > 1 << 28 ||
      p.K >= int64_t(1) << 37)
    return -1;
  int64_t grid = n * splits;
  if (grid > 0 && GRP == kGroupRows && TM == 256 && splits == 1) grid += kCus / 2;   // (tiles in halves)
  if (GRP == kGroupSums) {   // one for each that the chip holds at once, an equal number a XCD
    constexpr int64_t kPlaces = kCus * (TM == 128 ? 2 : 1);
    grid = (grid + kXcds - 1) / kXcds * kXcds;
    grid = grid < kPlaces ? grid : kPlaces;
  }
  return grid > kMaxWorkgroups ? -1 : grid;
}

template <int DT, int SRCA, int SRCB, int EPI, int GRP, int TM, int TN>
hipError_t launch_tile_of(const TileArgs& p, hipStream_t s) {
  const int64_t cols = EPI == kGated ? TN / 2 : TN;
  const int64_t MT = GRP == kGroupRows ? most_row_tiles(p.M, p.batch, TM) : (p.M + TM - 1) / TM;
  const int64_t NT = (p.N + cols - 1) / cols;
  const int64_t grid = tile_grid<GRP, TM>(p, MT, NT);
  if (grid == 0) return hipSuccess;
  if (grid < 0) return hipErrorInvalidConfiguration;
  auto kern = ffn_tile_kernel<DT, SRCA, SRCB, EPI, GRP, TM, TN>;
  hipLaunchKernelGGL(kern, dim3(unsigned(grid)), dim3(kTileWaves * kWave), 0, s, p,
                     uint32_t(p.batch * MT * NT), uint32_t(MT), uint32_t(NT));
  return hipGetLastError();
}

template <int DT, int SRCA, int SRCB, int EPI, int GRP = kWhole>
hipError_t launch_tile(const TileArgs& p, hipStream_t s) {
  switch (p.tile) {
    case kTile256: return launch_tile_of<DT, SRCA, SRCB, EPI, GRP, 256, 256>(p, s);
    case kTile256x128: return launch_tile_of<DT, SRCA, SRCB, EPI, GRP, 256, 128>(p, s);
    case kTile256x192: return launch_tile_of<DT, SRCA, SRCB, EPI, GRP, 256, 192>(p, s);
    default: return launch_tile_of<DT, SRCA, SRCB, EPI, GRP, 128, 128>(p, s);
  }
}

}  // namespace ffn
}  // namespace bmm
