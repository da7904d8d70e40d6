// The MFMA tile kernel of the feed-forward operators: D = A * B^T with the
// operands read where they lie, and the operator's own epilogue.
//
// A product here is one of
//   H  = act(X Wg^T) * (X Wu^T)      A rows,       B packed, two sources   gated
//   dX = [dG | dU] [Wg ; Wu]         A rows,       B packed, transposed    store
//   dW = [dG | dU]^T X               A transposed, B transposed            store
//   D  = A B^T, 4-bit                A, B 4-bit                            store
//   H  = act(..) * (..), 4-bit       A, B 4-bit, two sources               gated
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
#pragma once

#include <type_traits>

#include "ffn.h"

namespace bmm {
namespace ffn {

enum Src : int { kRows, kTrans, kPacked2, kPackedT2, kCodes, kCodes2 };
enum Epi : int { kStore, kGated };

constexpr uint32_t kXcds = 8;
// M tiles in a band: an XCD works on 4 x 8 tiles at a time, whose 12 panels share
// its L2. Gated 8192 x 4096 -> 8192: 4 746 us, 8 756, 16 763, 32 799.
constexpr uint32_t kGroupM = 4;
constexpr int kTileWaves = 4;
constexpr int kBufferFlags = 0x00020000;           // raw, untyped buffer
constexpr uint32_t kOutOfRange = 0x7fffffffu;      // an offset past every buffer's end

typedef short i16x4 __attribute__((ext_vector_type(4)));
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
    } else if constexpr (SRC == kPacked2) {
      k_lane = (lane & 16) + 8 * (lane & 1);
      step = 512;
      base0 = static_cast<const char*>(wave & 1 ? s1 : s0) + 2 * (batch_off + r0 * p.K);
#pragma unroll
      for (int r = 0; r < T / 64; ++r) {
        const int half = 2 * (2 * r + (wave >> 1)) + (lane >> 5);   // 8-column atom row
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
    } else if constexpr (SRC == kPacked2) {
      at[0] = 1024 * first + 512 * (i >> 3) + 256 * (g >> 1) + 32 * (i & 7) + 16 * (g & 1);
    } else {
      at[0] = 1024 * first + 16 * lane;
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
// against 843 us). Partial sums stay: the join reads them right after.
constexpr int kNonTemporal = 2;

// 256 rows: one workgroup a CU (a wave's 64 accumulators of 4 floats fill the
// accumulator registers, so 128 x 128 of D come from 16 fragment reads);
// 128 x 128: two workgroups a CU.
template <int DT, int SRCA, int SRCB, int EPI, int TM, int TN>
__global__ __launch_bounds__(kTileWaves* kWave)
__attribute__((amdgpu_waves_per_eu(TM == 256 ? 1 : 2, TM == 256 ? 1 : 2)))
void ffn_tile_kernel(TileArgs p, uint32_t n_tiles, uint32_t MT, uint32_t NT) {
  constexpr int kBM = TM / 32, kBN = TN / 32;   // 16-row and 16-column blocks a wave
  constexpr int kCols = EPI == kGated ? TN / 2 : TN;   // columns of D a tile
  static_assert((EPI == kGated) == two_sources(SRCB), "gated: two sources of B");
  // The ring. Separate objects, so that the compiler can tell the stages apart;
  // with rows, which come two slabs at a time, A's stages 0 and 1 are one, and 2
  // and 3.
  constexpr bool kPairs = Loader<SRCA, TM>::kSlabs == 2;
  __shared__ __attribute__((aligned(1024))) char b0[TN * 64], b1[TN * 64], b2[TN * 64], b3[TN * 64];
  __shared__ __attribute__((aligned(1024))) char a0[TM * (kPairs ? 128 : 64)],
      a2[TM * (kPairs ? 128 : 64)], a1[kPairs ? 16 : TM * 64], a3[kPairs ? 16 : TM * 64];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4;
  const uint32_t splits = p.splits > 1 ? p.splits : 1, total = n_tiles * splits;
  constexpr int kValues = slab_values(SRCA);
  const int64_t slabs = (p.K + kValues - 1) / kValues;

  Loader<SRCA, TM> la;
  Loader<SRCB, TN> lb;
  Scales ca, cb0, cb1;
  uint32_t work = xcd_run(blockIdx.x, total), split = 0;
  int64_t s0 = 0, s1 = slabs;   // the slabs to sum
  if (splits > 1) {
    split = work / n_tiles;
    work -= split * n_tiles;
    // (a split starts at an even slab: rows come two slabs at a time)
    const uint32_t pairs = uint32_t((slabs + 1) / 2), q = pairs / splits, r = pairs % splits;
    s0 = 2 * (int64_t(split) * q + (split < r ? split : r));
    if (split + 1 < splits) s1 = s0 + 2 * (q + (split < r ? 1 : 0));
  }
  const TileAt t = tile_at(work, MT, NT, p.batch > 1);
  const int64_t m0 = t.mt * TM, n0 = t.nt * kCols;
  la.init(p, p.a, nullptr, t.b * p.a_bs, p.lda, m0, p.M, s1, lane, wave);
  lb.init(p, p.b0, p.b1, t.b * p.b_bs, p.ldb, n0, p.N, s1, lane, wave);
  if constexpr (DT == kMX4) {
    ca.init(p.as, t.b * p.as_bs, p.K, m0, p.M);
    cb0.init(p.bs0, t.b * p.bs_bs, p.K, n0, p.N);
    if constexpr (EPI == kGated) cb1.init(p.bs1, t.b * p.bs_bs, p.K, n0, p.N);
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
  auto slab = [&](auto turn, int64_t s, const char* na, const char* nb, char* ta, char* tb,
                  const u32x4 (&Fc)[16], u32x4 (&Fn)[16]) {
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
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(kOpen, 0));
  };

  char* const r1 = kPairs ? a0 : a1;
  char* const r3 = kPairs ? a2 : a3;
  static_for<0, kWords>([&](auto i) { load_scale(i, 0); });
  __builtin_amdgcn_sched_barrier(0);
  issue_a(a0, kPairs ? s0 / 2 : s0);
  issue_b(b0, s0);
  if constexpr (!kPairs) issue_a(r1, s0 + 1);
  issue_b(b1, s0 + 1);
  issue_a(a2, kPairs ? s0 / 2 + 1 : s0 + 2);
  issue_b(b2, s0 + 2);
  if constexpr (!kPairs) issue_a(r3, s0 + 3);
  issue_b(b3, s0 + 3);
  take_scales();
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
  __builtin_amdgcn_s_waitcnt(waitcnt_imm((kPairs ? 1 : 2) * kLoadsA + 2 * kLoadsB, 15));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kBM + kBN; ++i) read(a0, 0, b0, F0, i);
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
  for (int64_t s = s0; s < s1; s += 4) {
    slab(std::integral_constant<int, 0>{}, s + 0, r1, b1, a0, b0, F0, F1);
    slab(std::integral_constant<int, 1>{}, s + 1, a2, b2, r1, b1, F1, F0);
    slab(std::integral_constant<int, 2>{}, s + 2, r3, b3, a2, b2, F0, F1);
    slab(std::integral_constant<int, 3>{}, s + 3, a0, b0, r3, b3, F1, F0);
    take_scales();
  }
  // No load may still be writing LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
  settle();
#pragma unroll
  for (int i = 0; i < kBM; ++i)
#pragma unroll
    for (int j = 0; j < kBN; ++j) asm volatile("" : "+a"(acc[i][j]));   // read from here on only
  const int64_t row = m0 + 16 * kBM * wm, col = n0 + (EPI == kGated ? 8 : 16) * kBN * wn;
  constexpr int kPairsN = EPI == kGated ? kBN / 4 : kBN / 2;   // 32-column pieces
  // float32 results: partial sums, and the 4-bit product's where it is asked for
  const bool wide = EPI == kStore && (DT == kMX4 ? p.out_type == BMM_ELEM_F32 : splits > 1);
  // (192 columns: 48 of H a wave, the last 16 by themselves)
  constexpr bool kLast = EPI == kGated && kBN % 4 != 0;
  u32x4 out[8][2];
  u32x2 last[8];
  if constexpr (EPI == kGated) {
    auto gate_all = [&](auto type, auto a) {
      constexpr int T = decltype(type)::value, A = decltype(a)::value;
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j)
          out[i][j] = join16<T>(gate<A>(acc[i][4 * j], acc[i][4 * j + 1]),
                                gate<A>(acc[i][4 * j + 2], acc[i][4 * j + 3]));
      if constexpr (kLast) {
#pragma unroll
        for (int i = 0; i < kBM; ++i) last[i] = pack4<T>(gate<A>(acc[i][kBN - 2], acc[i][kBN - 1]));
      }
    };
    auto gate_type = [&](auto a) {
      if constexpr (DT != kMX4) gate_all(std::integral_constant<int, DT>{}, a);
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

  // Offsets of this lane's columns in the first 16 rows; those outside are past
  // every buffer's end.
  const int64_t ld = EPI == kStore && splits > 1 ? p.N : p.ldd;
  const uint32_t row_bytes = uint32_t(ld) * (wide ? 4 : 2), step = 16 * row_bytes;
  uint32_t at[8];
  auto offsets = [&]() {
#pragma unroll
    for (int j = 0; j < (wide ? kBN : kPairsN); ++j) {
      const int c = wide ? 16 * j + 4 * g : 32 * j + 16 * (g & 1) + 8 * (g >> 1);
      at[j] = col + c < p.N ? (lane & 15) * row_bytes + (wide ? 4 : 2) * c : kOutOfRange;
    }
  };
  if constexpr (EPI == kGated) {
    auto store = [&](void* d, auto value, auto last_value) {
      const auto to = out_rows(static_cast<uint16_t*>(d) + (t.b * p.M + row) * ld + col,
                               row_bytes, p.M - row, 16 * kBM);
      offsets();
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(value(i, j), to, at[j] + i * step, 0, kNonTemporal);
      if constexpr (kLast) {
        const int c = 32 * kPairsN + 4 * g;
        const uint32_t at_last = col + c < p.N ? (lane & 15) * row_bytes + 2 * c : kOutOfRange;
#pragma unroll
        for (int i = 0; i < kBM; ++i)
          __builtin_amdgcn_raw_buffer_store_b64(last_value(i), to, at_last + i * step, 0, kNonTemporal);
      }
    };
    store(p.d, [&](int i, int j) { return out[i][j]; }, [&](int i) { return last[i]; });
    if constexpr (DT != kMX4) {
      if (p.d1) {
        store(p.d1, [&](int i, int j) { return join16<DT>(acc[i][4 * j], acc[i][4 * j + 2]); },
              [&](int i) { return pack4<DT>(acc[i][kBN - 2]); });
        store(p.d2, [&](int i, int j) { return join16<DT>(acc[i][4 * j + 1], acc[i][4 * j + 3]); },
              [&](int i) { return pack4<DT>(acc[i][kBN - 1]); });
      }
    }
  } else {
    // Rows below rows0 go to d, those from row1 (a multiple of 16) on to d1.
    const int size = wide ? 4 : 2;
    const bool parts = splits > 1;
    const char* d = parts ? reinterpret_cast<char*>(p.part + split * p.part_floats)
                          : static_cast<char*>(p.d);
    const int64_t rows = parts ? p.M : p.rows0;
    const auto to = out_rows(d + ((t.b * rows + row) * ld + col) * size, row_bytes,
                             rows - row, 16 * kBM);
    auto to1 = to;
    int second = kBM;   // first block of 16 rows that goes to d1
    if constexpr (SRCA == kTrans) {
      if (!parts && row + 16 * kBM > p.row1) {
        second = row < p.row1 ? int(p.row1 - row) / 16 : 0;
        to1 = out_rows(static_cast<char*>(p.d1) +
                           ((t.b * rows + row - p.row1) * ld + col) * size,
                       row_bytes, p.row1 + rows - row, 16 * kBM);
      }
    }
    offsets();
    auto store = [&](int i, int j, u32x4 v, auto nt) {
      __builtin_amdgcn_raw_buffer_store_b128(v, SRCA == kTrans && i >= second ? to1 : to,
                                             at[j] + i * step, 0, decltype(nt)::value);
    };
    float rescale = 1.f;
    if constexpr (DT == kF16) rescale = p.rescale ? *p.rescale : 1.f;
    auto result = [&](f32x4 acc) {
      const f32x4 v = sum(acc);
      return DT == kF16 ? v * rescale : v;
    };
    auto store16 = [&](auto type) {
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kPairsN; ++j)
          store(i, j, join16<decltype(type)::value>(result(acc[i][2 * j]), result(acc[i][2 * j + 1])),
                std::integral_constant<int, kNonTemporal>{});
    };
    auto store32 = [&](auto nt) {
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kBN; ++j) store(i, j, __builtin_bit_cast(u32x4, acc[i][j]), nt);
    };
    if constexpr (DT != kMX4) {
      if (wide) store32(std::integral_constant<int, 0>{});
      else store16(std::integral_constant<int, DT>{});
    } else {
      if (wide) store32(std::integral_constant<int, kNonTemporal>{});
      else if (p.out_type == BMM_ELEM_BF16) store16(std::integral_constant<int, kBF16>{});
      else store16(std::integral_constant<int, kF16>{});
    }
  }
}

template <int DT, int SRCA, int SRCB, int EPI, int TM, int TN>
hipError_t launch_tile_of(const TileArgs& p, hipStream_t s) {
  const int64_t cols = EPI == kGated ? TN / 2 : TN;
  const int64_t MT = (p.M + TM - 1) / TM, NT = (p.N + cols - 1) / cols;
  const int64_t n = p.batch * MT * NT;
  const int64_t splits = p.splits > 1 ? p.splits : 1;
  if (n == 0) return hipSuccess;
  if (n * splits > 0x7fffffff || NT > 1 << 28 || p.K >= int64_t(1) << 37)
    return hipErrorInvalidConfiguration;
  auto kern = ffn_tile_kernel<DT, SRCA, SRCB, EPI, TM, TN>;
  hipLaunchKernelGGL(kern, dim3(unsigned(n * splits)), dim3(kTileWaves * kWave), 0, s, p,
                     uint32_t(n), uint32_t(MT), uint32_t(NT));
  return hipGetLastError();
}

template <int DT, int SRCA, int SRCB, int EPI>
hipError_t launch_tile(const TileArgs& p, hipStream_t s) {
  switch (p.tile) {
    case kTile256: return launch_tile_of<DT, SRCA, SRCB, EPI, 256, 256>(p, s);
    case kTile256x128: return launch_tile_of<DT, SRCA, SRCB, EPI, 256, 128>(p, s);
    case kTile256x192: return launch_tile_of<DT, SRCA, SRCB, EPI, 256, 192>(p, s);
    default: return launch_tile_of<DT, SRCA, SRCB, EPI, 128, 128>(p, s);
  }
}

}  // namespace ffn
}  // namespace bmm
