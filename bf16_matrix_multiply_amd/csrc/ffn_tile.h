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
// piece, so that the reads that follow are spread over all banks:
// - packed and 4-bit: the piece is a fragment in lane order;
// - rows: 16 rows x 64 bytes; the 16-byte chunk c of row r lies at chunk
//   c ^ (r / 4 % 4), so the 16 lanes that read chunk c of 16 rows meet 16
//   different bank groups;
// - transposed: [64-column block][32 summed rows][128 bytes], read with the
//   hardware's transposing LDS read (ds_read_b64_tr_b16: of 16 lanes, lane
//   4 k + a reads four columns 4a .. 4a + 3 of summed row k, and lane i
//   receives column i of the four rows). Pairs of 16-byte chunks of summed row
//   k are exchanged by k's bits 1 and 3, so that the eight rows which half a
//   wave reads lie in different banks.
// What lies outside the matrices is read as zero: such lanes are given an
// address past the buffer's end, so no memory is touched.
#pragma once

#include <type_traits>

#include "ffn.h"

namespace bmm {
namespace ffn {

enum Src : int { kRows, kTrans, kPacked2, kPackedT2, kCodes, kCodes2 };
enum Epi : int { kStore, kGated };

constexpr int kXcds = 8;
constexpr int kGroupM = 8;
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

struct TileAt {
  int64_t b, mt, nt;
};

// Linear workgroup id -> work index, each XCD taking a contiguous run.
__device__ __forceinline__ int64_t xcd_run(int64_t w, int64_t n) {
  const int64_t q = n / kXcds, r = n % kXcds;
  const int64_t xcd = w % kXcds, k = w / kXcds;
  return xcd * q + (xcd < r ? xcd : r) + k;
}

// Linear tile index -> (batch, M tile, N tile), in bands of kGroupM M tiles.
__device__ __forceinline__ TileAt tile_at(int64_t t, int64_t MT, int64_t NT) {
  const int64_t per_batch = MT * NT;
  const int64_t b = t / per_batch, u = t % per_batch;
  const int64_t group = kGroupM * NT;
  const int64_t first_m = (u / group) * kGroupM;
  const int64_t gm = MT - first_m < kGroupM ? MT - first_m : kGroupM;
  const int64_t v = u % group;
  return {b, first_m + v % gm, v / gm};
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(kOutOfRange), kBufferFlags);
}

// Bits 1 and 3 of a summed row's index within its slab: the exchange of chunk
// pairs of the transposed image.
__device__ __forceinline__ int trans_swizzle(int k) { return ((k >> 1) & 1) | ((k >> 2) & 2); }

// The loads of one operand: piece f = 4 r + wave of T / 16, r < T / 64.
template <int SRC, int T>
struct Loader {
  const char* base0;       // slab 0, source 0 (or this wave's source)
  const char* base1;       // kPackedT2: slab 0 of source 1
  int64_t step;            // bytes from slab to slab
  int64_t n_sum;           // summed values (kPackedT2: of one source)
  int64_t n_rows;          // kPackedT2: summed values that exist in one source
  int k_lane;              // this lane's first summed value within a slab
  uint32_t off[4];         // fixed size: T / 64 are used

  // r0: first row (column of D for B) of the tile; n: rows that exist.
  __device__ __forceinline__ void init(const TileArgs& p, const void* s0, const void* s1,
                                       int64_t batch_off, int64_t ld, int64_t r0, int64_t n,
                                       int lane, int wave) {
    n_sum = p.K;
    n_rows = 0;
    base1 = nullptr;
    if constexpr (SRC == kRows) {
      const int row = lane >> 2, c = (lane & 3) ^ ((lane >> 4) & 3);
      k_lane = 8 * c;
      step = 64;
      base0 = static_cast<const char*>(s0) + 2 * (batch_off + r0 * ld);
#pragma unroll
      for (int r = 0; r < T / 64; ++r) {
        const int i = 16 * (4 * r + wave) + row;
        off[r] = r0 + i < n ? uint32_t(i * ld * 2 + 16 * c) : kOutOfRange;
      }
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
      const int kk = lane >> 3;
      k_lane = 8 * wave + kk;
      const int e = (lane & 7) ^ (2 * trans_swizzle(k_lane));
      step = 64 * n;
      n_sum = p.b_sum;
      n_rows = p.b_rows;
      base0 = static_cast<const char*>(s0) + 2 * batch_off + 16 * r0;
      base1 = static_cast<const char*>(s1) + 2 * batch_off + 16 * r0;
#pragma unroll
      for (int r = 0; r < T / 64; ++r)
        off[r] = r0 + 64 * r + 8 * e < n
                     ? uint32_t(wave * n * 16 + (4 * r + (e >> 1)) * 256 + kk * 32 + (e & 1) * 16)
                     : kOutOfRange;
    } else if constexpr (SRC == kPacked2) {
      const int c = lane & 15, g = lane >> 4;
      k_lane = 8 * g;
      step = 512;
      base0 = static_cast<const char*>(wave & 1 ? s1 : s0) + 2 * (batch_off + r0 * p.K);
#pragma unroll
      for (int r = 0; r < T / 64; ++r) {
        const int cb = 2 * r + (wave >> 1);   // 16-column block of this piece
        off[r] = r0 + 16 * cb + (c & 8) < n
                     ? uint32_t((2 * cb + (c >> 3)) * p.K * 16 + (g >> 1) * 256 + (c & 7) * 32 +
                                (g & 1) * 16)
                     : kOutOfRange;
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

  // Slab k into the operand's stage (T / 16 pieces of 1 KB).
  __device__ __forceinline__ void issue(char* stage, int64_t k, int wave) const {
    constexpr int kValues = slab_values(SRC);
    bool ok;
    const char* at;
    if constexpr (SRC == kPackedT2) {
      const int64_t per = n_sum / 32;
      const int64_t j = k < per ? k : k - per;
      at = (k < per ? base0 : base1) + j * step;
      ok = k < 2 * per && 32 * j + k_lane < n_rows;
    } else {
      at = base0 + k * step;
      ok = kValues * k + k_lane < n_sum;
    }
    const __amdgpu_buffer_rsrc_t rsrc = buffer(at);
#pragma unroll
    for (int r = 0; r < T / 64; ++r)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(stage + 1024 * (4 * r + wave)),
                                               16, ok ? off[r] : kOutOfRange, 0, 0, 0);
  }
};

// This lane's 16 bytes of fragment f (rows 16 f .. of the tile) in a stage.
template <int SRC>
struct Reader {
  int base;       // byte offset of the lane within a piece
  int pair[4];    // transposed: the four exchanges of chunk pairs

  __device__ __forceinline__ void init(int lane) {
    if constexpr (SRC == kRows) {
      const int m = lane & 15;
      base = 16 * (4 * m + ((lane >> 4) ^ ((m >> 2) & 3)));
    } else if constexpr (SRC == kTrans || SRC == kPackedT2) {
      const int i = lane & 15, k = 8 * (lane >> 4) + (i >> 2), a = i & 3;
      base = 128 * k + 16 * (a >> 1) + 8 * (a & 1);
#pragma unroll
      for (int b = 0; b < 4; ++b) pair[b] = 32 * (b ^ trans_swizzle(k));
    } else {
      base = 16 * lane;
    }
  }

  __device__ __forceinline__ u32x4 read(const char* stage, int f) const {
    if constexpr (SRC == kTrans || SRC == kPackedT2) {
      const char* at = stage + 4096 * (f >> 2) + pair[f & 3] + base;
      const u32x2 lo = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at));
      const u32x2 hi = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(at + 512)));
      return u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      return *(const volatile lds_u32x4*)(stage + 1024 * f + base);
    }
  }
};

// Scales of 16-row group r16 for four slabs: one word a lane.
__device__ __forceinline__ const uint32_t* scale_words(const uint8_t* scales, int64_t batch_off,
                                                       int64_t K, int64_t r16, int lane) {
  return reinterpret_cast<const uint32_t*>(scales + batch_off +
                                           r16 * ((K + 511) / 512) * 256) + lane;
}

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 b, u32x4 a, f32x4 acc) {
  return mfma_16x16x32<DT>(b, a, acc);
}
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

// Writes blocks (v0, v1) at columns col0 .. col0 + 31 of the row at `row`
// (null: the row does not exist), as out_type; n: columns that exist (a
// multiple of 8).
__device__ __forceinline__ void store_pair(void* row, int64_t col0, int64_t n, int out_type,
                                           f32x4 v0, f32x4 v1, int g) {
  if (out_type == BMM_ELEM_F32) {
    const int64_t c = col0 + 4 * g;
    float* at = static_cast<float*>(row) + c;
    if (row && c < n) store16f(at, v0);
    if (row && c + 16 < n) store16f(at + 16, v1);
  } else {
    const u32x4 o = out_type == BMM_ELEM_BF16 ? join16<kBF16>(v0, v1) : join16<kF16>(v0, v1);
    const int64_t c = col0 + 16 * (g & 1) + 8 * (g >> 1);
    if (row && c < n) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(row) + c) = o;
  }
}

template <int ACT>
__device__ __forceinline__ f32x4 gate(f32x4 g, f32x4 u) {
  f32x4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = act<ACT>(g[i]) * u[i];
  return h;
}

// Row pointer of an output of the given type, or null where the row is outside.
__device__ __forceinline__ char* row_at(void* d, int64_t row, int64_t ld, int out_type, bool ok) {
  const int64_t bytes = out_type == BMM_ELEM_F32 ? 4 : 2;
  return ok ? static_cast<char*>(d) + row * ld * bytes : nullptr;
}

template <int ACT>
__device__ __forceinline__ void gated_blocks(const TileArgs& p, int64_t b, int64_t m, int64_t col0,
                                             const f32x4 (&acc)[8], int blocks, int g) {
  const bool ok = m < p.M;
  const int64_t row = b * p.M + m;
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    if (j >= blocks) break;
    const int64_t c = col0 + 8 * j;
    store_pair(row_at(p.d, row, p.ldd, p.out_type, ok), c, p.N, p.out_type,
               gate<ACT>(acc[j], acc[j + 1]), gate<ACT>(acc[j + 2], acc[j + 3]), g);
    if (p.d1) {
      store_pair(row_at(p.d1, row, p.ldd, p.out_type, ok), c, p.N, p.out_type, acc[j], acc[j + 2], g);
      store_pair(row_at(p.d2, row, p.ldd, p.out_type, ok), c, p.N, p.out_type, acc[j + 1],
                 acc[j + 3], g);
    }
  }
}

template <int DT, int SRCA, int SRCB, int EPI, int TM, int TN>
__global__ __launch_bounds__(kTileWaves* kWave) void ffn_tile_kernel(TileArgs p, int64_t n_tiles,
                                                                     int64_t MT, int64_t NT) {
  constexpr int kBM = TM / 32, kBN = TN / 32;   // 16-row and 16-column blocks a wave
  constexpr int kCols = EPI == kGated ? TN / 2 : TN;   // columns of D a tile
  static_assert((EPI == kGated) == two_sources(SRCB), "gated: two sources of B");
  __shared__ __attribute__((aligned(1024))) char sa[TM * 64], sb[TN * 64];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4;
  const int64_t splits = p.splits > 1 ? p.splits : 1;
  const int64_t work = xcd_run(int64_t(blockIdx.y) * n_tiles + blockIdx.x, n_tiles * splits);
  const int64_t split = work / n_tiles;
  const TileAt t = tile_at(work % n_tiles, MT, NT);
  const int64_t m0 = t.mt * TM, n0 = t.nt * kCols;

  Loader<SRCA, TM> la;
  Loader<SRCB, TN> lb;
  la.init(p, p.a, nullptr, t.b * p.a_bs, p.lda, m0, p.M, lane, wave);
  lb.init(p, p.b0, p.b1, t.b * p.b_bs, p.ldb, n0, p.N, lane, wave);
  Reader<SRCA> ra;
  Reader<SRCB> rb;
  ra.init(lane);
  rb.init(lane);

  f32x4 acc[8][8];   // [16-row block][16-column block], kBM x kBN used
#pragma unroll
  for (int i = 0; i < kBM; ++i)
#pragma unroll
    for (int j = 0; j < kBN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // 4-bit: where this wave's scale words start, one pointer a 16-row group
  // (groups outside read the last one; their outputs are not stored)
  const uint32_t* wa[8];
  const uint32_t* wb[8];
  if constexpr (DT == kMX4) {
#pragma unroll
    for (int i = 0; i < kBM; ++i) {
      const int64_t r = m0 / 16 + kBM * wm + i, last = (p.M + 15) / 16 - 1;
      wa[i] = scale_words(p.as, t.b * p.as_bs, p.K, r < last ? r : last, lane);
    }
#pragma unroll
    for (int j = 0; j < kBN; ++j) {
      const int cb = EPI == kGated ? (kBN * wn + j) >> 1 : kBN * wn + j;
      const int64_t r = n0 / 16 + cb, last = (p.N + 15) / 16 - 1;
      wb[j] = scale_words(EPI == kGated && (j & 1) ? p.bs1 : p.bs0, t.b * p.bs_bs, p.K,
                          r < last ? r : last, lane);
    }
  }

  constexpr int kValues = slab_values(SRCA);
  const int64_t slabs = (p.K + kValues - 1) / kValues;
  const int64_t s0 = split * slabs / splits, s1 = (split + 1) * slabs / splits;
  for (int64_t s = s0; s < s1; ++s) {
    la.issue(sa, s, wave);
    lb.issue(sb, s, wave);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
    __syncthreads();
    u32x4 fa[8], fb[8];
#pragma unroll
    for (int i = 0; i < kBM; ++i) fa[i] = ra.read(sa, kBM * wm + i);
#pragma unroll
    for (int j = 0; j < kBN; ++j) fb[j] = rb.read(sb, kBN * wn + j);
    if constexpr (DT == kMX4) {
      uint32_t xa[8], xb[8];
      const int shift = 8 * int(s & 3);
#pragma unroll
      for (int i = 0; i < kBM; ++i) xa[i] = wa[i][(s >> 2) * 64] >> shift;
#pragma unroll
      for (int j = 0; j < kBN; ++j) xb[j] = wb[j][(s >> 2) * 64] >> shift;
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kBN; ++j)
          acc[i][j] = mfma_mx4<0>(fb[j], fa[i], xb[j], xa[i], acc[i][j]);
    } else {
#pragma unroll
      for (int i = 0; i < kBM; ++i)
#pragma unroll
        for (int j = 0; j < kBN; ++j) acc[i][j] = mfma<DT>(fb[j], fa[i], acc[i][j]);
    }
    __syncthreads();
  }

  const int64_t wave_m = m0 + 16 * kBM * wm + (lane & 15);
  if constexpr (EPI == kGated) {
    const int64_t col0 = n0 + 8 * kBN * wn;
    auto rows = [&](auto a) {
#pragma unroll
      for (int i = 0; i < kBM; ++i)
        gated_blocks<decltype(a)::value>(p, t.b, wave_m + 16 * i, col0, acc[i], kBN, g);
    };
    switch (p.act) {
      case BMM_ACT_SILU: rows(std::integral_constant<int, BMM_ACT_SILU>{}); break;
      case BMM_ACT_GELU: rows(std::integral_constant<int, BMM_ACT_GELU>{}); break;
      case BMM_ACT_GELU_TANH: rows(std::integral_constant<int, BMM_ACT_GELU_TANH>{}); break;
      default: rows(std::integral_constant<int, BMM_ACT_RELU>{});
    }
  } else {
    const int64_t col0 = n0 + 16 * kBN * wn;
#pragma unroll
    for (int i = 0; i < kBM; ++i) {
      const int64_t m = wave_m + 16 * i;
      char* row;
      int out_type = p.out_type;
      if (splits > 1) {
        row = m < p.M ? reinterpret_cast<char*>(p.part + split * p.part_floats +
                                                (t.b * p.M + m) * p.N)
                      : nullptr;
        out_type = BMM_ELEM_F32;
      } else if (m < p.rows0) {
        row = row_at(p.d, t.b * p.rows0 + m, p.ldd, out_type, true);
      } else {
        const int64_t r = m - p.row1;
        row = row_at(p.d1, t.b * p.rows0 + r, p.ldd, out_type, r >= 0 && r < p.rows0);
      }
#pragma unroll
      for (int j = 0; j < kBN; j += 2)
        store_pair(row, col0 + 16 * j, p.N, out_type, acc[i][j], acc[i][j + 1], g);
    }
  }
}

template <int DT, int SRCA, int SRCB, int EPI, int TM, int TN>
hipError_t launch_tile(const TileArgs& p, hipStream_t s) {
  const int64_t cols = EPI == kGated ? TN / 2 : TN;
  const int64_t MT = (p.M + TM - 1) / TM, NT = (p.N + cols - 1) / cols;
  const int64_t n = p.batch * MT * NT;
  if (n > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (n == 0) return hipSuccess;
  auto kern = ffn_tile_kernel<DT, SRCA, SRCB, EPI, TM, TN>;
  hipLaunchKernelGGL(kern, dim3(unsigned(n), unsigned(p.splits > 1 ? p.splits : 1)),
                     dim3(kTileWaves * kWave), 0, s, p, n, MT, NT);
  return hipGetLastError();
}

}  // namespace ffn
}  // namespace bmm
