// The product kernel of the feed-forward operators for few rows (tokens being
// decoded): bound by reading the weights once.
//
// A workgroup makes MR groups of 16 rows by NB blocks of 16 columns (gated: NB / 2
// blocks of both weights, alternating); its W waves share the summed axis. A wave
// streams its part of the weights from memory to registers, a round of four steps
// (32 16-bit or 128 4-bit values each) at a time: 4 NB loads of 1 KB in flight, and
// with 16 waves on a CU more than the memory needs to keep busy (8 TB/s x 1.5 us =
// 47 KB a CU). X is small, read by every workgroup and cached. The partial sums
// meet in LDS, the upper half of the waves first, then the lower half in order: the
// same result on every run.
//
// Measured on MI355X, weights cold: one token through 2 x 8192 x 4096 bf16 22.4 us =
// 6.0 TB/s, through 16384 x 16384 4-bit weights 23.7 us = 6.0 TB/s; a long read (1
// GiB and more) reaches 7.1. Eight steps at a time, 16 waves, a second set of
// registers for the next round, or loads that stay in the caches changed it by -1 to
// +4 us. 8-bit weights: 16384 x 16384 43 us = 6.2 TB/s. By groups: 64 rows of 8
// groups gated 4096 -> 8192 bf16 156-162 us = 6.6-6.9 TB/s, 14 rows of 7 with 8-bit
// weights 76 us = 6.2 TB/s.
//
// Fragments as in ffn_tile.h: lane l supplies row l % 16 and the 16 bytes of
// summed chunk l / 16, and holds D[m = l % 16][n = 4 (l / 16) .. + 3]. Loads go
// through buffers, so that lanes outside the matrices read zeros without a branch.
#pragma once

#include "ffn_tile.h"

namespace bmm {
namespace ffn {

__device__ __forceinline__ u32x4 load_at(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, int aux) {
  return aux ? __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, kNonTemporal)
             : __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0);
}

// 16 x 16 x 64 8-bit integers; the sums are whole numbers held in acc's bits.
__device__ __forceinline__ f32x4 mfma_i8(u32x4 b, u32x4 a, f32x4 acc) {
  return __builtin_bit_cast(
      f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b),
                                                   __builtin_bit_cast(i32x4, a),
                                                   __builtin_bit_cast(i32x4, acc), 0, 0, 0));
}

// Sums of two waves.
template <int DT>
__device__ __forceinline__ f32x4 add(f32x4 x, f32x4 y) {
  if constexpr (DT == kI8)
    return __builtin_bit_cast(f32x4, __builtin_bit_cast(i32x4, x) + __builtin_bit_cast(i32x4, y));
  else
    return x + y;
}

template <int DT, int EPI, int GRP, int MR, int NB, int W>
__global__ __launch_bounds__(W* kWave) void ffn_skinny_kernel(TileArgs p) {
  constexpr bool k4 = DT == kMX4;
  constexpr int kSteps = 4;                           // steps whose loads are sent together
  constexpr int kValues = k4 ? 128 : 32;              // summed values a step
  constexpr int kBytesB = k4 ? 1024 : 512;            // of a lane's row, from step to step
  constexpr int kBytesA = k4 ? 1024 : 64;
  // Whether the waves take the rounds in turns, so that together they read on in
  // each row, or each a range of its own. Measured, in turns / ranges (us, launches
  // from a graph, weights cold):
  //   rows                              1          16         32         64
  //   16 bits, 4096 -> 8192             24.1/24.8  23.8/25.4  34.2/34.0  47.0/47.4
  //   16 bits, 8192 -> 4096             26.3/27.9  27.2/28.2  38.6/38.0  47.4/48.1
  //   16 bits, 2048 -> 5464             11.2/12.3  12.4/13.5  16.4/16.7  24.0/24.7
  //   16 bits, 8192 -> 1024             14.6/14.2  17.5/17.4  31.8/31.2  41.8/41.5
  //   4-bit product, 16384 -> 16384     24.8/27.5  24.7/28.6  29.1/33.2  32.4/34.4
  //   4-bit product, 4096 -> 16384      8.5/8.5    8.6/8.6    10.5/10.3  12.5/12.5
  //   4-bit product, 8192 -> 1024       5.6/5.6    6.3/6.3    10.6/10.6  13.7/13.8
  //   4-bit gated, 8192 -> 16384        24.9/24.8  25.5/25.5  28.5/27.4  31.7/30.9
  //   4-bit gated, 4096 -> 8192         8.6/8.7    8.6/8.7    10.8/10.8  12.4/12.4
  //   4-bit gated, 2048 -> 5464         5.2/5.4    5.5/5.7    6.5/6.6    8.5/9.1
  constexpr bool kTurns = !k4 || EPI == kStore;
  // Whether the compiler is kept from moving products between a round's loads. 4-bit
  // product, kept / not: one row 16384 -> 16384 24.8/27.0 us, 8192 -> 1024 5.6/7.6;
  // 64 rows 32.4/36.6, 13.7/15.5. Gated: one row 8192 -> 16384 24.8/26.2, 8192 -> 1024
  // 6.6/7.4, but 64 rows 35.0/30.9 (registers: two waves a SIMD instead of four).
  constexpr bool kTogether = k4 && (EPI == kStore || MR == 1);
  __shared__ __attribute__((aligned(16))) f32x4 red[W / 2][MR][NB][kWave];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane & 15, g = lane >> 4;
  int64_t batch = blockIdx.z;
  int64_t m0 = int64_t(blockIdx.y) * (16 * MR);
  int64_t d_row = batch * p.M, a_off = batch * p.a_bs;   // first row of D; elements
  bool empty = false;
  if constexpr (GRP == kGroupRows) {
    Groups groups;
    groups.init(p.ends, int(p.batch), int(p.M), lane);
    const auto tiles = groups.tiles<16 * MR>(p.zero_tail);
    if (int(blockIdx.y) >= tiles.total) return;
    const Group at = groups.find<16 * MR>(tiles, int(blockIdx.y));
    empty = at.e == int(p.batch);   // the rows behind the last group: an empty sum
    batch = empty ? 0 : at.e;
    m0 = at.tile * (16 * MR);
    d_row = at.start;
    a_off = at.start * p.lda;
    p.M = at.rows;
    if (empty) p.K = 0;
  }
  const int64_t n0 = int64_t(blockIdx.x) * (EPI == kGated ? 8 : 16) * NB;
  auto column = [&](int j) { return n0 + 16 * (EPI == kGated ? j >> 1 : j); };

  // offsets of this lane's bytes in step 0 of each block, from the tile's start
  const int64_t row16_b = k4 ? (p.K + 127) / 128 * 1024 : p.K * 32;   // 16 columns
  const int64_t row16_a = k4 ? row16_b : p.lda * 32;
  const char* bases_b[2];
  bases_b[0] = static_cast<const char*>(p.b0) + (k4 ? 1 : 2) * batch * p.b_bs + n0 / 16 * row16_b;
  bases_b[1] = EPI == kGated ? static_cast<const char*>(p.b1) + (k4 ? 1 : 2) * batch * p.b_bs +
                                   n0 / 16 * row16_b
                             : bases_b[0];
  const char* const base_a =
      static_cast<const char*>(p.a) + (k4 ? 1 : 2) * a_off + m0 / 16 * row16_a;
  uint32_t ob[4], oa[4];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t col = column(j) - n0;
    const bool ok = column(j) + (k4 ? 0 : c & 8) < p.N;
    const int64_t at = k4 ? 16 * lane
                          : (c >> 3) * (p.K * 16) + (g >> 1) * 256 + (c & 7) * 32 + (g & 1) * 16;
    ob[j] = ok ? uint32_t(col / 16 * row16_b + at) : kOutOfRange;
  }
#pragma unroll
  for (int i = 0; i < MR; ++i) {
    const bool ok = m0 + 16 * i + c < p.M;
    oa[i] = ok ? uint32_t(i * row16_a + (k4 ? 16 * lane : c * p.lda * 2 + 16 * g)) : kOutOfRange;
  }
  Scales ca, cb[2];
  if constexpr (k4) {
    ca.init(p.as, batch * p.as_bs, p.K, m0, p.M);
    cb[0].init(p.bs0, batch * p.bs_bs, p.K, n0, p.N);
    if constexpr (EPI == kGated) cb[1].init(p.bs1, batch * p.bs_bs, p.K, n0, p.N);
  }

  f32x4 acc[4][4];   // MR x NB used
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int64_t rounds = (p.K + kSteps * kValues - 1) / (kSteps * kValues);
  const int64_t q0 = kTurns ? wave : wave * rounds / W, q1 = kTurns ? rounds : (wave + 1) * rounds / W;
  for (int64_t q = q0; q < q1; q += kTurns ? W : 1) {
    u32x4 fb[kSteps][4], fa[kSteps][4];
    uint32_t xa[4], xb[4];
    const auto rb0 = buffer(bases_b[0] + q * (kSteps * kBytesB));
    const auto rb1 = buffer(bases_b[1] + q * (kSteps * kBytesB));
    const auto ra = buffer(base_a + q * (kSteps * kBytesA));
    const int64_t left64 = p.K - q * (kSteps * kValues);
    const int left = int(left64 < kSteps * kValues ? left64 : kSteps * kValues);
    // The last round may be short: a lane past the end, by its first value, reads zeros.
    // (4 bits: so for X; the codes that pad the weights' K meet those zeros)
    const int first = k4 ? 0 : 8 * g, first_a = (k4 ? 32 : 8) * g;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const bool ok = u * kValues + first < left, ok_a = u * kValues + first_a < left;
#pragma unroll
      for (int j = 0; j < NB; ++j)
        fb[u][j] = load_at(EPI == kGated && (j & 1) ? rb1 : rb0,
                           ok ? ob[j] + u * kBytesB : kOutOfRange, 1);
#pragma unroll
      for (int i = 0; i < MR; ++i)
        fa[u][i] = load_at(ra, ok_a ? oa[i] + u * kBytesA : kOutOfRange, 0);
    }
    if constexpr (k4) {
#pragma unroll
      for (int i = 0; i < MR; ++i) xa[i] = ca.word(i, q, lane);
#pragma unroll
      for (int j = 0; j < NB; ++j)
        xb[j] = EPI == kGated ? cb[j & 1].word(j >> 1, q, lane) : cb[0].word(j, q, lane);
    }
    if constexpr (kTogether) __builtin_amdgcn_sched_barrier(0);
    static_for<0, kSteps>([&](auto step) {
      constexpr int u = decltype(step)::value;
#pragma unroll
      for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if constexpr (k4)
            acc[i][j] = mfma_mx4<u>(fb[u][j], fa[u][i], xb[j], xa[i], acc[i][j]);
          else if constexpr (DT == kI8)
            acc[i][j] = mfma_i8(fb[u][j], fa[u][i], acc[i][j]);
          else
            acc[i][j] = mfma_16x16x32<DT>(fb[u][j], fa[u][i], acc[i][j]);
    });
  }

  // ---- the waves' sums ----
  auto put = [&](int slot) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) red[slot][i][j][lane] = acc[i][j];
  };
  if (wave >= W / 2) put(wave - W / 2);
  __syncthreads();
  if (wave < W / 2) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = add<DT>(acc[i][j], red[wave][i][j][lane]);
    put(wave);
  }
  __syncthreads();
  auto total = [&](int i, int j, int l) {
    f32x4 v = red[0][i][j][l];
#pragma unroll
    for (int w = 1; w < W / 2; ++w) v = add<DT>(v, red[w][i][j][l]);
    return v;
  };
  auto store = [&](void* d, int64_t at, f32x4 v) {
    if (p.out_type == BMM_ELEM_F32) {
      store16f(static_cast<float*>(d) + at, v);
    } else {
      const bool bf = p.out_type == BMM_ELEM_BF16;
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(d) + at) =
          u32x2{bf ? pack2<kBF16>(v[0], v[1]) : pack2<kF16>(v[0], v[1]),
                bf ? pack2<kBF16>(v[2], v[3]) : pack2<kF16>(v[2], v[3])};
    }
  };
  constexpr int kOuts = EPI == kGated ? NB / 2 : NB;
  for (int o = threadIdx.x; o < MR * kOuts * kWave; o += W * kWave) {
    const int l = o % kWave, j = o / kWave % kOuts, i = o / kWave / kOuts;
    const int64_t m = m0 + 16 * i + (l & 15), n = n0 + 16 * j + 4 * (l >> 4);
    if (m >= p.M || n >= p.N) continue;
    const int64_t at = (d_row + m) * p.ldd + n;
    // 8-bit integers: the sums times the scales of their row and columns
    auto scaled = [&](f32x4 v, const float* sb) {
      if constexpr (DT == kI8) {
        if (empty) return v;   // zeros, whatever the tail's scales hold
        const float x = p.sa[d_row + m];
        const f32x4 y = load16f(sb + batch * p.N + n);
        const i32x4 q = __builtin_bit_cast(i32x4, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = float(q[e]) * x * y[e];
      }
      return v;
    };
    if constexpr (EPI == kGated) {
      const f32x4 gv = scaled(total(i, 2 * j, l), p.sb0), uv = scaled(total(i, 2 * j + 1, l), p.sb1);
      f32x4 h;
      switch (p.act) {
        case BMM_ACT_SILU: h = gate<BMM_ACT_SILU>(gv, uv); break;
        case BMM_ACT_GELU: h = gate<BMM_ACT_GELU>(gv, uv); break;
        case BMM_ACT_GELU_TANH: h = gate<BMM_ACT_GELU_TANH>(gv, uv); break;
        default: h = gate<BMM_ACT_RELU>(gv, uv);
      }
      store(p.d, at, h);
      if (p.d1) {
        store(p.d1, at, gv);
        store(p.d2, at, uv);
      }
    } else {
      store(p.d, at, scaled(total(i, j, l), p.sb0));
    }
  }
}

template <int DT, int EPI, int GRP, int MR, int NB, int W>
hipError_t launch_skinny_of(const TileArgs& p, hipStream_t s) {
  const int64_t cols = (EPI == kGated ? 8 : 16) * NB;
  const int64_t x = (p.N + cols - 1) / cols;
  const int64_t y = GRP == kGroupRows ? most_row_tiles(p.M, p.batch, 16 * MR)
                                      : (p.M + 16 * MR - 1) / (16 * MR);
  const int64_t z = GRP == kGroupRows ? 1 : p.batch;
  if (x > 0x7fffffff || y > 65535 || z > 65535) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((ffn_skinny_kernel<DT, EPI, GRP, MR, NB, W>),
                     dim3(unsigned(x), unsigned(y), unsigned(z)), dim3(W * kWave), 0, s, p);
  return hipGetLastError();
}

// Blocks a workgroup: two (512 workgroups for 8192 gated columns); for 4 bits and more
// than 16 rows four, so that fewer workgroups read X. Two / four, us, launches from a
// graph, weights cold:
//   rows                              24         32         48         64
//   16 bits gated, 4096 -> 8192       31.2/29.0  33.9/30.2  40.2/38.8  46.8/41.3
//   16 bits gated, 2048 -> 5464       15.4/14.2  16.5/14.9  20.8/19.8  24.1/21.1
//   16 bits gated, 8192 -> 1024       30.5/40.8  31.7/43.4  38.2/62.0  41.7/66.9
//   4-bit gated, 8192 -> 16384        29.2/27.8  30.0/28.0  38.4/30.4  40.0/31.2
//   4-bit gated, 4096 -> 8192         9.6/10.7   10.0/10.9  11.6/12.4  12.2/12.5
//   4-bit gated, 8192 -> 1024         8.2/9.9    8.3/10.5   9.8/13.9   9.9/14.2
//   4-bit product, 16384 -> 16384     28.3/29.6  29.7/30.3  38.8/32.4  38.8/33.0
//   4-bit product, 4096 -> 16384      9.4/10.3   9.8/10.5   13.8/12.1  14.6/12.6
//   4-bit product, 8192 -> 1024       7.5/10.1   7.8/10.5   9.4/12.7   10.1/13.7
// What decides is the number of workgroups more than the type. The rule by type avoids
// the largest loss of the other choice (16 bits 66.9 against 41.7, 4 bits 40.0 against
// 31.2) and costs up to a seventh on wide 16-bit blocks, two fifths on narrow 4-bit ones.
// 8 bits as 16: one row 16384 -> 16384 with its quantisation 47.8 us in two blocks by 8
// waves, 53.7 by 4 waves, 81.5 in four blocks; 14 rows of 7 groups gated 4096 -> 8192 76.4,
// 76.1 and 78.5.
template <int DT, int EPI>
hipError_t launch_skinny(const TileArgs& p, hipStream_t s) {
  constexpr int kWide = DT == kMX4 ? 4 : 2;
  if (p.M <= 16) return launch_skinny_of<DT, EPI, kWhole, 1, 2, 8>(p, s);
  if (p.M <= 32) return launch_skinny_of<DT, EPI, kWhole, 2, kWide, 8>(p, s);
  return launch_skinny_of<DT, EPI, kWhole, 4, kWide, 8>(p, s);
}

// By groups: blocks of 16 rows, or of 64 where the groups that have rows have more than
// 16 in the mean (the host does not know the groups, only T and E); but of 16 as long as
// that gives a chip that would stay half empty more workgroups. 16 / 64 (us, launches from
// a graph, weights cold):
//   rows a group                      6          12         20         32         48
//   4 x 4096 -> 1024, 128 wide        11.6/15.1  12.8/15.5  12.0/20.1  19.3/23.8  20.2/23.0
//   4 gated the same, 256             14.0/18.3  13.8/19.0  19.3/22.3  27.2/24.0  33.3/24.1
//   16 x 2048 -> 1024, 512            14.6/15.6  17.0/18.7  21.2/18.9  24.6/25.2  32.3/28.8
//   8 x 8192 -> 4096, 1024            91.5/102   115/106    163/120    230/149    302/186
// ("wide": workgroups of one block of rows a group). Blocks of 32 were never the best by
// more than 4%.
template <int DT, int EPI>
hipError_t launch_skinny_groups(const TileArgs& p, hipStream_t s) {
  const int64_t groups = p.batch < p.M ? p.batch : p.M, mean = groups > 0 ? p.M / groups : 0;
  const int64_t wide = groups * ((p.N + (EPI == kGated ? 15 : 31)) / (EPI == kGated ? 16 : 32));
  if (mean <= 16 || (mean <= 48 && wide <= 128))
    return launch_skinny_of<DT, EPI, kGroupRows, 1, 2, 8>(p, s);
  return launch_skinny_of<DT, EPI, kGroupRows, 4, 2, 8>(p, s);
}

}  // namespace ffn
}  // namespace bmm
