// The backward pass of H = act(G) * U, G = X Wg^T, U = X Wu^T:
//   dG = dH U act'(G),  dU = dH act(G)
//   dX = dG Wg + dU Wu = [dG | dU] [Wg ; Wu]
//   dWg = dG^T X, dWu = dU^T X: [dG | dU]^T X
//
// One pass makes [dG | dU] (16 bits a value), then two products read it: dX
// along its rows, the weight gradients along its columns. Rounding dG and dU
// to the operands' type is what lets the matrix cores multiply them; the error
// it adds to a gradient (a half step of each of many independent terms) is the
// size of that gradient's own last rounding. For f16 that holds only inside its
// range (2^-14 to 65504), which products of three f16 values leave on both
// sides: a pass before finds the largest finite magnitude of dG and dU, both are
// multiplied by the power of two that brings it to [2^14, 2^15), and the products
// take that out of their float32 sums, which is exact. Values down to 2^-28 of the
// largest then keep all their digits, and what vanishes is below 2^-39 of it. No
// operand is transposed or repacked in memory: the products read X, [dG | dU]
// and the packed weights through the transposing LDS reads.
#include "ffn_split.h"

namespace bmm {
namespace {

constexpr int kThreads = 256;

// dG and dU of 8 columns in one row, at element `at` of dH, G and U: fn(w, e, dG, dU)
// for the values of each word.
template <int DT, int ACT, class Fn>
__device__ __forceinline__ void slopes_of_eight(const uint16_t* dh, const uint16_t* g,
                                                const uint16_t* u, int64_t at, Fn fn) {
  const u32x4 vh = *reinterpret_cast<const u32x4*>(dh + at);
  const u32x4 vg = *reinterpret_cast<const u32x4*>(g + at);
  const u32x4 vu = *reinterpret_cast<const u32x4*>(u + at);
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t sh = 16 * e;
      const float h = half_bits_to_f32<DT>((vh[w] >> sh) & 0xffffu);
      const float x = half_bits_to_f32<DT>((vg[w] >> sh) & 0xffffu);
      const float y = half_bits_to_f32<DT>((vu[w] >> sh) & 0xffffu);
      float a, slope;
      act_and_slope<ACT>(x, a, slope);
      fn(w, e, h * y * slope, h * a);
    }
}

// The largest of the workgroup's values, in every thread.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
  __shared__ uint32_t of_wave[kThreads / kWave];
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) x = umax(x, uint32_t(__shfl_xor(int(x), d, kWave)));
  if (threadIdx.x % kWave == 0) of_wave[threadIdx.x / kWave] = x;
  __syncthreads();
  x = of_wave[0];
#pragma unroll
  for (int w = 1; w < kThreads / kWave; ++w) x = umax(x, of_wave[w]);
  return x;
}

// n items, per_row a row, of which those of the groups' rows count (what lies behind the
// last group is not read). Every lane of the wave takes part.
__device__ __forceinline__ int64_t rows_until(GroupEnds ends, int64_t n, int64_t per_row) {
  if (!ends.at) return n;
  return ffn::rows_of_groups(ends.at, ends.groups, ends.rows, threadIdx.x % kWave) * per_row;
}

// The largest finite magnitude of dG and dU that each workgroup meets, as float32
// bits (which are ordered like the values). Bound by memory: 8192 x 8192 72-79 us = 5.1-5.6
// TB/s; of the whole backward pass 45 x 528 -> 1368 3 of 26 us, 32773 x 512 -> 1024
// 37-45 of 238.
template <int DT, int ACT>
__global__ __launch_bounds__(kThreads) void peaks_kernel(uint32_t* __restrict__ peaks,
                                                         const uint16_t* __restrict__ dh,
                                                         const uint16_t* __restrict__ g,
                                                         const uint16_t* __restrict__ u, int64_t n,
                                                         int64_t F, int64_t ld,
                                                         GroupEnds ends) {
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  const int64_t per_row = F / 8;
  n = rows_until(ends, n, per_row);
  uint32_t top = 0;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {
    const int64_t row = i / per_row, f = 8 * (i % per_row);
    slopes_of_eight<DT, ACT>(dh, g, u, row * ld + f, [&](int, int, float dg, float du) {
      const uint32_t a = __builtin_bit_cast(uint32_t, dg) & 0x7fffffffu;
      const uint32_t b = __builtin_bit_cast(uint32_t, du) & 0x7fffffffu;
      top = umax(top, umax(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
    });
  }
  top = block_max(top);
  if (threadIdx.x == 0) peaks[blockIdx.x] = top;
}

// One thread: 8 columns of dG and of dU in one row. Read dH, G and U once, write
// both halves: 10 bytes a column. Bound by memory: 8192 x 8192 113 us = 5.9 TB/s.
// f16: the values are scaled as above by the largest of n_peaks peaks, and rescale
// receives the factor that undoes it.
template <int DT, int ACT>
__global__ __launch_bounds__(kThreads) void slopes_kernel(uint16_t* __restrict__ dgu,
                                                          const uint16_t* __restrict__ dh,
                                                          const uint16_t* __restrict__ g,
                                                          const uint16_t* __restrict__ u,
                                                          int64_t n, int64_t F, int64_t Fp,
                                                          int64_t ld,
                                                          GroupEnds ends,
                                                          const uint32_t* __restrict__ peaks,
                                                          int n_peaks,
                                                          float* __restrict__ rescale) {
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  const int64_t per_row = Fp / 8;
  n = rows_until(ends, n, per_row);
  float scale = 1.f;
  if constexpr (DT == kF16) {
    uint32_t top = 0;
    for (int i = threadIdx.x; i < n_peaks; i += kThreads) top = umax(top, peaks[i]);
    top = block_max(top);
    // 2^k with k = 14 - floor(log2 top); held at 2^126, so that 2^-k is a normal float
    // (f16 operands give -18 at the least)
    const int k = 14 + 127 - int(top >> 23), held = k < 126 ? k : 126;
    scale = __builtin_bit_cast(float, uint32_t(127 + held) << 23);
    if (blockIdx.x == 0 && threadIdx.x == 0)
      *rescale = __builtin_bit_cast(float, uint32_t(127 - held) << 23);
  }
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += stride) {
    const int64_t row = i / per_row, f = 8 * (i % per_row);
    u32x4 og = {0, 0, 0, 0}, ou = {0, 0, 0, 0};
    if (f < F) {
      float dg[4][2], du[4][2];
      slopes_of_eight<DT, ACT>(dh, g, u, row * ld + f, [&](int w, int e, float a, float b) {
        dg[w][e] = DT == kF16 ? a * scale : a;
        du[w][e] = DT == kF16 ? b * scale : b;
      });
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        og[w] = pack2<DT>(dg[w][0], dg[w][1]);
        ou[w] = pack2<DT>(du[w][0], du[w][1]);
      }
    }
    uint16_t* out = dgu + row * 2 * Fp + f;
    *reinterpret_cast<u32x4*>(out) = og;
    *reinterpret_cast<u32x4*>(out + Fp) = ou;
  }
}

unsigned grid_for(int64_t n) {
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  return unsigned(blocks < 8192 ? blocks : 8192);
}

}  // namespace

int64_t gated_peaks(int64_t rows, int64_t F) {
  const int64_t blocks = (rows * F / 8 + kThreads - 1) / kThreads;
  return blocks < 1024 ? blocks : 1024;   // four workgroups a CU keep the memory busy
}

hipError_t launch_gated_slopes(uint16_t* dgu, const uint16_t* dh, const uint16_t* g,
                               const uint16_t* u, int64_t rows, int64_t F, int64_t ld, int dtype,
                               int act, GroupEnds ends, uint32_t* peaks, float* rescale,
                               hipStream_t s) {
  const int64_t Fp = (F + 31) / 32 * 32, n = rows * Fp / 8;
  if (n == 0) return hipSuccess;
  auto by_act = [&](auto fn) {
    switch (act) {
      case BMM_ACT_SILU: return fn(std::integral_constant<int, BMM_ACT_SILU>{});
      case BMM_ACT_GELU: return fn(std::integral_constant<int, BMM_ACT_GELU>{});
      case BMM_ACT_GELU_TANH: return fn(std::integral_constant<int, BMM_ACT_GELU_TANH>{});
      default: return fn(std::integral_constant<int, BMM_ACT_RELU>{});
    }
  };
  const int n_peaks = int(gated_peaks(rows, F));
  if (dtype == kF16) {
    hipLaunchKernelGGL(by_act([](auto a) { return peaks_kernel<kF16, decltype(a)::value>; }),
                       dim3(unsigned(n_peaks)), dim3(kThreads), 0, s, peaks, dh, g, u, rows * F / 8,
                       F, ld, ends);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  auto kern = dtype == kBF16 ? by_act([](auto a) { return slopes_kernel<kBF16, decltype(a)::value>; })
                             : by_act([](auto a) { return slopes_kernel<kF16, decltype(a)::value>; });
  hipLaunchKernelGGL(kern, dim3(grid_for(n)), dim3(kThreads), 0, s, dgu, dh, g, u, n, F, Fp, ld, ends,
                     peaks, n_peaks, rescale);
  return hipGetLastError();
}

hipError_t launch_gated_dx(const TileArgs& a, int dtype, hipStream_t s) {
  return dtype == kBF16 ? ffn::product<kBF16, ffn::kRows, ffn::kPackedT2>(a, s)
                        : ffn::product<kF16, ffn::kRows, ffn::kPackedT2>(a, s);
}

hipError_t launch_gated_dw(const TileArgs& a, int dtype, hipStream_t s) {
  return dtype == kBF16 ? ffn::product<kBF16, ffn::kTrans, ffn::kTrans>(a, s)
                        : ffn::product<kF16, ffn::kTrans, ffn::kTrans>(a, s);
}

hipError_t launch_grouped_dx(const TileArgs& a, int dtype, hipStream_t s) {
  return dtype == kBF16 ? ffn::product<kBF16, ffn::kRows, ffn::kPackedT2, ffn::kGroupRows>(a, s)
                        : ffn::product<kF16, ffn::kRows, ffn::kPackedT2, ffn::kGroupRows>(a, s);
}

hipError_t launch_grouped_both(const TileArgs& dx, const TileArgs& dw, int dtype, hipStream_t s) {
  return dtype == kBF16 ? ffn::both_gradients<kBF16>(dx, dw, s)
                        : ffn::both_gradients<kF16>(dx, dw, s);
}

hipError_t launch_grouped_dw(const TileArgs& a, int dtype, hipStream_t s) {
  return dtype == kBF16 ? ffn::product<kBF16, ffn::kTrans, ffn::kTrans, ffn::kGroupSums>(a, s)
                        : ffn::product<kF16, ffn::kTrans, ffn::kTrans, ffn::kGroupSums>(a, s);
}

// The plan that a simple model finds fastest. A tile of each size takes so many
// nanoseconds a slab and so many besides (its first loads and its results) on a full
// chip (256 workgroups; 128 x 128: 512). The tiles run in rounds; one that fills a
// share f of the chip takes a + (1 - a) f of a full one, with another a for the first
// round than for a later one, which starts while the one before it ends. Split sums are
// written and read once, 8 bytes at 5 TB/s, and joined by one more launch. The
// constants are a fit to 60 products measured on MI355X (16-bit and 4-bit, 200 to 32773
// rows): 7% off in the mean, and within 3% of the fastest size in all but two. For
// example gated K = 2048 -> 5464 by tiles of 128 x 128, 256 x 128, 256 x 192 and 256 x
// 256: 777 rows 45.5, 52.3, 39.0 and 43.2 us, 1500 rows 70, 83, 77 and 92, 4095 rows
// 163, 172, 164 and 148; the weight gradients of 32773 x 512 -> 1024 by 128 x 128 tiles
// 258 us, by 256 x 128 tiles and 8 splits 72. Of 98 products and gated blocks of 8-bit
// integers (80 to 8192 rows, 1024 -> 4096 to 14336 -> 4096), which it does not tell
// from 16-bit ones of as many slabs, it takes a size within 3% of the fastest in 94, at
// worst 10% off. Outside of those products it is rougher. Below 128 rows it expects too
// little (96 x 4096 -> 8192: 38 us, measured 45), without a worse choice. It does not
// know that a gated call keeps its projections: where the sum is short, 128 x 128 tiles
// are then often the better ones (kept, 4096 x 256 -> 4096: 47 us, chosen 256 x 256 56;
// 16384 x 256 -> 2048: 83, chosen 97; but 8192 x 256 -> 8192: 230, chosen 159), and 256
// x 192 tiles, which write the last columns in pieces of 32 bytes, the slowest (369
// there).
namespace {

// row_tiles(tm): tiles of tm rows; most(tm): as many at most; outputs: values that a split
// sum is held in. A size whose tiles are more than one launch may have is not taken.
// The first so many sizes. `extra`: nanoseconds of a tile of each size besides those of its slabs that are added.
template <class Fn, class Most>
TilePlan plan_of(Fn row_tiles, Most most, int64_t N, int64_t slabs, double outputs, bool may_split,
                 const double (&extra)[4], int sizes = 4) {
  struct Size {
    int64_t tm, tn, places;
    double slab, besides, first, later;
  };
  static constexpr Size kSizes[] = {{128, 128, 512, 475, 3600, .45, .08},
                                    {256, 128, 256, 418, 4900, .74, .60},
                                    {256, 192, 256, 525, 7900, .77, .87},
                                    {256, 256, 256, 672, 9300, .77, .56}};
  static constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
  TilePlan best{kTile128, 1, 0};
  bool any = false;
  for (int size = 0; size < sizes; ++size) {
    const Size& z = kSizes[size];
    const double cols = double((N + z.tn - 1) / z.tn), tiles = row_tiles(z.tm) * cols;
    for (int splits : kSplits) {
      if (splits > 1 && (!may_split || slabs / splits < 8)) break;
      if (most(z.tm) * cols * splits + 128 > kMaxWorkgroups) break;   // (128: tiles in halves)
      const double tile = double((slabs + splits - 1) / splits) * z.slab + z.besides + extra[size];
      const double fill = tiles * splits / z.places, rounds = fill < 1e12 ? double(int64_t(fill)) : fill;
      const double a = rounds > 0 ? z.later : z.first;
      double cost = rounds * tile;
      if (fill > rounds) cost += tile * (a + (1 - a) * (fill - rounds));
      if (splits > 1) cost += 4000 + 8e-3 / 5 * splits * outputs;
      if (!any || cost < best.ns) best = {size, splits, cost};
      any = true;
    }
  }
  return best;
}

constexpr double kNoExtra[4] = {0, 0, 0, 0};

}  // namespace

TilePlan plan_tiles(int64_t batch, int64_t M, int64_t N, int64_t slabs, bool may_split) {
  auto row_tiles = [&](int64_t tm) { return double(batch) * ((M + tm - 1) / tm); };
  return plan_of(row_tiles, row_tiles, N, slabs, double(batch) * M * N, may_split, kNoExtra);
}

// The host knows T rows and E groups, not how the rows fall on them: groups that have
// rows have n in the mean, and the last tile of one is half full. Of 78 8-bit products and
// gated blocks by groups that differ by half in size (400 rows of 8 to 24576 of 64) the size
// is within 3% of the fastest in 62 and 2.8% off in the mean; worst where few columns make
// few tiles: 16384 rows of 4 groups, 4320 -> 416, by 128 x 128 tiles 57 us, by 256 x 192 42.
TilePlan plan_group_rows(int64_t E, int64_t T, int64_t N, int64_t slabs, bool may_split) {
  const double some = double(E < T ? E : T), n = some > 0 ? T / some : 0;
  auto row_tiles = [&](int64_t tm) {
    const double tiles = n / tm + (E > 1 ? 0.5 : 0);
    return some * (tiles > 1 ? tiles : 1);
  };
  auto most = [&](int64_t tm) { return double(ffn::most_row_tiles(T, E, tm)); };
  return plan_of(row_tiles, most, N, slabs, double(T) * N, may_split, kNoExtra);
}

// Sums over the rows of E groups of T. Their many results make the difference between the
// sizes: 24576 rows of 64 groups, 2048 x 1408, by tiles of 128 x 128, 256 x 128, 256 x 192
// and 256 x 256: 252, 251, 232 and 211 us; 16384 rows of 16 groups, 8192 x 2048: 694, 643,
// 559 and 529 us. Of 55 sums (1 to 128 groups, 2000 to 32768 rows, 512 x 1024 to 4096 x 4096)
// the plan is within 3% of the fastest size in 40 and 2.9% off in the mean; worst 8192 rows
// of 32 groups, 2048 x 2048, by 256 x 256 tiles 144 us, by 256 x 192 118, and 512 x 1024 27,
// by 128 x 128 22.
TilePlan plan_group_sums(int64_t E, int64_t T, int64_t M, int64_t N, bool small) {
  static constexpr double kExtra[4] = {2300, 1100, 500, 700};
  auto row_tiles = [&](int64_t tm) { return double(E) * ((M + tm - 1) / tm); };
  const int64_t slabs = E > 0 ? (T + 32 * E - 1) / (32 * E) : 0;   // of the mean group
  auto most = [](int64_t) { return 0.0; };   // (a workgroup makes as many as there are)
  return plan_of(row_tiles, most, N, slabs, double(E) * M * N, true, kExtra, small ? 1 : 4);
}

// Few rows: the weights are read once for up to 64 rows. Few-rows kernel / 128 x 128
// tiles, the better of the others (us, launches from a graph, weights cold):
//   rows                             33         48         64         65         128
//   gated 4096 -> 8192, 16 bits      34.2/43.1  41.0/43.1  47.8/43.5  66.7/43.9  88.3/46.6
//   gated 2048 -> 5464, 16 bits      18.0/21.7  21.2/21.8  24.4/21.9  29.6/21.9  34.7/22.7
//   gated 8192 -> 1024, 16 bits      35.4/69.6  38.7/69.6  41.8/69.9  40.9/70.0  41.2/73.1
//   gated 4096 -> 512, 16 bits       18.9/27.7  20.3/27.7  22.3/27.7  21.3/27.7  21.8/28.0
//   gated 4096 -> 8192, 4 bits       12.8/13.6  12.9/13.6  13.0/13.7  17.3/13.8  18.0/14.3
//   gated 8192 -> 1024, 4 bits       13.9/18.4  13.9/18.5  14.0/18.6  13.0/18.5  13.6/18.7
//   product 16384 -> 16384, 4 bits   33.1/47.6  33.5/42.3  33.4/43.1  57.1/43.3  61.6/46.4
// One limit for all: a wide 16-bit block would change at 56 rows (a tenth at 64), and a
// narrow one, whose tiles leave most of the chip empty, not before 256.
int plan_forward(int64_t batch, int64_t M, int64_t N, int64_t slabs) {
  if (M <= 64 && batch <= 65535) return kSkinny;
  return plan_tiles(batch, M, N, slabs, false).tile;
}

// By groups: up to which rows a group (in the mean) the few-rows kernel is the faster
// one goes by how much of the chip tiles of 128 x 128 would fill. Few-rows kernel, the
// better of its two blocks / the best tiles (us, launches from a graph, weights cold):
//   rows a group                      6           12          20          48          96
//   32 tiles: 4 x 4096 -> 1024        11.6/38.6   12.8/38.8   12.0/39.0   20.2/39.2   25.8/39.5
//   64 tiles: 4 gated the same        14.0/39.3   13.8/39.8   19.3/39.8   24.1/39.9   44.7/40.5
//   128 tiles: 16 x 2048 -> 1024      14.6/22.6   17.0/22.9   18.9/23.0   28.8/24.1   43.9/25.0
//   256 tiles: 8 x 8192 -> 4096       91.5/110    106/113     119/117     186/123     327/149
//   512 tiles: 8 x 4096 -> 8192       87.0/93.4   101/92.3    113/93.3    172/97.5    325/123
//   1024 tiles: 64 x 1408 -> 2048     62.4/66.3   80.2/67.9   91.7/69.9   131/78.1    219/89.1
// and with 8-bit operands alike (8 x 4096 -> 8192: 43.2/48.6, 52.8/47.9, 56.1/48.9). The
// groups there differ by half in size, and one with more than 16 rows reads its weight
// twice. Where tiles fill the chip, the few-rows kernel's time over the best tiles' with
// such groups and with equal ones:
//   rows a group                      7          8          10         11         14
//   512 tiles: 8 x 4096 -> 8192       0.85/0.86  0.96/0.86  0.97/0.87  1.08/0.88  1.09/0.92
//   512 tiles: 16 x 2048 -> 4096      0.90/0.89  0.93/0.88  1.03/0.89  0.95/0.89  1.13/0.92
//   1024 tiles: 8 gated 4096 -> 8192  0.92/0.92  1.03/0.92  1.02/0.91  1.13/0.91  1.13/0.92
//   1024 tiles: 64 x 1408 -> 2048     0.86/0.85  0.88/0.85  0.96/0.87  0.99/0.91  1.14/0.98
//   1408 tiles: 64 gated 2048 -> 1408 0.94/0.96  0.99/0.97  1.05/0.97  1.06/0.98  1.16/0.97
//   8 bits, 8 x 4096 -> 8192          0.86/0.87  0.95/0.85  0.96/0.87  1.04/0.87  1.04/0.89
//   8 bits, 8 gated 4096 -> 8192      0.93/0.94  1.04/0.93  1.04/0.94  1.13/0.94  1.14/0.95
// With different groups the two are even at 8 to 11 rows, with equal ones the few-rows
// kernel stays ahead: up to 10 rows are its own everywhere, which costs at most 5%, and
// beyond them equal groups pay up to 15%. Rows behind the last group count among a
// group's (the host cannot tell them): 64 rows of 8 groups gated 4096 -> 8192 take 158 us
// with a tail of 16 and 183 with one of 24.
int plan_group_forward(int64_t E, int64_t T, int64_t N, int64_t slabs) {
  const int64_t some = E < T ? E : T, tiles = some * ((N + 127) / 128);
  if (tiles > 0) {
    const int64_t rows = 4096 / tiles, limit = rows < 10 ? 10 : rows > 96 ? 96 : rows;
    if (T / some <= limit && T / 16 + some < 65535) return kSkinny;
  }
  return plan_group_rows(E, T, N, slabs, false).tile;
}

}  // namespace bmm
