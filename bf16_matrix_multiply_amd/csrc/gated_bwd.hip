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
#include "ffn_tile.h"

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

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

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

// The largest finite magnitude of dG and dU that each workgroup meets, as float32
// bits (which are ordered like the values). Bound by memory: 8192 x 8192 72-79 us = 5.1-5.6
// TB/s; of the whole backward pass 45 x 528 -> 1368 3 of 26 us, 32773 x 512 -> 1024
// 37-45 of 238.
template <int DT, int ACT>
__global__ __launch_bounds__(kThreads) void peaks_kernel(uint32_t* __restrict__ peaks,
                                                         const uint16_t* __restrict__ dh,
                                                         const uint16_t* __restrict__ g,
                                                         const uint16_t* __restrict__ u, int64_t n,
                                                         int64_t F, int64_t ld) {
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  const int64_t per_row = F / 8;
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
                                                          const uint32_t* __restrict__ peaks,
                                                          int n_peaks,
                                                          float* __restrict__ rescale) {
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  const int64_t per_row = Fp / 8;
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

// The partial sums of a split product, added in order and rounded once (f16: after
// the factor at p.rescale). Rows
// as in TileArgs: r < rows0 to d, row1 <= r < row1 + rows0 to d1.
template <int DT>
__global__ __launch_bounds__(kThreads) void join_kernel(TileArgs p, int64_t n8) {
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n8; i += stride) {
    const int64_t row = 8 * i / p.N, col = 8 * i % p.N;
    const int64_t b = row / p.M, m = row % p.M;
    const bool second = m >= p.row1;
    const int64_t r = second ? m - p.row1 : m;
    if (r >= p.rows0) continue;
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    for (int s = 0; s < p.splits; ++s) {
      const float* at = p.part + s * p.part_floats + 8 * i;
      lo += load16f_nt(at);
      hi += load16f_nt(at + 4);
    }
    if constexpr (DT == kF16) {
      const float z = p.rescale ? *p.rescale : 1.f;
      lo *= z;
      hi *= z;
    }
    const u32x4 o = {pack2<DT>(lo[0], lo[1]), pack2<DT>(lo[2], lo[3]), pack2<DT>(hi[0], hi[1]),
                     pack2<DT>(hi[2], hi[3])};
    uint16_t* d = static_cast<uint16_t*>(second ? p.d1 : p.d);
    *reinterpret_cast<u32x4*>(d + (b * p.rows0 + r) * p.ldd + col) = o;
  }
}

unsigned grid_for(int64_t n) {
  const int64_t blocks = (n + kThreads - 1) / kThreads;
  return unsigned(blocks < 8192 ? blocks : 8192);
}

template <int DT>
hipError_t join(const TileArgs& a, hipStream_t s) {
  const int64_t n8 = a.batch * a.M * a.N / 8;
  hipLaunchKernelGGL(join_kernel<DT>, dim3(grid_for(n8)), dim3(kThreads), 0, s, a, n8);
  return hipGetLastError();
}

template <int DT, int SRCA, int SRCB>
hipError_t product(const TileArgs& a, hipStream_t s) {
  hipError_t e = ffn::launch_tile<DT, SRCA, SRCB, ffn::kStore>(a, s);
  if (e == hipSuccess && a.splits > 1) e = join<DT>(a, s);
  return e;
}

}  // namespace

int64_t gated_peaks(int64_t rows, int64_t F) {
  const int64_t blocks = (rows * F / 8 + kThreads - 1) / kThreads;
  return blocks < 1024 ? blocks : 1024;   // four workgroups a CU keep the memory busy
}

hipError_t launch_gated_slopes(uint16_t* dgu, const uint16_t* dh, const uint16_t* g,
                               const uint16_t* u, int64_t rows, int64_t F, int64_t ld, int dtype,
                               int act, uint32_t* peaks, float* rescale, hipStream_t s) {
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
                       F, ld);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  auto kern = dtype == kBF16 ? by_act([](auto a) { return slopes_kernel<kBF16, decltype(a)::value>; })
                             : by_act([](auto a) { return slopes_kernel<kF16, decltype(a)::value>; });
  hipLaunchKernelGGL(kern, dim3(grid_for(n)), dim3(kThreads), 0, s, dgu, dh, g, u, n, F, Fp, ld, peaks,
                     n_peaks, rescale);
  return hipGetLastError();
}

hipError_t launch_gated_dx(const TileArgs& a, int dtype, hipStream_t s) {
  return dtype == kBF16 ? product<kBF16, ffn::kRows, ffn::kPackedT2>(a, s)
                        : product<kF16, ffn::kRows, ffn::kPackedT2>(a, s);
}

hipError_t launch_gated_dw(const TileArgs& a, int dtype, hipStream_t s) {
  return dtype == kBF16 ? product<kBF16, ffn::kTrans, ffn::kTrans>(a, s)
                        : product<kF16, ffn::kTrans, ffn::kTrans>(a, s);
}

// The plan that a simple model finds fastest. A tile of each size takes so many
// nanoseconds a slab and so many besides (its first loads and its results) on a
// full chip (256 workgroups; 128 x 128: 512). The tiles run in rounds; one that
// fills a share f of the chip takes a + (1 - a) f of a full one, with another a for
// the first round than for a later one, which starts while the one before it ends.
// Split sums are written and read once, 8 bytes at 5 TB/s, and joined by one more
// launch. The constants are a fit to 60 products measured on MI355X (16-bit and
// 4-bit, 200 to 32773 rows): 7% off in the mean, and within 3% of the fastest size
// in all but two. For example gated K = 2048 -> 5464 by tiles of 128 x 128, 256 x
// 128, 256 x 192 and 256 x 256: 777 rows 45.5, 52.3, 39.0 and 43.2 us, 1500 rows
// 70, 83, 77 and 92, 4095 rows 163, 172, 164 and 148; the weight gradients of 32773
// x 512 -> 1024 by 128 x 128 tiles 258 us, by 256 x 128 tiles and 8 splits 72.
// Outside of those products it is rougher. Below 128 rows it expects too little (96
// x 4096 -> 8192: 38 us, measured 45), without a worse choice. It does not know that a
// gated call keeps its projections: where the sum is short, 128 x 128 tiles are then
// often the better ones (kept, 4096 x 256 -> 4096: 47 us, chosen 256 x 256 56; 16384 x
// 256 -> 2048: 83, chosen 97; but 8192 x 256 -> 8192: 230, chosen 159), and 256 x 192
// tiles, which write the last columns in pieces of 32 bytes, the slowest (369 there).
TilePlan plan_tiles(int64_t batch, int64_t M, int64_t N, int64_t slabs, bool may_split) {
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
  for (int size = 0; size < 4; ++size) {
    const Size& z = kSizes[size];
    const double tiles = double(batch) * ((M + z.tm - 1) / z.tm) * ((N + z.tn - 1) / z.tn);
    for (int splits : kSplits) {
      if (splits > 1 && (!may_split || slabs / splits < 8)) break;
      const double tile = double((slabs + splits - 1) / splits) * z.slab + z.besides;
      const double fill = tiles * splits / z.places, rounds = fill < 1e12 ? double(int64_t(fill)) : fill;
      const double a = rounds > 0 ? z.later : z.first;
      double cost = rounds * tile;
      if (fill > rounds) cost += tile * (a + (1 - a) * (fill - rounds));
      if (splits > 1) cost += 4000 + 8e-3 / 5 * splits * batch * double(M) * N;
      if ((size == 0 && splits == 1) || cost < best.ns) best = {size, splits, cost};
    }
  }
  return best;
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

}  // namespace bmm
