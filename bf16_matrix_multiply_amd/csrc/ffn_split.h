// Products whose sum may be split over workgroups: the tile kernel, and where it
// left partial sums the kernel that joins them.
#pragma once

#include "ffn_tile.h"

namespace bmm {
namespace ffn {

constexpr int kJoinThreads = 256;

// The partial sums of a split product, added in order and rounded once (f16: after
// the factor at p.rescale). Rows
// as in TileArgs: r < rows0 to d, row1 <= r < row1 + rows0 to d1. By groups of rows
// those behind the last one stay as they are unless they are to be zero.
template <int DT, int GRP>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(TileArgs p, int64_t n8) {
  const int64_t stride = int64_t(gridDim.x) * kJoinThreads;
  for (int64_t i = int64_t(blockIdx.x) * kJoinThreads + threadIdx.x; i < n8; i += stride) {
    const int64_t row = 8 * i / p.N, col = 8 * i % p.N;
    const int64_t b = row / p.M, m = row % p.M;
    const bool second = m >= p.row1;
    const int64_t r = second ? m - p.row1 : m;
    if (r >= p.rows0) continue;
    if (GRP == kGroupRows && !p.zero_tail && (p.batch == 0 || m >= p.ends[p.batch - 1])) continue;
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

template <int DT, int GRP>
hipError_t join(const TileArgs& a, hipStream_t s) {
  const int64_t n8 = (GRP == kGroupRows ? 1 : a.batch) * a.M * a.N / 8;
  const int64_t blocks = (n8 + kJoinThreads - 1) / kJoinThreads;
  hipLaunchKernelGGL((join_kernel<DT, GRP>), dim3(unsigned(blocks < 8192 ? blocks : 8192)),
                     dim3(kJoinThreads), 0, s, a, n8);
  return hipGetLastError();
}

template <int DT, int SRCA, int SRCB, int GRP = kWhole>
hipError_t product(const TileArgs& a, hipStream_t s) {
  hipError_t e = launch_tile<DT, SRCA, SRCB, kStore, GRP>(a, s);
  if (e == hipSuccess && a.splits > 1) e = join<DT, GRP>(a, s);
  return e;
}

}  // namespace ffn
}  // namespace bmm
