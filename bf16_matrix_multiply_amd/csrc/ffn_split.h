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
  int64_t rows = p.M;   // that have a result
  if (GRP == kGroupRows && !p.zero_tail)
    rows = rows_of_groups(p.ends, int(p.batch), int(p.M), threadIdx.x % kWave);
  for (int64_t i = int64_t(blockIdx.x) * kJoinThreads + threadIdx.x; i < n8; i += stride) {
    const int64_t row = 8 * i / p.N, col = 8 * i % p.N;
    const int64_t b = row / p.M, m = row % p.M;
    const bool second = m >= p.row1;
    const int64_t r = second ? m - p.row1 : m;
    if (r >= p.rows0) continue;
    if (GRP == kGroupRows && m >= rows) continue;
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

// Both gradients of a product by groups in one launch, for products so small that
// either leaves most of the chip idle: workgroups below n_dx make tiles of dX, the
// others of dW. (777 rows of 5 groups, 528 -> 1000 f16: 14.6 us a call, 21.7 with two.)
template <int DT>
__global__ __launch_bounds__(kTileWaves* kWave) __attribute__((amdgpu_waves_per_eu(2, 2)))
void grads_kernel(TileArgs dx, TileArgs dw, uint32_t n_dx, uint32_t NT_dx, uint32_t n_dw,
                  uint32_t MT_dw, uint32_t NT_dw) {
  constexpr int kSide = 128;
  __shared__ __attribute__((aligned(1024))) char b0[kSide * 64], b1[kSide * 64], b2[kSide * 64],
      b3[kSide * 64], a0[kSide * 128], a1[kSide * 64], a2[kSide * 128], a3[kSide * 64];
  const Ring ring{b0, b1, b2, b3, a0, a1, a2, a3};
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  SumList list;
  if (blockIdx.x < n_dx) {
    Place<kGroupRows> at;
    bool small;
    if (!locate_rows<kSide, kSide>(dx, blockIdx.x, NT_dx, 32, lane, at, small)) return;
    make_tile<DT, kRows, kPackedT2, kStore, kGroupRows, kSide, kSide, 0>(dx, at, list, ring, lane,
                                                                        wave);
  } else {
    Place<kGroupSums> at;
    list.init(dw, blockIdx.x - n_dx, n_dw, MT_dw, NT_dw, lane);
    if (list.template locate<kSide, kSide>(dw, 0, 32, at))
      make_tile<DT, kTrans, kTrans, kStore, kGroupSums, kSide, kSide, 1>(dw, at, list, ring, lane,
                                                                        wave);
    fill_empty<1>(list);
  }
}

// Workgroups that make dW's tiles beside n_dx that make one of dX each, of n_dw that the
// chip would hold alone. Those that find no place start when tiles of dX end, and the call
// then lasts as long as such a tile and their tiles of dW together; fewer, in the places
// that dX leaves, last as long as the longer of the two. The shorter is taken, by the
// times of plan_tiles' 128 x 128 tile. As many as the chip holds / in the places left (us):
// gated block 768 -> 512, 610 rows of 16 groups 24.9 / 20.1; product 1352 -> 128, 216 rows
// of 41 19.2 / 16.0; and where as many are taken 1024 -> 640, 900 rows of 24 23.0 / 25.0,
// 3728 -> 120, 105 rows of 95 63 / 83.
inline int64_t dw_places(const TileArgs& dx, const TileArgs& dw, int64_t n_dx, int64_t n_dw,
                         int64_t tiles_dw) {
  constexpr int64_t kPlaces = 2 * kCus;
  const int64_t left = kPlaces - n_dx;
  if (left < kXcds || n_dw <= left) return n_dw;
  auto slabs = [](int64_t n, int64_t parts) { return (n + 32 * parts - 1) / (32 * parts); };
  const int64_t one_dx = 3600 + 475 * slabs(dx.K, dx.splits);
  const int64_t one_dw = 5900 + 475 * slabs(dw.K, dw.batch * dw.splits);
  auto rounds = [&](int64_t places) { return (tiles_dw + places - 1) / places; };
  const int64_t beside = rounds(left) * one_dw;
  return (beside > one_dx ? beside : one_dx) < one_dx + rounds(n_dw) * one_dw ? left : n_dw;
}

template <int DT>
hipError_t both_gradients(const TileArgs& dx, const TileArgs& dw, hipStream_t s) {
  const int64_t MT = (dw.M + 127) / 128, NT_dx = (dx.N + 127) / 128, NT_dw = (dw.N + 127) / 128;
  int64_t n_dx = tile_grid<kGroupRows, 128>(dx, most_row_tiles(dx.M, dx.batch, 128), NT_dx);
  int64_t n_dw = tile_grid<kGroupSums, 128>(dw, MT, NT_dw);
  if (n_dx < 0 || n_dw < 0) return hipErrorInvalidConfiguration;
  n_dx = (n_dx + kXcds - 1) / kXcds * kXcds;
  if (n_dx + n_dw > kMaxWorkgroups) return hipErrorInvalidConfiguration;
  n_dw = dw_places(dx, dw, n_dx, n_dw, dw.batch * MT * NT_dw * dw.splits);
  if (n_dx + n_dw == 0) return hipSuccess;
  hipLaunchKernelGGL(grads_kernel<DT>, dim3(unsigned(n_dx + n_dw)), dim3(kTileWaves * kWave), 0, s,
                     dx, dw, uint32_t(n_dx), uint32_t(NT_dx), uint32_t(n_dw), uint32_t(MT),
                     uint32_t(NT_dw));
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && dx.splits > 1) e = join<DT, kGroupRows>(dx, s);
  if (e == hipSuccess && dw.splits > 1) e = join<DT, kGroupSums>(dw, s);
  return e;
}

template <int DT, int SRCA, int SRCB, int GRP = kWhole>
hipError_t product(const TileArgs& a, hipStream_t s) {
  hipError_t e = launch_tile<DT, SRCA, SRCB, kStore, GRP>(a, s);
  if (e == hipSuccess && a.splits > 1) e = join<DT, GRP>(a, s);
  return e;
}

}  // namespace ffn
}  // namespace bmm
