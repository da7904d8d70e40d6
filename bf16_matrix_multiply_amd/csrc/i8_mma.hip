// Products of 8-bit integers with a scale for every row of both operands:
//   D[m][n] = sa[m] sb[n] (sum over k of A[m][k] B[n][k])
// and the gated block of two of them, of one weight or by groups. The sums are
// exact (K < 2^17: below 2^31); the scales are applied to them in float32, row's
// first, and the result is rounded once.
//
// One 16x16x64 MFMA takes 16 bytes a lane and row like the 16-bit ones, so the
// operands lie, travel and are read as 16-bit values with half the K. Measured at the
// two kernels.
#include "ffn_skinny.h"

namespace bmm {

hipError_t launch_i8_mma(const TileArgs& a, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny)
    return a.ends ? launch_skinny_groups<kI8, kStore>(a, s) : launch_skinny<kI8, kStore>(a, s);
  return a.ends ? launch_tile<kI8, kRows, kPacked, kStore, kGroupRows>(a, s)
                : launch_tile<kI8, kRows, kPacked, kStore>(a, s);
}

hipError_t launch_i8_gated(const TileArgs& a, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny)
    return a.ends ? launch_skinny_groups<kI8, kGated>(a, s) : launch_skinny<kI8, kGated>(a, s);
  return a.ends ? launch_tile<kI8, kRows, kPacked2, kGated, kGroupRows>(a, s)
                : launch_tile<kI8, kRows, kPacked2, kGated>(a, s);
}

}  // namespace bmm
