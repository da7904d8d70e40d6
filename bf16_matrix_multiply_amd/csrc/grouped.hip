// Products by groups of rows, the rows of each expert of a mixture with the
// expert's own weights:
//   Y = X W_e^T,  H = act(X Wg_e^T) * (X Wu_e^T)
// The tiles and the few-rows kernel of the gated block, each workgroup finding its
// group by itself (ffn_groups.h): one launch, and nothing for the host to wait for.
// Six rows of 6 of 64 groups, 1408 -> 2048 bf16, 8 us on the GPU, 34.6 MB of weights;
// longer products at the two kernels.
#include "ffn_skinny.h"

namespace bmm {

hipError_t launch_grouped_mma(const TileArgs& a, int dtype, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny)
    return dtype == kBF16 ? launch_skinny_groups<kBF16, kStore>(a, s)
                          : launch_skinny_groups<kF16, kStore>(a, s);
  return dtype == kBF16 ? launch_tile<kBF16, kRows, kPacked, kStore, kGroupRows>(a, s)
                        : launch_tile<kF16, kRows, kPacked, kStore, kGroupRows>(a, s);
}

hipError_t launch_grouped_gated(const TileArgs& a, int dtype, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny)
    return dtype == kBF16 ? launch_skinny_groups<kBF16, kGated>(a, s)
                          : launch_skinny_groups<kF16, kGated>(a, s);
  return dtype == kBF16 ? launch_tile<kBF16, kRows, kPacked2, kGated, kGroupRows>(a, s)
                        : launch_tile<kF16, kRows, kPacked2, kGated, kGroupRows>(a, s);
}

}  // namespace bmm
