// H = act(X Wg^T) * (X Wu^T): both projections of a gated feed-forward block,
// the activation and the product in one kernel.
//
// The columns of a tile alternate between the two weights, 16 columns of Wg
// and the same 16 of Wu, so a lane ends with both projections of the same
// outputs in its registers and the gate is applied there: G and U reach memory
// only when a training step keeps them.
#include "ffn_skinny.h"

namespace bmm {

hipError_t launch_gated(const TileArgs& a, int dtype, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny)
    return dtype == kBF16 ? launch_skinny<kBF16, kGated>(a, s) : launch_skinny<kF16, kGated>(a, s);
  return dtype == kBF16 ? launch_tile<kBF16, kRows, kPacked2, kGated>(a, s)
                        : launch_tile<kF16, kRows, kPacked2, kGated>(a, s);
}

}  // namespace bmm
