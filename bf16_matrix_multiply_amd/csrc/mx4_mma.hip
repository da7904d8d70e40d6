// Products of 4-bit operands: D = A B^T, and the gated block
// H = act(X Wg^T) * (X Wu^T), on the scaled 16x16x128 MFMA.
#include "ffn_skinny.h"

namespace bmm {

hipError_t launch_mx4_mma(const TileArgs& a, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny) return launch_skinny<kMX4, kStore>(a, s);
  return launch_tile<kMX4, kCodes, kCodes, kStore>(a, s);
}

hipError_t launch_mx4_gated(const TileArgs& a, hipStream_t s) {
  using namespace ffn;
  if (a.tile == kSkinny) return launch_skinny<kMX4, kGated>(a, s);
  return launch_tile<kMX4, kCodes, kCodes2, kGated>(a, s);
}

}  // namespace bmm
