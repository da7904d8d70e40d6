// Counting rows, tiles and slabs of the products by groups: plain arithmetic, the same
// on the host and in the kernels, without an overflow up to 2^31 - 1 rows (rounded up in
// unsigned arithmetic: a signed sum would pass 2^31 there, and a negative count of
// slabs leads a loader out of its matrix).
#pragma once

#include <stdint.h>

namespace bmm {
namespace ffn {

// The tiles that n rows take: of TM rows, the last one perhaps not full; with tiles of
// 256 rows a last one of at most 128 is a small one, of 128 rows.
template <int TM>
constexpr int full_tiles(int n) {
  return int((uint32_t(n) + (TM == 256 ? 127 : TM - 1)) / TM);
}
template <int TM>
constexpr int small_tiles(int n) {
  return TM == 256 && n % 256 > 0 && n % 256 <= 128;
}

// The most tiles, small ones among them, that T rows in E groups and a tail can take.
constexpr int64_t most_row_tiles(int64_t T, int64_t E, int64_t TM) {
  const int64_t some = E + 1 < T ? E + 1 : T;
  return (T + some * (TM - 1)) / TM;
}

// Slabs of so many values that a sum of K takes. (32 bits: by groups.)
constexpr int32_t slab_count(int32_t K, int values) {
  return int32_t((uint32_t(K) + (values - 1)) / values);
}
constexpr int64_t slab_count(int64_t K, int values) { return (K + (values - 1)) / values; }

// The slabs from first up to end that part `split` of `splits` sums of K values. A part
// starts at an even slab: rows come two slabs at a time.
template <class Int>
struct SlabRange {
  Int first, end;
};
template <class Int>
constexpr SlabRange<Int> slab_range(Int K, int values, uint32_t split, uint32_t splits) {
  const Int slabs = slab_count(K, values);
  SlabRange<Int> r{0, slabs};
  if (splits > 1) {
    const uint32_t pairs = uint32_t((slabs + 1) / 2), q = pairs / splits, more = pairs % splits;
    r.first = 2 * (Int(split) * q + (split < more ? split : more));
    if (split + 1 < splits) r.end = r.first + 2 * (q + (split < more ? 1 : 0));
  }
  return r;
}

}  // namespace ffn
}  // namespace bmm
