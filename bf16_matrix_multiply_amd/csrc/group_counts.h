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

constexpr uint32_t kCus = 256;

// How the row tiles of a product by groups lie, `full` ones and `small` ones of 128 rows
// (tiles of 256 rows only) across NT tiles of columns. Where the small ones are few, they
// come last, and if the full ones would leave the chip at most half full in their last
// round and the small ones find room beside them, those of the last round are made in two
// halves. Where they are many, they stay beside their group's full ones, whose weight
// they share.
struct RowLayout {
  uint32_t full, last;   // row tiles: those of the groups in turn, and small ones after them
  bool mixed;            // the small ones are among the full ones
  uint32_t cut;          // tiles made in halves
};
template <int TM>
constexpr RowLayout row_layout(uint32_t full, uint32_t small, uint32_t NT, uint32_t splits) {
  RowLayout l{full, small, TM == 256 && 4 * small >= full, 0};
  if (l.mixed) {
    l.full += small;
    l.last = 0;
  }
  const uint32_t over = l.full * NT * splits % kCus;
  if (TM == 256 && splits == 1 && !l.mixed && over <= kCus / 2 && 2 * over + l.last * NT <= kCus)
    l.cut = over;
  return l;
}

// Tile v of the k x NT tiles of one group, whose rows are taken in bands of 6 at most
// and as equal as can be, so that the tiles of a band that run together share the
// group's weight: its row and column. Bands of at most 2, 4, 6, 8 and any number (us):
// 16384 rows of 8 groups 8192 -> 4096 917, 889, 888, 883, 887; gated 4096 -> 4096 911, 879,
// 870, 862, 864; of one group 4096 -> 4096 401, 379, 381, 380, 408; 32768 rows of 16, 4096
// -> 1024 245, 246, 250, 251, 251; 24576 of 64 the same with each. From 4 to 8 it matters
// little.
struct BandTile {
  uint32_t row, col;
};
constexpr BandTile band_tile(uint32_t v, uint32_t k, uint32_t NT) {
  const uint32_t bands = (k + 5) / 6, low = k / bands, more = k % bands;
  uint32_t rows = low + 1, row = 0;
  if (v >= more * rows * NT) {
    v -= more * rows * NT;
    row = more * rows;
    rows = low;
  }
  const uint32_t band = v / (rows * NT);
  v -= band * (rows * NT);
  const uint32_t col = v / rows;
  return {row + band * rows + v - col * rows, col};
}

}  // namespace ffn
}  // namespace bmm
