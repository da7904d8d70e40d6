// Groups of rows (the experts' rows of a mixture): which rows a group has, and
// which group a tile of rows falls in.
//
// ends[e] is the first row behind group e; group e starts where group e - 1 ends,
// the first at row 0. The host does not know the values, so every workgroup reads
// them: each wave by itself, a run of consecutive groups a lane, with a running
// maximum and a running sum over the lanes (one load's latency and about 20 short
// instructions; up to 64 groups are one a lane). Ends are held to 0 .. T and to be
// no smaller than the ones before, so that no value of theirs leads out of the
// matrices.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "group_counts.h"

namespace bmm {
namespace ffn {

// Inclusive scan over the 64 lanes (row_shr 1, 2, 4, 8, then row broadcasts).
template <class Fn>
__device__ __forceinline__ int lanes_scan(int x, int identity, Fn fn) {
  x = fn(x, __builtin_amdgcn_update_dpp(identity, x, 0x111, 0xf, 0xf, false));
  x = fn(x, __builtin_amdgcn_update_dpp(identity, x, 0x112, 0xf, 0xf, false));
  x = fn(x, __builtin_amdgcn_update_dpp(identity, x, 0x114, 0xf, 0xf, false));
  x = fn(x, __builtin_amdgcn_update_dpp(identity, x, 0x118, 0xf, 0xf, false));
  x = fn(x, __builtin_amdgcn_update_dpp(identity, x, 0x142, 0xa, 0xf, false));
  x = fn(x, __builtin_amdgcn_update_dpp(identity, x, 0x143, 0xc, 0xf, false));
  return x;
}
__device__ __forceinline__ int lanes_max(int x) {
  return lanes_scan(x, 0, [](int a, int b) { return a > b ? a : b; });
}
__device__ __forceinline__ int lanes_sum(int x) {
  return lanes_scan(x, 0, [](int a, int b) { return a + b; });
}
// The rows of E groups in all, as Groups holds their ends, in every lane.
__device__ __forceinline__ int rows_of_groups(const int32_t* ends, int E, int T, int lane) {
  int top = 0;
  for (int e = lane; e < E; e += kWave) {
    const int x = ends[e] < T ? ends[e] : T;
    top = x > top ? x : top;
  }
  return __builtin_amdgcn_readlane(lanes_max(top), kWave - 1);
}
// The value of the lane before; lane 0: 0.
__device__ __forceinline__ int lane_before(int x) {
  return __builtin_amdgcn_update_dpp(0, x, 0x138, 0xf, 0xf, false);   // wave_shr:1
}

// A group, the same in every lane: its index, its first row and its rows, and the
// number of a tile within the group.
struct Group {
  int e, start, rows, tile;
};

struct Groups {
  const int32_t* ends;
  int E, T, per;       // groups, rows, groups a lane
  int lane, before;    // where this lane's first group starts
  int rank;            // this lane's group in the order of size (sort)
  int filled, own;     // groups that have rows, and this lane's (sort)
  int end0;            // and its end as read (kept: with 64 groups or fewer nothing is read again)

  __device__ __forceinline__ int end(int i, int from) const {   // this lane's i-th group
    int x = i == 0 ? end0 : ends[lane * per + i];
    x = x < T ? x : T;
    return x > from ? x : from;
  }
  __device__ __forceinline__ void init(const int32_t* ends_, int E_, int T_, int lane_) {
    ends = ends_;
    E = E_;
    T = T_;
    lane = lane_;
    per = (E + kWave - 1) / kWave;
    end0 = lane * per < E ? ends[lane * per] : 0;
    int top = 0;
    for (int i = 0; i < per; ++i)
      if (lane * per + i < E) top = end(i, top);
    before = lane_before(lanes_max(top));
  }

  // fn(e, start, rows) for this lane's groups.
  template <class Fn>
  __device__ __forceinline__ void each(Fn fn) const {
    int from = before;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) {
        const int to = end(i, from);
        fn(e, from, to - from);
        from = to;
      }
    }
  }

  // Group e.
  __device__ __forceinline__ Group at(int e) const {
    int start = 0, rows = 0;
    each([&](int i, int s, int n) {
      if (i == e) {
        start = s;
        rows = n;
      }
    });
    const int l = e / per;
    return {e, __builtin_amdgcn_readlane(start, l), __builtin_amdgcn_readlane(rows, l), 0};
  }

  // Orders the groups: up to 64 by size, the largest first, and rank is the place of
  // this lane's group; more as they are, but those without rows last, and rank is the
  // place of the first of this lane's that has rows.
  __device__ __forceinline__ void sort() {
    own = 0;
    if (per > 1) {
      each([&](int, int, int n) { own += n > 0; });
      const int sum = lanes_sum(own);
      rank = sum - own;
      filled = __builtin_amdgcn_readlane(sum, kWave - 1);
      return;
    }
    int rows = -1;
    each([&](int, int, int n) { rows = n; });
    int before_it = 0;
    for (int j = 0; j < E; ++j) {
      const int n = __builtin_amdgcn_readlane(rows, j);
      before_it += n > rows || (n == rows && j < lane);
    }
    rank = lane < E ? before_it : kWave;
    filled = __builtin_popcountll(__builtin_amdgcn_ballot_w64(rows > 0));
  }
  // The slot-th group in that order.
  __device__ __forceinline__ Group sorted(int slot) const {
    if (per > 1) {
      if (slot < filled) return search(slot, rank, own, [](int n) { return int(n > 0); });
      const int first = lane * per < E ? lane * per : E, left = E - first;
      return search(slot - filled, first - rank, (left < per ? left : per) - own,
                    [](int n) { return int(n == 0); });
    }
    return at(__builtin_ctzll(__builtin_amdgcn_ballot_w64(rank == slot)));
  }

  // Tiles: those of group 0, of group 1, ...; with `tail`, then those of the rows behind
  // the last group, as group E. Small ones are counted by themselves.
  template <int TM>
  struct Tiles {
    int first, own;        // tiles before this lane's groups, and theirs
    int first_small, own_small;
    int grouped, total;    // tiles of all groups; with the tail's
    int grouped_small, total_small;
    int end_all;           // the first row behind the last group
  };
  template <int TM>
  __device__ __forceinline__ Tiles<TM> tiles(bool tail) const {
    Tiles<TM> t;
    int last = before;
    t.own = t.own_small = 0;
    each([&](int, int s, int n) {
      t.own += full_tiles<TM>(n);
      t.own_small += small_tiles<TM>(n);
      last = s + n;
    });
    t.end_all = __builtin_amdgcn_readlane(last, kWave - 1);
    const int behind = tail ? T - t.end_all : 0;
    int sum = lanes_sum(t.own);
    t.first = sum - t.own;
    t.grouped = __builtin_amdgcn_readlane(sum, kWave - 1);
    t.total = t.grouped + full_tiles<TM>(behind);
    t.first_small = t.grouped_small = t.total_small = 0;
    if constexpr (TM == 256) {
      sum = lanes_sum(t.own_small);
      t.first_small = sum - t.own_small;
      t.grouped_small = __builtin_amdgcn_readlane(sum, kWave - 1);
      t.total_small = t.grouped_small + small_tiles<TM>(behind);
    }
    return t;
  }
  // The group of row tile r, with its number among the group's; of the full ones, of the
  // small ones, or of both in the groups' order, the small one last. (find: also of the
  // tail's, after the groups'.)
  template <int TM>
  __device__ __forceinline__ Group find(const Tiles<TM>& t, int r) const {
    if (r >= t.grouped) return behind(t, r - t.grouped);
    return search(r, t.first, t.own, [](int n) { return full_tiles<TM>(n); });
  }
  template <int TM>
  __device__ __forceinline__ Group find_small(const Tiles<TM>& t, int r) const {
    return search(r, t.first_small, t.own_small, [](int n) { return small_tiles<TM>(n); });
  }
  template <int TM>
  __device__ __forceinline__ Group find_any(const Tiles<TM>& t, int r) const {
    return search(r, t.first + t.first_small, t.own + t.own_small,
                  [](int n) { return full_tiles<TM>(n) + small_tiles<TM>(n); });
  }
  // The rows behind the last group.
  template <int TM>
  __device__ __forceinline__ Group behind(const Tiles<TM>& t, int tile) const {
    return {E, t.end_all, T - t.end_all, tile};
  }

 private:
  // The group of item r, of which each group has items(rows) and this lane's `own` from
  // `first` on, and the item's number in the group.
  template <class Fn>
  __device__ __forceinline__ Group search(int r, int first, int own, Fn items) const {
    int e = 0, start = 0, rows = 0, item = 0, left = r - first;
    each([&](int i, int s, int n) {
      const int k = items(n);
      if (left >= 0 && left < k) {
        e = i;
        start = s;
        rows = n;
        item = left;
      }
      left -= k;
    });
    const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(r >= first && r < first + own));
    return {__builtin_amdgcn_readlane(e, l), __builtin_amdgcn_readlane(start, l),
            __builtin_amdgcn_readlane(rows, l), __builtin_amdgcn_readlane(item, l)};
  }
};

}  // namespace ffn
}  // namespace bmm
