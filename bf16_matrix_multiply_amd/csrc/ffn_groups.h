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
// The value of the lane before; lane 0: 0.
__device__ __forceinline__ int lane_before(int x) {
  return __builtin_amdgcn_update_dpp(0, x, 0x138, 0xf, 0xf, false);   // wave_shr:1
}

// Tiles of TM rows that n rows take.
template <int TM>
__device__ __forceinline__ int row_tiles(int n) {
  return n / TM + (n % TM != 0);
}

// A group, the same in every lane: its index, its first row and its rows, and the
// tile's index among the group's tiles.
struct Group {
  int e, start, rows, tile;
};

struct Groups {
  const int32_t* ends;
  int E, T, per;       // groups, rows, groups a lane
  int lane, before;    // where this lane's first group starts
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

  // The slot-th group (up to 64 groups) when those of one and a half times the mean
  // rows or more come first, then those of the mean or more, of half of it, and the
  // others: work that takes as long as a group has rows is better begun with the
  // largest, and the four classes cost a few instructions where a sort would cost as
  // much as a tile of a small group.
  __device__ __forceinline__ Group large_first(int slot) const {
    if (per > 1) return at(slot);
    int start = 0, rows = -1;
    each([&](int, int s, int n) {
      start = s;
      rows = n;
    });
    const int mean = T / E, border[4] = {mean + mean / 2, mean, mean / 2, 0};
    int rank = -1, before_class = 0;
    bool free = rows >= 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool here = free && rows >= border[c];
      const uint64_t mask = __builtin_amdgcn_ballot_w64(here);
      const int below = __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32),
                                                  __builtin_amdgcn_mbcnt_lo(uint32_t(mask), 0));
      if (here) rank = before_class + below;
      before_class += __builtin_popcountll(mask);
      free = free && !here;
    }
    const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(rank == slot));
    return {l, __builtin_amdgcn_readlane(start, l), __builtin_amdgcn_readlane(rows, l), 0};
  }

  // Tiles of TM rows: those of group 0, of group 1, ...; with `tail`, then those of
  // the rows behind the last group, as group E.
  template <int TM>
  struct Tiles {
    int first, own;        // tiles before this lane's groups, and theirs
    int grouped, total;    // tiles of all groups; with the tail's
    int end_all;           // the first row behind the last group
  };
  template <int TM>
  __device__ __forceinline__ Tiles<TM> tiles(bool tail) const {
    Tiles<TM> t;
    int own = 0, last = before;
    each([&](int, int s, int n) {
      own += row_tiles<TM>(n);
      last = s + n;
    });
    const int sum = lanes_sum(own);
    t.own = own;
    t.first = sum - own;
    t.grouped = __builtin_amdgcn_readlane(sum, kWave - 1);
    t.end_all = __builtin_amdgcn_readlane(last, kWave - 1);
    t.total = t.grouped + (tail ? row_tiles<TM>(T - t.end_all) : 0);
    return t;
  }
  // The group of row tile r < total.
  template <int TM>
  __device__ __forceinline__ Group find(const Tiles<TM>& t, int r) const {
    if (r >= t.grouped) return {E, t.end_all, T - t.end_all, r - t.grouped};
    int e = 0, start = 0, rows = 0, tile = 0, left = r - t.first;
    each([&](int i, int s, int n) {
      const int k = row_tiles<TM>(n);
      if (left >= 0 && left < k) {
        e = i;
        start = s;
        rows = n;
        tile = left;
      }
      left -= k;
    });
    const uint64_t here = __builtin_amdgcn_ballot_w64(r >= t.first && r < t.first + t.own);
    const int l = __builtin_ctzll(here);
    return {__builtin_amdgcn_readlane(e, l), __builtin_amdgcn_readlane(start, l),
            __builtin_amdgcn_readlane(rows, l), __builtin_amdgcn_readlane(tile, l)};
  }
};

// The most tiles of TM rows that T rows in E groups and a tail can take.
inline int64_t most_row_tiles(int64_t T, int64_t E, int64_t TM) {
  const int64_t some = E + 1 < T ? E + 1 : T;
  return (T + some * (TM - 1)) / TM;
}

}  // namespace ffn
}  // namespace bmm
