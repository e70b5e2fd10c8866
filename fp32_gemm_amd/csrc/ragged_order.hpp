// ragged_order.hpp -- which tile a workgroup of a grouped product takes.
//
// The offsets stay on the device, so every workgroup finds its tile from them:
// a wave looks at 64 groups at a time, a lane each.  The functions are written
// over a wave type W, whose Int holds a value of every lane: DeviceWave is the
// wave itself, and ragged_host_wave.hpp has one for the host, with which the
// same code lists the order of all tiles.
#pragma once

#include <hip/hip_runtime.h>

namespace fp32gemm {

// Rows of group e, whatever the offsets hold: within 0 .. rows, never negative.
struct RowSpan { int lo, hi; };
struct Groups {
  const int* offsets;  // groups + 1 row numbers; null: one group of all rows
  int groups, rows;
  __host__ __device__ __forceinline__ RowSpan span(int e) const {
    if (offsets == nullptr) return {0, rows};
    auto inside = [&](int v, int low) {
      const int least = v > low ? v : low;
      return least < rows ? least : rows;
    };
    const int lo = inside(offsets[e], 0);
    return {lo, inside(offsets[e + 1], lo)};
  }
  // The most tiles of bm rows there are when the groups follow one another.
  // Offsets out of order may count more; such a launch computes nothing, so that
  // every tile found is one of a group's.  No sum passes an int on the way: a
  // launch has fewer than 2^24 workgroups, hence whole tiles of all rows, and 64
  // groups hold all rows 32 times at most, as the step back between two times
  // is an empty group.
  __host__ __device__ __forceinline__ int most(int bm) const {
    return rows / bm + (groups < rows ? groups : rows);
  }
};

struct DeviceWave {
  using Int = int;
  struct Spans { int lo, hi; };
  int lane;
  // The spans of groups e0 + lane, empty past the last.
  __device__ __forceinline__ Spans spans(const Groups& g, int e0) const {
    const RowSpan s = e0 + lane < g.groups ? g.span(e0 + lane) : RowSpan{0, 0};
    return {s.lo, s.hi};
  }
  // The sum over this and all lower lanes.
  static __device__ __forceinline__ int sum_below(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // from 1, 2, 4 and 8 lanes below,
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // within rows of sixteen,
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // a row's last lane to the next row,
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // and lane 31 to the upper half
    return v;
  }
  static __device__ __forceinline__ int at(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
  static __device__ __forceinline__ unsigned long long where(bool f) { return __ballot(f); }
  // How many lower lanes are in m, and whether this one is.
  static __device__ __forceinline__ int rank(unsigned long long m) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(m >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(m), 0));
  }
  __device__ __forceinline__ bool in(unsigned long long m) const { return m >> lane & 1; }
  __device__ __forceinline__ int lanes() const { return lane; }
};

// Consecutive workgroups run on the eight dies in turn, each with its own L2:
// die x takes the x-th run of consecutive tiles.  Returns -1 past the last.
__host__ __device__ __forceinline__ int die_order(int w, int tiles) {
  const int x = w & 7, i = w >> 3, q = tiles >> 3, r = tiles & 7;
  return i < q + (x < r) ? x * q + (x < r ? x : r) + i : -1;
}

// Within a group, tiles go down BAND row tiles before the next column, so that
// tiles in flight on a die share operand rows and columns in its L2.
struct TileRow { int m, n; };
constexpr int tile_band(int bm) { return bm >= 256 ? 4 : 8; }
template <int BAND>
__host__ __device__ __forceinline__ TileRow band_order(int id, int tm, int tn) {
  const int band = id / (BAND * tn), first = band * BAND, rows = BAND < tm - first ? BAND : tm - first;
  const int in = id - first * tn;
  return {first + in % rows, in / rows};
}

// The tile of workgroup w: its group, first row, the group's end and its
// column; group -1 past the last.  Group after group, the last row tile of each
// partly filled.  A lane counts a group, 64 at a time.
struct TileAt { int group, row, hi, n; };
template <int BM, int BAND, class W>
__host__ __device__ __forceinline__ TileAt tile_in_order(const W& wave, const Groups& p, int w, int tiles_n) {
  typename W::Spans s{};
  typename W::Int upto{}, n{};
  int before = 0, e0 = 0;
  auto count = [&] {
    s = wave.spans(p, e0);
    n = (s.hi - s.lo + (BM - 1)) / BM;
    upto = wave.sum_below(n) + before;
  };
  for (;; e0 += 64) {
    count();
    before = wave.at(upto, 63);
    if (before > p.most(BM)) return {-1, 0, 0, 0};
    if (e0 + 64 >= p.groups) break;
  }
  const int id = die_order(w, before * tiles_n);
  if (id < 0) return {-1, 0, 0, 0};
  const int want = id / tiles_n;  // the group's row tiles include the want-th of all
  if (p.groups > 64) {
    for (e0 = 0, before = 0;; e0 += 64) {
      count();
      const int end = wave.at(upto, 63);
      if (end > want) break;
      before = end;
    }
  }
  const int l = __builtin_ctzll(wave.where(upto > want)), tm = wave.at(n, l);
  const TileRow at = band_order<BAND>(id - (wave.at(upto, l) - tm) * tiles_n, tm, tiles_n);
  return {e0 + l, wave.at(s.lo, l) + at.m * BM, wave.at(s.hi, l), at.n};
}

// The same for tiles whose time goes by their filled part.  Whole row tiles
// come first.  The rows that are left of each group make partly filled tiles,
// which take less time the fewer blocks of CLASS rows they hold; they come
// last, the fullest first, so that the workgroups that finish early fill up
// with the short ones.  The dies take them in turn, kDeal columns at a time,
// which share the rows.
constexpr int kDeal = 4;
template <int BM, int CLASS, int BAND, class W>
__host__ __device__ __forceinline__ TileAt tile_by_fill(const W& wave, const Groups& p, int w, int tiles_n) {
  constexpr int NC = BM / CLASS;
  const int x = w & 7, i = w >> 3;
  typename W::Spans s{};
  typename W::Int whole{}, upto{};     // whole row tiles of the lane's group, and of all up to it
  unsigned long long members[NC];      // groups with c + 1 started blocks left
  int wholes = 0, parts[NC] = {};      // in the chunks before, and after the first pass in all
  int e0 = 0;
  auto count = [&] {
    s = wave.spans(p, e0);
    const typename W::Int n = s.hi - s.lo, left = (n % BM + (CLASS - 1)) / CLASS;
    whole = n / BM;
    upto = wave.sum_below(whole);
#pragma unroll
    for (int c = 0; c < NC; ++c) members[c] = wave.where(left == c + 1);
  };
  for (;; e0 += 64) {
    count();
    wholes += wave.at(upto, 63);
    if (wholes > p.most(BM)) return {-1, 0, 0, 0};
#pragma unroll
    for (int c = 0; c < NC; ++c) parts[c] += __builtin_popcountll(members[c]);
    if (e0 + 64 >= p.groups) break;
  }
  const int here = wholes * tiles_n / 8 + (x < wholes * tiles_n % 8);  // whole tiles of this die
  const bool in_whole = i < here;
  int id, want, n, kind = 0;  // the row tile among the whole ones, or among those of class `kind`
  if (in_whole) {
    id = die_order(w, wholes * tiles_n);
    want = id / tiles_n;
    n = 0;
  } else {
    const int deals = (tiles_n + kDeal - 1) / kDeal;  // of a row tile
    id = (i - here) / kDeal * 8 + (7 - x);
    want = id / deals;
    n = id % deals * kDeal + (i - here) % kDeal;
    for (kind = NC - 1; kind >= 0; --kind) {
      int all = 0;
#pragma unroll
      for (int c = 0; c < NC; ++c) all = c == kind ? parts[c] : all;
      if (want < all) break;
      want -= all;
    }
    if (kind < 0 || n >= tiles_n) return {-1, 0, 0, 0};
  }
  unsigned long long hit;
  int before = 0;
  auto look = [&] {  // the lane whose group holds the tile, counting this chunk's from `before`
    unsigned long long m = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) m = c == kind ? members[c] : m;
    hit = in_whole ? wave.where(upto + before > want) : wave.where(wave.in(m) & (wave.rank(m) + before == want));
    return in_whole ? wave.at(upto, 63) : __builtin_popcountll(m);
  };
  if (p.groups <= 64) {
    look();
  } else {
    for (e0 = 0;; e0 += 64) {
      count();
      const int these = look();
      if (hit != 0 || e0 + 64 >= p.groups) break;
      before += these;
    }
  }
  const int l = __builtin_ctzll(hit), tm = wave.at(whole, l);
  int row = tm;
  if (in_whole) {
    const TileRow at = band_order<BAND>(id - (before + wave.at(upto, l) - tm) * tiles_n, tm, tiles_n);
    row = at.m;
    n = at.n;
  }
  return {e0 + l, wave.at(s.lo, l) + row * BM, wave.at(s.hi, l), n};
}

// Tiles of 256 rows differ in time by how far they are filled.
template <int BM, class W>
__host__ __device__ __forceinline__ TileAt tile_of_rows(const W& wave, const Groups& p, int w, int tiles_n) {
  if constexpr (BM == 256) return tile_by_fill<BM, BM / 4, tile_band(BM)>(wave, p, w, tiles_n);
  else return tile_in_order<BM, tile_band(BM)>(wave, p, w, tiles_n);
}

// The group whose length is the `rank`-th largest (the lower one of equals), so
// that the longest reductions start first.  Past 64 groups: as they come.
template <class W>
__host__ __device__ __forceinline__ int by_length(const W& wave, const Groups& p, int rank) {
  if (p.groups > 64) return rank;
  const typename W::Spans s = wave.spans(p, 0);
  const typename W::Int n = s.hi - s.lo;
  typename W::Int above{};
  for (int e = 0; e < p.groups; ++e) {
    const int o = wave.at(n, e);
    above += (n < o) | ((n == o) & (wave.lanes() > e));
  }
  return __builtin_ctzll(wave.where((wave.lanes() < p.groups) & (above == rank)));
}

// The tile of a weight gradient: its group, row tile (of BM outputs) and column.
// Each group's tiles are dealt out over all dies: groups differ in length.
template <int BM, class W>
__host__ __device__ __forceinline__ TileAt tile_of_group(const W& wave, const Groups& p, int w, int tiles_m,
                                                         int tiles_n, bool longest_first) {
  const unsigned each = tiles_m * tiles_n, room = (each + 7) & ~7u, u = w;
  int group = u / room;
  if (longest_first) group = by_length(wave, p, group);
  const int id = die_order(u % room, each);
  if (id < 0) return {-1, 0, 0, 0};
  const TileRow at = band_order<tile_band(BM)>(id, tiles_m, tiles_n);
  return {group, at.m, 0, at.n};
}

}  // namespace fp32gemm
