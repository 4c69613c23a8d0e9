// Which tile of which expert a workgroup takes: the tasks are sorted by expert,
// each expert's tasks are cut into row tiles, and those into column tiles.
#pragma once
#include "device.hpp"

namespace omni {

// Found by every wave for itself: lane l counts the tiles of q consecutive
// experts, a prefix sum over the lanes gives the total and the lane that owns
// row tile `rt`, and that lane's experts are walked.  Offsets are clamped to
// [0, M] and to ascending order, so no value of theirs can lead a read or
// write outside the row lists.  A launch has fewer than 2^24 workgroups and
// offsets in order no more tiles than that; offsets that overlap can ask for any
// number, so counts are cut off there: the sum over the lanes then fits 31 bits,
// and a tile that is found lies within its lane's experts still.
constexpr int kMostTiles = 1 << 24;
struct ExpertTile {
  int e, m0, m1;  // expert, first task of the tile, end of the tile (m0 == m1: none)
};
__device__ __forceinline__ void expert_range(const int32_t* off, int e, int M, int& lo, int& hi) {
  lo = min(max(off[e], 0), M);
  hi = min(max(off[e + 1], lo), M);
}
struct ExpertScan {
  int mine, upto, total;
  int lo, hi;  // tasks of this lane's last expert (its only one up to 64 experts)
};
__device__ __forceinline__ ExpertScan scan_experts(const int32_t* off, int E, int M, int bm) {
  const int l = lane(), q = (E + kWave - 1) / kWave;
  ExpertScan s{0, 0, 0, 0, 0};
  for (int i = 0; i < q; ++i) {
    const int e = l * q + i;
    if (e < E) {
      expert_range(off, e, M, s.lo, s.hi);
      s.mine = min(s.mine + (s.hi - s.lo + bm - 1) / bm, kMostTiles);
    }
  }
  s.upto = wave_prefix_sum(s.mine);
  s.total = __builtin_amdgcn_readlane(s.upto, 63);
  return s;
}
// row tiles times column tiles, cut off likewise
__device__ __forceinline__ int all_tiles(const ExpertScan& s, int n_nt) {
  return static_cast<int>(min(static_cast<long long>(s.total) * n_nt, 64ll * kMostTiles));
}
// Tile `id` of the n_nt column tiles of every row tile.  An expert's tiles run
// in bands of kBand column tiles, each down all its row tiles: the tiles that
// an XCD works on at a time (32 of the largest) then form a block of about
// kBand x kBand, whose rows and weights its L2 fetches once.
constexpr int kBand = 6;
struct TilePlace {
  ExpertTile t;
  int nt;
};
__device__ __forceinline__ TilePlace place_in_expert(int e, int lo, int hi, int bm, int n_nt,
                                                     int id) {
  const int mt = (hi - lo + bm - 1) / bm;
  const int band = id / (mt * kBand), width = min(kBand, n_nt - band * kBand);
  const int rest = id - band * mt * kBand, rt = rest / width;
  return {{e, lo + rt * bm, min(hi, lo + (rt + 1) * bm)}, band * kBand + rest - rt * width};
}
__device__ __forceinline__ TilePlace find_tile(const ExpertScan& s, const int32_t* off, int E,
                                               int M, int bm, int n_nt, int id) {
  const int q = (E + kWave - 1) / kWave, row = id / n_nt;
  const uint64_t past = __ballot(s.upto > row);
  if (past == 0) return {{0, 0, 0}, 0};
  const int owner = __ffsll(static_cast<long long>(past)) - 1;
  int left = row - (__builtin_amdgcn_readlane(s.upto, owner) -
                    __builtin_amdgcn_readlane(s.mine, owner));
  if (q == 1)
    return place_in_expert(owner, __builtin_amdgcn_readlane(s.lo, owner),
                           __builtin_amdgcn_readlane(s.hi, owner), bm, n_nt,
                           id - (row - left) * n_nt);
  for (int i = 0; i < q; ++i) {
    const int e = owner * q + i;
    if (e >= E) break;
    int lo, hi;
    expert_range(off, e, M, lo, hi);
    const int mt = (hi - lo + bm - 1) / bm;
    if (left < mt) return place_in_expert(e, lo, hi, bm, n_nt, id - (row - left) * n_nt);
    left -= mt;
  }
  return {{0, 0, 0}, 0};
}
// The expert at position pos when every run of 64 experts is put in order of
// its task counts, most first (ties by id), and its tasks.
__device__ __forceinline__ int expert_by_size(const int32_t* off, int E, int M, int pos, int& lo,
                                              int& hi) {
  const int first = pos & ~63, e = first + lane();
  int l = 0, h = -1;  // past the last expert: behind those without tasks
  if (e < E) expert_range(off, e, M, l, h);
  const int count = h - l;
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < 64; ++j) {
    const int c = __builtin_amdgcn_readlane(count, j);
    rank += c > count || (c == count && j < lane()) ? 1 : 0;
  }
  const int at = __ffsll(static_cast<long long>(__ballot(rank == pos - first))) - 1;
  lo = __builtin_amdgcn_readlane(l, at);
  hi = __builtin_amdgcn_readlane(h, at);
  return first + at;
}
// Workgroup b runs on XCD b % 8: give every XCD a contiguous run of the tiles
// there are, so that neighbours share rows and weights in that XCD's L2.
__device__ __forceinline__ int xcd_tile(int b, int total) {
  const int per = total >> 3, rem = total & 7, xcd = b & 7;
  return xcd * per + min(xcd, rem) + (b >> 3);
}
__device__ __forceinline__ bool xcd_has(int b, int total) {
  return (b >> 3) < (total >> 3) + ((b & 7) < (total & 7) ? 1 : 0);
}
// The workgroup's tile of those that experts of `offsets` (NULL: one of all M
// tasks) have; an empty one (m0 == m1) where there is none for it.
__device__ __forceinline__ TilePlace my_tile(int block, int blocks, const int32_t* offsets, int E,
                                             int M, int bm, int n_nt) {
  if (!offsets) return place_in_expert(0, 0, M, bm, n_nt, xcd_tile(block, blocks));
  const ExpertScan s = scan_experts(offsets, E, M, bm);
  const int total = all_tiles(s, n_nt);
  if (!xcd_has(block, total)) return {{0, 0, 0}, 0};
  return find_tile(s, offsets, E, M, bm, n_nt, xcd_tile(block, total));
}

// A part of an expert's tasks and a tile of its weight gradient.
struct WgradPart {
  int e, lo, hi;  // lo == hi: none
  int slot;       // where the sum goes: a partial sum, or -1: dW itself (an expert in one part)
  int tile;
};

// Slots of the experts in several parts come one after the other, by id.
__device__ __forceinline__ int parts_of(int count, int part) {
  return (count + part - 1) / part;
}
// first partial slot of expert e
__device__ __forceinline__ int first_slot(const int32_t* off, int E, int M, int part, int e) {
  const int l = lane(), q = (E + kWave - 1) / kWave;
  int before = 0;  // slots of this lane's experts below e
  for (int i = 0; i < q; ++i) {
    const int f = l * q + i;
    if (f < e) {
      int lo, hi;
      expert_range(off, f, M, lo, hi);
      const int n = parts_of(hi - lo, part);
      before = min(before + (n > 1 ? n : 0), kMostTiles);
    }
  }
  return __builtin_amdgcn_readlane(wave_prefix_sum(before), 63);
}
__device__ __forceinline__ WgradPart my_part(int block, const int32_t* off, int E, int M, int part,
                                             int slots, int tiles) {
  const ExpertScan s = scan_experts(off, E, M, part);
  const int total = all_tiles(s, tiles);
  if (!xcd_has(block, total)) return {0, 0, 0, 0, 0};
  const int id = xcd_tile(block, total), p = id / tiles;
  // a part is a row tile of `part` rows; with one column tile each
  const TilePlace at = find_tile(s, off, E, M, part, 1, p);
  WgradPart w = {at.t.e, at.t.m0, at.t.m1, -1, id - p * tiles};
  if (w.lo >= w.hi) return {0, 0, 0, 0, 0};
  int lo, hi;
  expert_range(off, w.e, M, lo, hi);
  if (hi - lo > part) w.slot = first_slot(off, E, M, part, w.e) + (w.lo - lo) / part;
  if (w.slot >= slots) return {0, 0, 0, 0, 0};  // offsets that overlap
  return w;
}

}  // namespace omni
