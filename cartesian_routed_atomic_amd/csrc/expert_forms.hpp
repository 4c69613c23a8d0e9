// Which kernel and tile an expert product or weight gradient runs, from sizes and
// types alone (the routing is device data).  Host code.
#pragma once
#include "launch.hpp"

namespace omni {

// sum of ceil(c_e / bm) over at most min(E, M) experts with tasks
inline long long expert_row_tiles(int M, int E, int bm) {
  const long long used = E < M ? E : M;
  return (M + used * (bm - 1)) / bm;
}
inline int output_width(const ExpertMatmulArgs& a) { return a.transpose ? a.k : a.n; }
inline int used_experts(const ExpertMatmulArgs& a) { return a.E < a.M ? a.E : a.M; }
// Tiles to expect: an expert's last row tile is half full on average.
inline double expected_tiles(const ExpertMatmulArgs& a, int bm, int bno) {
  const int used = used_experts(a);
  const long long rt = used == 1 ? (a.M + bm - 1ll) / bm
                                 : (a.M + static_cast<long long>(used) * (bm / 2)) / bm;
  return static_cast<double>(rt > used ? rt : used) * ((output_width(a) + bno - 1) / bno);
}

// The forms of the product: rows kernels of 16 x 16, 32 x 32 and 64 x 32, and
// tiles, each tasks x rows of W (with SWIGLU half as many outputs, the 16 x 16
// one then 16 x 32 rows of W).
enum ProductForm {
  kRows16, kRows32, kRows64, kTileF32, kTileSmall, kTileMid, kTileWide, kTileBig
};
struct FormShape {
  int bm, bn, threads;
};
inline FormShape form_shape(ProductForm f, int swiglu) {
  switch (f) {
    case kRows16: return {16, swiglu ? 32 : 16, 512};
    case kRows32: return {32, 32, 512};
    case kRows64: return {64, 32, 512};
    case kTileF32: return {64, 64, 256};
    case kTileSmall: return {64, 128, 256};
    case kTileMid: return {128, 128, 256};
    case kTileWide: return {128, 256, 512};
    default: return {256, 256, 512};
  }
}
inline long long form_blocks(const ExpertMatmulArgs& a, ProductForm f) {
  const FormShape h = form_shape(f, a.swiglu);
  const int bno = a.swiglu ? h.bn / 2 : h.bn;
  return expert_row_tiles(a.M, a.E, h.bm) * ((output_width(a) + bno - 1) / bno);
}

// Which tile, for bf16 and int8: the one whose tiles take the least time, in
// units of one round of 256 x 256 tiles (one per CU).  A 128 x 256 tile is
// alone on a CU as well, of the two smaller ones two and three share one; a
// large tile needs less LDS and L2 traffic per MFMA, a small one wastes less
// where there are few tiles or few rows.  Fitted to (us, 2048 inputs):
//   tiles of 256 x 256       64 (int8)  128 (int8)  80    144   1700
//   256 x 256                30         32          28    30    425
//   128 x 256                21         25          20    37    490
//   128 x 128                17         27          22    34    518
//   64 x 128                 19         32          23    34    650
inline ProductForm pick_tile(const ExpertMatmulArgs& a) {
  const int h = a.swiglu ? 2 : 1;
  const double t1 = expected_tiles(a, 256, 256 / h), t2 = expected_tiles(a, 128, 256 / h),
               t4 = expected_tiles(a, 128, 128 / h), t5 = expected_tiles(a, 64, 128 / h);
  auto rounds = [](double t) { return t <= 1024 ? static_cast<int>((t + 255) / 256) : t / 256; };
  const double big = rounds(t1);
  const double wide = t2 <= 768 ? 0.72 * rounds(t2) : 0.61 * t2 / 256 + 0.3;
  const double mid = t4 <= 256 ? 0.55 : t4 <= 512 ? 0.83 : 0.62 * t4 / 512 + 0.3;
  const double small = t5 <= 256 ? 0.46 : 0.55 * t5 / 768 + 0.35;
  if (big <= wide && big <= mid && big <= small) return kTileBig;
  if (wide <= mid && wide <= small) return kTileWide;
  return mid <= small ? kTileMid : kTileSmall;
}
inline ProductForm pick_form(const ExpertMatmulArgs& a) {
  const bool f32 = a.type == kRowsF32;
  if (!a.transpose) {
    // Few rows r of an expert, or so few tiles that most CUs would idle (us;
    // the rows kernel taken against 64 x 128 tiles):
    //   64 experts, 1408 outputs, 2048 inputs, 1 / 4 / 8 rows    44 74 90 / 54 75 79
    //   1 expert, 2048 outputs, 2048 inputs, 16 / 128 / 512      7.5 12.6 34 / 14 16 18
    //   4 experts, 512 outputs, 1024 inputs, 8 / 64 / 256        5.5 8.0 16 / 9.5 10 11
    // float32 against its 64 x 64 tiles:
    //   16 experts, 1024 outputs, 1024 inputs, 1 / 8 / 16        14 23 28 / 22 22 23
    //   4 experts, 512 outputs, 512 inputs, 30 / 200             7.6 13.3 / 13.7 14.2
    //   32 experts, 128 outputs, 344 inputs, 64 / 128            9.1 13.8 / 11.2 11.4
    const int r = a.M / used_experts(a);
    const double t = expected_tiles(a, 64, (f32 ? 64 : 128) / (a.swiglu ? 2 : 1));
    if (t < (f32 ? 128 : 48)) return r <= 32 ? kRows16 : r <= 128 ? kRows32 : kRows64;
    if (r <= (f32 ? 4 : t < 256 ? 8 : 2)) return kRows16;
  }
  // float32 is bound by its MFMAs at any tile: a small one balances best (64 x
  // 64 against 64 x 128: 20-40 % less time up to 1000 tiles, the same beyond)
  return f32 ? kTileF32 : pick_tile(a);
}
// How a weight gradient runs: its square tile, and the tasks of a part (0: no
// parts).  A tile of 256 where experts and parts of 1024 tasks give enough of
// them for the chip, else the smaller ones; float32, bound by its MFMAs, always
// takes the smallest, and experts of few tasks, bound by writing dW, not the
// largest (us, tiles of 64 / 128 / 256):
//   64 experts, 1408 x 2048, 1024 tasks each, bf16       - / 688 / 512
//   1 expert, 512 x 512, 8192 tasks, bf16                26 / 32 / 41
//   100 experts, 256 x 1024, 4 tasks each, bf16          41 / 29 / 36
//   16 experts, 512 x 512, 500 tasks each, float32       79 / 139 / -
// Parts where the tiles are fewer than four times those that run at a time and
// experts have tasks enough (half a part's on average):
// long enough that one round of them holds all tasks, and at least 32 stages
// (their partial sums and the second launch cost about what 30 stages do).
struct WgradPlan {
  int tile, part, slots;
};
inline WgradPlan plan_wgrad(int bf16, int M, int E, int n, int k) {
  auto tiles = [&](int b) {
    return static_cast<long long>((n + b - 1) / b) * ((k + b - 1) / b);
  };
  const long long used = E < M ? E : M, least = bf16 ? 1024 : 512;
  const long long units = used > M / least ? used : M / least;
  WgradPlan p = {64, 0, 0};
  if (bf16 && units * tiles(256) >= 192 && M >= 64 * used) p.tile = 256;
  else if (bf16 && units * tiles(128) >= 256) p.tile = 128;
  const long long t = tiles(p.tile), round = p.tile == 256 ? 256 : p.tile == 128 ? 512 : 1024;
  if (M >= used * least / 2 && M > 0 && used * t < 4 * round) {
    // one large tile per CU: room in the round for every expert's short part
    const long long full = p.tile == 256 ? round - used * t / 2 : 0;
    long long part = (M * t + round - 1) / (full > round / 4 ? full : round);
    if (part < least) part = least;
    part = (part + 127) / 128 * 128;
    if (part < M) {
      p.part = static_cast<int>(part);
      const long long most = M / part + used, twice = 2ll * M / part;
      p.slots = static_cast<int>(most < twice ? most : twice);
    }
  }
  return p;
}
inline long long wgrad_blocks(const ExpertWgradArgs& a, int tile) {
  const long long nt = (a.n + tile - 1) / tile, kt = (a.k + tile - 1) / tile;
  if (a.part > 0) return expert_row_tiles(a.M, a.E, a.part) * nt * kt;
  return (a.E * nt + 7) / 8 * 8 * kt;
}
inline int wgrad_threads(int tile) { return tile == 256 ? 512 : 256; }

// ------------------------------------------------------------------ 4-bit rows

// The forms of the 4-bit product: rows kernels of 16 x 16 (with SWIGLU 16 x 32
// weight rows) and 32 x 32, and tiles of tasks x weight rows.
enum MxForm { kMxRows16, kMxRows32, kMxSmall, kMxMid, kMxWide, kMxBig };
inline FormShape mx_form_shape(MxForm f, int swiglu) {
  switch (f) {
    case kMxRows16: return {16, swiglu ? 32 : 16, 512};
    case kMxRows32: return {32, 32, 512};
    case kMxSmall: return {64, 128, 256};
    case kMxMid: return {128, 128, 256};
    case kMxWide: return {128, 256, 512};
    default: return {256, 256, 512};
  }
}
inline long long mx_tiles(const ExpertMatmulArgs& a, MxForm f) {
  const FormShape h = mx_form_shape(f, a.swiglu);
  const int bno = a.swiglu ? h.bn / 2 : h.bn;
  return expert_row_tiles(a.M, a.E, h.bm) * ((a.n + bno - 1) / bno);
}
// A workgroup runs its tiles in turn where a row has 16 bytes of scales to load at
// once (then it also has the two stages that the next tile's loads are ahead).
#ifdef __HIPCC__
__host__ __device__
#endif
inline bool mx_tiles_in_turn(int k) { return k > 384; }
// the workgroups that fit on the chip at a time
inline int mx_slots(MxForm f) { return f == kMxSmall || f == kMxMid ? 512 : 256; }
inline long long mx_blocks(const ExpertMatmulArgs& a, MxForm f) {
  const long long t = mx_tiles(a, f);
  const bool rows = f == kMxRows16 || f == kMxRows32;
  return rows || !mx_tiles_in_turn(a.k) || t < mx_slots(f) ? t : mx_slots(f);
}
// Which one: the tile of least expected time, in us: its rounds of the chip times a
// start and the stages of 256 elements of a tile.  Workgroups of two a CU share it:
// where the last round has few of them, those are faster, and so are 256 or fewer.
// Fitted over 170 shapes, where the tile chosen takes 0.5 % more than the best one in
// the geometric mean; some of them (us; tasks of all experts x outputs x inputs):
//   tiles of                          256 x 256   128 x 256   128 x 128   64 x 128
//   2048 x 2048 x 2048                20.3        14.4        11.6        11.9
//   8192 x 5632 x 2048                67.8        77.0        79.8        107
//   8192 x 2048 x 2048                27.0        28.4        29.6        35.4
//   12234 x 1408 x 704, 32 experts    28.8        21.2        19.3        23.3
//   4096 x 1408 x 2048, 64 experts    40.1        27.9        23.6        23.5
//   4096 x 4096 x 4096, 8 experts     69.4        65.6        59.7        70.5
// The rows kernels where their workgroups are few a CU (us; rows of 16 and of 32
// against 64 x 128 tiles, 2048 inputs; where the choice lies within 0.5 % of the best
// in the geometric mean of 170 shapes):
//   1 expert, 2048 outputs, 1 / 64 / 128 / 256     3.6 5.1 7.4 12 / 4.5 5.4 5.5 7.8 / 7.7 8.3 8.3 8.3
//   1 expert, 8192 outputs, 1 / 16 / 32 / 64       4.4 5.1 7.4 12 / 4.5 5.0 5.4 7.9 / 7.6 7.8 8.0 8.3
//   the same, SWIGLU                               5.7 6.5 9.9 17 / 6.3 7.0 7.9 13 / 8.4 8.5 8.6 8.7
//   64 experts, 1408 outputs, 1 / 8                29 43 / 30 39 / 19 20
inline MxForm pick_mx_form(const ExpertMatmulArgs& a) {
  const int h = a.swiglu ? 2 : 1, r = a.M / used_experts(a);
  const double nk = (a.k + 255) / 256;
  const double rows = expected_tiles(a, 16, 16);
  if (rows <= 300 || (r <= 16 && rows <= 1024)) return kMxRows16;
  if (expected_tiles(a, 32, 32 / h) <= 640) return kMxRows32;
  struct Rounds {
    double part, whole;
  };
  auto rounds = [](double tiles, int slots) {
    const double t = tiles / slots < 1 ? 1. : tiles / slots;
    const double up = t <= 64 ? static_cast<double>(static_cast<int>(t + 0.999)) : t;
    return Rounds{t, up < t ? t : up};
  };
  auto half = [](double tiles) { return tiles <= 256 ? 0.6 : 1.; };
  const double small = expected_tiles(a, 64, 128 / h), mid = expected_tiles(a, 128, 128 / h),
               wide = expected_tiles(a, 128, 256 / h), big = expected_tiles(a, 256, 256 / h);
  const Rounds r_small = rounds(small, 512), r_mid = rounds(mid, 512);
  const double t_small =
      3.3 + (0.5 * r_small.part + 0.5 * r_small.whole) * (0.825 * nk + 2.5) * half(small);
  const double t_mid = 3.1 + (0.75 * r_mid.part + 0.25 * r_mid.whole) * (1.12 * nk + 4.1) * half(mid);
  const double t_wide = 0.7 + rounds(wide, 256).whole * (0.94 * nk + 5.7);
  const double t_big = rounds(big, 256).whole * (1.47 * nk + 8.5);
  if (t_big <= t_wide && t_big <= t_mid && t_big <= t_small) return kMxBig;
  if (t_wide <= t_mid && t_wide <= t_small) return kMxWide;
  return t_mid <= t_small ? kMxMid : kMxSmall;
}

}  // namespace omni
