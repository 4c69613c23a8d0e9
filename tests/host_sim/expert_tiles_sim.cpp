// Runs the tile search of the expert operators (csrc/expert_tiles.hpp, compiled
// for the host against the wave model in hip/hip_runtime.h) for a list of
// workgroups, for tests/test_host_sim_expert_tiles.py.
//
//   expert_tiles_sim IN OUT
//   IN:  int32 mode, E, M, bm, n_nt, slots, blocks, count; block ids [count]; offsets [E + 1]
//   OUT: int32 [count, 5]
//        mode 0 (tiles): expert, first task, end, column tile, 0
//        mode 1 (parts of a weight gradient): expert, first task, end, slot, tile
//        mode 2 (experts by size, position = block id): expert, first task, end, 0, 0
// Only the offsets are memory: the number of tasks can be as large as a call's.
#include <cstdio>
#include <vector>

#include "hip/hip_runtime.h"
inline int __ffsll(long long v) { return __builtin_ffsll(v); }
#include "expert_tiles.hpp"

static void search(int mode, int block, int blocks, const int32_t* off, int E, int M, int bm,
                   int n_nt, int slots, int32_t* out) {
  int32_t r[5] = {0, 0, 0, 0, 0};
  if (mode == 0) {
    const omni::TilePlace p = omni::my_tile(block, blocks, off, E, M, bm, n_nt);
    r[0] = p.t.e, r[1] = p.t.m0, r[2] = p.t.m1, r[3] = p.nt;
  } else if (mode == 1) {
    const omni::WgradPart p = omni::my_part(block, off, E, M, bm, slots, n_nt);
    r[0] = p.e, r[1] = p.lo, r[2] = p.hi, r[3] = p.slot, r[4] = p.tile;
  } else {
    int lo, hi;
    r[0] = omni::expert_by_size(off, E, M, block, lo, hi);
    r[1] = lo, r[2] = hi;
  }
  if (OMNI_SIM_LANE == 0)
    for (int i = 0; i < 5; ++i) out[i] = r[i];
}

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  FILE* f = std::fopen(argv[1], "rb");
  if (!f) sim::fail("cannot open input");
  int32_t h[8];
  if (std::fread(h, 4, 8, f) != 8) sim::fail("short input file");
  std::vector<int32_t> ids(h[7]), off(h[1] + 1), out(5 * static_cast<size_t>(h[7]));
  if (std::fread(ids.data(), 4, ids.size(), f) != ids.size()) sim::fail("short input file");
  if (std::fread(off.data(), 4, off.size(), f) != off.size()) sim::fail("short input file");
  std::fclose(f);
  for (int i = 0; i < h[7]; ++i)
    sim::launch(search, dim3(1), dim3(64), 0, nullptr, h[0], ids[i], h[6], off.data(), h[1], h[2],
                h[3], h[4], h[5], out.data() + 5 * static_cast<size_t>(i));
  FILE* o = std::fopen(argv[2], "wb");
  if (!o || std::fwrite(out.data(), 4, out.size(), o) != out.size()) sim::fail("short write");
  return std::fclose(o);
}
