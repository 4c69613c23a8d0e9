// Rows in 4-bit floating point with a power-of-two scale for each 32 elements,
// and products of them on the scaled matrix-core instruction.
#include "device.hpp"
#include "expert_forms.hpp"
#include "expert_pipeline.hpp"
#include "expert_tiles.hpp"
#include "launch.hpp"

namespace omni {

constexpr int kMxBlock = 32;
__host__ __device__ inline int mx_scale_bytes(int k) { return (k + 127) / 128 * 4; }

// ------------------------------------------------------------------ rows made 4-bit

// Sixteen consecutive elements of a lane.
struct F32Sixteen {
  float v[16];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      v[i] = f.x;
      v[i + 1] = f.y;
      v[i + 2] = f.z;
      v[i + 3] = f.w;
    }
  }
  // the largest magnitude, as bits: NaN above infinity above numbers
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) t = max(t, __float_as_uint(v[i]) & 0x7fffffffu);
    return t;
  }
  template <int I>
  __device__ __forceinline__ uint32_t four(float unit) const {  // elements 8 I .. 8 I + 7
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * I], v[8 * I + 1], unit, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * I + 2], v[8 * I + 3], unit, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * I + 4], v[8 * I + 5], unit, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[8 * I + 6], v[8 * I + 7], unit, 3);
  }
  __device__ __forceinline__ void lift() {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= 0x1p64f;
  }
};
// In pairs as they lie in memory: the maximum and the conversion take them so.
struct Bf16Sixteen {
  typedef unsigned short Pair __attribute__((ext_vector_type(2)));
  typedef __bf16 Bf16Pair __attribute__((ext_vector_type(2)));
  uint32_t v[8];
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = a.z;
    v[3] = a.w;
    v[4] = b.x;
    v[5] = b.y;
    v[6] = b.z;
    v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    Pair t = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t = __builtin_elementwise_max(t, __builtin_bit_cast(Pair, v[i] & 0x7fff7fffu));
    return static_cast<uint32_t>(max(t[0], t[1])) << 16;
  }
  template <int I>
  __device__ __forceinline__ uint32_t four(float unit) const {
    auto pair = [&](int i) { return __builtin_bit_cast(Bf16Pair, v[4 * I + i]); };
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(0), unit, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(1), unit, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(2), unit, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair(3), unit, 3);
  }
  __device__ __forceinline__ void lift() {  // bfloat16 has float32's exponents: exact
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float lo = bf_lo(v[i]) * 0x1p64f, hi = bf_hi(v[i]) * 0x1p64f;
      v[i] = __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
    }
  }
};

// Eight lanes take 128 elements of a row, sixteen each; two lanes share a block.  The
// conversion instruction rounds to nearest even and saturates, with a float32 scale
// that has to be a normal number: blocks whose scale is 2^-127 are lifted by 2^64
// (exact).  HBM-bound: 65536 x 2048 from bfloat16 in 58 us, 5.8 TB/s, 8192 x 2048 in
// 7.9; eight elements a lane, converted from float32, took 13.3.
template <typename T, typename Sixteen>
__global__ __launch_bounds__(256) void microscale_kernel(const T* x, uint8_t* q, uint8_t* scale,
                                                         int R, int k) {
  const uint32_t groups = (k + 127) / 128, l = threadIdx.x & 7;
  const uint32_t item = blockIdx.x * 32 + threadIdx.x / 8;  // below 2^28
  if (item >= static_cast<uint32_t>(R) * groups) return;
  const uint32_t row = item / groups, c = (item - row * groups) * 128 + l * 16;
  const bool in = c < static_cast<uint32_t>(k);
  Sixteen v = {};
  if (in) v.load(x + static_cast<size_t>(row) * k + c);
  uint32_t top = v.top();
  top = max(top, dpp_u<0xb1, 0xf>(0u, top));  // the neighbour: quad_perm 1 0 3 2
  const uint32_t ex = top >> 23;
  const uint32_t b = !in ? 127u : ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
  const bool tiny = b == 0u;
  if (__any(tiny)) {
    if (tiny) v.lift();
  }
  const float unit = __uint_as_float((tiny ? 64u : b) << 23);
  uint2 w = make_uint2(v.template four<0>(unit), v.template four<1>(unit));
  if (b == 255u) w = make_uint2(0u, 0u);
  // the four blocks' bytes, from lanes 0, 2, 4, 6
  uint32_t all = b << (l / 2 * 8);
  all |= dpp_u<0x4e, 0xf>(0u, all);   // quad_perm 2 3 0 1
  all |= dpp_u<0x141, 0xf>(0u, all);  // row_half_mirror
  if (in) *reinterpret_cast<uint2*>(q + static_cast<size_t>(row) * (k / 2) + c / 2) = w;
  if (l == 0) *reinterpret_cast<uint32_t*>(scale + static_cast<size_t>(item) * 4) = all;
}

hipError_t launch_microscale_rows(int bf16, int R, int k, const void* x, uint8_t* q,
                                  uint8_t* scale, hipStream_t s) {
  const size_t items = static_cast<size_t>(R) * ((k + 127) / 128);
  const unsigned nb = static_cast<unsigned>((items + 31) / 32);
  if (bf16)
    microscale_kernel<uint16_t, Bf16Sixteen>
        <<<nb, 256, 0, s>>>(static_cast<const uint16_t*>(x), q, scale, R, k);
  else
    microscale_kernel<float, F32Sixteen>
        <<<nb, 256, 0, s>>>(static_cast<const float*>(x), q, scale, R, k);
  return hipGetLastError();
}

// ------------------------------------------------------------------ the product

// 16 rows by 64 bytes of an operand: lane 16 g + r holds the 16 bytes of row r's
// g-th block of 32 elements, and their scale.
typedef float f32x16 __attribute__((ext_vector_type(16)));
struct MxFrag {
  i32x4 q;
  int scale;
};
__device__ __forceinline__ void mx_mma(f32x4& c, const MxFrag& q, const MxFrag& p) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 a = __builtin_shufflevector(q.q, q.q, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b = __builtin_shufflevector(p.q, p.q, 0, 1, 2, 3, -1, -1, -1, -1);
  // formats 4: e2m1; byte 0 of each lane's scale
  c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, q.scale, 0, p.scale);
}

// 16 RT tasks x 16 CT rows of W per workgroup, the contraction split over its KS
// waves, whose sums are added through LDS in wave order.  Bound by one memory latency:
// all of a wave's loads are out before its first MFMA.  One row by 11264 x 2048, 12.3
// MB of weights: 6.3 us, of which reading them at a copy's rate takes 2.4.
// SWIGLU: the first CT / 2 column tiles are gate rows, the others their up rows.
template <typename TO, bool SWIGLU, int RT, int CT, int KS, int U>
__global__ __launch_bounds__(KS * 64) void mx_rows_kernel(ExpertMatmulArgs a) {
  constexpr int BM = 16 * RT, H = SWIGLU ? 2 : 1, CO = CT / H, BNO = 16 * CO;
  static_assert(U == 2 || U == 4, "align_scales");
  static_assert(CT % H == 0, "gate and up tiles in pairs");
  __shared__ __attribute__((aligned(16))) f32x4 part[KS][RT * CT][64];
  const int wv = threadIdx.x >> 6, l = threadIdx.x & 63, fr = l & 15, g = l >> 4;
  const int N = a.n;
  const int n_nt = (N + BNO - 1) / BNO;
  const TilePlace at = my_tile(blockIdx.x, gridDim.x, a.offsets, a.E, a.M, BM, n_nt);
  const ExpertTile t = at.t;
  const int n0 = at.nt * BNO;
  if (t.m0 >= t.m1) return;
  const size_t row_bytes = static_cast<size_t>(a.k) / 2, row_scales = mx_scale_bytes(a.k);
  const size_t first = static_cast<size_t>(t.e) * H * N;
  const uint8_t *psrc[RT], *qsrc[CT], *pscale[RT], *qscale[CT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int m = min(t.m0 + i * 16 + fr, t.m1 - 1);
    const size_t row = min(max(a.x_row ? a.x_row[m] : m, 0), a.R - 1);
    psrc[i] = static_cast<const uint8_t*>(a.x) + row * row_bytes + g * 16;
    pscale[i] = a.x_mx + row * row_scales;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const size_t row = first + min(n0 + j % CO * 16 + fr, N - 1) + static_cast<size_t>(j / CO) * N;
    qsrc[j] = static_cast<const uint8_t*>(a.w) + row * row_bytes + g * 16;
    qscale[j] = a.w_mx + row * row_scales;
  }
  const int blocks = a.k / kMxBlock, nk = (blocks + 3) / 4;
  const int per = (nk + KS - 1) / KS, kb = min(nk, wv * per), ke = min(nk, kb + per);
  f32x4 acc[RT][CT] = {};
  // The scales of U steps from k0 on, a word each, in one load: a byte at a time they
  // took a quarter of the kernel (1 x 11264 x 2048: 7.3 us for 6.3).  A row's last
  // 4 U bytes are those of its last U steps.
  auto load_scales = [&](uint32_t (&w)[U], const uint8_t* scale, int k0) {
    if (nk < U) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        w[u] = k0 + u < nk ? *reinterpret_cast<const uint32_t*>(scale + (k0 + u) * 4) : 0u;
      return;
    }
    __builtin_memcpy(w, __builtin_assume_aligned(scale + min(k0, nk - U) * 4, 4), 4 * U);
  };
  // to step k0's first where the load began before it
  auto align_scales = [&](uint32_t (&w)[U], int k0) {
    const int early = nk < U ? 0 : k0 - min(k0, nk - U);
    if constexpr (U == 4) {
      if (early & 2) {
        w[0] = w[2];
        w[1] = w[3];
      }
    }
    if (early & 1) {
#pragma unroll
      for (int u = 0; u + 1 < U; ++u) w[u] = w[u + 1];
    }
  };
  // past the end of a row zeros with a scale of one
  auto inside = [&](int kt) { return kt < ke && kt * 4 + g < blocks; };
  auto fetch = [&](const uint8_t* src, int kt) {
    return inside(kt) ? *reinterpret_cast<const i32x4*>(src + static_cast<size_t>(kt) * 64)
                      : i32x4{0, 0, 0, 0};
  };
  for (int k0 = kb; k0 < ke; k0 += U) {
    i32x4 p[U][RT], q[U][CT];
    uint32_t ps[RT][U], qs[CT][U];
#pragma unroll
    for (int j = 0; j < CT; ++j) load_scales(qs[j], qscale[j], k0);
#pragma unroll
    for (int i = 0; i < RT; ++i) load_scales(ps[i], pscale[i], k0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < CT; ++j) q[u][j] = fetch(qsrc[j], k0 + u);
#pragma unroll
      for (int i = 0; i < RT; ++i) p[u][i] = fetch(psrc[i], k0 + u);
    }
#pragma unroll
    for (int j = 0; j < CT; ++j) align_scales(qs[j], k0);
#pragma unroll
    for (int i = 0; i < RT; ++i) align_scales(ps[i], k0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = inside(k0 + u);
      auto own = [&](uint32_t w) { return static_cast<int>(in ? w >> (8 * g) : 127u); };
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
          mx_mma(acc[i][j], {q[u][j], own(qs[j][u])}, {p[u][i], own(ps[i][u])});
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) part[wv][i * CT + j][l] = acc[i][j];
  __syncthreads();
  TO* out = static_cast<TO*>(a.out);
  const bool aligned = (N * sizeof(TO)) % 16 == 0;
  for (int o = wv; o < RT * CO; o += KS) {
    const int i = o / CO, j = o % CO, c0 = n0 + j * 16 + g * 4;
    f32x4 s[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      s[h] = part[0][i * CT + h * CO + j][l];
      for (int z = 1; z < KS; ++z) s[h] += part[z][i * CT + h * CO + j][l];
    }
    const int m = t.m0 + i * 16 + fr;
    if (m >= t.m1) continue;
    const int row = a.out_row ? a.out_row[m] : m, xr = a.x_row ? a.x_row[m] : m;
    if (row < 0 || row >= a.Ro) continue;
    const bool in = xr >= 0 && xr < a.R;
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = !in ? 0.f : SWIGLU ? silu_mul(s[0][q], s[H - 1][q]) : s[0][q];
    store_cols(out + static_cast<size_t>(row) * N, c0, N, aligned, v);
  }
}

// ------------------------------------------------------------------ tiles

__device__ __forceinline__ void mx_mma32(f32x16& c, i32x4 q, i32x4 p, int qs, int ps,
                                         std::false_type) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 a = __builtin_shufflevector(q, q, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b = __builtin_shufflevector(p, p, 0, 1, 2, 3, -1, -1, -1, -1);
  c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 0, qs, 0, ps);
}
__device__ __forceinline__ void mx_mma32(f32x16& c, i32x4 q, i32x4 p, int qs, int ps,
                                         std::true_type) {  // byte 2 of the scales
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 a = __builtin_shufflevector(q, q, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b = __builtin_shufflevector(p, p, 0, 1, 2, 3, -1, -1, -1, -1);
  c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, 2, qs, 2, ps);
}
// Row i of an MFMA's 32 weight rows is row mx_row(i) of the tile's 32: a lane's
// results are then 16 consecutive columns.
__device__ __forceinline__ int mx_row(int i) {
  return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
}
// A row of a stage is 128 bytes, eight chunks, chunk c of row r stored at c ^
// mx_swz(r).  A 16-byte-per-lane read is served
// sixteen lanes at a time (0-3, 12-15, 20-23, 24-27 and the other sixteen, then the
// same of the upper half) from the 256 bytes of the banks; their rows, of tasks and
// by mx_row of weights, then lie on sixteen distinct 16-byte slots.
__device__ __forceinline__ int mx_swz(int r) { return (r >> 1) & 7; }

// Direct global -> LDS load of 4 bytes per lane to dst + 4 lane (dst uniform).
__device__ __forceinline__ void load_lds4(const void* src, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
                   :
                   : "v"(src), "s"(dst)
                   : "memory");
}

__device__ __forceinline__ TilePlace same_in_wave(TilePlace p) {
  p.t.e = __builtin_amdgcn_readfirstlane(p.t.e);
  p.t.m0 = __builtin_amdgcn_readfirstlane(p.t.m0);
  p.t.m1 = __builtin_amdgcn_readfirstlane(p.t.m1);
  p.nt = __builtin_amdgcn_readfirstlane(p.nt);
  return p;
}

// Tile BM tasks x BN columns, WM x WN waves, ring of S stages of 128 bytes (256
// elements, a cache line: with 64 every line was fetched twice, 76 us for 70) a row.  A
// workgroup runs its tiles one after the other as one stream of stages: the next
// tile's first stages are under way while this one's last run and its results are
// stored (8192 x 5632 x 2048 in a launch's workgroup per tile: 83 us for 72).
// 8192 x 5632 x 2048: 67 us, 2.8 POP/s, 39 % of the MFMAs' cycles at the 1.7 GHz that
// power leaves (64 without its loads, 56 without its stores, 49 without either); 8192
// x 8192 x 8192: 313 us, 3.5 POP/s; 2048 tasks of 64 experts of 1408 x 2048, 98 MB of
// weights and scales: 27 us, 3.6 TB/s.
template <typename TO, bool SWIGLU, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64, 2) void mx_tile_kernel(ExpertMatmulArgs a) {
  constexpr int NW = WM * WN, S = 2;
  constexpr int TI = BM / WM / 32, TJ = BN / WN / 32;
  constexpr int IP = BM / 8 / NW, IQ = BN / 8 / NW, I = IP + IQ;  // 1-KiB loads per wave, stage
  constexpr int IS = (BM + BN + NW * 64 - 1) / (NW * 64);  // loads of 64 rows' scales
  constexpr int STAGE = (BM + BN) * 128, SCALES = (BM + BN) * 16;
  constexpr int BNO = SWIGLU ? BN / 2 : BN;            // output columns of a tile
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "loads split evenly");
  static_assert((BM + BN) % 64 == 0 && BM <= NW * 64, "whole loads of scales and row numbers");
  static_assert(TI >= 1 && TJ >= (SWIGLU ? 2 : 1) && TJ % (SWIGLU ? 2 : 1) == 0, "column pairs");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE + S * SCALES + BM * 4];

  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int N = a.n, n_nt = (N + BNO - 1) / BNO;
  const ExpertScan scan = a.offsets ? scan_experts(a.offsets, a.E, a.M, BM) : ExpertScan{};
  // offsets that overlap ask for more tiles than there can be: those are left out
  const int most = static_cast<int>((a.M + static_cast<long long>(min(a.E, a.M)) * (BM - 1)) / BM);
  const int total = min(a.offsets ? all_tiles(scan, n_nt) : most * n_nt, most * n_nt);
  auto place = [&](int v) -> TilePlace {
    if (!xcd_has(v, total)) return {{0, 0, 0}, 0};
    const int id = xcd_tile(v, total);
    TilePlace p = a.offsets ? find_tile(scan, a.offsets, a.E, a.M, BM, n_nt, id)
                            : place_in_expert(0, 0, a.M, BM, n_nt, id);
    return same_in_wave(p);
  };
  int v = blockIdx.x;
  TilePlace at = place(v);
  if (at.t.m0 >= at.t.m1) return;

  const int row_bytes = a.k / 2, G = mx_scale_bytes(a.k), blocks = a.k / kMxBlock;
  const int nk = (blocks + 7) / 8, left = blocks - (nk - 1) * 8;  // blocks of the last stage
  const int cut = left < 8 ? nk - 1 : -1;                         // the stage that is not whole
  const bool wide = G >= 16;
  const bool in_turn = mx_tiles_in_turn(a.k);
  const uint32_t ring = lds_address(smem), scales = ring + S * STAGE;
  int32_t* rows = reinterpret_cast<int32_t*>(smem + S * STAGE + S * SCALES);

  // Sources of this lane's direct loads.  Rows past the end and rows out of range
  // re-read a valid one: their results are not stored (or stored as zeros).
  // SWIGLU: every 64 rows of a tile's weights are 32 gate rows, then the same 32 up.
  const uint8_t *psrc[IP], *ssrc[IS], *qbase;
  uint32_t qoff[IQ];  // from the tile's first weight row
  auto sources = [&](const TilePlace& p, auto task_row) {
    // the lane, opaque: what follows from it alone would otherwise be kept in
    // registers throughout
    int l = tid & 63;
    __asm__ volatile("" : "+v"(l));
    const int n0 = p.nt * BNO;
    const size_t first = static_cast<size_t>(p.t.e) * (SWIGLU ? 2 : 1) * N + n0;
    auto x_row = [&](int r) -> size_t { return min(max(task_row(r), 0), a.R - 1); };
    auto w_row = [&](int r) {
      return min(SWIGLU ? (r >> 6) * 32 + (r & 31) : r, N - 1 - n0) + (SWIGLU ? (r >> 5) & 1 : 0) * N;
    };
#pragma unroll
    for (int u = 0; u < IP; ++u) {
      const int r = (wv * IP + u) * 8 + (l >> 3);
      psrc[u] = static_cast<const uint8_t*>(a.x) + x_row(r) * row_bytes + ((l & 7) ^ mx_swz(r)) * 16;
    }
#pragma unroll
    for (int u = 0; u < IQ; ++u) {
      const int r = (wv * IQ + u) * 8 + (l >> 3);
      qoff[u] = w_row(r) * static_cast<uint32_t>(row_bytes) + ((l & 7) ^ mx_swz(r)) * 16;
    }
    qbase = static_cast<const uint8_t*>(a.w) + first * row_bytes;
#pragma unroll
    for (int u = 0; u < IS; ++u) {
      const int r = min((u * NW + wv) * 64 + l, BM + BN - 1);
      ssrc[u] = r < BM ? a.x_mx + x_row(r) * G : a.w_mx + (first + w_row(r - BM)) * G;
    }
  };
  auto listed_row = [&](const TilePlace& p, int r) {
    const int m = min(p.t.m0 + r, p.t.m1 - 1);
    return a.x_row ? a.x_row[m] : m;
  };
  // Scales come 16 bytes of a row at a time, those of two stages, with the first of
  // the two.  A row's last 16 bytes start at G - 16.
  auto first_scale = [&](int j) { return min(j * 16, max(G - 16, 0)); };
  auto issue_scales = [&](int j, int slot) {
#pragma unroll
    for (int u = 0; u < IS; ++u)
      if ((u * NW + wv) * 64 < BM + BN)
        load_lds16(ssrc[u] + first_scale(j), scales + slot * SCALES + (u * NW + wv) * 1024);
  };
  // load u of stage kt into the slot of the stream's q-th
  auto issue = [&](int kt, int q, int u) {
    const uint32_t st = ring + (q % S) * STAGE, at = static_cast<uint32_t>(kt) * 128;
    if (u < IP) {
      load_lds16(psrc[u] + at, st + (wv * IP + u) * 1024);
    } else {
      u -= IP;
      load_lds16(qbase, qoff[u] + at, st + BM * 128 + (wv * IQ + u) * 1024);
    }
  };
  // Before the stage that is not whole: past the end of a row the tasks' data are
  // zeros; the weights', which are finite whatever their bits, are the row's start.
  auto end_rows = [&] {
    int ll = l;
    __asm__ volatile("" : "+v"(ll));  // opaque, as above
#pragma unroll
    for (int u = 0; u < IP; ++u)
      if (((ll & 7) ^ mx_swz((wv * IP + u) * 8 + (ll >> 3))) >= left)
        psrc[u] = reinterpret_cast<const uint8_t*>(kZeroChunk) - static_cast<size_t>(cut) * 128;
#pragma unroll
    for (int u = 0; u < IQ; ++u) {
      const int c = (ll & 7) ^ mx_swz((wv * IQ + u) * 8 + (ll >> 3));
      if (c >= left) qoff[u] -= static_cast<uint32_t>(cut) * 128 + c * 16;
    }
  };

  const int i32 = l & 31, h = l >> 5;
  int wm, wn;
  wave_place<WM, WN>(wv, wm, wn);
  const int prow = wm * (BM / WM) + i32, qrow = wn * (BN / WN) + mx_row(i32);
  // chunk 2 s + h of the lane's row in step s of a stage's four, 64 elements each:
  // the swizzle leaves the four apart by an exclusive or with 32 s
  const uint32_t pread = kept(ring + prow * 128 + ((h ^ mx_swz(prow)) << 4));
  const uint32_t qread = kept(ring + (BM + qrow) * 128 + ((h ^ mx_swz(qrow)) << 4));
  const uint32_t pscale = kept(scales + prow * 16), qscale = kept(scales + (BM + qrow) * 16);
  struct Frags {
    i32x4 p[TI], q[TJ];
  };
  struct Scales {
    int p[TI], q[TJ];  // bytes 0 and 2: of the lane's two chunks
  };
  Frags f0, f1;
  Scales sc, next;
  auto read_row = [&](Frags& f, int q, int s, int i, int of) {  // share i of `of`
    const uint32_t st = (q % S) * STAGE, pat = (pread + st) ^ (32 * s), qat = (qread + st) ^ (32 * s);
#pragma unroll
    for (int j = i * TJ / of; j < (i + 1) * TJ / of; ++j)
      f.q[j] = lds_read<i32x4>(qat + j * 32 * 128);
#pragma unroll
    for (int r = i * TI / of; r < (i + 1) * TI / of; ++r)
      f.p[r] = lds_read<i32x4>(pat + r * 32 * 128);
  };
  // of steps 2 half and 2 half + 1 of stage kt
  auto read_scales = [&](Scales& d, int kt, int half, int slot) {
    const uint32_t base = slot * SCALES + (kt * 8 + half * 4 - first_scale(kt / 2));
#pragma unroll
    for (int i = 0; i < TI; ++i) d.p[i] = lds_read<int>(base + pscale + i * 32 * 16);
#pragma unroll
    for (int i = 0; i < TJ; ++i) d.q[i] = lds_read<int>(base + qscale + i * 32 * 16);
  };
  // past the end of a row the data are zeros, and so that they stay zeros whatever
  // the last four scales' rest holds, their scale is one
  auto use_scales = [&](int kt, int half) {
    const int whole = min(max(left - half * 4, 0), 4);
    const uint32_t keep = kt == cut && whole < 4 ? (1u << (8 * whole)) - 1u : ~0u;
    const uint32_t one = 0x7f7f7f7fu & ~keep;
#pragma unroll
    for (int i = 0; i < TI; ++i)
      sc.p[i] = static_cast<int>(((static_cast<uint32_t>(next.p[i]) & keep) | one) >> (8 * h));
#pragma unroll
    for (int i = 0; i < TJ; ++i)
      sc.q[i] = static_cast<int>(((static_cast<uint32_t>(next.q[i]) & keep) | one) >> (8 * h));
  };
  f32x16 acc[TI][TJ];
  auto mma_row = [&](const Frags& f, int i, auto step) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      mx_mma32(acc[i][j], f.q[j], f.p[i], sc.q[j], sc.p[i], step);
    // keeps the MFMAs here, between the reads ahead of and behind them
#pragma unroll
    for (int j = 0; j < TJ; ++j) __asm__ volatile("" : "+v"(acc[i][j])::"memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Lane (i32, h) holds row 32 i + i32, columns 32 j + 16 h + 0..15.  Two rows sixteen
  // apart change halves, so that four lanes store a row's 32 columns side by side: with
  // 16 bytes of every row at a time 8192 x 5632 x 2048 took 70.4 us for 67.8, and in
  // tiles of 128 x 128 8192 x 8192 x 8192 416 for 370.
  auto store = [&](const TilePlace& p) {
    TO* out = static_cast<TO*>(a.out);
    const bool aligned = (N * sizeof(TO)) % 16 == 0;
    constexpr int W = 16 * sizeof(TO) / 4;  // 32-bit words of a lane's columns
    const int lo = l & 15, quarter = l >> 4;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int m = p.t.m0 + wm * (BM / WM) + i * 32;
      int row[2];  // where the lane stores: rows lo and 16 + lo
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = m + 16 * e + lo;
        row[e] = at >= p.t.m1 ? -1 : a.out_row ? a.out_row[at] : at;
        if (row[e] >= a.Ro) row[e] = -1;
      }
      bool in = true;  // a row out of range gives zeros
      if (a.x_row) {
        const int xr = a.x_row[min(m + i32, p.t.m1 - 1)];
        in = xr >= 0 && xr < a.R;
      }
#pragma unroll
      for (int j = 0; j < TJ; j += SWIGLU ? 2 : 1) {
        uint32_t w[W];
#pragma unroll
        for (int c = 0; c < 16; c += 4 / static_cast<int>(sizeof(TO))) {
          auto value = [&](int e) {
            if constexpr (SWIGLU) return in ? silu_mul(acc[i][j][e], acc[i][j + 1][e]) : 0.f;
            else return in ? acc[i][j][e] : 0.f;
          };
          if constexpr (sizeof(TO) == 2) w[c / 2] = bf16_pair(value(c), value(c + 1));
          else w[c] = __float_as_uint(value(c));
        }
        // pieces of 16 bytes: 0, 1, .. of a lane's own row; odd ones change places
#pragma unroll
        for (int b = 0; b < W; b += 8)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const auto both = __builtin_amdgcn_permlane16_swap(w[b + c], w[b + 4 + c], false, false);
            w[b + c] = both[0];
            w[b + 4 + c] = both[1];
          }
        const int c0 = p.nt * BNO + wn * (BNO / WN) + (SWIGLU ? j / 2 : j) * 32 +
                       (quarter >> 1) * 16 + (quarter & 1) * (16 / static_cast<int>(sizeof(TO)));
#pragma unroll
        for (int b = 0; b < W; b += 4) {
          const int to = row[(b >> 2) & 1], c = c0 + (b >> 3) * 8;
          if (to < 0) continue;
          TO* dst = out + static_cast<size_t>(to) * N;
          constexpr int N4 = 16 / sizeof(TO);
          if (aligned && c + N4 <= N) {
            *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[b], w[b + 1], w[b + 2], w[b + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < N4; ++e) {
              if (c + e >= N) continue;
              if constexpr (sizeof(TO) == 2) dst[c + e] = static_cast<TO>(w[b + e / 2] >> (16 * (e & 1)));
              else dst[c + e] = __uint_as_float(w[b + e]);
            }
          }
        }
      }
    }
  };

  sources(at, [&](int r) { return listed_row(at, r); });
  if (wide) {
    issue_scales(0, 0);
  } else {  // rows of fewer than 16 scales: at most two stages, both in the first slot
    for (int r = tid; r < BM + BN; r += NW * 64) {
      uint32_t b[4] = {0, 0, 0, 0};
      // of this lane's own sources where they are its rows: row (u NW + wv) 64 + l is tid's
#pragma unroll
      for (int u = 0; u < IS; ++u)
        if (r == (u * NW + wv) * 64 + l) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c * 4 < G) b[c] = *reinterpret_cast<const uint32_t*>(ssrc[u] + c * 4);
        }
      *reinterpret_cast<uint4*>(smem + S * STAGE + r * 16) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (s < nk) {
      if (s == cut) end_rows();
#pragma unroll
      for (int u = 0; u < I; ++u) issue(s, s, u);
    }
  wait_stages<I, S + 1>(min(S, nk) - 1);
  lds_barrier();
  read_row(f0, 0, 0, 0, 1);
  read_scales(next, 0, 0, 0);
  int q0 = 0, slot0 = 0;  // of the tile's first stage: its number in the stream, its scales' slot
  for (;;) {
    // the same for all lanes, which the compiler loses sight of behind the stores
    at = same_in_wave(at);
    q0 = __builtin_amdgcn_readfirstlane(q0);
    slot0 = __builtin_amdgcn_readfirstlane(slot0);
    v = __builtin_amdgcn_readfirstlane(v) + gridDim.x;
    const TilePlace then = in_turn ? place(v) : TilePlace{{0, 0, 0}, 0};
    const bool more = then.t.m0 < then.t.m1;
    const int slot1 = (slot0 + (nk + 1) / 2) % S;
    if (more && a.x_row && wv * 64 < BM)
      load_lds4(a.x_row + min(then.t.m0 + wv * 64 + l, then.t.m1 - 1),
                lds_address(rows) + wv * 256);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = f32x16{};
    // A step's MFMAs run while the fragments of the next one are read.  Before the
    // last step the next stage has to have landed, after which nobody needs this
    // one's slot: it is refilled with the stage S further on (of the next tile past
    // this one's end).
    for (int kt = 0; kt < nk; ++kt) {
      const int q = q0 + kt;
      const bool own = kt + S < nk, end = kt + 1 == nk;
      const int in = own ? kt + S : kt + S - nk;
      use_scales(kt, 0);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        read_row(f1, q, 1, i, TI);
        mma_row(f0, i, std::false_type{});
      }
      read_scales(next, kt, 1, (slot0 + kt / 2) % S);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        read_row(f0, q, 2, i, TI);
        mma_row(f1, i, std::true_type{});
      }
      use_scales(kt, 1);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        read_row(f1, q, 3, i, TI);
        mma_row(f0, i, std::false_type{});
      }
      wait_vm_lds<0>();
      lds_barrier();
      if (kt + S == nk && more)
        sources(then, [&](int r) {
          return a.x_row ? rows[r] : min(then.t.m0 + r, then.t.m1 - 1);
        });
      if (in == cut && (own || more)) end_rows();
      if (in % 2 == 0 && (own || more)) issue_scales(in / 2, ((own ? slot0 : slot1) + in / 2) % S);
      read_scales(next, end ? 0 : kt + 1, 0, end ? slot1 : (slot0 + (kt + 1) / 2) % S);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        if (own || more) {
#pragma unroll
          for (int u = i * I / TI; u < (i + 1) * I / TI; ++u) issue(in, q + S, u);
        }
        read_row(f0, q + 1, 0, i, TI);
        mma_row(f1, i, std::true_type{});
      }
    }
    store(at);
    if (!more) break;
    at = then;
    q0 += nk;
    slot0 = slot1;
  }
}

// ------------------------------------------------------------------ dispatch

bool microscaled_matmul_fits(const ExpertMatmulArgs& a) {
  // offsets within a tile's weights are 32 bits, and so is an expert's number rounded up to 64
  if (a.n > 1 << 22 || a.k > 1 << 22 || a.E > 1 << 30) return false;
  // an up row is n rows behind its gate row
  if (a.swiglu && (a.n + 256ll) * (a.k / 2) >= 1ll << 32) return false;
  return a.M == 0 || mx_tiles(a, pick_mx_form(a)) < (1ll << 32) / 512;
}
template <typename TO, bool SW>
static hipError_t run_mx(const ExpertMatmulArgs& a, hipStream_t s) {
  const MxForm f = pick_mx_form(a);
  const unsigned nb = static_cast<unsigned>(mx_blocks(a, f));
  // steps of a wave at a time: two where a wave has no more (1 x 4096 x 4096: 4.7 us
  // with four, 4.9 with two; 1 x 11264 x 2048: 6.4 and 6.3)
  const bool more = a.k > 2048;
  if (f == kMxRows16) {
    if (more) mx_rows_kernel<TO, SW, 1, SW ? 2 : 1, 8, 4><<<nb, 512, 0, s>>>(a);
    else mx_rows_kernel<TO, SW, 1, SW ? 2 : 1, 8, 2><<<nb, 512, 0, s>>>(a);
  } else if (f == kMxRows32) {
    if (more) mx_rows_kernel<TO, SW, 2, 2, 8, 4><<<nb, 512, 0, s>>>(a);
    else mx_rows_kernel<TO, SW, 2, 2, 8, 2><<<nb, 512, 0, s>>>(a);
  }
  else if (f == kMxSmall) mx_tile_kernel<TO, SW, 64, 128, 2, 2><<<nb, 256, 0, s>>>(a);
  else if (f == kMxMid) mx_tile_kernel<TO, SW, 128, 128, 2, 2><<<nb, 256, 0, s>>>(a);
  else if (f == kMxWide) mx_tile_kernel<TO, SW, 128, 256, 2, 4><<<nb, 512, 0, s>>>(a);
  else mx_tile_kernel<TO, SW, 256, 256, 2, 4><<<nb, 512, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_microscaled_matmul(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.out_bf16) return a.swiglu ? run_mx<uint16_t, true>(a, s) : run_mx<uint16_t, false>(a, s);
  return a.swiglu ? run_mx<float, true>(a, s) : run_mx<float, false>(a, s);
}

}  // namespace omni
