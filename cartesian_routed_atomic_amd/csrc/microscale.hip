// Rows in 4-bit floating point with a power-of-two scale for each 32 elements,
// and products of them on the scaled matrix-core instruction.
#include "device.hpp"
#include "expert_pipeline.hpp"
#include "expert_tiles.hpp"
#include "launch.hpp"

namespace omni {

constexpr int kMxBlock = 32;
__host__ __device__ inline int mx_scale_bytes(int k) { return (k + 127) / 128 * 4; }

// ------------------------------------------------------------------ rows made 4-bit

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = a.z;
  v[3] = a.w;
  v[4] = b.x;
  v[5] = b.y;
  v[6] = b.z;
  v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  v[0] = bf_lo(u.x);
  v[1] = bf_hi(u.x);
  v[2] = bf_lo(u.y);
  v[3] = bf_hi(u.y);
  v[4] = bf_lo(u.z);
  v[5] = bf_hi(u.z);
  v[6] = bf_lo(u.w);
  v[7] = bf_hi(u.w);
}

// Sixteen lanes take 128 elements of a row, eight each; four lanes share a block.
template <typename T>
__global__ __launch_bounds__(256) void microscale_kernel(const T* x, uint8_t* q, uint8_t* scale,
                                                         int R, int k) {
  const int groups = (k + 127) / 128, l = threadIdx.x & 15;
  const size_t item = static_cast<size_t>(blockIdx.x) * 16 + threadIdx.x / 16;
  if (item >= static_cast<size_t>(R) * groups) return;
  const size_t row = item / groups;
  const int c = static_cast<int>(item - row * groups) * 128 + l * 8;
  const bool in = c < k;
  float v[8] = {};
  if (in) load8(x + row * k + c, v);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1)));
  top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2)));
  const uint32_t ex = top >> 23;
  const uint32_t b = !in ? 127u : ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
  // 2^-127 is no normal number: such blocks are lifted by 2^64 (exact)
  const float lift = b == 0u ? 0x1p64f : 1.f;
  const float unit = __uint_as_float((b == 0u ? 64u : b) << 23);
  uint32_t w = 0;
  if (b != 255u) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * lift, v[1] * lift, unit, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * lift, v[3] * lift, unit, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * lift, v[5] * lift, unit, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * lift, v[7] * lift, unit, 3);
  }
  uint32_t all = b << (l / 4 * 8);
  all |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), 4));
  all |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(all), 8));
  if (in) *reinterpret_cast<uint32_t*>(q + row * (k / 2) + c / 2) = w;
  if (l == 0) *reinterpret_cast<uint32_t*>(scale + item * 4) = all;
}

hipError_t launch_microscale_rows(int bf16, int R, int k, const void* x, uint8_t* q,
                                  uint8_t* scale, hipStream_t s) {
  const size_t items = static_cast<size_t>(R) * ((k + 127) / 128);
  const unsigned nb = static_cast<unsigned>((items + 15) / 16);
  if (bf16) microscale_kernel<<<nb, 256, 0, s>>>(static_cast<const uint16_t*>(x), q, scale, R, k);
  else microscale_kernel<<<nb, 256, 0, s>>>(static_cast<const float*>(x), q, scale, R, k);
  return hipGetLastError();
}

// ------------------------------------------------------------------ the product

// 16 rows by 64 bytes of an operand: lane 16 g + r holds the 16 bytes of row r's
// g-th block of 32 elements, and their scale.
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
// waves, whose sums are added through LDS in wave order.
// SWIGLU: the first CT / 2 column tiles are gate rows, the others their up rows.
template <typename TO, bool SWIGLU, int RT, int CT, int KS, int U>
__global__ __launch_bounds__(KS * 64) void mx_rows_kernel(ExpertMatmulArgs a) {
  constexpr int BM = 16 * RT, H = SWIGLU ? 2 : 1, CO = CT / H, BNO = 16 * CO;
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
    pscale[i] = a.x_mx + row * row_scales + g;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const size_t row = first + min(n0 + j % CO * 16 + fr, N - 1) + static_cast<size_t>(j / CO) * N;
    qsrc[j] = static_cast<const uint8_t*>(a.w) + row * row_bytes + g * 16;
    qscale[j] = a.w_mx + row * row_scales + g;
  }
  const int blocks = a.k / kMxBlock, nk = (blocks + 3) / 4;
  const int per = (nk + KS - 1) / KS, kb = min(nk, wv * per), ke = min(nk, kb + per);
  f32x4 acc[RT][CT] = {};
  // past the end of a row zeros with a scale of one
  auto fetch = [&](const uint8_t* src, const uint8_t* scale, int kt) {
    MxFrag f = {{0, 0, 0, 0}, 127};
    if (kt < ke && kt * 4 + g < blocks) {
      f.q = *reinterpret_cast<const i32x4*>(src + static_cast<size_t>(kt) * 64);
      f.scale = scale[kt * 4];
    }
    return f;
  };
  for (int k0 = kb; k0 < ke; k0 += U) {
    MxFrag p[U][RT], q[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < CT; ++j) q[u][j] = fetch(qsrc[j], qscale[j], k0 + u);
#pragma unroll
      for (int i = 0; i < RT; ++i) p[u][i] = fetch(psrc[i], pscale[i], k0 + u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) mx_mma(acc[i][j], q[u][j], p[u][i]);
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

static long long mx_rows_blocks(const ExpertMatmulArgs& a) {
  const long long used = a.E < a.M ? a.E : a.M;
  return (a.M + used * 15) / 16 * ((a.n + 15) / 16);
}
bool microscaled_matmul_fits(const ExpertMatmulArgs& a) {
  if (a.n > 1 << 22 || a.k > 1 << 22 || a.E > 1 << 30) return false;
  return a.M == 0 || mx_rows_blocks(a) < (1ll << 32) / 512;
}
template <typename TO>
static void run_mx(const ExpertMatmulArgs& a, hipStream_t s) {
  const unsigned nb = static_cast<unsigned>(mx_rows_blocks(a));
  if (a.swiglu) mx_rows_kernel<TO, true, 1, 2, 8, 2><<<nb, 512, 0, s>>>(a);
  else mx_rows_kernel<TO, false, 1, 1, 8, 2><<<nb, 512, 0, s>>>(a);
}
hipError_t launch_microscaled_matmul(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.out_bf16) run_mx<uint16_t>(a, s);
  else run_mx<float>(a, s);
  return hipGetLastError();
}

}  // namespace omni
