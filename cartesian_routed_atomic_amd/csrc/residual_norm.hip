// The norm after a block with its gate and residual scale, fused with the norm
// before the next block, and the backward of both:
//   n = y, or y b post_w with b = 1 / sqrt(mean y^2 + eps)
//   r1 = r + alpha g n,   x = r1 a w with a = 1 / sqrt(mean r1^2 + eps)
// and, for p = dx w,
//   dr = dr_out + a p - r1 a^3 mean(p r1),   dw = sum_rows dx r1 a
//   dgate = alpha dr n,   dn = alpha g dr,   q = dn post_w
//   dy = b q - y b^3 mean(q y),   dpost_w = sum_rows dn y b
// Both are HBM-bound: a row is read once, kept in registers, and written once.
#include "device.hpp"
#include "launch.hpp"

namespace omni {

template <int U>
__device__ __forceinline__ void load_unit(const float* p, float (&v)[U]) {
#pragma unroll
  for (int i = 0; i < U; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    v[i] = f.x;
    v[i + 1] = f.y;
    v[i + 2] = f.z;
    v[i + 3] = f.w;
  }
}
template <int U>
__device__ __forceinline__ void load_unit(const uint16_t* p, float (&v)[U]) {
  static_assert(U == 8, "16 bytes");
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
template <int U>
__device__ __forceinline__ void store_unit(float* p, const float (&v)[U]) {
#pragma unroll
  for (int i = 0; i < U; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {  // nearest even
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(a))) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
}
template <int U>
__device__ __forceinline__ void store_unit(uint16_t* p, const float (&v)[U]) {
  static_assert(U == 8, "16 bytes");
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                            bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

// Sums over the NT threads of a row, in a fixed order.  Every call takes an LDS
// array of its own (no barrier between a read of one and a write of the next).
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[16]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NT > kWave) {
    if (lane() == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < NT / kWave; ++w) v[i] += part[i][w];
    }
  }
}

// NT threads per row (a wave, or the whole workgroup), EPT columns of it each, in
// units of 16 bytes of the row's type.
template <typename T, typename TY, int NT, int EPT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_kernel(ResidualNormArgs a) {
  constexpr int U = 16 / sizeof(T), NV = EPT / U, ROWS = NT < 256 ? 256 / NT : 1;
  __shared__ float part[2][1][16];
  const int t = threadIdx.x % NT, d = a.d;
  const size_t row = static_cast<size_t>(blockIdx.x) * ROWS + threadIdx.x / NT;
  if (row >= static_cast<size_t>(a.L)) return;  // NT >= 256: never
  const size_t base = row * d;
  const T* gate = static_cast<const T*>(a.gate);
  float r[NV][U];
  auto column = [&](int u) { return (u * NT + t) * U; };
#pragma unroll
  for (int u = 0; u < NV; ++u) {
#pragma unroll
    for (int i = 0; i < U; ++i) r[u][i] = 0.f;
    if (column(u) < d) load_unit(static_cast<const T*>(a.r) + base + column(u), r[u]);
  }
  const float over = 1.f / d;
  if (a.y) {
    float n[NV][U];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
#pragma unroll
      for (int i = 0; i < U; ++i) n[u][i] = 0.f;
      if (column(u) < d) load_unit(static_cast<const TY*>(a.y) + base + column(u), n[u]);
    }
    float s = a.alpha;
    if (a.gate_kind == kGateToken) s *= load_one(gate + row);
    if (a.post) {
      float v[1] = {0.f};
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int i = 0; i < U; ++i) v[0] = fmaf(n[u][i], n[u][i], v[0]);
      row_sums<NT>(v, part[0]);
      s *= rsqrtf(fmaf(v[0], over, a.eps));
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (column(u) >= d) continue;
      if (a.post_w) {
        float w[U];
        load_unit(static_cast<const T*>(a.post_w) + column(u), w);
#pragma unroll
        for (int i = 0; i < U; ++i) n[u][i] *= w[i];
      }
      if (a.gate_kind == kGateColumn || a.gate_kind == kGateFull) {
        float g[U];
        load_unit(gate + (a.gate_kind == kGateFull ? base : 0) + column(u), g);
#pragma unroll
        for (int i = 0; i < U; ++i) n[u][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < U; ++i) r[u][i] = fmaf(s, n[u][i], r[u][i]);
      store_unit(static_cast<T*>(a.r_out) + base + column(u), r[u]);
    }
  }
  if (!a.x) return;
  float v[1] = {0.f};
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int i = 0; i < U; ++i) v[0] = fmaf(r[u][i], r[u][i], v[0]);
  row_sums<NT>(v, part[1]);
  const float s = rsqrtf(fmaf(v[0], over, a.eps));
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    if (column(u) >= d) continue;
    float w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) w[i] = 1.f;
    if (a.w) load_unit(static_cast<const T*>(a.w) + column(u), w);
#pragma unroll
    for (int i = 0; i < U; ++i) w[i] *= r[u][i] * s;
    store_unit(static_cast<T*>(a.x) + base + column(u), w);
  }
}

// Sums over rows: every workgroup adds up the rows it takes (its first, then every
// G-th) in registers and leaves a partial sum of each column.
constexpr int kNormParts = 512;
constexpr int kSumW = 0, kSumPost = 1, kSumGate = 2;
__host__ __device__ inline int norm_parts(int L, int rows) {
  const int n = (L + rows - 1) / rows;
  return n < kNormParts ? n : kNormParts;
}

template <typename T, typename TY, typename TX, int NT, int EPT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_backward_kernel(
    ResidualNormBackwardArgs a, float* sums) {
  constexpr int U = 16 / sizeof(T), NV = EPT / U, ROWS = NT < 256 ? 256 / NT : 1;
  __shared__ float part[2][2][3][16];
  const int t = threadIdx.x % NT, sub = threadIdx.x / NT, d = a.d;
  const T* gate = static_cast<const T*>(a.gate);
  const float over = 1.f / d;
  auto column = [&](int u) { return (u * NT + t) * U; };
  float total[3][NV][U] = {};
  int turn = 0;
  for (size_t row = static_cast<size_t>(blockIdx.x) * ROWS + sub; row < static_cast<size_t>(a.L);
       row += static_cast<size_t>(gridDim.x) * ROWS, turn ^= 1) {
    const size_t base = row * d;
    float dr[NV][U], r[NV][U], dx[NV][U], y[NV][U];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
#pragma unroll
      for (int i = 0; i < U; ++i) dr[u][i] = r[u][i] = dx[u][i] = y[u][i] = 0.f;
      if (column(u) >= d) continue;
      if (a.dr_out) load_unit(static_cast<const T*>(a.dr_out) + base + column(u), dr[u]);
      if (a.dx) {
        load_unit(static_cast<const T*>(a.r_out) + base + column(u), r[u]);
        load_unit(static_cast<const TX*>(a.dx) + base + column(u), dx[u]);
      }
      if (a.y) load_unit(static_cast<const TY*>(a.y) + base + column(u), y[u]);
    }
    float v[3] = {0.f, 0.f, 0.f};  // sums of r1^2, p r1, y^2
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) w[i] = 1.f;
      if (a.w && column(u) < d) load_unit(static_cast<const T*>(a.w) + column(u), w);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        v[0] = fmaf(r[u][i], r[u][i], v[0]);
        v[1] = fmaf(dx[u][i] * w[i], r[u][i], v[1]);
        v[2] = fmaf(y[u][i], y[u][i], v[2]);
      }
    }
    row_sums<NT>(v, part[turn][0]);
    if (a.dx) {
      const float s = rsqrtf(fmaf(v[0], over, a.eps)), c = s * s * s * (v[1] * over);
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float w[U];
#pragma unroll
        for (int i = 0; i < U; ++i) w[i] = 1.f;
        if (a.w && column(u) < d) load_unit(static_cast<const T*>(a.w) + column(u), w);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          dr[u][i] += s * (dx[u][i] * w[i]) - c * r[u][i];
          total[kSumW][u][i] = fmaf(dx[u][i], r[u][i] * s, total[kSumW][u][i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (column(u) < d) store_unit(static_cast<T*>(a.dr) + base + column(u), dr[u]);
    if (!a.y) continue;
    const float b = a.post ? rsqrtf(fmaf(v[2], over, a.eps)) : 1.f;
    float row_gate = a.alpha;
    if (a.gate_kind == kGateToken) row_gate *= load_one(gate + row);
    float m[2] = {0.f, 0.f};  // sums of q y, dr n
    float q[NV][U];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float w[U], g[U], dg[U];
#pragma unroll
      for (int i = 0; i < U; ++i) w[i] = g[i] = 1.f;
      if (column(u) < d) {
        if (a.post_w) load_unit(static_cast<const T*>(a.post_w) + column(u), w);
        if (a.gate_kind == kGateColumn || a.gate_kind == kGateFull)
          load_unit(gate + (a.gate_kind == kGateFull ? base : 0) + column(u), g);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float dn = row_gate * g[i] * dr[u][i], yb = y[u][i] * b;
        q[u][i] = dn * w[i];
        dg[i] = a.alpha * dr[u][i] * (yb * w[i]);
        m[0] = fmaf(q[u][i], y[u][i], m[0]);
        m[1] += dg[i];
        total[kSumPost][u][i] = fmaf(dn, yb, total[kSumPost][u][i]);
        total[kSumGate][u][i] += dg[i];
      }
      if (a.gate_kind == kGateFull && a.dgate && column(u) < d)
        store_unit(static_cast<T*>(a.dgate) + base + column(u), dg);
    }
    const bool gate_sum = a.gate_kind == kGateToken && a.dgate;
    if (a.post || gate_sum) row_sums<NT>(m, part[turn][1]);
    if (gate_sum && t == 0) static_cast<float*>(a.dgate)[row] = m[1];
    if (!a.dy) continue;
    const float c = a.post ? b * b * b * (m[0] * over) : 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (column(u) >= d) continue;
#pragma unroll
      for (int i = 0; i < U; ++i) q[u][i] = b * q[u][i] - c * y[u][i];
      store_unit(static_cast<TY*>(a.dy) + base + column(u), q[u]);
    }
  }
  if (!sums) return;
  // the ROWS rows at a time of a workgroup are parts of their own
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (column(u) < d)
        store_unit(sums + ((static_cast<size_t>(blockIdx.x) * ROWS + sub) * 3 + k) * d + column(u),
                   total[k][u]);
}

// The partial sums in part order; 64 columns by 16 runs of the parts a workgroup.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* sums, int parts, int d,
                                                        float* dw, float* dpost, float* dgate) {
  __shared__ float4 run[16][17];
  float* out = blockIdx.y == kSumW ? dw : blockIdx.y == kSumPost ? dpost : dgate;
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 15) * 4, z = threadIdx.x >> 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d) {
    const int per = (parts + 15) / 16, end = min(parts, (z + 1) * per);
    for (int p = z * per; p < end; ++p) {
      const float4 v =
          *reinterpret_cast<const float4*>(sums + (static_cast<size_t>(p) * 3 + blockIdx.y) * d + c);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  run[z][threadIdx.x & 15] = s;
  __syncthreads();
  if (z != 0 || c >= d) return;
  for (int i = 1; i < 16; ++i) {
    const float4 v = run[i][threadIdx.x];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  *reinterpret_cast<float4*>(out + c) = s;
}

template <typename T, typename TY>
static void run_norm(const ResidualNormArgs& a, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.L), quads = (rows + 3) / 4;
  if (a.d <= 512) residual_norm_kernel<T, TY, 64, 8><<<quads, 256, 0, s>>>(a);
  else if (a.d <= 1024) residual_norm_kernel<T, TY, 64, 16><<<quads, 256, 0, s>>>(a);
  else if (a.d <= 2048) residual_norm_kernel<T, TY, 256, 8><<<rows, 256, 0, s>>>(a);
  else if (a.d <= 4096) residual_norm_kernel<T, TY, 256, 16><<<rows, 256, 0, s>>>(a);
  else if (a.d <= 8192) residual_norm_kernel<T, TY, 256, 32><<<rows, 256, 0, s>>>(a);
  else residual_norm_kernel<T, TY, 1024, 16><<<rows, 1024, 0, s>>>(a);
}

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t s) {
  if (!a.bf16) run_norm<float, float>(a, s);
  else if (a.y_bf16) run_norm<uint16_t, uint16_t>(a, s);
  else run_norm<uint16_t, float>(a, s);
  return hipGetLastError();
}

static int norm_rows_at_a_time(int d) { return d <= 512 ? 4 : 1; }
size_t residual_norm_backward_ws_bytes(int bf16, int L, int d) {
  const int rows = norm_rows_at_a_time(d);
  return static_cast<size_t>(norm_parts(L, rows)) * rows * 3 * d * 4;
}
template <typename T, typename TY, typename TX>
static void run_norm_backward(const ResidualNormBackwardArgs& a, float* sums, hipStream_t s) {
  const unsigned nb = norm_parts(a.L, norm_rows_at_a_time(a.d));
  if (a.d <= 512) residual_norm_backward_kernel<T, TY, TX, 64, 8><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 2048)
    residual_norm_backward_kernel<T, TY, TX, 256, 8><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 4096)
    residual_norm_backward_kernel<T, TY, TX, 256, 16><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 8192)
    residual_norm_backward_kernel<T, TY, TX, 1024, 8><<<nb, 1024, 0, s>>>(a, sums);
  else
    residual_norm_backward_kernel<T, TY, TX, 1024, 16><<<nb, 1024, 0, s>>>(a, sums);
}
hipError_t launch_residual_norm_backward(const ResidualNormBackwardArgs& a, float* ws,
                                         hipStream_t s) {
  float* dgate = a.gate_kind == kGateColumn ? static_cast<float*>(a.dgate) : nullptr;
  float* sums = a.dw || a.dpost_w || dgate ? ws : nullptr;
  if (a.L > 0) {
    if (!a.bf16) run_norm_backward<float, float, float>(a, sums, s);
    else if (a.y_bf16 && a.dx_bf16) run_norm_backward<uint16_t, uint16_t, uint16_t>(a, sums, s);
    else if (a.y_bf16) run_norm_backward<uint16_t, uint16_t, float>(a, sums, s);
    else if (a.dx_bf16) run_norm_backward<uint16_t, float, uint16_t>(a, sums, s);
    else run_norm_backward<uint16_t, float, float>(a, sums, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dw || a.dpost_w || dgate) {
    const int rows = norm_rows_at_a_time(a.d), parts = norm_parts(a.L, rows) * rows;
    norm_sums_kernel<<<dim3((a.d + 63) / 64, 3), 256, 0, s>>>(sums, parts, a.d, a.dw, a.dpost_w,
                                                              dgate);
  }
  return hipGetLastError();
}

}  // namespace omni
