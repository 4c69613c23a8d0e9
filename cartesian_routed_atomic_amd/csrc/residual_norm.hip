// The norm after a block with its gate and residual scale, fused with the norm
// before the next block, and the backward of both:
//   n = y, or y b post_w with b = 1 / sqrt(mean y^2 + eps)
//   r1 = r + alpha g n,   x = r1 a w with a = 1 / sqrt(mean r1^2 + eps)
// and, for p = dx w,
//   dr = dr_out + a p - r1 a^3 mean(p r1),   dw = sum_rows dx r1 a
//   dgate = alpha dr n,   dn = alpha g dr,   q = dn post_w
//   dy = b q - y b^3 mean(q y),   dpost_w = sum_rows dn y b
// Both are HBM-bound: a row is read once, kept in registers, and written once.
// 8192 x 2048, bfloat16 with a float32 y: forward 34 us, 4.9 TB/s; backward with
// float32 dx 60 us, 5.0 TB/s, and 6 for the join of the column sums.
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
  for (int i = 0; i < N; ++i) {
    if constexpr (NT >= kWave) {
      v[i] = wave_sum(v[i]);
    } else {
#pragma unroll
      for (int o = NT / 2; o > 0; o >>= 1) v[i] += __shfl_xor(v[i], o);
    }
  }
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
      for (int w = 0; w < NT / kWave; ++w) v[i] += part[i][threadIdx.x / NT * (NT / kWave) + w];
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
constexpr int kSumW = 0, kSumPost = 1, kSumGate = 2;

// 16 bytes of a row as loaded
template <typename T, int U>
struct Unit {
  uint4 v[U * sizeof(T) / 16];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(U * sizeof(T) / 16); ++i)
      v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(U * sizeof(T) / 16); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&f)[U]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < U; i += 4) {
        f[i] = __uint_as_float(v[i / 4].x);
        f[i + 1] = __uint_as_float(v[i / 4].y);
        f[i + 2] = __uint_as_float(v[i / 4].z);
        f[i + 3] = __uint_as_float(v[i / 4].w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; i += 8) {
        const uint4 u = v[i / 8];
        f[i] = bf_lo(u.x);
        f[i + 1] = bf_hi(u.x);
        f[i + 2] = bf_lo(u.y);
        f[i + 3] = bf_hi(u.y);
        f[i + 4] = bf_lo(u.z);
        f[i + 5] = bf_hi(u.z);
        f[i + 6] = bf_lo(u.w);
        f[i + 7] = bf_hi(u.w);
      }
    }
  }
};

// NT threads per row, as in the forward.  The row's sums are formed in one pass and
// meet once: with t = g post_w y, the mean of q y is that of alpha t dr, and dr's
// three terms give three sums.  What a row's registers hold:
// kAhead: the row and what belongs to its columns, and the next row's loads are under
//   way meanwhile;
// kHeld: the row (longer ones);
// kTwice: nothing, it is read again for the results, from the L2 or the chip's last
//   cache (longer still, where holding spills: 1024 x 16384 from bfloat16 with float32
//   dx and y 217 us for 403, 2048 x 8192 float32 118 for 121, but from bfloat16, which
//   does not spill, 85 for 80; without a y 1024 x 16384 float32 71 for 57).
enum RowIn { kAhead, kHeld, kTwice };
// Y: there is a y, and with it what belongs to it.  A norm alone takes half the registers:
// 11984 x 632 from bfloat16 17 us where the kernel for both took 27.
template <typename T, typename TY, typename TX, int NT, int EPT, RowIn IN, bool Y>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_norm_backward_kernel(
    ResidualNormBackwardArgs a, float* sums) {
  constexpr int U = 16 / sizeof(T), NV = EPT / U, ROWS = NT < 256 ? 256 / NT : 1;
  constexpr int NS = Y ? 6 : 2, SUMS = Y ? 3 : 1;
  __shared__ float part[2][NS][16];
  __shared__ __attribute__((aligned(16))) float joined[ROWS > 1 ? ROWS * NT * EPT : 4];
  int t = threadIdx.x % NT;
  const int sub = threadIdx.x / NT, d = a.d;
  const T* gate = static_cast<const T*>(a.gate);
  const float over = 1.f / d;
  auto column = [&](int u) { return (u * NT + t) * U; };
  struct Column {
    Unit<T, U> w, pw, g;  // ones where there are none
  };
  Column kept[NV];
  auto of_column = [&](Column& v, int u) {
    constexpr uint32_t kOne = sizeof(T) == 4 ? 0x3f800000u : 0x3f803f80u;
    v.w.v[0] = v.pw.v[0] = v.g.v[0] = make_uint4(kOne, kOne, kOne, kOne);
    if (column(u) >= d) return;
    if (a.w) v.w.load(static_cast<const T*>(a.w) + column(u));
    if constexpr (Y) {
      if (a.post_w) v.pw.load(static_cast<const T*>(a.post_w) + column(u));
      if (a.gate_kind == kGateColumn) v.g.load(gate + column(u));
    }
  };
  if constexpr (IN == kAhead) {
#pragma unroll
    for (int u = 0; u < NV; ++u) of_column(kept[u], u);
  }
  struct RowUnit {
    Unit<T, U> dr, r, g;
    Unit<TX, U> dx;
    Unit<TY, U> y;
  };
  struct Row {
    RowUnit u[NV];
    float gate;
  };
  auto fetch_unit = [&](RowUnit& v, size_t row, int u) {
    const size_t base = row * d;
    v.dr.clear();
    v.r.clear();
    v.dx.clear();
    v.y.clear();
    v.g.clear();
    if (row >= static_cast<size_t>(a.L) || column(u) >= d) return;
    if (a.dr_out) v.dr.load(static_cast<const T*>(a.dr_out) + base + column(u));
    if (a.dx) {
      v.r.load(static_cast<const T*>(a.r_out) + base + column(u));
      v.dx.load(static_cast<const TX*>(a.dx) + base + column(u));
    }
    if constexpr (Y) {
      v.y.load(static_cast<const TY*>(a.y) + base + column(u));
      if (a.gate_kind == kGateFull) v.g.load(gate + base + column(u));
    }
  };
  auto fetch_gate = [&](size_t row) {
    return Y && row < static_cast<size_t>(a.L) && a.gate_kind == kGateToken ? load_one(gate + row)
                                                                           : 1.f;
  };
  auto fetch = [&](Row& v, size_t row) {
    v.gate = fetch_gate(row);
#pragma unroll
    for (int u = 0; u < NV; ++u) fetch_unit(v.u[u], row, u);
  };
  float total[SUMS][NV][U] = {};
  const size_t step = static_cast<size_t>(gridDim.x) * ROWS;
  const bool full = Y && a.gate_kind == kGateFull;
  int turn = 0;
  // the rows of a workgroup's turn: all its threads take part in the same turns
  size_t row = static_cast<size_t>(blockIdx.x) * ROWS + sub;
  size_t first = static_cast<size_t>(blockIdx.x) * ROWS;
  Row now, then;
  if constexpr (IN != kTwice) fetch(now, row);
  for (; first < static_cast<size_t>(a.L); first += step, row += step, turn ^= 1) {
    const bool live = row < static_cast<size_t>(a.L);
    const size_t base = row * d;
    if constexpr (IN == kAhead) fetch(then, row + step);
    if constexpr (IN == kTwice) now.gate = fetch_gate(row);
    // a unit of the row and its columns' values
    auto unit = [&](int u, RowUnit& x, Column& k) {
      if constexpr (IN == kTwice) {
        // one unit after the other, its addresses formed anew
        __builtin_amdgcn_sched_barrier(0);
        __asm__ volatile("" : "+v"(t)::"memory");
        fetch_unit(x, row, u);
      } else {
        x = now.u[u];
      }
      if constexpr (IN == kAhead) k = kept[u];
      else of_column(k, u);
    };
    float v[NS] = {};  // sums of r1^2, p r1, y^2, t dr_out, t p, t r1
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float r[U], dx[U], y[U], dr[U], wf[U], pf[U], g[U];
      RowUnit x;
      Column k;
      unit(u, x, k);
      x.r.floats(r);
      x.dx.floats(dx);
      x.y.floats(y);
      x.dr.floats(dr);
      k.w.floats(wf);
      k.pw.floats(pf);
      (full ? x.g : k.g).floats(g);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float p = dx[i] * wf[i];
        v[0] = fmaf(r[i], r[i], v[0]);
        v[1] = fmaf(p, r[i], v[1]);
        if constexpr (Y) {
          const float q = g[i] * pf[i] * y[i];
          v[2] = fmaf(y[i], y[i], v[2]);
          v[3] = fmaf(q, dr[i], v[3]);
          v[4] = fmaf(q, p, v[4]);
          v[5] = fmaf(q, r[i], v[5]);
        }
      }
    }
    row_sums<NT>(v, part[turn]);
    const float s = a.dx ? rsqrtf(fmaf(v[0], over, a.eps)) : 0.f;
    // a mean of squares is taken out factor by factor: its root's cube leaves float32's
    // range long before the gradients do
    const float c = a.dx ? v[1] * over * s : 0.f;  // mean(p r1 a)
    float b = 1.f, row_gate = 0.f, back = 0.f;
    if constexpr (Y) {
      if (a.post) b = rsqrtf(fmaf(v[2], over, a.eps));
      // sum of t dr.  Without dx its other terms would be 0 times a y that may be infinite;
      // of finite numbers whose squares pass float32's range, so that a or b is 0, the
      // products may as well, and the row passes nothing
      float qy = a.dx && (s != 0.f || c != 0.f) ? v[3] + s * (v[4] - c * (s * v[5])) : v[3];
      if (b == 0.f && fabsf(v[3]) < INFINITY) qy = 0.f;
      row_gate = a.alpha * now.gate;
      if (a.post) back = row_gate * qy * over * b;  // mean(q y b)
      if (live && a.gate_kind == kGateToken && a.dgate && t == 0)
        static_cast<float*>(a.dgate)[row] = a.alpha * b * qy;
    }
    // a place beyond the last row has no part in the sums either: the root of its mean of
    // zeros may be infinite
    if (ROWS == 1 || live) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float r[U], dx[U], y[U], dr[U], wf[U], pf[U], g[U], dg[U];
        RowUnit x;
        Column k;
        unit(u, x, k);
        x.r.floats(r);
        x.dx.floats(dx);
        x.y.floats(y);
        x.dr.floats(dr);
        k.w.floats(wf);
        k.pw.floats(pf);
        (full ? x.g : k.g).floats(g);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float ra = r[i] * s;
          dr[i] += s * (dx[i] * wf[i] - c * ra);
          total[kSumW][u][i] = fmaf(dx[i], ra, total[kSumW][u][i]);
          if constexpr (Y) {
            const float dn = row_gate * g[i] * dr[i], yb = y[i] * b;
            dg[i] = a.alpha * dr[i] * (yb * pf[i]);
            total[kSumPost][u][i] = fmaf(dn, yb, total[kSumPost][u][i]);
            total[kSumGate][u][i] += dg[i];
            // without a post norm y has no part in dy, infinite or not
            y[i] = a.post ? b * (dn * pf[i] - back * yb) : dn;
          }
        }
        if (column(u) >= d) continue;
        store_unit(static_cast<T*>(a.dr) + base + column(u), dr);
        if constexpr (Y) {
          if (full && a.dgate) store_unit(static_cast<T*>(a.dgate) + base + column(u), dg);
          if (a.dy) store_unit(static_cast<TY*>(a.dy) + base + column(u), y);
        }
      }
    }
    if constexpr (IN == kAhead) now = then;
    if constexpr (IN == kHeld) fetch(now, row + step);
  }
  float* wanted[3] = {a.dw, a.dpost_w,
                      a.gate_kind == kGateColumn ? static_cast<float*>(a.dgate) : nullptr};
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
    if (!wanted[k]) continue;
    // one part is the sum
    float* out = gridDim.x == 1 ? wanted[k]
                                : sums + (static_cast<size_t>(blockIdx.x) * SUMS + k) * d;
    if constexpr (ROWS > 1) {  // the rows at a time of a workgroup, in order
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NV; ++u) store_unit(joined + sub * NT * EPT + column(u), total[k][u]);
      __syncthreads();
      for (int col = threadIdx.x; col < d; col += 256) {
        float x = joined[col];
#pragma unroll
        for (int i = 1; i < ROWS; ++i) x += joined[i * NT * EPT + col];
        out[col] = x;
      }
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (column(u) < d) store_unit(out + column(u), total[k][u]);
    }
  }
}

// The partial sums in part order: 16 columns by 64 runs of the parts a workgroup.
// kinds: sums of a part.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* sums, int parts, int kinds,
                                                        int d, float* dw, float* dpost,
                                                        float* dgate) {
  __shared__ float4 run[64][4];
  float* out = blockIdx.y == kSumW ? dw : blockIdx.y == kSumPost ? dpost : dgate;
  if (!out) return;
  const int l = threadIdx.x & 3, c = blockIdx.x * 16 + l * 4, z = threadIdx.x >> 2;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4& x, const float4& y) {
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  };
  if (c < d) {
    const int per = (parts + 63) / 64, end = min(parts, (z + 1) * per);
#pragma unroll 8
    for (int p = z * per; p < end; ++p)
      add(s, *reinterpret_cast<const float4*>(
                 sums + (static_cast<size_t>(p) * kinds + blockIdx.y) * d + c));
  }
  run[z][l] = s;
  __syncthreads();
  if (z >= 8) return;
  s = run[z * 8][l];
#pragma unroll
  for (int i = 1; i < 8; ++i) add(s, run[z * 8 + i][l]);
  // eight runs are left, in the first 32 lanes: 4 apart
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    const float4 y = make_float4(__shfl_down(s.x, o), __shfl_down(s.y, o), __shfl_down(s.z, o),
                                 __shfl_down(s.w, o));
    add(s, y);
  }
  if (z == 0 && c < d) *reinterpret_cast<float4*>(out + c) = s;
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

// As few threads to a row as hold it: 8192 x 1024 from bfloat16 takes 25 us with 128
// and 38 with 256.  Parts: as many workgroups as the chip holds at a time (two of 256 threads a CU; 8192 x
// 2048: 67 us, with twice the parts 75).
constexpr int kNormParts = 512;
static int norm_threads(int d) {  // of a row
  return d <= 256 ? 32 : d <= 512 ? 64 : d <= 1024 ? 128 : d <= 2048 ? 256 : d <= 8192 ? 512 : 1024;
}
// Rows that four turns of one workgroup hold are one part, without a second launch (4
// rows of 2048: 5.8 us, 10.5 with it).  A norm alone has room for twice the workgroups
// (8192 x 2048 from bfloat16 29 us, with three times as many 31).
static int norm_parts(int L, int d, bool y) {
  const int nt = norm_threads(d), rows = nt < 256 ? 256 / nt : 1, n = (L + rows - 1) / rows;
  const int most = (nt <= 256 ? kNormParts : kNormParts * 256 / nt) * (y ? 1 : 2);
  return n <= 4 ? (n < 1 ? n : 1) : n < most ? n : most;
}
// three sums of a part with a y, one without: those of both
size_t residual_norm_backward_ws_bytes(int bf16, int L, int d) {
  const int with = norm_parts(L, d, true), without = norm_parts(L, d, false);
  if (with <= 1) return 0;
  return static_cast<size_t>(with * 3 > without ? with * 3 : without) * d * 4;
}
template <typename T, typename TY, typename TX, bool Y>
static void run_norm_backward(const ResidualNormBackwardArgs& a, float* sums, hipStream_t s) {
  const unsigned nb = norm_parts(a.L, a.d, Y);
  if (a.d <= 256)
    residual_norm_backward_kernel<T, TY, TX, 32, 8, kAhead, Y><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 512)
    residual_norm_backward_kernel<T, TY, TX, 64, 8, kAhead, Y><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 1024)
    residual_norm_backward_kernel<T, TY, TX, 128, 8, kAhead, Y><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 2048)
    residual_norm_backward_kernel<T, TY, TX, 256, 8, kAhead, Y><<<nb, 256, 0, s>>>(a, sums);
  else if (a.d <= 4096)
    residual_norm_backward_kernel<T, TY, TX, 512, 8, kAhead, Y><<<nb, 512, 0, s>>>(a, sums);
  else if (a.d <= 8192)
    residual_norm_backward_kernel<T, TY, TX, 512, 16, sizeof(T) == 4 && Y ? kTwice : kHeld, Y>
        <<<nb, 512, 0, s>>>(a, sums);
  else
    residual_norm_backward_kernel<T, TY, TX, 1024, 16, sizeof(T) == 4 || Y ? kTwice : kHeld, Y>
        <<<nb, 1024, 0, s>>>(a, sums);
}
hipError_t launch_residual_norm_backward(const ResidualNormBackwardArgs& a, float* ws,
                                         hipStream_t s) {
  float* dgate = a.gate_kind == kGateColumn ? static_cast<float*>(a.dgate) : nullptr;
  float* sums = a.dw || a.dpost_w || dgate ? ws : nullptr;
  if (a.L > 0) {
    if (!a.y) {
      if (!a.bf16) run_norm_backward<float, float, float, false>(a, sums, s);
      else if (a.dx_bf16) run_norm_backward<uint16_t, uint16_t, uint16_t, false>(a, sums, s);
      else run_norm_backward<uint16_t, uint16_t, float, false>(a, sums, s);
    } else if (!a.bf16) run_norm_backward<float, float, float, true>(a, sums, s);
    else if (a.y_bf16 && a.dx_bf16) run_norm_backward<uint16_t, uint16_t, uint16_t, true>(a, sums, s);
    else if (a.y_bf16) run_norm_backward<uint16_t, uint16_t, float, true>(a, sums, s);
    else if (a.dx_bf16) run_norm_backward<uint16_t, float, uint16_t, true>(a, sums, s);
    else run_norm_backward<uint16_t, float, float, true>(a, sums, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int parts = norm_parts(a.L, a.d, a.y), kinds = a.y || a.L == 0 ? 3 : 1;
  if ((a.dw || a.dpost_w || dgate) && parts != 1)
    norm_sums_kernel<<<dim3((a.d + 15) / 16, kinds), 256, 0, s>>>(sums, parts, kinds, a.d, a.dw,
                                                                  a.dpost_w, dgate);
  return hipGetLastError();
}

}  // namespace omni
