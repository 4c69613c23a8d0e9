// Rows made 8-bit integers: s = max |x| / 127 (float32), q = x / s rounded to
// the nearest integer, ties to even.  The quotient is decided exactly: the
// remainder x - q s of a candidate q next to it fits in float32 (q has 7
// bits, and the remainder is a multiple of the smaller operand's last place
// no larger than s), so one fma gives it without rounding and a comparison
// with s / 2 settles the neighbour and the tie.  Candidates off by one are
// rare (quotients within float32 rounding of a half), so that part runs only
// where a lane of the wave needs it.
//
// The maximum keeps a NaN: a row with a NaN or an infinity has that as its scale
// and q 0, so that its products are NaN instead of a finite number.
//
// A row is read once, kept in registers and written once.  8192 x 2048 takes 15.0
// us from float32 (5.6 TB/s), bound by HBM, and 14.3 us from bf16 (3.5 TB/s): 10
// vector instructions per element are 4-5 us of the SIMDs, and since all 8192
// waves are resident at once they read (6.4 us at a copy's rate), compute and
// write (3.2 us) one after the other instead of side by side.
#include "device.hpp"
#include "launch.hpp"

namespace omni {

constexpr int kUnit = 16;  // consecutive elements of a lane: one 16-byte store

__device__ __forceinline__ void load_unit(const float* p, float (&v)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    v[i] = f.x;
    v[i + 1] = f.y;
    v[i + 2] = f.z;
    v[i + 3] = f.w;
  }
}
__device__ __forceinline__ void load_unit(const uint16_t* p, float (&v)[kUnit]) {
#pragma unroll
  for (int i = 0; i < kUnit; i += 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + i);
    v[i] = bf_lo(u.x);
    v[i + 1] = bf_hi(u.x);
    v[i + 2] = bf_lo(u.y);
    v[i + 3] = bf_hi(u.y);
    v[i + 4] = bf_lo(u.z);
    v[i + 5] = bf_hi(u.z);
    v[i + 6] = bf_lo(u.w);
    v[i + 7] = bf_hi(u.w);
  }
}

// The row's scale, and what its quotients are formed with: rows whose scale is
// tiny are lifted by 2^64 (exact), so that 1 / s and the remainders stay
// normal numbers.  A scale of 0 and one that is not finite have no quotients.
struct RowScale {
  float s, lift, lifted, inv;
  bool any;  // positive and finite
};
__device__ __forceinline__ RowScale row_scale(float top) {
  RowScale r;
  r.s = top / 127.f;
  r.any = r.s > 0.f && r.s < INFINITY;
  r.lift = r.s < 0x1p-90f ? 0x1p64f : 1.f;
  r.lifted = r.s * r.lift;
  r.inv = r.any ? 1.f / r.lifted : 0.f;
  return r;
}

// q of one unit with every case decided: scales without quotients (q is 0),
// tiny scales, halves
__device__ void exact_unit(const float (&x)[kUnit], const RowScale& s, uint32_t (&w)[kUnit / 4]) {
  const float half = 0.5f * s.lifted;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    const float v = x[i] * s.lift;
    float q = rintf(v * s.inv);
    const float r = fmaf(-q, s.lifted, v), a = fabsf(r);
    const bool odd = (static_cast<int>(q) & 1) != 0;
    if (a > half || (a == half && odd)) q += copysignf(1.f, r);
    const int n = s.any ? static_cast<int>(fminf(fmaxf(q, -127.f), 127.f)) : 0;
    const uint32_t b = static_cast<uint32_t>(n & 255) << (8 * (i & 3));
    w[i >> 2] = (i & 3) ? w[i >> 2] | b : b;
  }
}
// Adding 1.5 * 2^23 leaves x / s as an integer in the low bits: its low byte is
// q.  The vector work per element counts beside HBM, so the common case is one
// fma, one subtraction, one fma for the remainder and the packing (8192 x 2048
// bf16: 15.1 us when measured; 16.6 with every element decided on its own).
__device__ __forceinline__ void store_unit(int8_t* p, const float (&x)[kUnit], const RowScale& s) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  uint32_t t[kUnit], w[kUnit / 4];
  float worst = 0.f;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    const float m = fmaf(x[i], s.inv, kMagic);
    t[i] = __float_as_uint(m);
    worst = fmaxf(worst, fabsf(fmaf(kMagic - m, s.s, x[i])));
  }
  if (__any(!(worst < 0.5f * s.s) || s.lift != 1.f || !s.any)) {
    exact_unit(x, s, w);
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; i += 4) {
      const uint32_t lo = __builtin_amdgcn_perm(t[i + 1], t[i], 0x0c0c0400);
      const uint32_t hi = __builtin_amdgcn_perm(t[i + 3], t[i + 2], 0x04000c0c);
      w[i >> 2] = lo | hi;
    }
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float unit_max(const float (&v)[kUnit], float top) {
#pragma unroll
  for (int i = 0; i < kUnit; ++i) top = __builtin_elementwise_maximum(top, fabsf(v[i]));
  return top;
}

// NT threads per row (a wave, or a whole workgroup of 256), the row in NV units
// per thread; NV = 0: rows too long for that, read twice.
template <typename T, int NT, int NV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* __restrict__ x,
                                                            int8_t* __restrict__ q,
                                                            float* __restrict__ scale, int R,
                                                            int k) {
  __shared__ float part[4];
  const int t = threadIdx.x % NT;
  const size_t row = static_cast<size_t>(blockIdx.x) * (256 / NT) + threadIdx.x / NT;
  if (row >= static_cast<size_t>(R)) return;  // NT == 256: never
  const T* xr = x + row * k;
  int8_t* qr = q + row * k;
  float v[NV ? NV : 1][kUnit];
  float top = 0.f;
  if constexpr (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (u * NT + t) * kUnit;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[u][i] = 0.f;
      if (c < k) load_unit(xr + c, v[u]);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) top = unit_max(v[u], top);
  } else {
    // unsigned: rows may have up to 2^31 - 16 columns, and the last step ends past them
    for (uint32_t c = t * kUnit; c < static_cast<uint32_t>(k); c += NT * kUnit) {
      load_unit(xr + c, v[0]);
      top = unit_max(v[0], top);
    }
  }
  const bool any_nan = __any(top != top);
  top = any_nan ? __builtin_nanf("") : wave_max(top);
  if constexpr (NT > kWave) {
    if (lane() == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(part[0], part[1]),
                                        __builtin_elementwise_maximum(part[2], part[3]));
  }
  const RowScale s = row_scale(top);
  if (t == 0) scale[row] = s.s;
  if constexpr (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (u * NT + t) * kUnit;
      if (c < k) store_unit(qr + c, v[u], s);
    }
  } else {
    for (uint32_t c = t * kUnit; c < static_cast<uint32_t>(k); c += NT * kUnit) {
      load_unit(xr + c, v[0]);
      store_unit(qr + c, v[0], s);
    }
  }
}

// rows of up to 128 units: a wave each, longer ones a workgroup
long long quantize_rows_blocks(int R, int k) { return k / kUnit <= 128 ? (R + 3ll) / 4 : R; }

template <typename T>
static void run_quantize(const T* x, int8_t* q, float* scale, int R, int k, hipStream_t s) {
  const int units = k / kUnit;
  const unsigned nb = static_cast<unsigned>(quantize_rows_blocks(R, k));
  if (units <= 64) quantize_rows_kernel<T, 64, 1><<<nb, 256, 0, s>>>(x, q, scale, R, k);
  else if (units <= 128) quantize_rows_kernel<T, 64, 2><<<nb, 256, 0, s>>>(x, q, scale, R, k);
  else if (units <= 256) quantize_rows_kernel<T, 256, 1><<<nb, 256, 0, s>>>(x, q, scale, R, k);
  else if (units <= 512) quantize_rows_kernel<T, 256, 2><<<nb, 256, 0, s>>>(x, q, scale, R, k);
  else if (units <= 1024) quantize_rows_kernel<T, 256, 4><<<nb, 256, 0, s>>>(x, q, scale, R, k);
  else quantize_rows_kernel<T, 256, 0><<<nb, 256, 0, s>>>(x, q, scale, R, k);
}

hipError_t launch_quantize_rows(int bf16, int R, int k, const void* x, int8_t* q, float* scale,
                                hipStream_t s) {
  if (bf16) run_quantize(static_cast<const uint16_t*>(x), q, scale, R, k, s);
  else run_quantize(static_cast<const float*>(x), q, scale, R, k, s);
  return hipGetLastError();
}

}  // namespace omni
