// Rows made 8-bit integers: s = max |x| / 127 (float32), q = x / s rounded to
// the nearest integer, ties to even.  The quotient is decided exactly: the
// remainder x - q s of a candidate q next to it fits in float32 (q has 7
// bits, and the remainder is a multiple of the smaller operand's last place
// no larger than s), so one fma gives it without rounding and a comparison
// with s / 2 settles the neighbour and the tie.
#include "device.hpp"
#include "launch.hpp"

namespace omni {

__device__ __forceinline__ float4 qload4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 qload4(const uint16_t* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y));
}

// x / s rounded to the nearest integer, ties to even; |x| <= 127.5 s
__device__ __forceinline__ int nearest_quotient(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x), h = 0.5f * s;
  const float odd = fabsf(q) - 2.f * floorf(0.5f * fabsf(q));
  if (r > h || (r == h && odd != 0.f)) q += 1.f;
  else if (r < -h || (r == -h && odd != 0.f)) q -= 1.f;
  return static_cast<int>(fminf(fmaxf(q, -127.f), 127.f));
}

// one workgroup per row
template <typename T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* x, int8_t* q, float* scale,
                                                            int k) {
  __shared__ float part[4];
  const size_t row = blockIdx.x;
  const T* xr = x + row * k;
  float top = 0.f;
  for (int c = threadIdx.x * 4; c < k; c += 1024) {
    const float4 v = qload4(xr + c);
    top = fmaxf(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))), top);
  }
  top = wave_max(top);
  if (lane() == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float s = top / 127.f;
  if (threadIdx.x == 0) scale[row] = s;
  // rows whose scale is tiny are lifted by 2^64 (exact), so that 1 / s and
  // the remainders stay normal numbers
  const float lift = s < 0x1p-90f ? 0x1p64f : 1.f, ss = s * lift;
  const float inv = s > 0.f ? 1.f / ss : 0.f;
  for (int c = threadIdx.x * 4; c < k; c += 1024) {
    const float4 v = qload4(xr + c);
    char4 o;
    o.x = static_cast<signed char>(nearest_quotient(v.x * lift, ss, inv));
    o.y = static_cast<signed char>(nearest_quotient(v.y * lift, ss, inv));
    o.z = static_cast<signed char>(nearest_quotient(v.z * lift, ss, inv));
    o.w = static_cast<signed char>(nearest_quotient(v.w * lift, ss, inv));
    if (s == 0.f) o = make_char4(0, 0, 0, 0);
    *reinterpret_cast<char4*>(q + row * k + c) = o;
  }
}

hipError_t launch_quantize_rows(int bf16, int R, int k, const void* x, int8_t* q, float* scale,
                                hipStream_t s) {
  if (bf16)
    quantize_rows_kernel<<<R, 256, 0, s>>>(static_cast<const uint16_t*>(x), q, scale, k);
  else
    quantize_rows_kernel<<<R, 256, 0, s>>>(static_cast<const float*>(x), q, scale, k);
  return hipGetLastError();
}

}  // namespace omni
