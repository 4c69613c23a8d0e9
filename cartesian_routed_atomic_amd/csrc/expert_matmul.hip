// Products with experts that are matrices, the tasks sorted by expert:
//   out[o(m), :] = x[r(m), :] W[e]^T      for off[e] <= m < off[e + 1]
// (or times W[e], the input gradient), the weight gradient
//   dW[e] = sum_m dy[o(m), :]^T x[r(m), :]
// and the same forward product over 8-bit integers with a scale for each row
// of x and each row of W.
//
// First form: one 64 x 64 output tile per workgroup of 256 threads, 4 x 4
// sums per thread, 16 contraction steps at a time through LDS.
#include "device.hpp"
#include "launch.hpp"

namespace omni {

constexpr int TM = 64, TN = 64, TK = 16;

// Row tiles of the experts, found by every wave for itself: lane l counts the
// tiles of q consecutive experts, a prefix sum over the lanes finds the lane
// that owns row tile `rt`, and that lane's experts are walked.  Offsets are
// clamped to [0, M] and to ascending order, so no value of theirs can lead a
// read or write outside the row lists.
struct ExpertTile {
  int e, m0, m1;  // expert, first task of the tile, end of the tile (m0 == m1: none)
};
__device__ __forceinline__ void expert_range(const int32_t* off, int e, int M, int& lo, int& hi) {
  lo = min(max(off[e], 0), M);
  hi = min(max(off[e + 1], lo), M);
}
__device__ ExpertTile find_expert_tile(const int32_t* off, int E, int M, int bm, int rt) {
  const int l = lane(), q = (E + kWave - 1) / kWave;
  int mine = 0;
  for (int i = 0; i < q; ++i) {
    const int e = l * q + i;
    if (e < E) {
      int lo, hi;
      expert_range(off, e, M, lo, hi);
      mine += (hi - lo + bm - 1) / bm;
    }
  }
  const int upto = wave_prefix_sum(mine);
  const uint64_t past = __ballot(upto > rt);
  if (past == 0) return {0, 0, 0};
  const int owner = __ffsll(static_cast<long long>(past)) - 1;
  int left = rt - (__builtin_amdgcn_readlane(upto, owner) - __builtin_amdgcn_readlane(mine, owner));
  for (int i = 0; i < q; ++i) {
    const int e = owner * q + i;
    if (e >= E) break;
    int lo, hi;
    expert_range(off, e, M, lo, hi);
    const int t = (hi - lo + bm - 1) / bm;
    if (left < t) return {e, lo + left * bm, min(hi, lo + (left + 1) * bm)};
    left -= t;
  }
  return {0, 0, 0};
}

__device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ int to_acc(int8_t v) { return v; }
__device__ __forceinline__ float to_acc(uint16_t v) { return to_f(v); }
__device__ __forceinline__ float to_acc(float v) { return v; }
template <typename T> struct AccOf { using type = float; };
template <> struct AccOf<int8_t> { using type = int; };

// float32 -> bf16, nearest even (NaN stays NaN)
__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + __expf(-g)) * u; }

template <typename T, typename TO, bool TRANS, bool SWIGLU>
__global__ __launch_bounds__(256) void expert_tile_kernel(ExpertMatmulArgs a) {
  using Acc = typename AccOf<T>::type;
  __shared__ Acc sa[TK][TM + 1], sb[TK][TN + 1], sc[SWIGLU ? TK : 1][TN + 1];
  const int tid = threadIdx.x;
  // inner length, output width, and W's strides over (output column, inner)
  const int K = TRANS ? a.n : a.k, N = TRANS ? a.k : a.n;
  const int n_nt = (N + TN - 1) / TN;
  const int rt = blockIdx.x / n_nt, n0 = (blockIdx.x - rt * n_nt) * TN;
  ExpertTile t{0, rt * TM, min(a.M, (rt + 1) * TM)};
  if (a.offsets) t = find_expert_tile(a.offsets, a.E, a.M, TM, rt);
  if (t.m0 >= t.m1) return;
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w) +
               static_cast<size_t>(t.e) * (SWIGLU ? 2 : 1) * a.n * a.k;
  Acc acc[4][4] = {}, acu[4][4] = {};
  const int ty = tid >> 4, tx = tid & 15;
  for (int k0 = 0; k0 < K; k0 += TK) {
    for (int i = tid; i < TM * TK; i += 256) {
      const int r = i / TK, c = k0 + i % TK, m = t.m0 + r;
      Acc v = 0;
      if (m < t.m1 && c < K) {
        const int row = a.x_row ? a.x_row[m] : m;
        if (row >= 0 && row < a.R) v = to_acc(x[static_cast<size_t>(row) * K + c]);
      }
      sa[i % TK][r] = v;
    }
    for (int i = tid; i < TN * TK; i += 256) {
      const int j = TRANS ? i % TN : i / TK, c = TRANS ? i / TN : i % TK;
      const bool in = n0 + j < N && k0 + c < K;
      const size_t at = TRANS ? static_cast<size_t>(k0 + c) * a.k + (n0 + j)
                              : static_cast<size_t>(n0 + j) * a.k + (k0 + c);
      sb[c][j] = in ? to_acc(w[at]) : Acc(0);
      if constexpr (SWIGLU)
        sc[c][j] = in ? to_acc(w[at + static_cast<size_t>(a.n) * a.k]) : Acc(0);
    }
    __syncthreads();
    for (int c = 0; c < TK; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
          acc[i][j] += sa[c][ty * 4 + i] * sb[c][tx * 4 + j];
          if constexpr (SWIGLU) acu[i][j] += sa[c][ty * 4 + i] * sc[c][tx * 4 + j];
        }
    __syncthreads();
  }
  TO* out = static_cast<TO*>(a.out);
  for (int i = 0; i < 4; ++i) {
    const int m = t.m0 + ty * 4 + i;
    if (m >= t.m1) continue;
    const int row = a.out_row ? a.out_row[m] : m;
    if (row < 0 || row >= a.Ro) continue;
    const int xr = a.x_row ? a.x_row[m] : m;
    const float rs = a.x_scale && xr >= 0 && xr < a.R ? a.x_scale[xr] : 1.f;
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + tx * 4 + j;
      if (c >= N) continue;
      const float* ws = a.w_scale ? a.w_scale + static_cast<size_t>(t.e) * (SWIGLU ? 2 : 1) * a.n
                                  : nullptr;
      float v = static_cast<float>(acc[i][j]);
      if (ws) v = v * rs * ws[c];
      if constexpr (SWIGLU) {
        float u = static_cast<float>(acu[i][j]);
        if (ws) u = u * rs * ws[a.n + c];
        v = silu_mul(v, u);
      }
      put(out + static_cast<size_t>(row) * N + c, v);
    }
  }
}

// dW tile: 64 x 64 of one expert, its tasks in order
template <typename T>
__global__ __launch_bounds__(256) void expert_wgrad_kernel(ExpertWgradArgs a) {
  __shared__ float sa[TK][TM + 1], sb[TK][TN + 1];
  const int tid = threadIdx.x, n_kt = (a.k + TN - 1) / TN, n_nt = (a.n + TM - 1) / TM;
  const int e = blockIdx.x / (n_kt * n_nt), r = blockIdx.x - e * n_kt * n_nt;
  const int n0 = r / n_kt * TM, c0 = r % n_kt * TN;
  int lo, hi;
  expert_range(a.offsets, e, a.M, lo, hi);
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  float acc[4][4] = {};
  const int ty = tid >> 4, tx = tid & 15;
  for (int m0 = lo; m0 < hi; m0 += TK) {
    for (int i = tid; i < TK * 64; i += 256) {
      const int m = m0 + i / 64, c = i % 64;
      float va = 0.f, vb = 0.f;
      if (m < hi) {
        const int ry = a.dy_row ? a.dy_row[m] : m, rx = a.x_row ? a.x_row[m] : m;
        const bool in = ry >= 0 && ry < a.Ry && rx >= 0 && rx < a.R;
        if (in && n0 + c < a.n) va = to_f(dy[static_cast<size_t>(ry) * a.n + n0 + c]);
        if (in && c0 + c < a.k) vb = to_f(x[static_cast<size_t>(rx) * a.k + c0 + c]);
      }
      sa[i / 64][c] = va;
      sb[i / 64][c] = vb;
    }
    __syncthreads();
    for (int c = 0; c < TK; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[c][ty * 4 + i], sb[c][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int rr = n0 + ty * 4 + i, cc = c0 + tx * 4 + j;
      if (rr < a.n && cc < a.k)
        a.dw[(static_cast<size_t>(e) * a.n + rr) * a.k + cc] = acc[i][j];
    }
}

// sum of ceil(c_e / bm) over at most min(E, M) experts with tasks
static long long expert_row_tiles(int M, int E, int bm) {
  const long long used = E < M ? E : M;
  return (M + used * (bm - 1)) / bm;
}
static long long product_blocks(const ExpertMatmulArgs& a) {
  const int N = a.transpose ? a.k : a.n;
  return expert_row_tiles(a.M, a.E, TM) * ((N + TN - 1) / TN);
}
static long long wgrad_blocks(const ExpertWgradArgs& a) {
  return static_cast<long long>(a.E) * ((a.n + TM - 1) / TM) * ((a.k + TN - 1) / TN);
}
bool expert_matmul_grid_fits(const ExpertMatmulArgs& a) {
  return product_blocks(a) < (1ll << 32) / 256;
}
bool expert_wgrad_grid_fits(const ExpertWgradArgs& a) {
  return wgrad_blocks(a) < (1ll << 32) / 256;
}

template <typename T, typename TO>
static hipError_t run_product(const ExpertMatmulArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(product_blocks(a)));
  if (a.transpose) expert_tile_kernel<T, TO, true, false><<<grid, 256, 0, s>>>(a);
  else if (a.swiglu) expert_tile_kernel<T, TO, false, true><<<grid, 256, 0, s>>>(a);
  else expert_tile_kernel<T, TO, false, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_expert_matmul(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.type == kRowsI8)
    return a.out_bf16 ? run_product<int8_t, uint16_t>(a, s) : run_product<int8_t, float>(a, s);
  return a.type == kRowsBf16 ? run_product<uint16_t, uint16_t>(a, s)
                             : run_product<float, float>(a, s);
}

hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t s) {
  const long long nb = wgrad_blocks(a);
  if (a.bf16) expert_wgrad_kernel<uint16_t><<<static_cast<unsigned>(nb), 256, 0, s>>>(a);
  else expert_wgrad_kernel<float><<<static_cast<unsigned>(nb), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace omni
