// A token's experts and gates from its logits, and the gradient of the logits.
//
// What selects is the score plus the balance bias, s + b.  Scores of different
// experts can lie within float32's rounding of each other, so they are compared
// in float64; without a bias the score grows with the logit, which is compared
// as it stands.
#include "device.hpp"
#include "launch.hpp"

namespace omni {

__device__ __forceinline__ float load_logit(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float load_logit(const uint16_t* p, size_t i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}

// Order-preserving map float64 -> uint64 (never 0), -0 onto +0, NaN as -infinity.
__device__ __forceinline__ uint64_t dkey(double v) {
  if (!(v == v)) v = -INFINITY;
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }

// Gates' weights of a wave's K selected experts (lane k: the k-th's logit z, not
// read from lane K on) over their sum.  Scores are formed relative to the largest,
// so that scores too small for float32 still share out: softmax e^(z - m);
// sigmoid, times e^-m for m = min(largest z, 0): e^(z - m) / (1 + e^z), or
// 1 / (1 + e^-z) where z > 0 (then m = 0).
__device__ __forceinline__ float shared_weight(float z, bool mine, bool sigmoid) {
  const float top = wave_max(mine ? z : -INFINITY);
  float e;
  if (sigmoid) {
    const float m = fminf(top, 0.f);
    e = z > 0.f ? 1.f / (1.f + expf(-z)) : expf(z - m) / (1.f + expf(z));
  } else {
    e = expf(z - top);
  }
  if (!mine) e = 0.f;
  const float sum = wave_sum(e);
  return top == -INFINITY && !(sum > 0.f) && !__any(mine && z != z) ? 0.f : e / sum;
}

// One wave per token; lane l holds experts l, l + 64, ..  The K best are taken one
// at a time: every lane's best, the wave's best of those, which is then struck off.
template <typename T, int V>
__global__ __launch_bounds__(64) void expert_route_kernel(ExpertRouteArgs a) {
  __shared__ double value[V * 64];
  const int l = lane(), E = a.E;
  const size_t t = blockIdx.x;
  const T* row = static_cast<const T*>(a.logits) + t * E;
  float z[V];
  double s[V], c[V];
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l + v * 64;
    z[v] = e < E ? load_logit(row, e) : -INFINITY;
    bad |= z[v] != z[v] || z[v] == INFINITY;
    top = fmaxf(top, z[v]);
  }
  bad = __any(bad) && !a.sigmoid;
  if (!a.sigmoid) {
    top = wave_max(top);
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = z[v] == -INFINITY ? 0.0 : exp(static_cast<double>(z[v]) - top);
      sum += s[v];
    }
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = bad ? __builtin_nan("") : sum > 0.0 ? s[v] / sum : 0.0;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = sigmoid64(z[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l + v * 64;
    c[v] = a.bias && e < E ? s[v] + a.bias[e] : z[v];
    if (a.score && e < E) a.score[t * E + e] = static_cast<float>(s[v]);
  }
  uint64_t stay = ~0ull;
  const int size = E / a.groups;
  if (a.top_groups < a.groups) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const double m = !a.bias && a.group_best == 2 ? s[v] : c[v];
      value[l + v * 64] = m == m ? m : -INFINITY;
    }
    __syncthreads();
    double b1 = -INFINITY, b2 = -INFINITY;
    if (l < a.groups) {
      for (int i = 0; i < size; ++i) {
        const double m = value[l * size + i];
        b2 = fmax(b2, fmin(b1, m));
        b1 = fmax(b1, m);
      }
    }
    const uint64_t key = l < a.groups ? dkey(a.group_best == 2 && size > 1 ? b1 + b2 : b1) : 0;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
      const uint64_t other = __shfl(key, g);
      ahead += other > key || (other == key && g < l) ? 1 : 0;
    }
    stay = __ballot(l < a.groups && ahead < a.top_groups);
  }
  uint64_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l + v * 64;
    key[v] = e < E && (stay >> (e / size) & 1) ? dkey(c[v]) : 0;
  }
  if (a.top_groups == a.groups) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = l + v * 64 < E ? dkey(c[v]) : 0;
  }
  int mine = 0;
  for (int k = 0; k < a.K; ++k) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = l + v * 64;
      }
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t k2 = __shfl_xor(best, o);
      const int a2 = __shfl_xor(at, o);
      if (k2 > best || (k2 == best && a2 < at)) {
        best = k2;
        at = a2;
      }
    }
    if (l == k) mine = at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == l + v * 64) key[v] = 0;
  }
  const bool in = l < a.K;
  const float zk = in ? load_logit(row, mine) : 0.f;
  float w;
  if (a.renormalize) {
    w = shared_weight(zk, in, a.sigmoid);
  } else {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) value[l + v * 64] = s[v];
    __syncthreads();
    w = static_cast<float>(value[mine]);
  }
  if (in) {
    a.expert_idx[t * a.K + l] = mine;
    a.gate[t * a.K + l] = bad ? __builtin_nanf("") : a.scale * w;
  }
}

template <typename T>
__device__ __forceinline__ void store_logit(T* p, float v) {
  if constexpr (sizeof(T) == 4) *p = v;
  else *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// One wave per token, lane k the k-th selected expert.
template <typename T, int V>
__global__ __launch_bounds__(256) void expert_route_backward_kernel(ExpertRouteBackwardArgs a) {
  const int l = lane(), E = a.E;
  const size_t t = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (t >= static_cast<size_t>(a.L)) return;
  const T* row = static_cast<const T*>(a.logits) + t * E;
  int id = l < a.K ? a.expert_idx[t * a.K + l] : -1;
  const bool in = l < a.K && id >= 0 && id < E;
  if (!in) id = -1;
  float up = in ? a.scale * a.dgate[t * a.K + l] : 0.f;
  if (a.renormalize) {
    const float zk = in ? load_logit(row, id) : 0.f;
    const float w = shared_weight(zk, in, a.sigmoid);
    const float m = wave_sum(in ? w * up : 0.f);
    up = in ? w * (up - m) : 0.f;
    if (a.sigmoid && in) up *= 1.f / (1.f + expf(zk));
  }
  float u[V];
#pragma unroll
  for (int v = 0; v < V; ++v) u[v] = 0.f;
  for (int k = 0; k < a.K; ++k) {
    const int e = __builtin_amdgcn_readlane(id, k);
    const float x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(up), k));
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == l + v * 64) u[v] += x;
  }
  float s[V], ds[V], rest = 0.f;
  const bool dense = a.dscore || !a.renormalize;
  if (dense) {
    float z[V], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = l + v * 64;
      z[v] = e < E ? load_logit(row, e) : -INFINITY;
      top = fmaxf(top, z[v]);
      ds[v] = a.dscore && e < E ? a.dscore[(a.dscore_shared ? 0 : t * E) + e] : 0.f;
      if (!a.renormalize) ds[v] += u[v];
    }
    if (!a.sigmoid) {
      top = wave_max(top);
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = z[v] == -INFINITY ? 0.f : expf(z[v] - top);
        sum += s[v];
      }
      sum = wave_sum(sum);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] *= inv;
        dot = fmaf(s[v], ds[v], dot);
      }
      rest = wave_sum(dot);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = 1.f / (1.f + expf(-z[v])) * (1.f / (1.f + expf(z[v])));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = l + v * 64;
    if (e >= E) continue;
    const float dz = (dense ? s[v] * (ds[v] - rest) : 0.f) + (a.renormalize ? u[v] : 0.f);
    store_logit(static_cast<T*>(a.dlogits) + t * E + e, dz);
  }
}

template <typename T>
static void run_route(const ExpertRouteArgs& a, hipStream_t s) {
  const unsigned nb = static_cast<unsigned>(a.L);
  if (a.E <= 64) expert_route_kernel<T, 1><<<nb, 64, 0, s>>>(a);
  else if (a.E <= 128) expert_route_kernel<T, 2><<<nb, 64, 0, s>>>(a);
  else if (a.E <= 256) expert_route_kernel<T, 4><<<nb, 64, 0, s>>>(a);
  else if (a.E <= 512) expert_route_kernel<T, 8><<<nb, 64, 0, s>>>(a);
  else expert_route_kernel<T, 16><<<nb, 64, 0, s>>>(a);
}
hipError_t launch_expert_route(const ExpertRouteArgs& a, hipStream_t s) {
  if (a.bf16) run_route<uint16_t>(a, s);
  else run_route<float>(a, s);
  return hipGetLastError();
}
template <typename T>
static void run_route_backward(const ExpertRouteBackwardArgs& a, hipStream_t s) {
  const unsigned nb = (static_cast<unsigned>(a.L) + 3) / 4;
  if (a.E <= 64) expert_route_backward_kernel<T, 1><<<nb, 256, 0, s>>>(a);
  else if (a.E <= 128) expert_route_backward_kernel<T, 2><<<nb, 256, 0, s>>>(a);
  else if (a.E <= 256) expert_route_backward_kernel<T, 4><<<nb, 256, 0, s>>>(a);
  else if (a.E <= 512) expert_route_backward_kernel<T, 8><<<nb, 256, 0, s>>>(a);
  else expert_route_backward_kernel<T, 16><<<nb, 256, 0, s>>>(a);
}
hipError_t launch_expert_route_backward(const ExpertRouteBackwardArgs& a, hipStream_t s) {
  if (a.bf16) run_route_backward<uint16_t>(a, s);
  else run_route_backward<float>(a, s);
  return hipGetLastError();
}

}  // namespace omni
