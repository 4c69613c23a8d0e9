// A token's experts and gates from its logits, and the gradient of the logits.
//
// What selects is the score plus the balance bias, c = s + b.  The c of different
// experts can lie within float32's rounding of each other, so their order is that
// of float64.  For biased scores float32 nearly always tells it; where any two that
// had to be told apart are closer than twice its error, those are decided in float64
// (16384 tokens, 256 experts, 8 of them, sigmoid, groups: 17.6 us, with float64
// throughout 43.9).  Without a bias the score grows with the logit, which is compared
// as it stands; rows with equal logits among their best are decided the same way, and
// bfloat16 ones often are such: of 16384 normal rows of 256 experts, 8 of them, 40 %,
// and they take 24.3 us, float32 ones 10.3; 16 of them 81 %, 43.5 and 13.4.
//
// The error of c, in units of 2^-24.  e^x: the exponent's product with log2 e is off
// by 1.5 |x|, the exponential and a reciprocal by 2 each, relative; times e^-|x|, at
// most 2.1 of the largest term.  Sigmoid: s (1 - s) (1.5 |z| + 2) + 3 s < 3.7.
// Softmax: 2.1 and the sum's, which all of a row's scores share, 22 (at most 16 + 6
// additions) and 2, of the largest score.  c's own rounding adds 1 of c.  Twice that
// is below 2^-20 and below 2^-18 of the largest score, plus 2^-22 of c.
//
// Bound by instructions: a token's 256 logits and scores are 2 KiB, 6.6 us of HBM for
// 16384 tokens; the rounds of the selection are about 55 instructions each, of 1524 a
// wave.
#include "device.hpp"
#include "launch.hpp"

#include <type_traits>

namespace omni {

// T lanes (a DPP row, or the wave) share a token; lane l of them holds experts
// 4 T (v / 4) + 4 l + v % 4 in its slots v < V: four consecutive ones per load.
constexpr int kRow = 16;
template <int ctrl>
__device__ __forceinline__ uint32_t dpp_row(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), ctrl, 0xf, 0xf, true));
}
// lane `from` of the token's (T == kWave: the same one for all) as all of them see it
template <int T, typename V>
__device__ __forceinline__ V of_lane(V v, int from) {
  if constexpr (T != kWave) {
    return __shfl(v, from, T);
  } else if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), from));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), from);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), from);
    return __builtin_bit_cast(V, static_cast<uint64_t>(hi) << 32 | lo);
  }
}
// op over the token's lanes, the result in all of them; halves are added to halves,
// so every lane forms the same sum
template <int T, class Op>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v, Op op) {
  v = op(v, dpp_row<0x128>(v));  // row_ror 8, 4, 2, 1
  v = op(v, dpp_row<0x124>(v));
  v = op(v, dpp_row<0x122>(v));
  v = op(v, dpp_row<0x121>(v));
  if constexpr (T == kWave)
    v = op(op(of_lane<T>(v, 0), of_lane<T>(v, 16)), op(of_lane<T>(v, 32), of_lane<T>(v, 48)));
  return v;
}
template <int T>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(over_lanes<T>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int T>
__device__ __forceinline__ float lanes_max(float v) {
  return __uint_as_float(over_lanes<T>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int T>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return over_lanes<T>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int T>
__device__ __forceinline__ uint64_t lanes_max(uint64_t v) {
  const uint32_t hi = lanes_max<T>(static_cast<uint32_t>(v >> 32));
  const uint32_t lo = lanes_max<T>(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
// over the wave
__device__ __forceinline__ double lanes_sum(double v) {
  auto turned = [&](auto by) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_row<by()>(static_cast<uint32_t>(u));
    const uint32_t hi = dpp_row<by()>(static_cast<uint32_t>(u >> 32));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
  };
  v += turned(std::integral_constant<int, 0x128>{});
  v += turned(std::integral_constant<int, 0x124>{});
  v += turned(std::integral_constant<int, 0x122>{});
  v += turned(std::integral_constant<int, 0x121>{});
  return (of_lane<kWave>(v, 0) + of_lane<kWave>(v, 16)) +
         (of_lane<kWave>(v, 32) + of_lane<kWave>(v, 48));
}
// true in all of the token's lanes if in any
template <int T>
__device__ __forceinline__ bool lanes_any(bool v) {
  const uint64_t m = __ballot(v);
  if constexpr (T == kWave) return m != 0;
  return (m >> (lane() & ~(kRow - 1)) & 0xffffu) != 0;
}

__device__ __forceinline__ float load_logit(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float load_logit(const uint16_t* p, size_t i) {
  return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}
// Values e .. e + 3 of a row of E, `past` behind its end; vec: rows start at 4 elements
__device__ __forceinline__ void load4(const float* row, int e, int E, bool vec, float past,
                                      float* v) {
  if (vec && e < E) {
    const float4 f = *reinterpret_cast<const float4*>(row + e);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = e + i < E ? row[e + i] : past;
}
__device__ __forceinline__ void load4(const uint16_t* row, int e, int E, bool vec, float past,
                                      float* v) {
  if (vec && e < E) {
    const uint2 u = *reinterpret_cast<const uint2*>(row + e);
    v[0] = bf_lo(u.x);
    v[1] = bf_hi(u.x);
    v[2] = bf_lo(u.y);
    v[3] = bf_hi(u.y);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = e + i < E ? load_logit(row, e + i) : past;
}
__device__ __forceinline__ void store4(float* row, int e, int E, bool vec, const float* v) {
  if (vec && e < E) {
    *reinterpret_cast<float4*>(row + e) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (e + i < E) row[e + i] = v[i];
}
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ void store4(uint16_t* row, int e, int E, bool vec, const float* v) {
  if (vec && e < E) {
    *reinterpret_cast<uint2*>(row + e) = make_uint2(bf16_bits(v[0]) | bf16_bits(v[1]) << 16,
                                                    bf16_bits(v[2]) | bf16_bits(v[3]) << 16);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (e + i < E) row[e + i] = static_cast<uint16_t>(bf16_bits(v[i]));
}
template <typename P>
__device__ __forceinline__ bool fours(const P* p, int E) {  // rows of E start at 4 elements
  return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(P) - 1)) == 0;
}

// Order-preserving keys of what is compared: never 0, -0 onto +0, NaN as -infinity.
__device__ __forceinline__ uint32_t order_key(float v) { return fkey(v == v ? v : -INFINITY); }
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v == v)) v = -INFINITY;
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}

// Gates' weights of a token's selected experts (a lane each: logit z where mine) over
// their sum.  Scores are formed relative to the largest, so that scores too small
// for float32 still share out: softmax e^(z - m); sigmoid, times e^-m for m =
// min(largest z, 0): e^(z - m) / (1 + e^z), or 1 / (1 + e^-z) where z > 0 (then m = 0).
template <int T>
__device__ __forceinline__ float shared_weight(float z, bool mine, bool sigmoid) {
  const float top = lanes_max<T>(mine ? z : -INFINITY);
  float e;
  if (sigmoid) {
    const float m = fminf(top, 0.f);
    e = z > 0.f ? 1.f / (1.f + __expf(-z)) : __expf(z - m) / (1.f + __expf(z));
  } else {
    e = __expf(z - top);
  }
  if (!mine) e = 0.f;
  const float sum = lanes_sum<T>(e);
  // nothing but -infinity: weights of 0
  return top == -INFINITY && !lanes_any<T>(mine && z != z) ? 0.f : e / sum;
}

// The K best of the token's slots by key, a round each: the slot of round k holds k + 1
// afterwards, which is below every key.  Keys are taken to differ: equal ones share
// their round, and where the keys then run out, earlier rounds' slots are struck
// again.  seen(k, key): the key of round k, K or less if there was none.
template <int T, int V, class Seen>
__device__ __forceinline__ void strike_best(uint32_t (&key)[V], int K, Seen seen) {
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = lanes_max<T>(best);
    seen(k, best);
    const uint32_t taken = k + 1;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] == best ? taken : key[v];
  }
}
// The same over a wave by (key desc, expert asc): lane k gets the k-th expert.  Slot v of
// lane l is expert 64 v + l.
template <int V>
__device__ __forceinline__ int take_best(uint64_t (&key)[V], int K) {
  const int l = lane();
  int mine = 0;
  for (int k = 0; k < K; ++k) {
    uint64_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = lanes_max<kWave>(best);
    int at = 0;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) {
      const uint64_t m = __ballot(key[v] == best);
      if (m != 0) at = v * 64 + __ffsll(static_cast<long long>(m)) - 1;
    }
    if (l == k) mine = at;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] == best && at == v * 64 + l ? 0 : key[v];
  }
  return mine;
}

// Lanes that share a group (a power of two): as many as the token's lanes hold.
template <int T>
__device__ __forceinline__ int group_shift(int groups) {
  return 31 - __builtin_clz(static_cast<unsigned>(T / groups));
}
// Which groups stay, bit g << shift in the result for group g.  c: the token's E values
// in LDS, none of them NaN.  apart(a, b, size): values of the last that stays and the
// first that does not, and the sum of the absolute terms of both.
template <int T, typename F, class Apart>
__device__ __forceinline__ uint64_t best_groups(const F* c, const ExpertRouteArgs& a, int l,
                                                int shift, Apart apart) {
  const int size = a.E / a.groups, g = l >> shift, share = 1 << shift, part = l & (share - 1);
  F b1 = -INFINITY, b2 = -INFINITY;
  const int steps = (size + share - 1) >> shift;
  // started g steps further on: the groups' lanes then read different banks
  int n = g < steps ? g : g % steps;
  if (g < a.groups) {
#pragma unroll 4
    for (int i = 0; i < steps; ++i) {
      const int at = part + (n << shift);
      const F m = at < size ? c[g * size + at] : -INFINITY;
      b2 = max(b2, min(b1, m));
      b1 = max(b1, m);
      n = n + 1 == steps ? 0 : n + 1;
    }
  }
  for (int o = 1; o < share; o <<= 1) {
    const F m = __shfl_xor(b1, o, T), n2 = __shfl_xor(b2, o, T);
    b2 = max(min(b1, m), max(b2, n2));
    b1 = max(b1, m);
  }
  F value = a.group_best == 2 && size > 1 ? b1 + b2 : b1;
  if (!(value == value)) value = -INFINITY;  // infinities of both signs
  using Key = decltype(order_key(value));
  const bool mine = g < a.groups && part == 0;
  const Key key = order_key(value);
  int ahead = 0;
  for (int j = 0; j < a.groups; ++j) {
    const Key other = of_lane<T>(key, j << shift);
    ahead += other > key || (other == key && j < g) ? 1 : 0;
  }
  const int low = T == kWave ? 0 : lane() & ~(T - 1);  // the token's first lane
  auto lane_of = [&](int rank) {
    return __ffsll(static_cast<long long>(__ballot(mine && ahead == rank) >> low)) - 1;
  };
  const int last = lane_of(a.top_groups - 1), first = lane_of(a.top_groups);
  const F terms = a.group_best == 2 && size > 1 ? fabs(b1) + fabs(b2) : fabs(b1);
  apart(of_lane<T>(value, last), of_lane<T>(value, first),
        of_lane<T>(terms, last) + of_lane<T>(terms, first));
  const uint64_t stay = __ballot(mine && ahead < a.top_groups);
  return T == kWave ? stay : stay >> low & ((1ull << (T & 63)) - 1);
}

// One token decided in float64 by its whole wave; lane k gets the k-th expert.  slots:
// room for the token's values.
template <typename L, int V, bool GROUPS>
__device__ __forceinline__ int decide_exactly(const ExpertRouteArgs& a, size_t t, double* slots) {
  const int l = lane(), E = a.E;
  const L* row = static_cast<const L*>(a.logits) + t * E;
  float z[V];
  double d[V];
  bool bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    z[v] = v * 64 + l < E ? load_logit(row, v * 64 + l) : -INFINITY;
    bad |= z[v] != z[v] || z[v] == INFINITY;
    top = fmaxf(top, z[v]);
  }
  const bool sums = GROUPS && (a.bias || a.group_best == 2);
  if (a.bias || sums) {
    const double from = wave_max(top);
    double total = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(z[v])))
                       : z[v] == -INFINITY ? 0.0 : exp(z[v] - from);
      total += d[v];
    }
    if (!a.sigmoid) {
      bad = __any(bad);
      total = lanes_sum(total);
#pragma unroll
      for (int v = 0; v < V; ++v)
        d[v] = bad ? __builtin_nan("") : total > 0.0 ? d[v] / total : 0.0;
    }
    if (a.bias) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * 64 + l < E) d[v] += a.bias[v * 64 + l];
    }
  }
  uint64_t stay = ~0ull;
  int shift = 0;
  if constexpr (GROUPS) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const double m = sums ? d[v] : z[v];
      if (v * 64 + l < E) slots[v * 64 + l] = m == m ? m : -INFINITY;
    }
    wave_lds_fence();
    shift = group_shift<kWave>(a.groups);
    stay = best_groups<kWave>(slots, a, l, shift, [](double, double, double) {});
    wave_lds_fence();
  }
  const float per = GROUPS ? static_cast<float>(a.groups) / E : 0.f;
  uint64_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 64 + l;
    const bool in = e < E && (!GROUPS || (stay >> (static_cast<int>((e + 0.5f) * per) << shift) & 1) != 0);
    key[v] = in ? order_key(a.bias ? d[v] : static_cast<double>(z[v])) : 0ull;
  }
  return take_best<V>(key, a.K);
}

// Sigmoid scores with a bias whose order float32 leaves open: the slots that may be
// among the K best, those within what c is off of the K-th distinct c, go to a lane
// each, which forms c in float64 and counts those ahead of it.  open: of this token
// (the wave's others go along).  False where there are more than T of them.
template <typename L, int T, int V>
__device__ __forceinline__ bool rank_near(const ExpertRouteArgs& a, const L* row,
                                          const float (&c)[V], const uint32_t (&key)[V],
                                          float last, float close, bool open, int* ids, int l) {
  const float floor = last - (close + 0x1p-22f * fabsf(last));
  int count = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) count += key[v] != 0 && c[v] >= floor ? 1 : 0;
  // exclusive prefix over the token's lanes
  uint32_t upto = count;
  upto += dpp_u<0x111, 0xf>(0u, upto);  // row_shr 1, 2, 4, 8
  upto += dpp_u<0x112, 0xf>(0u, upto);
  upto += dpp_u<0x114, 0xf>(0u, upto);
  upto += dpp_u<0x118, 0xf>(0u, upto);
  if constexpr (T == kWave) {
    upto += dpp_u<0x142, 0xa>(0u, upto);
    upto += dpp_u<0x143, 0xc>(0u, upto);
  }
  const int n = of_lane<T>(static_cast<int>(upto), T - 1);
  const bool fits = n >= a.K && n <= T;
  int at = static_cast<int>(upto) - count;
  wave_lds_fence();
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (key[v] != 0 && c[v] >= floor) {
      if (open && fits) ids[at] = 4 * T * (v / 4) + 4 * l + v % 4;
      ++at;
    }
  wave_lds_fence();
  const bool in = open && fits && l < n;
  const int e = in ? ids[l] : 1 << 20;
  double exact = 0.0;
  if (in)
    exact = 1.0 / (1.0 + exp(-static_cast<double>(load_logit(row, e)))) + a.bias[e];
  const uint64_t mine = in ? order_key(exact) : 0ull;
  int ahead = 0;
  if constexpr (T == kRow) {
    uint32_t hi = static_cast<uint32_t>(mine >> 32), lo = static_cast<uint32_t>(mine), id = e;
#pragma unroll
    for (int r = 1; r < T; ++r) {
      hi = dpp_row<0x121>(hi);
      lo = dpp_row<0x121>(lo);
      id = dpp_row<0x121>(id);
      const uint64_t other = static_cast<uint64_t>(hi) << 32 | lo;
      ahead += other > mine || (other == mine && static_cast<int>(id) < e) ? 1 : 0;
    }
  } else {
    const int some = min(n, T);
    for (int j = 0; j < some; ++j) {
      const uint64_t other = of_lane<T>(mine, j);
      const int id = of_lane<T>(e, j);
      ahead += other > mine || (other == mine && id < e) ? 1 : 0;
    }
  }
  if (in && ahead < a.K) ids[ahead] = e;
  wave_lds_fence();
  return fits;
}

// T lanes per token, V slots each.
template <typename L, int T, int V, bool GROUPS>
__global__ __launch_bounds__(256) void expert_route_kernel(ExpertRouteArgs a) {
  constexpr int PER = kWave / T, ROOM = T * V + 8;  // tokens of a wave; 8: other banks each
  // a token's values, in float32 for all of a wave's tokens, in float64 for one
  constexpr int BYTES = !GROUPS ? 8 : PER * ROOM * 4 > ROOM * 8 ? PER * ROOM * 4 : ROOM * 8;
  __shared__ __attribute__((aligned(16))) uint8_t room[4][BYTES];
  __shared__ int list[4][kWave];
  const int l = lane() & (T - 1), E = a.E, wv = threadIdx.x >> 6, sub = lane() / T;
  const size_t first = (static_cast<size_t>(blockIdx.x) * 4 + wv) * PER, t0 = first + sub;
  const bool live = t0 < static_cast<size_t>(a.L);
  const size_t t = live ? t0 : a.L - 1;  // lanes without a token go along
  const L* row = static_cast<const L*>(a.logits) + t * E;
  const bool vec = fours(static_cast<const L*>(a.logits), E);
  auto expert = [&](int v) { return 4 * T * (v / 4) + 4 * l + v % 4; };
  float z[V], s[V];
#pragma unroll
  for (int v = 0; v < V; v += 4) load4(row, expert(v), E, vec, -INFINITY, z + v);
  float top = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, z[v]);
  top = lanes_max<T>(top);
  const float from = top == -INFINITY ? 0.f : top;  // a row of -infinity alone has scores of 0
  const bool biased = a.bias != nullptr;
  const bool sums = GROUPS && (biased || a.group_best == 2);  // groups compared by scores
  float largest = 1.f;  // score, or above it
  if (!a.sigmoid) {
    float parts[2] = {0.f, 0.f};  // of 16 each
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bad |= z[v] != z[v] || z[v] == INFINITY;
      s[v] = __expf(z[v] - from);
      parts[v / 16] += s[v];
    }
    bad = lanes_any<T>(bad);
    const float sum = lanes_sum<T>(parts[0] + parts[1]);
    largest = bad ? __builtin_nanf("") : sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] *= largest;
  } else if (a.score || biased || sums) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = __builtin_amdgcn_rcpf(1.f + __expf(-z[v]));
  }
  if (a.score && live) {
    float* out = a.score + t * E;
    const bool whole = fours(a.score, E);
#pragma unroll
    for (int v = 0; v < V; v += 4) store4(out, expert(v), E, whole, s + v);
  }
  // what is compared, in float32
  float c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = z[v];
  if (biased) {
    const bool whole = fours(a.bias, E);
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      float b[4];
      load4(a.bias, expert(v), E, whole, 0.f, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) c[v + i] = s[v + i] + b[i];
    }
  }
  const float close = largest * (a.sigmoid ? 0x1p-20f : 0x1p-18f);
  bool unsure = false;
  uint64_t stay = ~0ull;
  int shift = 0;
  if constexpr (GROUPS) {
    shift = group_shift<T>(a.groups);
    float* mine = reinterpret_cast<float*>(room[wv]) + sub * ROOM;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float m = sums && !biased ? s[v] : c[v];
      if (expert(v) < E) mine[expert(v)] = m == m ? m : -INFINITY;
    }
    wave_lds_fence();
    stay = best_groups<T>(mine, a, l, shift, [&](float x, float y, float terms) {
      if (sums) unsure |= !(x - y > 2 * close + 0x1p-22f * terms);
    });
  }
  // e / size of whole numbers up to 1024: the quotient of e + 1/2 is 1/1024 or more
  // from a whole number, far beyond float32's rounding
  const float per = GROUPS ? static_cast<float>(a.groups) / E : 0.f;
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert(v);
    const bool in = e < E && (!GROUPS || (stay >> (static_cast<int>((e + 0.5f) * per) << shift) & 1) != 0);
    key[v] = in ? order_key(c[v]) : 0u;
  }
  uint32_t before = ~0u;
  bool near = false;  // the best are the best, but their order or the last is in doubt
  auto apart = [&](uint32_t best) {  // from the round before's; not where one is no number
    const float x = fkey_inv(before), y = fkey_inv(best);
    near |= !(x - y > close + 0x1p-22f * fabsf(x));
  };
  strike_best<T, V>(key, a.K, [&](int k, uint32_t best) {
    unsure |= best <= static_cast<uint32_t>(a.K);  // equal keys left none for this round
    if (biased && k > 0) apart(best);
    before = best;
  });
  if (biased) {  // the first that is left has to be apart from the last taken
    uint32_t best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = max(best, key[v]);
    best = lanes_max<T>(best);
    if (best > static_cast<uint32_t>(a.K)) apart(best);
  }
  int* ids = list[wv] + sub * T;
  int count = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (key[v] - 1u < static_cast<uint32_t>(a.K)) {
      ids[key[v] - 1u] = expert(v);
      ++count;
    }
  }
  // equal keys shared a round: more slots than rounds.  Otherwise each of K rounds
  // struck one slot, and the list is whole.
  const bool shared = lanes_sum<T>(static_cast<float>(count)) != static_cast<float>(a.K);
  const bool doubt = shared || near;
  if (!biased || !a.sigmoid) {
    unsure |= doubt;
  } else {
    const float last = fkey_inv(before);
    unsure |= !(last > -INFINITY);  // what is not a number ranks there too
    if (__any(doubt && !unsure))
      unsure |= doubt && !rank_near<L, T, V>(a, row, c, key, last, close, doubt && !unsure, ids, l);
  }
  uint64_t open = __ballot(unsure && live);
  wave_lds_fence();
  while (open != 0) {
    const int at = __ffsll(static_cast<long long>(open)) - 1;  // a lane of the token
    const int which = at / T;
    const int id = decide_exactly<L, (T * V + 63) / 64, GROUPS>(
        a, first + which, reinterpret_cast<double*>(room[wv]));
    wave_lds_fence();
    if (lane() < a.K) list[wv][which * T + lane()] = id;
    wave_lds_fence();
    open &= T == kWave ? 0ull : ~(((1ull << (T & 63)) - 1) << (which * T));
  }
  const bool in = l < a.K && live;  // the list of no token may not be whole
  const int mine = in ? ids[l] : 0;
  const float zk = in ? load_logit(row, mine) : 0.f;
  float w;
  if (a.renormalize) w = shared_weight<T>(zk, in, a.sigmoid);
  else if (a.sigmoid) w = 1.f / (1.f + __expf(-zk));
  else w = largest * __expf(zk - from);
  if (in) {
    a.expert_idx[t * a.K + l] = mine;
    a.gate[t * a.K + l] = bad ? __builtin_nanf("") : a.scale * w;
  }
}

// T lanes per token; lane k also the k-th selected expert.  The selected experts'
// terms meet the token's row in LDS.  16384 tokens of 256 experts with a dense row, 34
// MB, in 10.5 us; comparing ids slot by slot took 18.4.  Bound by two latencies, the
// ids' and then their logits'.  Sigmoid gates that are not renormalised count as dense
// without a dscore too, though the selected logits would do (9.5 us; renormalised 7.5).
template <typename L, int T, int V>
__global__ __launch_bounds__(256) void expert_route_backward_kernel(ExpertRouteBackwardArgs a) {
  constexpr int PER = kWave / T, ROOM = T * V;
  __shared__ __attribute__((aligned(16))) float room[4 * PER * ROOM];
  const int l = lane() & (T - 1), E = a.E;
  const size_t t0 = static_cast<size_t>(blockIdx.x) * 4 * PER + threadIdx.x / T;
  const bool live = t0 < static_cast<size_t>(a.L);
  const size_t t = live ? t0 : a.L - 1;
  const L* row = static_cast<const L*>(a.logits) + t * E;
  const bool vec = fours(static_cast<const L*>(a.logits), E);
  auto expert = [&](int v) { return 4 * T * (v / 4) + 4 * l + v % 4; };
  const bool dense = a.dscore || !a.renormalize;
  float z[V], ds[V];
  if (dense) {
#pragma unroll
    for (int v = 0; v < V; v += 4) load4(row, expert(v), E, vec, -INFINITY, z + v);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) ds[v] = 0.f;
  if (a.dscore) {
    const float* up = a.dscore + (a.dscore_shared ? 0 : t * E);
    const bool whole = fours(a.dscore, E);
#pragma unroll
    for (int v = 0; v < V; v += 4) load4(up, expert(v), E, whole, 0.f, ds + v);
  }
  const int id = l < a.K ? a.expert_idx[t * a.K + l] : -1;
  const bool in = id >= 0 && id < E;
  float up = in ? a.scale * a.dgate[t * a.K + l] : 0.f;
  float* mine = room + (threadIdx.x / T) * ROOM;
#pragma unroll
  for (int v = 0; v < V; v += 4)
    *reinterpret_cast<float4*>(mine + expert(v)) = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.renormalize) {
    const float zk = in ? load_logit(row, id) : 0.f;
    const float w = shared_weight<T>(zk, in, a.sigmoid);
    const float m = lanes_sum<T>(in ? w * up : 0.f);
    up = in ? w * (up - m) : 0.f;
    if (a.sigmoid && in) up *= 1.f / (1.f + __expf(zk));
  }
  // the same expert more than once: each of its lanes forms the sum, in order
  float sum = 0.f;
  for (int k = 0; k < a.K; ++k) {
    const int other = of_lane<T>(id, k);
    const float x = of_lane<T>(up, k);
    if (other == id) sum += x;
  }
  wave_lds_fence();
  if (in) mine[id] = sum;
  wave_lds_fence();
  float u[V];
#pragma unroll
  for (int v = 0; v < V; v += 4) {
    const float4 f = *reinterpret_cast<const float4*>(mine + expert(v));
    u[v] = f.x;
    u[v + 1] = f.y;
    u[v + 2] = f.z;
    u[v + 3] = f.w;
  }
  float dz[V];
  if (dense) {
    if (!a.renormalize) {
#pragma unroll
      for (int v = 0; v < V; ++v) ds[v] += u[v];
    }
    if (!a.sigmoid) {
      float top = -INFINITY, total = 0.f, dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) top = fmaxf(top, z[v]);
      top = lanes_max<T>(top);
      if (top == -INFINITY) top = 0.f;  // scores of 0
#pragma unroll
      for (int v = 0; v < V; ++v) {
        z[v] = __expf(z[v] - top);
        total += z[v];
        dot = fmaf(z[v], ds[v], dot);
      }
      total = lanes_sum<T>(total);
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const float rest = lanes_sum<T>(dot) * inv;
#pragma unroll
      for (int v = 0; v < V; ++v) dz[v] = z[v] * inv * (ds[v] - rest);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        dz[v] = __builtin_amdgcn_rcpf(1.f + __expf(-z[v])) *
                __builtin_amdgcn_rcpf(1.f + __expf(z[v])) * ds[v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) dz[v] = (dense ? dz[v] : 0.f) + (a.renormalize ? u[v] : 0.f);
  if (live) {
    L* out = static_cast<L*>(a.dlogits) + t * E;
    const bool whole = fours(static_cast<const L*>(a.dlogits), E);
#pragma unroll
    for (int v = 0; v < V; v += 4) store4(out, expert(v), E, whole, dz + v);
  }
}

// Sixteen lanes per token, four tokens a wave, take fewer instructions, a wave per token
// is sooner done with it: sixteen where they hold the token's experts, groups and
// selection and the tokens are many; either way a token of up to 64 experts has four
// slots a lane.  us, sixteen lanes and 64, 8 selected, softmax scores:
//   tokens           1          1024       2048       4096       8192       16384
//   128 experts      3.8 3.5    4.1 3.9    4.1 4.2    4.2 5.2    4.5 7.7    5.9 12.6
//   256 experts      4.9 3.3    5.3 3.8    5.4 4.2    5.5 5.2    6.0 7.8    8.3 12.5
//   512 experts      7.5 4.0    7.9 4.5    7.9 4.9    8.0 6.5    9.1 10.0   13.2 17.0
static bool sixteen_lanes(int L, int E, int K, int groups) {
  return E <= 512 && K <= 16 && groups <= 16 && (E <= 64 || L > 16 * E);
}
template <typename L, bool GROUPS>
static void run_route(const ExpertRouteArgs& a, hipStream_t s) {
  const unsigned n = static_cast<unsigned>(a.L), few = (n + 15) / 16, many = (n + 3) / 4;
  if (sixteen_lanes(a.L, a.E, a.K, a.groups)) {
    if (a.E <= 64) expert_route_kernel<L, 16, 4, GROUPS><<<few, 256, 0, s>>>(a);
    else if (a.E <= 128) expert_route_kernel<L, 16, 8, GROUPS><<<few, 256, 0, s>>>(a);
    else if (a.E <= 256) expert_route_kernel<L, 16, 16, GROUPS><<<few, 256, 0, s>>>(a);
    else expert_route_kernel<L, 16, 32, GROUPS><<<few, 256, 0, s>>>(a);
  } else if (a.E <= 256) expert_route_kernel<L, 64, 4, GROUPS><<<many, 256, 0, s>>>(a);
  else if (a.E <= 512) expert_route_kernel<L, 64, 8, GROUPS><<<many, 256, 0, s>>>(a);
  else expert_route_kernel<L, 64, 16, GROUPS><<<many, 256, 0, s>>>(a);
}
hipError_t launch_expert_route(const ExpertRouteArgs& a, hipStream_t s) {
  const bool groups = a.top_groups < a.groups;
  if (a.bf16) groups ? run_route<uint16_t, true>(a, s) : run_route<uint16_t, false>(a, s);
  else groups ? run_route<float, true>(a, s) : run_route<float, false>(a, s);
  return hipGetLastError();
}
// As above; 2.4 us for 2.7 of one token of 256 experts, 7.7 for 5.8 of 16384.  Rows of
// more than 256 experts are a wave's: 17.6 us for 20.0 of 16384 of 512.
template <typename L>
static void run_route_backward(const ExpertRouteBackwardArgs& a, hipStream_t s) {
  const unsigned n = static_cast<unsigned>(a.L), few = (n + 15) / 16, many = (n + 3) / 4;
  if (a.E <= 256 && a.K <= 16 && (a.E <= 64 || a.L > 8 * a.E)) {
    if (a.E <= 64) expert_route_backward_kernel<L, 16, 4><<<few, 256, 0, s>>>(a);
    else if (a.E <= 128) expert_route_backward_kernel<L, 16, 8><<<few, 256, 0, s>>>(a);
    else expert_route_backward_kernel<L, 16, 16><<<few, 256, 0, s>>>(a);
  } else if (a.E <= 256) expert_route_backward_kernel<L, 64, 4><<<many, 256, 0, s>>>(a);
  else if (a.E <= 512) expert_route_backward_kernel<L, 64, 8><<<many, 256, 0, s>>>(a);
  else expert_route_backward_kernel<L, 64, 16><<<many, 256, 0, s>>>(a);
}
hipError_t launch_expert_route_backward(const ExpertRouteBackwardArgs& a, hipStream_t s) {
  if (a.bf16) run_route_backward<uint16_t>(a, s);
  else run_route_backward<float>(a, s);
  return hipGetLastError();
}

}  // namespace omni
