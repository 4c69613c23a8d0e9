// The matrix-core pipeline that the products over experts are tiles of: element
// types, stages of 64 bytes of the contraction in LDS filled by direct loads, the
// ring that overlaps them with the MFMAs, and the stores of an output tile.
#pragma once
#include <type_traits>

#include "device.hpp"

namespace omni {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ element types

struct Bf16Op {
  using Frag = bf16x8;
  using Acc = f32x4;
  using T = uint16_t;
  static constexpr int kBytes = 2, kSumBlock = 0;
  static __device__ __forceinline__ void mma(Acc& c, Frag q, Frag p) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q, p, c, 0, 0, 0);
  }
};
struct I8Op {
  using Frag = i32x4;
  using Acc = i32x4;
  using T = int8_t;
  static constexpr int kBytes = 1, kSumBlock = 0;
  static __device__ __forceinline__ void mma(Acc& c, Frag q, Frag p) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(q, p, c, 0, 0, 0);
  }
};
// A 16-byte fragment holds four consecutive contraction steps of a lane; the
// j-th of four MFMAs takes element j of both operands, so it contracts steps
// j, 4 + j, 8 + j and 12 + j of the stage.
struct F32Op {
  using Frag = f32x4;
  using Acc = f32x4;
  using T = float;
  static constexpr int kBytes = 4, kSumBlock = 8;
  static __device__ __forceinline__ void mma(Acc& c, Frag q, Frag p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(q[j], p[j], c, 0, 0, 0);
  }
};

// 16 bytes of zeros: where a lane of a direct load has nothing to fetch
__device__ __attribute__((aligned(16))) const uint32_t kZeroChunk[4] = {0, 0, 0, 0};

// ------------------------------------------------------------------ stages in LDS

// A stage of an operand whose contraction is contiguous in memory: one 64-byte
// row (four 16-byte chunks) per output row or column, chunk c of row r stored
// at c ^ swz.  A 16-byte-per-lane read is served eight lanes at a time from one
// 128-byte bank window; the swizzles below put the eight rows that such a
// group reads on eight distinct 16-byte slots.
//   P: rows r .. r + 7 (consecutive);  Q: rows 0-3 and 8-11 of a 32-row block
//   (tiles 2i and 2i + 1 take the columns 8 g + 0..3 and 8 g + 4..7 of their 32,
//   so a lane ends up with eight consecutive columns).
__device__ __forceinline__ int swz_p(int r) { return (r >> 1) & 3; }
__device__ __forceinline__ int swz_q(int r) { return ((r >> 1) & 1) | ((r >> 2) & 2); }
// A stage of an operand whose contraction is strided: one row of `cols`
// elements per contraction step, 16-byte chunk c of step kk at c ^ swz_cols(kk).
// bf16: the eight steps 0-3, 8-11 that half a transposing read takes at once
// land on eight 32-byte slots; float32: the steps 4 g + j of a read on four
// 64-byte slots.
// (64 bf16 columns are 128 bytes: the step's lowest bit then picks a half of
// the 256-byte bank window by itself.)
template <class Op, int COLS>
__device__ __forceinline__ int swz_cols(int kk) {
  static_assert(COLS * Op::kBytes >= 128 && (Op::kBytes == 2 || COLS >= 64), "row length");
  if (Op::kBytes == 4) return kk & 12;
  if (COLS == 64) return (((kk >> 1) & 1) | ((kk >> 2) & 2)) << 1;
  return ((kk & 3) | ((kk >> 1) & 4)) << 1;
}

template <int N>
__device__ __forceinline__ void wait_vm_lds() {  // vmcnt <= N, lgkmcnt = 0
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
// at most `after` stages of I loads each still in flight
template <int I, int S>
__device__ __forceinline__ void wait_stages(int after) {
  static_assert(S <= 5, "four stages at most");
  if (S > 4 && after >= 3) wait_vm_lds<(S > 4 ? 3 : 0) * I>();
  else if (S > 3 && after >= 2) wait_vm_lds<(S > 3 ? 2 : 0) * I>();
  else if (S > 2 && after >= 1) wait_vm_lds<(S > 2 ? 1 : 0) * I>();
  else wait_vm_lds<0>();
}
__device__ __forceinline__ void lds_barrier() {
  // a bare barrier: a fenced one would also wait for the stages in flight
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}
// Direct global -> LDS load: 16 bytes per lane to dst + 16 lane (dst uniform).
// It writes no register.  The builtin would make the compiler wait for every
// load in flight before each transposing read (it takes them to overlap); here
// the pipeline's own waits order them.  M0 needs one wait state before its use
// (nothing else in these kernels uses it).
__device__ __forceinline__ void load_lds16(const void* src, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                   :
                   : "v"(src), "s"(dst)
                   : "memory");
}
// the same from a uniform base and a lane's offset (a base that a vector
// instruction has just written needs five wait states)
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t offset, uint32_t dst) {
  __asm__ volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1"
                   :
                   : "v"(offset), "s"(base), "s"(dst)
                   : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) const void*)(p)));
}

// A fragment is read at the ring's address of its stage plus an offset that the
// lane keeps for the whole tile (and that the compiler is kept from taking
// apart again: one addition per fragment and stage instead of two or three).
// Fragments whose swizzle is the same are constants apart.
template <class Frag>
__device__ __forceinline__ Frag lds_read(uint32_t at) {
  return *(__attribute__((address_space(3))) const Frag*)static_cast<uintptr_t>(at);
}
__device__ __forceinline__ uint32_t kept(uint32_t v) {
  __asm__("" : "+v"(v));
  return v;
}
// K-contiguous stage: row r, chunk g
template <bool Q>
__device__ __forceinline__ uint32_t row_offset(int r, int g) {
  return kept(r * 64 + ((g ^ (Q ? swz_q(r) : swz_p(r))) << 4));
}
// Strided stage, rows of COLS elements, ROW bytes apart: columns c0 .. c0 + 15.
// bf16: a transposing read; lane 4 r + c of 16 names the 8 bytes of step r,
// columns 4 c .. 4 c + 3, and lane i receives the four steps of column i (the
// second read, four steps on, has the same swizzle).  float32: the lane's
// column at its first step; its others are ROW apart with the same swizzle.
template <class Op, int COLS, int ROW>
__device__ __forceinline__ uint32_t column_offset(int c0, int l) {
  const int i = l & 15, g = l >> 4;
  if constexpr (Op::kBytes == 2) {
    const int kk = g * 8 + (i >> 2), chunk = (c0 >> 3) + ((i & 3) >> 1);
    return kept(kk * ROW + ((chunk ^ swz_cols<Op, COLS>(kk)) << 4) + (i & 1) * 8);
  } else {
    const int c = c0 + i, kk = 4 * g;
    return kept(kk * ROW + (((c >> 2) ^ swz_cols<Op, COLS>(kk)) << 4) + (c & 3) * 4);
  }
}
template <class Op, int ROW>
__device__ __forceinline__ typename Op::Frag read_column(uint32_t at) {
  if constexpr (Op::kBytes == 2) {
    typedef __attribute__((address_space(3))) s16x4* Lds;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)static_cast<uintptr_t>(at));
    const s16x4 b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)static_cast<uintptr_t>(at + 4 * ROW));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = lds_read<float>(at + j * ROW);
    return v;
  }
}

// The pipeline of a tile: a ring of S stages in LDS, filled by direct
// global -> LDS loads (I of them per wave and stage).  Iteration kt: wait until
// stage kt + 1 has landed, barrier, then run stage kt's MFMAs (its fragments
// are in registers) while the slot of stage kt is refilled with stage kt + S
// and stage kt + 1's fragments are read into the other register set.  Loads and
// reads are issued between the MFMAs, one row of tiles at a time, the loads in
// the first half and the reads ahead of the last rows: issued together after
// the barrier they fill the load and LDS queues, and a wave that waits for room
// there issues no MFMA (up_train's shape: 442 us, spread as here 422).
//   issue(kt, u, may_end): load u of stage kt; may_end: it or the next may be the last
//   read_p(kt, i), read_q(kt, j): fragments of stage kt
// ACTIVE false: a wave whose part of the tile is empty; it only loads.
// The steady loop has no branch between a read and the MFMAs that use it: a
// join there makes the compiler wait for the reads just issued.
// float32 sums run in blocks of kSumBlock stages, each added to the total as the
// next begins, tile by tile between the MFMAs: a long sum of one accumulator
// rounds at its own size at every step (3424 steps: 1.0e-6 of the result, a
// library product 5.3e-7, blocks 2.3e-7).  That costs 3 % of a short product and
// 8 % of a long one (22 stages: 10.9 us without, 11.2 with, 11.6 with the blocks
// added between two stages).
template <class Op, int I, int S, bool ACTIVE, int TI, int TJ, class Issue, class ReadP,
          class ReadQ>
__device__ __forceinline__ void run_stages(int nk, Issue issue, ReadP read_p, ReadQ read_q,
                                           typename Op::Acc (&acc)[TI][TJ]) {
  using Frag = typename Op::Frag;
  constexpr int H = TI > 1 ? TI / 2 : 1, D = TI > 2 ? TI - 2 : 1;
  constexpr int kBlock = Op::kSumBlock;
  Frag p0[TI], q0[TJ], p1[TI], q1[TJ];
  typename Op::Acc block[kBlock ? TI : 1][kBlock ? TJ : 1] = {};
  // fresh: the first stage of a block
  auto mma_row = [&](int i, const Frag (&p)[TI], const Frag (&q)[TJ], auto fresh) {
    if constexpr (!ACTIVE) return;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if constexpr (kBlock == 0) {
        Op::mma(acc[i][j], q[j], p[i]);
      } else {
        if constexpr (fresh) {
          acc[i][j] += block[i][j];
          block[i][j] = typename Op::Acc{};
        }
        Op::mma(block[i][j], q[j], p[i]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read = [&](int kt, int i, int of, Frag (&np)[TI], Frag (&nq)[TJ]) {  // share i of `of`
    if constexpr (!ACTIVE) return;
#pragma unroll
    for (int j = i * TJ / of; j < (i + 1) * TJ / of; ++j) nq[j] = read_q(kt, j);
#pragma unroll
    for (int r = i * TI / of; r < (i + 1) * TI / of; ++r) np[r] = read_p(kt, r);
  };
  auto steady = [&](int kt, const Frag (&p)[TI], const Frag (&q)[TJ], Frag (&np)[TI],
                    Frag (&nq)[TJ], auto fresh) {
    wait_vm_lds<(S - 2) * I>();
    lds_barrier();
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      if (i < H) {
#pragma unroll
        for (int u = i * I / H; u < (i + 1) * I / H; ++u) issue(kt + S, u, false);
      }
      if (i < D) read(kt + 1, i, D, np, nq);
      mma_row(i, p, q, fresh);
    }
  };
  auto tail = [&](int kt, const Frag (&p)[TI], const Frag (&q)[TJ], Frag (&np)[TI],
                  Frag (&nq)[TJ]) {
    if (kt + 1 < nk) {
      wait_stages<I, S>(min(kt + S - 1, nk - 1) - (kt + 1));
      lds_barrier();
      if (kt + S < nk) {
#pragma unroll
        for (int u = 0; u < I; ++u) issue(kt + S, u, true);
      }
      read(kt + 1, 0, 1, np, nq);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) mma_row(i, p, q, std::false_type{});
  };
  read(0, 0, 1, p0, q0);
  int kt = 0;
  while (kt + S + 3 < nk) {
    int end = nk - S - 3;
    if constexpr (kBlock > 0) {
      end = min(end, kt + kBlock);
      steady(kt, p0, q0, p1, q1, std::true_type{});
      steady(kt + 1, p1, q1, p0, q0, std::false_type{});
      kt += 2;
    }
    for (; kt < end; kt += 2) {
      steady(kt, p0, q0, p1, q1, std::false_type{});
      steady(kt + 1, p1, q1, p0, q0, std::false_type{});
    }
  }
  for (; kt < nk; kt += 2) {
    tail(kt, p0, q0, p1, q1);
    if (kt + 1 < nk) tail(kt + 1, p1, q1, p0, q0);
  }
  if constexpr (kBlock > 0 && ACTIVE) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] += block[i][j];
  }
}
// active: uniform in a wave.  A tile of a ragged expert's last rows or of the
// last columns leaves waves without work; the other wave of their SIMD then
// has the matrix core to itself.
template <class Op, int I, int S, int TI, int TJ, class Issue, class ReadP, class ReadQ>
__device__ __forceinline__ void run_pipeline(int nk, bool active, Issue issue, ReadP read_p,
                                             ReadQ read_q, typename Op::Acc (&acc)[TI][TJ]) {
#pragma unroll
  for (int v = 0; v < S; ++v)
    if (v < nk) {
#pragma unroll
      for (int u = 0; u < I; ++u) issue(v, u, true);
    }
  wait_stages<I, S + 1>(min(S, nk) - 1);
  lds_barrier();
  if (active) run_stages<Op, I, S, true>(nk, issue, read_p, read_q, acc);
  else run_stages<Op, I, S, false>(nk, issue, read_p, read_q, acc);
}
// Waves w and w + 4 share a SIMD: of 2 x 4 waves the pair differs in both
// halves of the tile, so that where a half is empty every SIMD keeps one.
template <int WM, int WN>
__device__ __forceinline__ void wave_place(int wv, int& wm, int& wn) {
  wm = wv / WN;
  wn = WM == 2 && WN == 4 ? (wv + 2 * wm) % WN : wv % WN;
}

// ------------------------------------------------------------------ outputs

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {  // nearest even
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(a))) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
}
template <int N>
__device__ __forceinline__ void store_vec(uint16_t* p, const float (&v)[N]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                              bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store_one(uint16_t* p, float v) {
  *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
// N values of row `dst` at column c; aligned: the rows start at 16 bytes
template <typename TO, int N>
__device__ __forceinline__ void store_cols(TO* dst, int c, int width, bool aligned,
                                           const float (&v)[N]) {
  if (aligned && c + N <= width) {
    store_vec(dst + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < width) store_one(dst + c + i, v[i]);
  }
}
__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + __expf(-g)) * u; }

}  // namespace omni
