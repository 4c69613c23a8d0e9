// Products with experts that are matrices, the tasks sorted by expert:
//   out[o(m), :] = x[r(m), :] W[e]^T      for off[e] <= m < off[e + 1]
// (or times W[e], the input gradient), the weight gradient
//   dW[e] = sum_m dy[o(m), :]^T x[r(m), :]
// and the same forward product over 8-bit integers with a scale for each row
// of x and each row of W.
//
// All of them are tiles of one matrix-core pipeline.  An output tile has an
// operand P that runs over its rows (tasks) and an operand Q that runs over
// its columns (output features); a stage holds 64 bytes of the contraction
// (32 bf16, 64 int8 or 16 float32) of both.  Q is the MFMA's first operand and
// P its second, so a lane holds four consecutive columns of one output row and
// stores them without a pass through LDS.
#include "device.hpp"
#include "expert_forms.hpp"
#include "expert_pipeline.hpp"
#include "expert_tiles.hpp"
#include "launch.hpp"

namespace omni {

// ------------------------------------------------------------------ the product

// Tile BM tasks x BN columns, WM x WN waves, ring of S stages.  MFMA-bound with
// many rows per expert: 256 x 256 tiles of waves with 128 x 64 each read 12 KiB
// of fragments from LDS per 32 MFMAs, which the LDS just keeps up with (tiles
// of 64 x 64 per wave read 16 KiB); the matrix cores are busy 56 % of the
// kernel's cycles and the card lowers its clock under them.  65536 tasks of 61
// experts, 1408 x 2048, bf16: 400 us, 0.94 PFLOP/s; 8192 x 8192 x 8192: 843 us,
// 1.30 PFLOP/s (int8 446 us, 2.5 POP/s).  HBM-bound with few rows: 2048 tasks of
// 64 experts, 2 x 704 x 2048, 64 x 128 tiles: 82 us, 4.5 TB/s.
// QT: W is read as [contraction][columns] (the input gradient).
// SWIGLU: every 64 columns of Q are 32 gate rows, then the same 32 up rows.
template <class Op, typename TO, bool QT, bool SWIGLU, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM * WN * 64, 2) void expert_product_kernel(ExpertMatmulArgs a) {
  using Acc = typename Op::Acc;
  constexpr int NW = WM * WN, KE = 64 / Op::kBytes;
  constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
  constexpr int IP = BM / 16 / NW, IQ = BN / 16 / NW;  // 1-KiB loads per wave and stage
  constexpr int STAGE = (BM + BN) * 64;
  constexpr int BNO = SWIGLU ? BN / 2 : BN;            // output columns of a tile
  static_assert(BM % (16 * NW) == 0 && BN % (16 * NW) == 0, "loads split evenly");
  static_assert(TJ % (SWIGLU ? 4 : 2) == 0, "column pairs");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE];

  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int K = QT ? a.n : a.k, N = QT ? a.k : a.n;
  const int n_nt = (N + BNO - 1) / BNO;
  const TilePlace at = my_tile(blockIdx.x, gridDim.x, a.offsets, a.E, a.M, BM, n_nt);
  const ExpertTile t = at.t;
  const int n0 = at.nt * BNO;
  if (t.m0 >= t.m1) return;
  const uint8_t* x = static_cast<const uint8_t*>(a.x);
  const uint8_t* w = static_cast<const uint8_t*>(a.w) +
                     static_cast<size_t>(t.e) * (SWIGLU ? 2 : 1) * a.n * a.k * Op::kBytes;

  // Sources of this lane's direct loads.  Rows and columns past the end (and
  // rows out of range) re-read a valid one: their results are not stored (or
  // stored as zeros).  Contraction steps past the end fetch zeros.
  const int nk = (K + KE - 1) / KE;
  const int left = (K - (nk - 1) * KE) * Op::kBytes / 16;  // chunks of the last stage
  const uint8_t* psrc[IP];  // rows may lie anywhere: whole addresses
#pragma unroll
  for (int u = 0; u < IP; ++u) {
    const int r = (wv * IP + u) * 16 + (l >> 2);
    const int m = min(t.m0 + r, t.m1 - 1);
    const int row = min(max(a.x_row ? a.x_row[m] : m, 0), a.R - 1);
    psrc[u] = x + static_cast<size_t>(row) * K * Op::kBytes + ((l & 3) ^ swz_p(r)) * 16;
  }
  // W: a uniform base (the tile's first row; with SWIGLU the 16 rows of a load
  // are all of one half) and the lane's offset from it
  constexpr int CPR = BN * Op::kBytes / 16;  // QT: chunks per step
  const uint8_t* qbase[SWIGLU ? IQ : 1];
  uint32_t qoff[IQ];
  const size_t row_bytes = static_cast<size_t>(K) * Op::kBytes;
#pragma unroll
  for (int u = 0; u < IQ; ++u) {
    if constexpr (QT) {
      const int o = (wv * IQ + u) * 64 + l, kk = o / CPR, c = (o % CPR) ^ swz_cols<Op, BN>(kk);
      const int col = n0 + c * (16 / Op::kBytes);
      qoff[u] = (kk * static_cast<uint32_t>(N) + (col < N ? col : 0)) * Op::kBytes;
    } else {
      const int first = (wv * IQ + u) * 16, r = first + (l >> 2);
      const int row = SWIGLU ? (r >> 6) * 32 + (r & 31) : r;
      qoff[u] = static_cast<uint32_t>(min(row, N - 1 - n0)) * static_cast<uint32_t>(row_bytes) +
                ((l & 3) ^ swz_q(r)) * 16;
      if constexpr (SWIGLU)
        qbase[u] = w + (n0 + static_cast<size_t>((first >> 5) & 1) * N) * row_bytes;
    }
  }
  if constexpr (!SWIGLU) qbase[0] = QT ? w : w + n0 * row_bytes;
  const int q_left = QT ? K - (nk - 1) * KE : left;
  const size_t q_step = QT ? static_cast<size_t>(KE) * N * Op::kBytes : 64;
  const uint32_t ring = lds_address(smem);
  auto issue = [&](int kt, int u, bool may_end) {
    const uint32_t st = ring + (kt % S) * STAGE;
    // the lane, opaque where the last stage needs it: what follows from it
    // there would otherwise be kept in registers throughout
    int ll = l;
    if (may_end) __asm__ volatile("" : "+v"(ll));
    const bool last = may_end && kt == nk - 1;
    if (u < IP) {
      const void* src = psrc[u] + static_cast<size_t>(kt) * 64;
      if (last && ((ll & 3) ^ swz_p((wv * IP + u) * 16 + (ll >> 2))) >= left) src = kZeroChunk;
      load_lds16(src, st + (wv * IP + u) * 1024);
    } else {
      u -= IP;
      const uint8_t* base = qbase[SWIGLU ? u : 0] + kt * q_step;
      const uint32_t dst = st + BM * 64 + (wv * IQ + u) * 1024;
      if (last) {
        const int part = QT ? ((wv * IQ + u) * 64 + ll) / CPR
                            : (ll & 3) ^ swz_q((wv * IQ + u) * 16 + (ll >> 2));
        const void* src = base + qoff[u];
        load_lds16(part >= q_left ? static_cast<const void*>(kZeroChunk) : src, dst);
      } else {
        load_lds16(base, qoff[u], dst);
      }
    }
  };

  const int fr = l & 15, g = l >> 4;
  int wm, wn;
  wave_place<WM, WN>(wv, wm, wn);
  const uint32_t poff = row_offset<false>(wm * (BM / WM) + fr, g);
  uint32_t toff[QT ? TJ : 1];
  if constexpr (QT) {
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      toff[j] = column_offset<Op, BN, BN * Op::kBytes>(wn * (BN / WN) + j * 16, l);
  } else {
    toff[0] = row_offset<true>(wn * (BN / WN) + (fr >> 2) * 8 + (fr & 3), g);
  }
  using Frag = typename Op::Frag;
  auto read_p = [&](int kt, int i) {
    return lds_read<Frag>(ring + (kt % S) * STAGE + poff + i * 16 * 64);
  };
  auto read_q = [&](int kt, int j) {
    const uint32_t st = ring + (kt % S) * STAGE + BM * 64;
    if constexpr (QT) return read_column<Op, BN * Op::kBytes>(st + toff[j]);
    else return lds_read<Frag>(st + toff[0] + ((j >> 1) * 32 + (j & 1) * 4) * 64);
  };
  Acc acc[TI][TJ] = {};
  const bool active = t.m0 + wm * (BM / WM) < t.m1 && n0 + wn * (BNO / WN) < N;
  run_pipeline<Op, IP + IQ, S>(nk, active, issue, read_p, read_q, acc);
  if (!active) return;

  // lane (fr, g) holds row i * 16 + fr; columns: QT 16 j + 4 g + 0..3, else
  // 32 (j / 2) + 8 g + 0..7 of tiles j, j + 1
  TO* out = static_cast<TO*>(a.out);
  const bool aligned = (N * sizeof(TO)) % 16 == 0;
  const float* ws = a.w_scale ? a.w_scale + static_cast<size_t>(t.e) * (SWIGLU ? 2 : 1) * a.n
                              : nullptr;
  // scale of the weight row behind this lane's value q of column tile j
  float wsc[Op::kBytes == 1 ? TJ : 1][4];
  if constexpr (Op::kBytes == 1) {
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int half = SWIGLU ? (j >> 1) & 1 : 0;
        const int c = n0 + wn * (BNO / WN) + (SWIGLU ? j >> 2 : j >> 1) * 32 + g * 8 + (j & 1) * 4 + q;
        wsc[j][q] = c < N ? ws[half * N + c] : 0.f;
      }
  }
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int m = t.m0 + wm * (BM / WM) + i * 16 + fr;
    if (m >= t.m1) continue;
    const int row = a.out_row ? a.out_row[m] : m, xr = a.x_row ? a.x_row[m] : m;
    if (row < 0 || row >= a.Ro) continue;
    const bool in = xr >= 0 && xr < a.R;
    float rs = 0.f;
    if constexpr (Op::kBytes == 1) rs = in ? a.x_scale[xr] : 0.f;
    TO* dst = out + static_cast<size_t>(row) * N;
    auto value = [&](int j, int q) {
      const float v = static_cast<float>(acc[i][j][q]);
      // a row out of range gives zeros, whatever the weights and their scales hold
      if constexpr (Op::kBytes == 1) return in ? v * rs * wsc[j][q] : 0.f;
      else return in ? v : 0.f;
    };
    if constexpr (QT) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = value(j, q);
        store_cols(dst, n0 + wn * (BN / WN) + j * 16 + g * 4, N, true, v);
      }
    } else if constexpr (SWIGLU) {
#pragma unroll
      for (int b = 0; b < TJ / 4; ++b) {  // blocks of 32 gate and 32 up columns
        const int c = n0 + wn * (BN / WN / 2) + b * 32 + g * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int j = b * 4 + (q >> 2);
          v[q] = silu_mul(value(j, q & 3), value(j + 2, q & 3));
        }
        store_cols(dst, c, N, aligned, v);
      }
    } else {
#pragma unroll
      for (int b = 0; b < TJ / 2; ++b) {
        const int c = n0 + wn * (BN / WN) + b * 32 + g * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = value(b * 2 + (q >> 2), q & 3);
        store_cols(dst, c, N, aligned, v);
      }
    }
  }
}

// ------------------------------------------------------------------ the weight gradient

// Tile BM output features (columns of dy) x BN inputs (columns of x) of one
// expert; the contraction runs over its tasks in order, whose rows of dy and x
// are gathered by the same ring of direct loads: a stage holds, task by task,
// BM columns of the task's dy row and then BN columns of its x row, so that a
// load takes both of one task (BM = BN = 256, bf16) or of a few.  The row
// numbers are read one stage ahead as constants at uniform addresses (scalar
// loads: the vector-memory counter stays with the ring), and the address work
// is kept to a few instructions per load: at two waves per SIMD the
// instructions between the MFMAs bound this kernel: 65536 tasks, 64 experts of
// 1408 x 2048 take 511 us (0.74 PFLOP/s) with 54 scalar and 60 vector ones per
// stage and wave (the whole kernel's by its stages), took 543 with 74 vector ones
// and 630 with 105 scalar ones besides.  Memory is not far behind: 1.88e7 L2
// misses, 2.4 GB (4.7 TB/s), 0.74 of it dW; the x rows of an expert are fetched by
// every XCD that has one of its column blocks of dy.
// bf16 sums stay in one accumulator (an MFMA adds 32 tasks, so it rounds 8 times
// less often than float32's): relative error 2.9e-7 at 8192 tasks in parts, 1.6e-6
// at 65536 tasks uncut, where a float32 library product has 9.6e-7 and 3.5e-6.
// Where either row is out of range both are fetched as zeros, which removes the
// task's term whatever the other row holds: the comparison's lane mask is folded
// onto both halves of the task (a test of each task's two row numbers took 525 us).
template <class Op, int BM, int BN, int WM, int WN, int S, bool LISTS>
__global__ __launch_bounds__(WM * WN * 64, 2) void expert_wgrad_kernel(ExpertWgradArgs a) {
  using Acc = typename Op::Acc;
  constexpr int NW = WM * WN, KE = 64 / Op::kBytes;
  constexpr int TI = BM / WM / 16, TJ = BN / WN / 16;
  constexpr int ROW = (BM + BN) * Op::kBytes;  // bytes of a task in a stage
  constexpr int STAGE = KE * ROW;
  constexpr int I = STAGE / 1024 / NW;          // loads per wave and stage
  constexpr int TPI = 1024 / ROW;               // tasks of a load
  constexpr int NT = I * TPI;                   // tasks of a wave and stage
  static_assert(TPI >= 1 && I >= 1 && I * NW * 1024 == STAGE, "loads split evenly");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE];

  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 63;
  const int n_nt = (a.n + BM - 1) / BM, n_kt = (a.k + BN - 1) / BN;
  WgradPart w;
  int n0, c0;
  if (a.part > 0) {
    w = my_part(blockIdx.x, a.offsets, a.E, a.M, a.part, a.slots, n_nt * n_kt);
    if (w.lo >= w.hi) return;
    n0 = w.tile / n_kt * BM;
    c0 = w.tile % n_kt * BN;
  } else {
    // The n_kt tiles of one expert and one dy column block are a group: they
    // share dy's columns and x's rows in an L2.  Groups are dealt to the XCDs
    // in turn, the experts with the most tasks first (of every 64), so that
    // long contractions neither pile up on one XCD nor start last.
    const int slot = blockIdx.x >> 3, group = slot / n_kt * 8 + (blockIdx.x & 7);
    if (group >= a.E * n_nt) return;
    w.e = expert_by_size(a.offsets, a.E, a.M, group / n_nt, w.lo, w.hi);
    w.slot = -1;
    n0 = group % n_nt * BM;
    c0 = slot % n_kt * BN;
  }
  const int lo = __builtin_amdgcn_readfirstlane(w.lo), hi = __builtin_amdgcn_readfirstlane(w.hi);
  const int nk = (hi - lo + KE - 1) / KE;

  // This lane's part of a load: which of the load's rows, and where in it.  The
  // tasks of a wave's load u are TPI (wv I + u) .. + TPI - 1 of the stage.
  const int sub = l * 16 / ROW, in = l * 16 % ROW;
  const bool is_x = in >= BM * Op::kBytes;
  const int pos = is_x ? in - BM * Op::kBytes : in;  // byte in its operand's part of the row
  const uint32_t limit = is_x ? a.R : a.Ry;
  const uint32_t stride = (is_x ? a.k : a.n) * Op::kBytes;
  const uint8_t* base[I];
#pragma unroll
  for (int u = 0; u < I; ++u) {
    const int kk = (wv * I + u) * TPI + sub;
    const int col = (is_x ? c0 : n0) + ((pos >> 4) ^ swz_cols<Op, BM>(kk)) * (16 / Op::kBytes);
    base[u] = static_cast<const uint8_t*>(is_x ? a.x : a.dy) +
              (col < (is_x ? a.k : a.n) ? col : 0) * static_cast<size_t>(Op::kBytes);
  }
  static_assert(BM == BN, "one swizzle for both halves of a task");

  typedef const int32_t __attribute__((address_space(4))) ConstInt;
  ConstInt* xl = (ConstInt*)reinterpret_cast<uintptr_t>(a.x_row);
  ConstInt* yl = (ConstInt*)reinterpret_cast<uintptr_t>(a.dy_row);
  int raw_y[NT], raw_x[NT];
  // may_end: the stage may reach past the last task (or the lists' end)
  auto fetch_rows = [&](int kt, bool may_end) {
    const int first = lo + kt * KE + wv * NT;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const int m = may_end ? min(first + r, a.M - 1) : first + r;
      if constexpr (LISTS) {
        raw_y[r] = yl[m];
        raw_x[r] = xl[m];
      } else {
        raw_y[r] = a.dy_row ? yl[m] : m;
        raw_x[r] = a.x_row ? xl[m] : m;
      }
      if (may_end && first + r >= hi) raw_y[r] = raw_x[r] = -1;
    }
  };
  const uint32_t ring = lds_address(smem);
  auto issue = [&](int kt, int u, bool may_end) {
    uint32_t row = 0;
#pragma unroll
    for (int r = 0; r < TPI; ++r) {
      const uint32_t ry = raw_y[u * TPI + r], rx = raw_x[u * TPI + r], mine = is_x ? rx : ry;
      row = r == 0 || sub == r ? mine : row;
    }
    const uint8_t* src = base[u] + static_cast<uint64_t>(row) * stride;
    // lanes whose row and whose task's other row are in range
    constexpr int W = BM * Op::kBytes / 16;  // lanes of a task's dy row; as many of its x row
    static_assert(W == 8 || W == 16 || W == 32, "a wave holds whole tasks");
    constexpr uint64_t kDy = W == 32 ? 0xffffffffull : W == 16 ? 0x0000ffff0000ffffull
                                                               : 0x00ff00ff00ff00ffull;
    const uint64_t in_range = __builtin_amdgcn_ballot_w64(row < limit);
    const uint64_t both = in_range & in_range >> W & kDy;
    const bool ok = __builtin_amdgcn_inverse_ballot_w64(both | both << W);
    load_lds16(ok ? src : reinterpret_cast<const uint8_t*>(kZeroChunk),
               ring + (kt % S) * STAGE + (wv * I + u) * 1024);
    if (u == I - 1) fetch_rows(kt + 1, may_end);
  };
  const int fr = l & 15, g = l >> 4;
  int wm, wn;
  wave_place<WM, WN>(wv, wm, wn);
  uint32_t poff[TI], toff[TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
    poff[i] = column_offset<Op, BM, ROW>(wm * (BM / WM) + i * 16, l);
#pragma unroll
  for (int j = 0; j < TJ; ++j)
    toff[j] = column_offset<Op, BN, ROW>(wn * (BN / WN) + j * 16, l);
  auto read_p = [&](int kt, int i) {
    return read_column<Op, ROW>(ring + (kt % S) * STAGE + poff[i]);
  };
  auto read_q = [&](int kt, int j) {
    return read_column<Op, ROW>(ring + (kt % S) * STAGE + BM * Op::kBytes + toff[j]);
  };
  Acc acc[TI][TJ] = {};
  if (nk > 0) {
    fetch_rows(0, true);
    run_pipeline<Op, I, S>(nk, n0 + wm * (BM / WM) < a.n && c0 + wn * (BN / WN) < a.k, issue, read_p,
                           read_q, acc);
  }
  float* out = w.slot < 0 ? a.dw + static_cast<size_t>(w.e) * a.n * a.k
                          : a.partial + static_cast<size_t>(w.slot) * a.n * a.k;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int r = n0 + wm * (BM / WM) + i * 16 + fr;
    if (r >= a.n) continue;
    float* dst = out + static_cast<size_t>(r) * a.k;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int c = c0 + wn * (BN / WN) + j * 16 + g * 4;
      if (c < a.k)
        *reinterpret_cast<float4*>(dst + c) = make_float4(acc[i][j][0], acc[i][j][1],
                                                          acc[i][j][2], acc[i][j][3]);
    }
  }
}

// Experts cut into parts: dW = the sum of their partial sums in part order;
// zeros for experts without tasks.  A workgroup covers 4096 sums of one expert:
// most find an expert in one part and end there, so few of them are launched
// (47 experts of 960 x 584, one of them cut: 11 us with 1024 sums each, 7.4 now).
constexpr int kReduce = 4096;
__global__ __launch_bounds__(256) void expert_wgrad_reduce_kernel(ExpertWgradArgs a) {
  const int e = blockIdx.y;
  int lo, hi;
  expert_range(a.offsets, e, a.M, lo, hi);
  const int parts = parts_of(hi - lo, a.part);
  if (parts == 1) return;
  const size_t size = static_cast<size_t>(a.n) * a.k;
  const int first = parts > 1 ? max(first_slot(a.offsets, a.E, a.M, a.part, e), 0) : 0;
  const int n = min(parts, a.slots - first);  // fewer: offsets that overlap
#pragma unroll
  for (int u = 0; u < kReduce / 1024; ++u) {
    const size_t at = static_cast<size_t>(blockIdx.x) * kReduce + (u * 256 + threadIdx.x) * 4;
    if (at >= size) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int z = 0; z < n; ++z) {
      const float4 v = *reinterpret_cast<const float4*>(a.partial + (first + z) * size + at);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    *reinterpret_cast<float4*>(a.dw + e * size + at) = s;
  }
}

// ------------------------------------------------------------------ few rows per expert

// 16 RT tasks x 16 CT rows of W per workgroup, the contraction split over its
// KS waves: both operands go from memory to the MFMA's registers, U stages of
// 64 bytes ahead, and the waves' sums are added through LDS in wave order.
// SWIGLU: the first CT / 2 column tiles are gate rows, the others their up rows.
// Bound by HBM latency and bandwidth: no barrier stands between a wave's loads,
// and splitting the contraction gives one token's eight experts 2816 waves.
// That token's gate and up halves (2 x 704 x 2048, bf16, 46 MB): 12 us, 3.8 TB/s,
// of which about 4 us are the launch and finding the tile; 4 or 8 waves and 2 to
// 16 stages ahead measure the same.  Each wave sums its share of the contraction
// in one accumulator (float32: an eighth of the steps, not blocks of 128).
template <class Op, typename TO, bool SWIGLU, int RT, int CT, int KS, int U>
__global__ __launch_bounds__(KS * 64) void expert_rows_kernel(ExpertMatmulArgs a) {
  using Frag = typename Op::Frag;
  using Acc = typename Op::Acc;
  constexpr int BM = 16 * RT, H = SWIGLU ? 2 : 1, CO = CT / H, BNO = 16 * CO;
  static_assert(CT % H == 0, "gate and up tiles in pairs");
  __shared__ __attribute__((aligned(16))) Acc part[KS][RT * CT][64];
  const int wv = threadIdx.x >> 6, l = threadIdx.x & 63, fr = l & 15, g = l >> 4;
  const int K = a.k, N = a.n;
  const int n_nt = (N + BNO - 1) / BNO;
  const TilePlace at = my_tile(blockIdx.x, gridDim.x, a.offsets, a.E, a.M, BM, n_nt);
  const ExpertTile t = at.t;
  const int n0 = at.nt * BNO;
  if (t.m0 >= t.m1) return;
  const size_t row_bytes = static_cast<size_t>(K) * Op::kBytes;
  const uint8_t* w = static_cast<const uint8_t*>(a.w) +
                     static_cast<size_t>(t.e) * H * N * row_bytes;
  const uint8_t* psrc[RT];
  const uint8_t* qsrc[CT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int m = min(t.m0 + i * 16 + fr, t.m1 - 1);
    const int row = min(max(a.x_row ? a.x_row[m] : m, 0), a.R - 1);
    psrc[i] = static_cast<const uint8_t*>(a.x) + row * row_bytes + g * 16;
  }
#pragma unroll
  for (int j = 0; j < CT; ++j)
    qsrc[j] = w + (min(n0 + j % CO * 16 + fr, N - 1) + static_cast<size_t>(j / CO) * N) * row_bytes +
              g * 16;

  // chunks of 16 bytes; this wave's stages are [kb, ke)
  const int chunks = static_cast<int>(row_bytes / 16), nk = (chunks + 3) / 4;
  const int per = (nk + KS - 1) / KS, kb = min(nk, wv * per), ke = min(nk, kb + per);
  Acc acc[RT][CT] = {};
  auto fetch = [&](const uint8_t* src, int kt) {
    const bool ok = kt < ke && kt * 4 + g < chunks;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) v = *reinterpret_cast<const uint4*>(src + static_cast<size_t>(kt) * 64);
    return __builtin_bit_cast(Frag, v);
  };
  for (int k0 = kb; k0 < ke; k0 += U) {
    Frag p[U][RT], q[U][CT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < CT; ++j) q[u][j] = fetch(qsrc[j], k0 + u);
#pragma unroll
      for (int i = 0; i < RT; ++i) p[u][i] = fetch(psrc[i], k0 + u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) Op::mma(acc[i][j], q[u][j], p[u][i]);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) part[wv][i * CT + j][l] = acc[i][j];
  __syncthreads();
  // the output tiles are finished by the waves in turn
  TO* out = static_cast<TO*>(a.out);
  const bool aligned = (N * sizeof(TO)) % 16 == 0;
  for (int o = wv; o < RT * CO; o += KS) {
    const int i = o / CO, j = o % CO, c0 = n0 + j * 16 + g * 4;
    Acc s[H];
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
    for (int q = 0; q < 4; ++q) {
      float z[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        z[h] = in ? static_cast<float>(s[h][q]) : 0.f;
        if constexpr (Op::kBytes == 1)
          if (in)
            z[h] = z[h] * a.x_scale[xr] *
                   a.w_scale[(static_cast<size_t>(t.e) * H + h) * N + min(c0 + q, N - 1)];
      }
      v[q] = SWIGLU ? silu_mul(z[0], z[H - 1]) : z[0];
    }
    store_cols(out + static_cast<size_t>(row) * N, c0, N, aligned, v);
  }
}

// ------------------------------------------------------------------ dispatch

bool expert_matmul_fits(const ExpertMatmulArgs& a) {
  // a tile's offsets within W are 32 bits, and so is an expert's number rounded up to 64
  if (a.n > 1 << 22 || a.k > 1 << 22 || a.E > 1 << 30) return false;
  if (a.M == 0) return true;
  const ProductForm f = pick_form(a);
  return form_blocks(a, f) < (1ll << 32) / form_shape(f, a.swiglu).threads;
}
template <class Op, typename TO, bool QT, bool SW>
static hipError_t run_form(const ExpertMatmulArgs& a, hipStream_t s) {
  ProductForm f = pick_form(a);
  const unsigned nb = static_cast<unsigned>(form_blocks(a, f));
  const int nt = form_shape(f, SW).threads;
  if constexpr (!QT) {
    if (f == kRows16)
      expert_rows_kernel<Op, TO, SW, 1, SW ? 2 : 1, 8, 4><<<nb, nt, 0, s>>>(a);
    else if (f == kRows32)
      expert_rows_kernel<Op, TO, SW, 2, 2, 8, 4><<<nb, nt, 0, s>>>(a);
    else if (f == kRows64)
      expert_rows_kernel<Op, TO, SW, 4, 2, 8, 2><<<nb, nt, 0, s>>>(a);
  }
  if constexpr (Op::kBytes != 4) {
    if (f == kTileBig)
      expert_product_kernel<Op, TO, QT, SW, 256, 256, 2, 4, 4><<<nb, nt, 0, s>>>(a);
    else if (f == kTileWide)
      expert_product_kernel<Op, TO, QT, SW, 128, 256, 2, 4, 4><<<nb, nt, 0, s>>>(a);
    else if (f == kTileMid)
      expert_product_kernel<Op, TO, QT, SW, 128, 128, 2, 2, 4><<<nb, nt, 0, s>>>(a);
  }
  if constexpr (Op::kBytes == 4) {
    if (f == kTileF32)
      expert_product_kernel<Op, TO, QT, SW, 64, 64, 4, 1, 4><<<nb, nt, 0, s>>>(a);
  } else {
    if (f == kTileSmall)
      expert_product_kernel<Op, TO, QT, SW, 64, 128, 2, 2, 4><<<nb, nt, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <class Op, typename TO>
static hipError_t run_product(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.swiglu) return run_form<Op, TO, false, true>(a, s);
  if constexpr (Op::kBytes != 1)
    if (a.transpose) return run_form<Op, TO, true, false>(a, s);
  return run_form<Op, TO, false, false>(a, s);
}

hipError_t launch_expert_matmul(const ExpertMatmulArgs& a, hipStream_t s) {
  if (a.type == kRowsI8)
    return a.out_bf16 ? run_product<I8Op, uint16_t>(a, s) : run_product<I8Op, float>(a, s);
  return a.type == kRowsBf16 ? run_product<Bf16Op, uint16_t>(a, s)
                             : run_product<F32Op, float>(a, s);
}

size_t expert_wgrad_ws_bytes(int bf16, int M, int E, int n, int k) {
  return static_cast<size_t>(plan_wgrad(bf16, M, E, n, k).slots) * n * k * 4;
}
bool expert_wgrad_fits(const ExpertWgradArgs& a) {
  // row lengths in bytes are 32 bits, and so is a task's number rounded up to a part or stage
  if (a.n > 1 << 22 || a.k > 1 << 22 || a.M > 1 << 30) return false;
  ExpertWgradArgs b = a;
  const WgradPlan p = plan_wgrad(a.bf16, a.M, a.E, a.n, a.k);
  b.part = p.part;
  return wgrad_blocks(b, p.tile) < (1ll << 32) / wgrad_threads(p.tile) &&
         a.E < (p.part ? 65536 : 1 << 30) &&
         static_cast<long long>(a.n) * a.k / 4 < (1ll << 32) - 1024;
}

template <class Op, int B, int WM, int WN>
static hipError_t run_wgrad(const ExpertWgradArgs& a, hipStream_t s) {
  static_assert(WM * WN <= (B == 256 ? 8 : 4), "wgrad_threads");
  const unsigned nb = static_cast<unsigned>(wgrad_blocks(a, B));
  if (a.x_row && a.dy_row)
    expert_wgrad_kernel<Op, B, B, WM, WN, 4, true><<<nb, WM * WN * 64, 0, s>>>(a);
  else
    expert_wgrad_kernel<Op, B, B, WM, WN, 4, false><<<nb, WM * WN * 64, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_expert_wgrad(const ExpertWgradArgs& args, float* ws, hipStream_t s) {
  ExpertWgradArgs a = args;
  const WgradPlan p = plan_wgrad(a.bf16, a.M, a.E, a.n, a.k);
  a.part = p.part;
  a.slots = p.slots;
  a.partial = ws;
  hipError_t e;
  if (p.tile == 256) e = run_wgrad<Bf16Op, 256, 2, 4>(a, s);
  else if (p.tile == 128) e = run_wgrad<Bf16Op, 128, 2, 2>(a, s);
  else
    e = a.bf16 ? run_wgrad<Bf16Op, 64, 2, 2>(a, s) : run_wgrad<F32Op, 64, 2, 2>(a, s);
  if (e != hipSuccess || a.part == 0) return e;
  const unsigned nb =
      static_cast<unsigned>((static_cast<size_t>(a.n) * a.k + kReduce - 1) / kReduce);
  expert_wgrad_reduce_kernel<<<dim3(nb, a.E), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace omni
