// Products of two matrices tile by tile, for kernels that go on with a tile in registers:
//   acc[n][m] += sum over k of A[m][k] * B[k][n]
// A workgroup of four waves makes a tile of BM x BN, a wave TM x TN blocks of 32x32 of it. An operand
// is given in rows along k (ROWS) or in rows of one k each (COLS; LDS delivers it transposed), and
// either as a matrix of rows or in panels: 64 bytes of every row, one row after the other, panel
// after panel (_P). A step takes 64 bytes along k: of a matrix that is half a cache line of each
// row, of panels it is one piece, which halves the requests to L2 (8192 x 30522 x 768 in bf16 with
// tiles of 128 x 256, rows in panels: 69.6 million requests became 46, and 424 us 395). Steps go from
// memory straight into a ring of STAGES places in LDS, swizzled so that the reads meet no bank
// twice; a place is filled again one step after it was read, so that STAGES - 1 steps are under way
// and one barrier a step does.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

constexpr int GEMM_THREADS = 256;
constexpr int PANEL = 64;  // bytes of a row in a panel

enum { SIDE_ROWS, SIDE_COLS, SIDE_ROWS_P, SIDE_COLS_P };

// One operand's steps. R: its rows, or columns (of the result's side).
template <int DT, int R, int KIND> struct GemmSide {
  static constexpr int eb = Elem<DT>::bytes;
  static constexpr int BK = 64 / eb;  // of a step
  static constexpr bool along_k = KIND == SIDE_ROWS || KIND == SIDE_ROWS_P;
  using L = RowLayout<DT, KIND == SIDE_COLS ? R : BK>;  // a row in LDS
  static constexpr int bytes = R * 64;
  static constexpr int pieces = R / 64 < 1 ? 1 : R / 64;  // 16 bytes a thread each
  static constexpr bool partial = R < 64;                  // fewer pieces than threads
  uint32_t at[pieces];
  uint64_t base, step;  // and the bytes from one step to the next
  uint32_t stride;      // of rows, or of k rows

  // Piece i of this thread: its row in LDS and the byte within that row; and for panels of columns
  // the panel.
  struct Place {
    int row, byte, panel;
  };
  __device__ __forceinline__ static Place place(int i) {
    const int p = threadIdx.x + i * GEMM_THREADS, q = p / L::chunks;
    const int r = KIND == SIDE_COLS_P ? q % BK : q;
    return {r, (p % L::chunks * 16) ^ L::f(r), q / BK};
  }
  // first: row or column 0 of the tile at k = 0, of which `exist` rows, or bytes of columns, exist (the
  // last row, or 16 bytes, is repeated). `by`: a matrix's bytes from row to row, or panels' from one
  // to the next.
  __device__ __forceinline__ void start(const char *first, int64_t by, int exist) {
    start(first, by, exist, [](int row) { return row; });
  }
  // row(i): which of the matrix's rows is row i (ROWS).
  template <typename Row> __device__ __forceinline__ void start(const char *first, int64_t by, int exist, Row row) {
    base = (uint64_t)uniform((int64_t)(uintptr_t)first);
    stride = KIND == SIDE_ROWS || KIND == SIDE_COLS ? (uint32_t)by : PANEL;
    step = KIND == SIDE_ROWS ? 64 : KIND == SIDE_ROWS_P ? (uint64_t)by : (uint64_t)BK * stride;
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const Place p = place(i);
      if constexpr (along_k) {
        at[i] = (uint32_t)row(p.row < exist ? p.row : exist - 1) * stride + p.byte;
      } else {
        int c = KIND == SIDE_COLS ? p.byte : p.panel * PANEL + p.byte;
        c = c < exist ? c : exist - 16;
        at[i] = (uint32_t)p.row * stride + (KIND == SIDE_COLS ? (uint32_t)c : (uint32_t)(c / PANEL * by) + c % PANEL);
      }
    }
  }
  // The last step: `left` bytes (ROWS) or k rows (COLS) of it exist, the last ones are repeated.
  __device__ __forceinline__ void narrow(int left) {
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const Place p = place(i);
      if constexpr (along_k) {
        if (p.byte >= left) at[i] -= (uint32_t)(p.byte - left + 16);
      } else {
        if (p.row >= left) at[i] -= (uint32_t)(p.row - left + 1) * stride;
      }
    }
  }
  __device__ __forceinline__ void go(int to, int wave) {
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const int p = wave * 64 + i * GEMM_THREADS;
      if (partial && p >= R * 4) break;
      asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                   :
                   : "{m0}"(uniform(to + p * 16)), "v"(at[i]), "s"(uniform((int64_t)base)));
    }
    base += step;
  }
  // Loads of one wave (uniform): a partial tile's last waves have none.
  __device__ __forceinline__ static int loads(int wave) {
    return partial ? (wave * 64 < R * 4 ? 1 : 0) : pieces;
  }

  // Zeros for what lies past `left` bytes of every row of a step that is in LDS (ROWS).
  __device__ __forceinline__ static void clear_past(char *tile, int left) {
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const int p = threadIdx.x + i * GEMM_THREADS;
      if (p < R * 4 && (int)place(i).byte >= left) *(u32x4_t *)(tile + p * 16) = u32x4_t{0, 0, 0, 0};
    }
  }

  // This lane's place in a block of 32 rows or columns, and the operand of step t (of two) of block
  // `b`: k = 16 t + 8 h + 0 .. 7 (fp32: 8 t + 4 h + 0 .. 3) in lanes of half h.
  __device__ __forceinline__ static int lane_offset() {
    const int l = threadIdx.x & 63, h = l >> 5;
    if constexpr (along_k) {
      return (l & 31) * L::bytes + ((h * 16) ^ L::f(l & 31));
    } else if constexpr (DT == DT_FP32) {
      // columns of panels: 16 to a panel
      const int c = KIND == SIDE_COLS ? l & 31 : l & 15;
      return 4 * h * L::bytes + ((c * 4) ^ L::f(4 * h)) + (KIND == SIDE_COLS ? 0 : ((l >> 4) & 1) * BK * PANEL);
    } else {
      const int row = 8 * h + ((l & 15) >> 2);
      return row * L::bytes + ((((l >> 4) & 1) * 32 + (l & 2) * 8) ^ L::f(row)) + (l & 1) * 8;
    }
  }
  __device__ __forceinline__ static u32x4_t operand(const char *tile, int lane, int b, int t) {
    if constexpr (along_k) {
      return load16(tile + b * 32 * L::bytes + L::along(lane, 32 * t));
    } else if constexpr (DT == DT_FP32) {
      u32x4_t x;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int row = 8 * t + e, in = lane ^ L::f(row);
        x[e] = *(const uint32_t *)(tile + row * L::bytes +
                                   (KIND == SIDE_COLS ? L::along(in, b * 128) : in + b * 2 * BK * PANEL));
      }
      return x;
    } else {
      // rows 8 h .. 8 h + 3 and the four after them, whose f differs in its lowest bit
      const char *at = tile + 16 * t * L::bytes + (KIND == SIDE_COLS ? 0 : b * BK * PANEL);
      const int by = KIND == SIDE_COLS ? b * 64 : 0;
      const s16x4_t lo = read_tr(at + L::along(lane, by));
      const s16x4_t hi = read_tr(at + 4 * L::bytes + L::along(lane ^ 16, by));
      return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

template <int DT, int BM, int BN, int WM, int AKIND, int BKIND, int STAGES> struct TileGemm {
  static constexpr int WN = 4 / WM;
  static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  static_assert(TM * WM * 32 == BM && TN * WN * 32 == BN, "whole blocks");
  using A = GemmSide<DT, BM, AKIND>;
  using B = GemmSide<DT, BN, BKIND>;
  static constexpr int stage = A::bytes + B::bytes;
  static constexpr int lds = STAGES * stage;
  static constexpr int BK = A::BK;

  // fp32 sums of tiles that leave registers go in two levels: a place's 16 entries along k are added up
  // first. One chain of d / 2 sums costs digits that fp32 operands have (scale 5: 137 rows, 929 x 728,
  // gradients off by 2.7e-6 of their size and 0.9e-6 so; 24 rows, 13649 x 528, 2.9e-6 and 1.2e-6), for 6 to 9
  // in 100 of the time (32 rows, 30522 x 768: 32.0 us and 34.0; 78 rows, 25314 x 712: 64 and 70). All
  // kernels that make the same logits do it alike: errors that differ do not cancel in z - lse (as much
  // as 3e-6). 16-bit operands take 16 products at a time.
  static constexpr bool two_levels = DT == DT_FP32 && TM * TN <= 4;

  A a;
  B b;
  f32x16_t acc[TN][TM];

  // Until at most n of this wave's loads are under way, its LDS reads are done, and so is every
  // other wave. s_waitcnt takes a constant: counts other than the tiles' own wait for all.
  __device__ __forceinline__ static void wait(int n) {
    asm volatile("" ::: "memory");
    switch (n) {
#define MAXSIM_WAIT(N) case N: __builtin_amdgcn_s_waitcnt(0x0070 | ((N) & 15) | ((N) >> 4) << 14); break;
    MAXSIM_WAIT(6) MAXSIM_WAIT(8) MAXSIM_WAIT(20) MAXSIM_WAIT(30)
#undef MAXSIM_WAIT
    default: __builtin_amdgcn_s_waitcnt(0x0070); break;
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < TN; n++)
#pragma unroll
      for (int m = 0; m < TM; m++) acc[n][m] = zero16();
  }

  // The two steps of a place in the ring. All operands are read before the first product: a wave
  // waits once a place, and the other one of its SIMD fills that in.
  __device__ __forceinline__ void multiply(const char *tile, int la, int lb, int wm, int wn) {
    u32x4_t x[2][TM], y[2][TN];
#pragma unroll
    for (int t = 0; t < 2; t++) {
#pragma unroll
      for (int m = 0; m < TM; m++) {
        if (m < TN) y[t][m] = B::operand(tile + A::bytes, lb, wn * TN + m, t);
        x[t][m] = A::operand(tile, la, wm * TM + m, t);
      }
#pragma unroll
      for (int n = TM; n < TN; n++) y[t][n] = B::operand(tile + A::bytes, lb, wn * TN + n, t);
    }
    keep_order();
    if constexpr (two_levels) {
      f32x16_t part[TN][TM];
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int n = 0; n < TN; n++)
#pragma unroll
          for (int m = 0; m < TM; m++) part[n][m] = mma_rows<DT>(x[t][m], y[t][n], t ? part[n][m] : zero16());
#pragma unroll
      for (int n = 0; n < TN; n++)
#pragma unroll
        for (int m = 0; m < TM; m++) acc[n][m] += part[n][m];
    } else {
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int n = 0; n < TN; n++)
#pragma unroll
          for (int m = 0; m < TM; m++) acc[n][m] = mma_rows<DT>(x[t][m], y[t][n], acc[n][m]);
    }
    keep_order();
  }

  // ---- all steps of a tile (at least one): begin, then finish ----
  // What exists of the last step along k: a_last and b_last bytes (ROWS; 64 for all) or k rows (COLS;
  // BK for all). The last bytes or rows are repeated, so one side has to hold zeros there, or B is
  // cleared there (finish).
  int steps, fetched, a_last, b_last, to;

  __device__ __forceinline__ void fetch(int ring_at, int wave) {
    if (fetched == steps - 1) {
      if (a_last < (A::along_k ? 64 : BK)) a.narrow(a_last);
      if (b_last < (B::along_k ? 64 : BK)) b.narrow(b_last);
    }
    a.go(ring_at + to, wave);
    b.go(ring_at + to + A::bytes, wave);
    fetched++;
    to = to == (STAGES - 1) * stage ? 0 : to + stage;
  }
  // The first STAGES - 1 steps' loads, to the first places of a ring that nobody reads; the last
  // place stays free until finish.
  __device__ __forceinline__ void begin(char *ring, int n_steps, int last_a, int last_b) {
    steps = n_steps;
    a_last = last_a;
    b_last = last_b;
    fetched = to = 0;
    const int wave = uniform((int)threadIdx.x >> 6), ring_at = lds_address(ring);
    for (int i = 0; i < STAGES - 1; i++)
      if (fetched < steps) fetch(ring_at, wave);
  }
  // The ring is free again afterwards. CLEAR: with zeros for what B has not got of the last step.
  template <bool CLEAR = false> __device__ __forceinline__ void finish(char *ring) {
    const int wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
    const int la = A::lane_offset(), lb = B::lane_offset();
    const int ring_at = lds_address(ring);
    const int loads = A::loads(wave) + B::loads(wave);
    int from = 0;
    for (int i = 0; i < steps; i++) {
      const int ahead = fetched - i - 1;
      wait(ahead >= STAGES - 2 ? (STAGES - 2) * loads : 0);
      if (fetched < steps) fetch(ring_at, wave);
      if (CLEAR && i == steps - 1 && b_last < 64) {
        B::clear_past(ring + from + A::bytes, b_last);
        __syncthreads();
      }
      multiply(ring + from, la, lb, wm, wn);
      from = from == (STAGES - 1) * stage ? 0 : from + stage;
    }
    wait(0);
  }
};

// The number of blocks of `per` in n.
__device__ __host__ __forceinline__ int64_t blocks_of(int64_t n, int64_t per) { return (n + per - 1) / per; }

}  // namespace maxsim
