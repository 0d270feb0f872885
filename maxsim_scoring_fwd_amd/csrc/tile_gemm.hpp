// Products of two matrices tile by tile, for kernels that go on with a tile in registers:
//   acc[n][m] += sum over k of A[m][k] * B[k][n]
// A workgroup of four waves makes a tile of BM x BN, a wave TM x TN blocks of 32x32 of it. Either
// operand is given in rows along k (ROWS) or in rows of one k each (COLS): the second is what
// LDS delivers transposed. Tiles of 64 bytes along k go from memory straight into a ring of STAGES
// places in LDS, swizzled so that neither kind of read meets a bank twice; a place is filled again
// one step after it was read, so that STAGES - 1 tiles are under way and one barrier a step does.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

constexpr int GEMM_THREADS = 256;

// One operand's tiles. R: its rows (of the result's side), COLS: rows of one k each.
template <int DT, int R, bool COLS> struct GemmSide {
  static constexpr int eb = Elem<DT>::bytes;
  static constexpr int BK = 64 / eb;  // of a step
  using L = RowLayout<DT, COLS ? R : BK>;
  static constexpr int bytes = R * 64;
  static constexpr int pieces = R / 64 < 1 ? 1 : R / 64;  // 16 bytes a thread each
  static constexpr bool partial = R < 64;                  // fewer pieces than threads
  uint32_t at[pieces];
  uint64_t base;
  uint32_t step;  // bytes from one step to the next

  // ROWS: `first` is row 0 of the tile at k = 0, of which `rows` exist (the last is repeated), with
  // rows `stride` bytes apart. COLS: `first` is column 0 of the tile at k = 0, of which `rows`
  // bytes exist (the last 16 are repeated); k rows `stride` bytes apart.
  __device__ __forceinline__ void start(const char *first, int64_t stride, int rows) {
    base = (uint64_t)uniform((int64_t)(uintptr_t)first);
    step = COLS ? (uint32_t)(BK * stride) : 64u;
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const int p = threadIdx.x + i * GEMM_THREADS;
      const int r = p / L::chunks, c = (p % L::chunks * 16) ^ L::f(r);
      if (COLS) at[i] = (uint32_t)(r * stride) + (c < rows ? c : rows - 16);
      else at[i] = (uint32_t)((r < rows ? r : rows - 1) * stride) + c;
    }
  }
  // The last step: `left` bytes (ROWS) or k rows (COLS) of it exist, the last ones are repeated.
  __device__ __forceinline__ void narrow(int left, int64_t stride) {
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const int p = threadIdx.x + i * GEMM_THREADS;
      const int r = p / L::chunks, c = (p % L::chunks * 16) ^ L::f(r);
      if (COLS) {
        if (r >= left) at[i] -= (uint32_t)((r - left + 1) * stride);
      } else if (c >= left) {
        at[i] -= (uint32_t)(c - left + 16);
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
  // ROWS: zeros past `left` bytes along k.
  __device__ __forceinline__ static void clear_from(char *tile, int left) {
#pragma unroll
    for (int i = 0; i < pieces; i++) {
      const int p = threadIdx.x + i * GEMM_THREADS;
      const int r = p / L::chunks, c = (p % L::chunks * 16) ^ L::f(r);
      if (p < R * 4 && c >= left) *(u32x4_t *)(tile + p * 16) = u32x4_t{0, 0, 0, 0};
    }
  }
  // Loads of one wave (uniform): a partial tile's last waves have none.
  __device__ __forceinline__ static int loads(int wave) {
    return partial ? (wave * 64 < R * 4 ? 1 : 0) : pieces;
  }

  // This lane's place in a block of 32 rows, and the operand of step t (of two) of block `b`.
  __device__ __forceinline__ static int lane_offset() {
    const int l = threadIdx.x & 63, h = l >> 5;
    if constexpr (!COLS) return (l & 31) * L::bytes + ((h * 16) ^ L::f(l & 31));
    else if constexpr (DT == DT_FP32) return 4 * h * L::bytes + (((l & 31) * 4) ^ L::f(4 * h));
    else {
      const int row = 8 * h + ((l & 15) >> 2);
      return row * L::bytes + ((((l >> 4) & 1) * 32 + (l & 2) * 8) ^ L::f(row)) + (l & 1) * 8;
    }
  }
  __device__ __forceinline__ static u32x4_t operand(const char *tile, int lane, int b, int t) {
    if constexpr (!COLS) {
      return load16(tile + b * 32 * L::bytes + L::along(lane, 32 * t));
    } else if constexpr (DT == DT_FP32) {
      u32x4_t x;
#pragma unroll
      for (int e = 0; e < 4; e++)
        x[e] = *(const uint32_t *)(tile + (8 * t + e) * L::bytes + L::along(lane ^ L::f(8 * t + e), b * 128));
      return x;
    } else {
      // rows 8 h .. 8 h + 3 and the four after them, whose f differs in its lowest bit
      const char *at = tile + 16 * t * L::bytes;
      const s16x4_t lo = read_tr(at + L::along(lane, b * 64));
      const s16x4_t hi = read_tr(at + 4 * L::bytes + L::along(lane ^ 16, b * 64));
      return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

template <int DT, int BM, int BN, int WM, bool ACOLS, bool BCOLS, int STAGES> struct TileGemm {
  static constexpr int WN = 4 / WM;
  static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  static_assert(TM * WM * 32 == BM && TN * WN * 32 == BN, "whole blocks");
  using A = GemmSide<DT, BM, ACOLS>;
  using B = GemmSide<DT, BN, BCOLS>;
  static constexpr int stage = A::bytes + B::bytes;
  static constexpr int lds = STAGES * stage;
  static constexpr int BK = A::BK;

  A a;
  B b;
  f32x16_t acc[TN][TM];

  // Until at most n of this wave's loads are under way, its LDS reads are done, and so is every
  // other wave: s_waitcnt takes a constant.
  __device__ __forceinline__ static void wait(int n) {
    asm volatile("" ::: "memory");
    switch (n) {
    case 0: __builtin_amdgcn_s_waitcnt(0x0070); break;
#define MAXSIM_WAIT(N) case N: __builtin_amdgcn_s_waitcnt(0x0070 | ((N) & 15) | ((N) >> 4) << 14); break;
    MAXSIM_WAIT(1) MAXSIM_WAIT(2) MAXSIM_WAIT(3) MAXSIM_WAIT(4) MAXSIM_WAIT(5) MAXSIM_WAIT(6)
    MAXSIM_WAIT(8) MAXSIM_WAIT(10) MAXSIM_WAIT(12) MAXSIM_WAIT(15) MAXSIM_WAIT(16)
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

  // The two steps of a place in the ring.
  __device__ __forceinline__ void multiply(const char *tile, int la, int lb, int wm, int wn) {
#pragma unroll
    for (int t = 0; t < 2; t++) {
      u32x4_t x[TM], y[TN];
#pragma unroll
      for (int m = 0; m < TM; m++) x[m] = A::operand(tile, la, wm * TM + m, t);
#pragma unroll
      for (int n = 0; n < TN; n++) y[n] = B::operand(tile + A::bytes, lb, wn * TN + n, t);
#pragma unroll
      for (int n = 0; n < TN; n++)
#pragma unroll
        for (int m = 0; m < TM; m++) acc[n][m] = mma_rows<DT>(x[m], y[n], acc[n][m]);
    }
  }

  // All steps (at least one). Bytes along k that exist in the last step of ROWS operands: `left` (64
  // for all); k rows that exist in that of COLS operands: a_last and b_last, the last is repeated.
  // The ring is free again afterwards.
  __device__ __forceinline__ void run(char *ring, int steps, int left, int a_last, int b_last, int64_t a_stride,
                                      int64_t b_stride) {
    const int wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
    const int la = A::lane_offset(), lb = B::lane_offset();
    const int ring_at = lds_address(ring);
    const int loads = A::loads(wave) + B::loads(wave);
    int fetched = 0, to = 0;
    auto fetch = [&]() {
      if (fetched == steps - 1) {
        if (ACOLS ? a_last < BK : left < 64) a.narrow(ACOLS ? a_last : left, a_stride);
        if (BCOLS ? b_last < BK : left < 64) b.narrow(BCOLS ? b_last : left, b_stride);
      }
      a.go(ring_at + to, wave);
      b.go(ring_at + to + A::bytes, wave);
      fetched++;
      to = to == (STAGES - 1) * stage ? 0 : to + stage;
    };
    for (int i = 0; i < STAGES - 1; i++)
      if (fetched < steps) fetch();
    int from = 0;
    for (int i = 0; i < steps; i++) {
      const int ahead = fetched - i - 1;
      wait(ahead >= STAGES - 2 ? (STAGES - 2) * loads : 0);
      if (fetched < steps) fetch();
      if (!ACOLS && i == steps - 1 && left < 64) {
        // what the last step lacks along k counts as 0: the same loop serves it
        A::clear_from(ring + from, left);
        if (!BCOLS) B::clear_from(ring + from + A::bytes, left);
        wait(0);
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
