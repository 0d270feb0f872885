// Pieces shared by the attention kernels (include/maxsim.h, maxsim_attention).
//
// All matrix work runs on 32x32 tiles. Accumulator layout: lane l holds column l % 32, and
// element r of it is row (r & 3) + 8 * (r >> 2) + 4 * (l / 32). Operands: A's lane holds row
// l % 32, B's lane column l % 32, and each lane half a share of the contraction index.
//
// The kernels compute scores so that the index they reduce over next runs along the
// accumulator's rows, i.e. along a lane's own registers: S^T = K Q^T in the forward and dQ
// kernels (a lane holds one query's scores), S = Q K^T in the dK / dV kernel (a lane holds one
// key's). Then 8 consecutive registers are, as they stand, a B operand of the following
// product: half 0 holds rows 0-3 and 8-11 of 16, half 1 rows 4-7 and 12-15. The A operand of
// that product has to come in the same row order, which two transposing LDS reads deliver
// (each gives a 16-lane group 4 rows x 16 columns, lane i the 4 values of column i).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "doc_lookup.hpp"

namespace maxsim {

// Score forms: plain scale; scale and distance bias; scale and tanh cap; all of them; and 16-bit
// types' caps above ATTN_NEAR_CAP, with or without a bias (whose slope is 0 then).
enum { ATTN_PLAIN = 0, ATTN_BIAS = 1, ATTN_CAP = 2, ATTN_CAP_BIAS = 3, ATTN_FAR_CAP = 4 };
constexpr bool has_cap(int mode) { return mode >= ATTN_CAP; }
constexpr bool has_bias(int mode) { return mode == ATTN_BIAS || mode >= ATTN_CAP_BIAS; }

// Largest cap of the 16-bit types' tanh in stages (tanh_stages). Its error, up to 2^-22 of the cap
// whatever the score, is then at most 2^-13 of a weight, a quarter of half a step of fp16. Larger
// caps take tanhf, whose error is relative to the score, and which takes longer: 16 pages of 1045
// tokens, 16 heads of 128 on 4, bf16, forward 190 and 257 us, backward 697 and 941.
constexpr float ATTN_NEAR_CAP = 512.0f;
// Above this one the capped score is the score itself in 32 bits for all scores below 2^88, and
// cap * log2 e and scale / cap would leave the range of fp32: no cap is applied.
constexpr float ATTN_NO_CAP = 1.2676506e30f;  // 2^100

struct AttnArgs {
  const char *q, *k, *v;
  int64_t q_doc, k_doc, v_doc;     // byte strides of documents (fixed layout)
  int64_t q_head, k_head, v_head;  // of heads
  int q_tok, k_tok, v_tok;         // of tokens
  const int64_t *offsets;
  int64_t n_tokens, n_docs;
  int nd;
  const int32_t *lens;
  const int32_t *prefix;
  int heads, kv_heads, group, d, causal;  // group: heads / kv_heads
  float softcap, scale;
  const float *slopes;
  char *o;                 // [rows][heads][d]
  float *lse;              // [heads][rows]
  int64_t rows;            // rows of o: all tokens
  uint32_t slots;          // tiles along the tokens
  FastDiv tiles_per_doc;   // fixed layout
  FastDiv per_kv, per_group;  // workgroups of a key/value head; of one tile of it
  uint32_t base, total;    // first workgroup of this launch, workgroups of all launches
  // backward
  const char *dO;          // [rows][heads][d]
  const float2 *stats;     // [heads][rows]: where S and dP start (attn_delta.hpp)
  const float *grad_scale; // fp16: power of two that dS is scaled by before its rounding
  char *dq, *dk, *dv;      // [rows][heads or kv_heads][d]
};

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// fp16 weights of the backward are rounded 2^8 times too large: over thousands of keys they would
// be subnormal.
constexpr float ATTN_WEIGHT_SHIFT = 8.0f;
constexpr int ATTN_THREADS = 256;
constexpr int ATTN_ROWS = 128;  // tokens of a workgroup's tile: 32 to a wave

template <int DT> struct AttnElem;
template <> struct AttnElem<DT_BF16> { using type = __bf16; };
template <> struct AttnElem<DT_FP16> { using type = _Float16; };
template <> struct AttnElem<DT_FP32> { using type = float; };

__device__ __forceinline__ f32x16_t zero16() {
  f32x16_t z;
#pragma unroll
  for (int i = 0; i < 16; i++) z[i] = 0.0f;
  return z;
}

// One 32-byte step of rows of A times rows of B: half h of the wave holds bytes 16 h .. 16 h + 15
// of the step. The same bytes feed the same contraction index on both sides.
template <int DT> __device__ __forceinline__ f32x16_t mma_rows(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else if constexpr (DT == DT_FP16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a),
                                                  __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  } else {
    const uint32_t a0 = a.x, a1 = a.y, a2 = a.z, a3 = a.w, b0 = b.x, b1 = b.y, b2 = b.z, b3 = b.w;
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a0), __uint_as_float(b0), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a1), __uint_as_float(b1), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a2), __uint_as_float(b2), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a3), __uint_as_float(b3), c, 0, 0, 0);
    return c;
  }
}

// A 32x32 accumulator as the B operand of the next product: rounded to the storage type (to
// nearest even) for the 16-bit types, as it is for fp32.
template <int DT> struct Packed {
  static constexpr int n = 2;  // operands of mma_cols that 32 rows make
  u32x4_t f[2];
  __device__ __forceinline__ void set_half(const f32x16_t &s, int t) {
    using T = typename AttnElem<DT>::type;
    typedef T v8 __attribute__((ext_vector_type(8)));
    v8 x;
#pragma unroll
    for (int e = 0; e < 8; e++) x[e] = (T)s[8 * t + e];
    f[t] = __builtin_bit_cast(u32x4_t, x);
  }
  __device__ __forceinline__ void set(const f32x16_t &s) {
    set_half(s, 0);
    set_half(s, 1);
  }
};
template <> struct Packed<DT_FP32> {
  static constexpr int n = 4;
  f32x16_t f;
  __device__ __forceinline__ void set(const f32x16_t &s) { f = s; }
};

// Rows of a head in LDS: DP columns (the head's size rounded up), no padding. LDS serves 16 lanes
// of a 16-byte read, or 32 lanes of an 8-byte one, a clock, if they fall on different 16 bytes of
// 256. A row's 16-byte chunks are stored at chunk ^ f(row): 16 rows of one chunk (an operand in
// rows) then lie on 16 different places, and so do 4 consecutive rows x 4 chunks (the transposing
// reads). f is linear: f(a ^ b) = f(a) ^ f(b).
template <int DT, int DP> struct RowLayout {
  static constexpr int eb = Elem<DT>::bytes;
  static constexpr int chunks = DP * eb / 16;  // 16-byte chunks of a row
  static constexpr int steps = DP * eb / 32;   // mma_rows steps of a row
  static constexpr int bytes = DP * eb;
  // bits of a byte offset that f(row) reaches: as many as divide the row
  static constexpr int mask = chunks % 16 == 0 ? 255 : chunks % 8 == 0 ? 127 : 63;
  // f(row) in bytes. Rows that differ by 16 share it, and row + 8 flips bit 5.
  __device__ __forceinline__ static constexpr int f(int row) {
    const int high = (row >> 2) & 3;
    return 16 * (mask == 255 ? (row & 3) << 2 | high : mask == 127 ? (row & 2) << 1 | high : high);
  }
  // A byte offset `at` plus `by` bytes along the row, where at contains f(row).
  __device__ __forceinline__ static int along(int at, int by) {
    return (at ^ (by & mask)) + (by & ~mask);
  }
};

// This lane's place in a tile for read_cols.
template <int DT, int DP> __device__ __forceinline__ int tr_lane_offset() {
  using L = RowLayout<DT, DP>;
  const int l = threadIdx.x & 63, h = l >> 5;
  if constexpr (DT == DT_FP32) return 4 * h * L::bytes + (((l & 31) * 4) ^ L::f(4 * h));
  const int row = 4 * h + ((l & 15) >> 2);
  return row * L::bytes + ((((l >> 4) & 1) * 32 + (l & 2) * 8) ^ L::f(row)) + (l & 1) * 8;
}

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ s16x4_t read_tr(const char *p) {
  typedef __attribute__((address_space(3))) char lds_char;
  typedef __attribute__((address_space(3))) s16x4_t lds_v4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(lds_char *)p);
}

// Operand `s` of 32 rows of an LDS tile (mma_rows' step s): lane is row_lane_offset.
template <int DT, int DP> __device__ __forceinline__ int row_lane_offset() {
  using L = RowLayout<DT, DP>;
  const int l = threadIdx.x & 63;
  return (l & 31) * L::bytes + ((l >> 5) * 16 ^ L::f(l));
}
template <int DT, int DP>
__device__ __forceinline__ u32x4_t read_rows(const char *tile, int lane, int s) {
  return load16(tile + RowLayout<DT, DP>::along(lane, 32 * s));
}
// Operand t of columns c0 .. c0 + 31 of a tile, transposed: for 16-bit types rows 16 t .. 16 t + 15,
// for fp32 rows 8 t .. 8 t + 7 (this lane's half of them). lane is tr_lane_offset.
template <int DT, int DP>
__device__ __forceinline__ u32x4_t read_cols(const char *tile, int lane, int c0, int t) {
  using L = RowLayout<DT, DP>;
  if constexpr (DT == DT_FP32) {
    u32x4_t x;
#pragma unroll
    for (int e = 0; e < 4; e++)  // row 8 t + e of this half's, whose f is on top of the lane's
      x[e] = *(const uint32_t *)(tile + (8 * t + e) * L::bytes + L::along(lane ^ L::f(8 * t + e), c0 * 4));
    return x;
  } else {
    const char *at = tile + 16 * t * L::bytes;
    const s16x4_t lo = read_tr(at + L::along(lane, c0 * 2));
    const s16x4_t hi = read_tr(at + 8 * L::bytes + L::along(lane ^ 32, c0 * 2));
    return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}
// acc += X^T[columns, operand t's rows] * P
template <int DT>
__device__ __forceinline__ f32x16_t mma_cols(u32x4_t x, const Packed<DT> &p, int t, f32x16_t acc) {
  if constexpr (DT == DT_FP32) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const uint32_t v = x[e];
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(v), p.f[4 * t + e], acc, 0, 0, 0);
    }
    return acc;
  } else {
    return mma_rows<DT>(x, p.f[t], acc);
  }
}

// Copies tiles of 32 rows of a head, one after the other, from global memory straight into LDS, in
// `n` pieces a tile: a wave's piece is 64 chunks that lie side by side in LDS, and each lane fetches
// the one that belongs there. Rows past the last one repeat it, and columns past the head's size
// its last 16 bytes: nothing outside is read, what follows stays finite, and those columns meet
// zeros (Held) or are not stored. Past the last tile one row is fetched again and again, which
// keeps branches out of the loops. Arrival is waited for by tile_barrier.
template <int DT, int DP> struct Carry {
  using L = RowLayout<DT, DP>;
  static constexpr int total = 32 * L::chunks;
  static constexpr int n = (total + ATTN_THREADS - 1) / ATTN_THREADS;
  uint32_t at[n];  // byte offset of this lane's chunks in the tile
  uint64_t base;   // first row of the tile (uniform, as what follows)
  int left;        // rows from there on
  int stride, row_bytes;

  __device__ __forceinline__ uint32_t column(int i) const {
    const int p = threadIdx.x + i * ATTN_THREADS;
    const int c = (p % L::chunks * 16) ^ L::f(p / L::chunks);
    return c < row_bytes ? c : row_bytes - 16;
  }
  __device__ __forceinline__ void init(int row_stride, int bytes) {
    stride = row_stride;
    row_bytes = bytes;
  }
  // The first tile: `rows` rows (at least one) from `first` on.
  __device__ __forceinline__ void start(const char *first, int rows) {
    base = (uint64_t)uniform((int64_t)(uintptr_t)first);
    left = uniform(rows);
#pragma unroll
    for (int i = 0; i < n; i++)
      at[i] = (uint32_t)((threadIdx.x + i * ATTN_THREADS) / L::chunks * stride) + column(i);
    if (left < 32) narrow();
  }
  __device__ __forceinline__ void narrow() {
    if (left < 1) {
      base -= (uint64_t)(uint32_t)(32 * stride);
      left = 1;
    }
    const uint32_t last = (uint32_t)(left - 1) * (uint32_t)stride;
#pragma unroll
    for (int i = 0; i < n; i++) {
      const uint32_t most = last + column(i);
      at[i] = at[i] < most ? at[i] : most;
    }
  }
  __device__ __forceinline__ void next() {
    base += (uint64_t)(uint32_t)(32 * stride);
    left -= 32;
    if (left < 32) narrow();
  }
  // Piece i of the tile, to LDS address `to`. wave: this wave's number (uniform).
  __device__ __forceinline__ void go(int to, int wave, int i) const {
    const int p = wave * 64 + i * ATTN_THREADS;
    if (total % ATTN_THREADS != 0 && p >= total) return;
    // The instruction itself: beside the builtin the compiler waits for every LDS read in flight
    // wherever it needs one. It has no result in registers, and tile_barrier waits for it.
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "{m0}"(uniform(to + p * 16)), "v"(at[i]), "s"(uniform((int64_t)base)));
  }
  __device__ __forceinline__ void all(int to, int wave) const {
#pragma unroll
    for (int i = 0; i < n; i++) go(to, wave, i);
  }
};

__device__ __forceinline__ int lds_address(const char *p) {
  typedef __attribute__((address_space(3))) char lds_char;
  return uniform((int)(uintptr_t)(lds_char *)p);
}

// Every wave's carried pieces and LDS writes have arrived, and its LDS reads are done.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // no loads, no LDS accesses outstanding
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// This lane's share of 32 rows as an mma_rows operand held in registers: row l % 32 (clamped to
// the last valid one), every step's 16 bytes; columns past the head's size are zero.
template <int DT, int DP> struct Held {
  using L = RowLayout<DT, DP>;
  u32x4_t f[L::steps];
  __device__ __forceinline__ void load(const char *base, int64_t stride, int row, int row_bytes) {
    const int h = (threadIdx.x & 63) >> 5;
    const char *p = base + row * stride;
#pragma unroll
    for (int s = 0; s < L::steps; s++) {
      u32x4_t z = {0, 0, 0, 0};
      if (s * 32 + h * 16 < row_bytes) z = load16(p + s * 32 + h * 16);
      f[s] = z;
    }
  }
};

// Nothing moves across: the compiler would put every LDS read right before its use, and a wave
// would wait out the latency of each.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// Until at most n of this wave's LDS reads are under way.
__device__ __forceinline__ void wait_reads(int n) {
  constexpr int NONE = 0xc07f;  // counters that are not waited for
  switch (n) {
  case 2: __builtin_amdgcn_s_waitcnt(NONE | 2 << 8); break;
  case 3: __builtin_amdgcn_s_waitcnt(NONE | 3 << 8); break;
  case 4: __builtin_amdgcn_s_waitcnt(NONE | 4 << 8); break;
  }
}

// N matrix instructions in order, their operands read from LDS AHEAD instructions before, with a
// share of other work beside each: read(i) gives operand i, mma(i, operand) uses it, work(i) is
// the i-th share. The compiler waits for every operand by itself; with the number of LDS reads that
// make operand i, reads(i), two are waited for at once, which saves a wave an instruction in eight
// or so where it is alone on its SIMD.
template <int N, int AHEAD, typename Read, typename Mma, typename Work, typename Reads>
__device__ __forceinline__ void pipeline(Read read, Mma mma, Work work, Reads reads) {
  constexpr int A = AHEAD < N ? AHEAD : N;
  u32x4_t x[A];
#pragma unroll
  for (int i = 0; i < A; i++) x[i] = read(i);
#pragma unroll
  for (int i = 0; i < N; i++) {
    keep_order();
    if (i % 2 == 0 && i + A <= N && reads(0)) {
      int after = 0;
#pragma unroll
      for (int e = 2; e < A; e++) after += reads(i + e);
      wait_reads(after);
      keep_order();
    }
    mma(i, x[i % A]);
    if (i + A < N) x[i % A] = read(i + A);
    work(i);
  }
  keep_order();
}

// 32 rows of an LDS tile times held columns, added to acc.
template <int DT, int DP>
__device__ __forceinline__ f32x16_t mma_tile(const char *tile, const Held<DT, DP> &b, f32x16_t acc) {
  using L = RowLayout<DT, DP>;
  const int lane = row_lane_offset<DT, DP>();
#pragma unroll
  for (int s = 0; s < L::steps; s++)
    acc = mma_rows<DT>(read_rows<DT, DP>(tile, lane, s), b.f[s], acc);
  return acc;
}

__device__ __forceinline__ int acc_row(int r) { return (r & 3) + 8 * (r >> 2); }

// Whether a tanh goes in stages (tanh_stages).
template <int DT, int MODE> constexpr bool staged = has_cap(MODE) && MODE != ATTN_FAR_CAP && DT != DT_FP32;

// Constants of the scores, in units of log 2 (the exponentials are powers of two).
struct ScoreForm {
  float a, b, slope;
  float c;  // the constant term that score_of_tanh leaves out
};
template <int DT, int MODE>
__device__ __forceinline__ ScoreForm score_form(const AttnArgs &a, int head) {
  ScoreForm f;
  f.slope = has_bias(MODE) && (MODE != ATTN_FAR_CAP || a.slopes) ? a.slopes[head] * LOG2E : 0.0f;
  f.a = a.scale * LOG2E;
  f.b = f.c = 0.0f;
  if (has_cap(MODE)) {
    f.a = a.scale / a.softcap * (staged<DT, MODE> ? 2.0f * LOG2E : 1.0f);
    f.a = __builtin_fminf(f.a, __FLT_MAX__);  // a tiny cap: 0 stays 0, the rest saturates
    f.b = a.softcap * LOG2E;
    f.c = staged<DT, MODE> ? f.b : 0.0f;
  }
  return f;
}

constexpr float NOTHING = -0.0f;  // x + NOTHING is x for every x, so the compiler drops the sum

// q.k (x) to a score, plus off; dist: the tokens' distance. keep: the cap's slope. 16-bit types
// take their tanh in stages, below, up to ATTN_NEAR_CAP.
template <int DT, int MODE>
__device__ __forceinline__ float score(const ScoreForm &f, float x, float dist, float off, float *keep) {
  float y;
  if constexpr (has_cap(MODE)) {
    const float t = tanhf(x * f.a);
    y = f.b * t + off;
    if (keep) *keep = __builtin_fmaf(-t, t, 1.0f);
  } else {
    y = x * f.a + off;
  }
  if constexpr (has_bias(MODE)) y = __builtin_fmaf(-f.slope, __builtin_fabsf(dist), y);
  return y;
}

// tanh x = 1 + 2 u, u = -1 / (1 + e^2x): a reciprocal and an exponential. Near 0 it loses relative
// accuracy: a score is off by up to 2^-22 of the cap, see ATTN_NEAR_CAP.
// Elements from .. to - 1 of x: each goes from q.k to u, one step of it beside another element's
// next, so that none waits for the one before; then done(r) takes it on.
template <typename Done>
__device__ __forceinline__ void tanh_stages(const ScoreForm &f, f32x16_t &x, int from, int to, Done done) {
#pragma unroll
  for (int r = from; r < to; r++) {
    if (r >= 2) done(r - 2);
    if (r >= 1) x[r - 1] = __builtin_amdgcn_rcpf(-1.0f - x[r - 1]);
    x[r] = __builtin_amdgcn_exp2f(x[r] * f.a);
  }
  if (to == 16) {
    x[15] = __builtin_amdgcn_rcpf(-1.0f - x[15]);
    done(14);
    done(15);
  }
}
// u to a score less its constant term, plus off, and the cap's slope over slope_unit.
template <int MODE>
__device__ __forceinline__ float score_of_tanh(const ScoreForm &f, float u, float dist, float off) {
  float y = __builtin_fmaf(2.0f * f.b, u, off);
  if constexpr (has_bias(MODE)) y = __builtin_fmaf(-f.slope, __builtin_fabsf(dist), y);
  return y;
}
__device__ __forceinline__ float slope_of_tanh(float u) { return __builtin_fmaf(-u, u, -u); }
template <int DT, int MODE> constexpr float slope_unit = staged<DT, MODE> ? 4.0f : 1.0f;

// Where a workgroup works: a tile of a document's rows, and a head.
struct AttnTile {
  int64_t row0;    // first row of the document, among all rows
  int64_t q, k, v; // byte offsets of the document's rows
  int rows;        // rows of the span (its length, or nd)
  int len;         // tokens that exist
  int first;       // first row of the tile
  int prefix;      // keys below it are visible to every row; len for no causal mask
  int head;
};

// Workgroups of one key/value head follow each other on one XCD (workgroups are dealt to the 8
// XCDs in turn), so that its L2 serves the keys and values that they share.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t n) {
  const uint32_t x = id & 7, per = n >> 3, more = n & 7;
  return x * per + (x < more ? x : more) + (id >> 3);
}

// False where the tile does not exist.
__device__ __forceinline__ bool locate(const AttnArgs &a, int rows, AttnTile &t) {
  const uint32_t id = xcd_order(a.base + blockIdx.x, a.total);
  const uint32_t kv = a.per_kv(id), in = id - kv * a.per_kv.d;
  uint32_t slot = a.per_group(in);
  t.head = kv * a.per_group.d + (in - slot * a.per_group.d);
  // with a causal mask the last tiles have the most keys: they start first
  if (a.causal) slot = a.slots - 1 - slot;
  int64_t doc;
  if (a.offsets) {
    const TileSpan s = find_tile(a.offsets, a.n_docs, a.n_tokens, slot, rows);
    if (s.first >= s.len) return false;
    t.row0 = s.begin;
    t.rows = (int)s.len;
    t.len = s.doc < 0 ? 0 : t.rows;
    t.first = (int)s.first;
    doc = s.doc;
    t.q = t.row0 * a.q_tok;
    t.k = t.row0 * a.k_tok;
    t.v = t.row0 * a.v_tok;
  } else {
    const uint32_t b = a.tiles_per_doc(slot);
    doc = b;
    t.first = (int)(slot - b * a.tiles_per_doc.d) * rows;
    t.row0 = doc * a.nd;
    t.rows = a.nd;
    const int n = a.lens ? uniform(a.lens[doc]) : a.nd;
    t.len = n < 0 ? 0 : (n < a.nd ? n : a.nd);
    t.q = doc * a.q_doc;
    t.k = doc * a.k_doc;
    t.v = doc * a.v_doc;
  }
  t.prefix = t.len;
  if (a.causal) {
    const int p = a.prefix && doc >= 0 ? a.prefix[doc] : 0;
    t.prefix = p < 0 ? 0 : (p < t.len ? p : t.len);
  }
  t.row0 = uniform(t.row0);
  t.q = uniform(t.q);
  t.k = uniform(t.k);
  t.v = uniform(t.v);
  t.rows = uniform(t.rows);
  t.len = uniform(t.len);
  t.first = uniform(t.first);
  t.prefix = uniform(t.prefix);
  t.head = uniform(t.head);
  return true;
}

// Keys that row i sees: those below the result.
__device__ __forceinline__ int visible(const AttnArgs &a, const AttnTile &t, int i) {
  if (!a.causal) return t.len;
  const int n = i + 1 > t.prefix ? i + 1 : t.prefix;
  return n < t.len ? n : t.len;
}

// Stores 32 rows of a wave's transposed accumulators, each lane's row times f (0 for rows that do
// not exist), through the wave's own 32 rows of LDS: a lane holds 4 columns of a row here and
// there, memory wants whole rows. out: the wave's first row, rows `stride` bytes apart, the first
// `rows` of them written.
template <int DT, int DP, int OT>
__device__ __forceinline__ void store_rows(char *lds, const f32x16_t (&acc)[OT], float f, char *out,
                                           int64_t stride, int rows, int row_bytes) {
  using L = RowLayout<DT, DP>;
  using T = typename AttnElem<DT>::type;
  typedef T v4 __attribute__((ext_vector_type(4)));
  int l = threadIdx.x & 63;
  asm volatile("" : "+v"(l));  // nothing of this is kept in registers from before the main loop
  const int row = l & 31, h = l >> 5;
#pragma unroll
  for (int c = 0; c < OT; c++)
#pragma unroll
    for (int g = 0; g < 4; g++) {
      v4 x;
#pragma unroll
      for (int e = 0; e < 4; e++) x[e] = (T)(acc[c][4 * g + e] * f);
      const int at = (c * 32 + 8 * g + 4 * h) * L::eb;
      *(v4 *)(lds + row * L::bytes + ((at & ~15) ^ L::f(row)) + (at & 15)) = x;
    }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < (32 * L::chunks) / 64; i++) {
    const int p = i * 64 + l, r = p / L::chunks, c = p % L::chunks * 16;
    const u32x4_t x = *(const u32x4_t *)(lds + r * L::bytes + (c ^ L::f(r)));
    if (r < rows && c < row_bytes) *(u32x4_t *)(out + r * stride + c) = x;
  }
  wave_lds_sync();
}

// Zeros in a tile's rows of out [rows][heads][d].
template <int DT>
__device__ __forceinline__ void zero_tile(char *out, int heads, const AttnTile &t, int tile_rows, int d) {
  const int chunks = d * Elem<DT>::bytes / 16, left = t.rows - t.first;
  const int rows = left < tile_rows ? left : tile_rows;
  const u32x4_t z = {0, 0, 0, 0};
  for (int e = threadIdx.x; e < rows * chunks; e += ATTN_THREADS) {
    const int r = e / chunks, c = e - r * chunks;
    *(u32x4_t *)(out + ((t.row0 + t.first + r) * heads + t.head) * (chunks * 16) + c * 16) = z;
  }
}

__device__ __forceinline__ float half_max(float v) {
  uint32_t a, b;
  row_pair<32>(__float_as_uint(v), a, b);
  return __builtin_fmaxf(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float half_sum(float v) {
  uint32_t a, b;
  row_pair<32>(__float_as_uint(v), a, b);
  return __uint_as_float(a) + __uint_as_float(b);
}

}  // namespace maxsim
