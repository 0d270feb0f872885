// MaxSim scores of 4-bit microscaled vectors (include/maxsim.h, maxsim_score_mx4).
//
// One wave takes a document at a time, 16 tokens a tile (32 or 64 of rows of 64 or 32 entries), as in the dense kernel: persistent waves
// with contiguous, token-balanced document ranges, a ring of P tiles in flight, rows past a
// document's end clamped to its last token (a duplicate does not change a maximum), the running
// maxima in one register per 16 query tokens. The products run on the scaled matrix instruction
// 16x16x128: lane l of an operand holds 32 entries of row l % 16 (16 bytes of codes), block
// l / 16 of the row's 128 entries, and that block's exponent, so that a tile's rows go from memory
// to the operand as they lie: 16 bytes and one byte a lane, the whole 64-byte rows of 128 entries
// side by side in one instruction. Each product of two entries and their powers of two is exact in
// 32 bits. Rows shorter than whole 128 entries: the lanes past the end fetch the row's first block
// (finite, in range) and meet zeros in the query's operand. The read of the documents bounds it: on
// one MI355X 100000 documents of 128 tokens, d = 128, take 129 to 132 us (870 MB at 6.7 TB/s), and
// 20000 of 20 to 300 tokens, d = 96, 34 us (163 MB at 4.8 TB/s, of which the search for a wave's
// documents and the last tiles are some 10 us). Wide rows have few documents a wave, and the longest share
// sets the time (10000 documents of 128 tokens: d = 256 42 us, 4.1 TB/s, 512 83 us, 4.2; 5000, d = 1024
// 91 us, 3.8). With a long query LDS and the matrix cores share it (5000 documents of 180 tokens, d = 128,
// 300 query tokens: 44 us for 12 of bytes; LDS busy 41 in 100 cycles, the matrix cores 26).
#pragma once

#include "dense_kernel.hpp"
#include "doc_lookup.hpp"

namespace maxsim {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

struct Mx4Args {
  DenseArgs doc;  // documents: D (codes), offsets, n_docs, nd, doc_lens, contiguous, out
  const uint8_t *d_scale, *q_scale;
  const char *Q;
  int q_len;
  int blocks;  // of 32 entries in a row
};

__device__ __forceinline__ f32x4_t mfma_mx4(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x4_t c) {
  const i32x8_t x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  constexpr int FP4 = 4;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, FP4, FP4, 0, (int)sa, 0, (int)sb);
}

// The document boundaries nearest to the token targets lo and hi, as nearest_boundary finds one: the
// halves of the wave search for one each, which takes half as many loads that wait for each other.
__device__ __forceinline__ void nearest_boundaries(const int64_t *off, int64_t n_docs, int64_t lo, int64_t hi,
                                                   int lane, int64_t &first, int64_t &end) {
  const int64_t target = lane < 32 ? lo : hi;
  int64_t a = 0, b = n_docs + 1;  // the first offset that is not below the target lies in [a, b]
  while (__any(a < b)) {
    const int64_t step = (b - a + 31) / 32, at = a + (lane & 31) * step;
    const bool less = at < b && off[at] < target;  // these are a prefix of the probes
    const uint64_t all = __ballot(less);
    const int n = __popc((uint32_t)(all >> (lane & 32)));
    if (a < b) {
      const int64_t next = a + n * step;
      if (n == 0) {
        b = a;
      } else {
        a = next - step + 1;
        b = next < b ? next : b;
      }
    }
  }
  if (a > 0) {
    const int64_t below = off[a - 1], above = a <= n_docs ? off[a] : below;
    if (a > n_docs || target - below < above - target) a--;
  }
  first = lane_value(a, 0);
  end = lane_value(a, 32);
}

// KS: steps of 128 entries in a row; QB: blocks of 16 query tokens; P: tiles in flight; QLDS: the
// query's operands come from LDS, else they stay in registers. SUB: rows of 128 / SUB entries, of which
// an operand holds SUB sixteens side by side, and the query stands in its own part of SUB operands
// beside zeros: as many products, but whole loads (documents of 128 tokens, 60000 with d = 64: 72 us
// with SUB = 1, 56 with 2; 100000 with d = 32: 80 with 1, 45 with 4). A block that is not a number
// meets the zeros too, and takes out the tokens of its document that lie 16, 32 and 48 places away.
template <int KS, int QB, int P, bool QLDS, int SUB>
__global__ void __launch_bounds__(DENSE_THREADS) mx4_score_kernel(Mx4Args a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & (WAVE - 1);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t wave = uniform((int64_t)blockIdx.x * DENSE_WAVES + (threadIdx.x >> 6));
  const int64_t nwaves = (int64_t)gridDim.x * DENSE_WAVES;
  const int64_t RB = (int64_t)a.blocks * 16;  // bytes of a row's codes
  const int q_len = a.q_len;
  static_assert(SUB == 1 || (KS == 1 && !QLDS), "narrow rows, short queries");

  // this lane's block of every step, or block 0 where the row has none there; and which of the
  // tile's rows it holds
  constexpr int ROWS = 16 * SUB;
  const int part = SUB == 1 ? 0 : g * SUB / 4, tile_row = part * 16 + r16;
  uint32_t blk[KS];
  bool has[KS];
#pragma unroll
  for (int c = 0; c < KS; c++) {
    const int at = c * 4 + (SUB == 1 ? g : g % (4 / SUB));
    has[c] = at < a.blocks;
    blk[c] = has[c] ? at : 0;
  }
  auto query = [&](int qb, int c, int sub, uint32_t &s) {
    const int qi = qb * 16 + r16;
    u32x4_t v = {0u, 0u, 0u, 0u};
    s = 0;
    if (qi < q_len && has[c] && sub == part) {
      v = load16(a.Q + (int64_t)qi * RB + blk[c] * 16);
      s = a.q_scale[(int64_t)qi * a.blocks + blk[c]];
    }
    return v;
  };
  u32x4_t qreg[QLDS ? 1 : QB][QLDS ? 1 : KS * SUB];
  uint32_t qs[QLDS ? 1 : QB][QLDS ? 1 : KS * SUB];
  // operands of block qb, step c in LDS: 64 lanes x 16 bytes, then, after all of those, exponents
  constexpr int OPERAND = WAVE * 16;
  if constexpr (QLDS) {
    for (int i = threadIdx.x >> 6; i < QB * KS; i += DENSE_WAVES) {
      // the step is a run-time number here: its block is worked out again
      const int qb = i / KS, at = i % KS * 4 + g, qi = qb * 16 + r16;
      u32x4_t v = {0u, 0u, 0u, 0u};
      uint8_t s = 0;
      if (qi < q_len && at < a.blocks) {
        v = load16(a.Q + (int64_t)qi * RB + at * 16);
        s = a.q_scale[(int64_t)qi * a.blocks + at];
      }
      *(u32x4_t *)(lds + i * OPERAND + lane * 16) = v;
      lds[QB * KS * OPERAND + i * WAVE + lane] = (char)s;
    }
    __syncthreads();
  } else {
#pragma unroll
    for (int qb = 0; qb < QB; qb++)
#pragma unroll
      for (int c = 0; c < KS; c++)
#pragma unroll
        for (int sub = 0; sub < SUB; sub++) qreg[qb][c * SUB + sub] = query(qb, c, sub, qs[qb][c * SUB + sub]);
  }

  // ---- producer: the (document, tile) sequence of this wave ----
  int64_t pb = wave, pend = a.doc.n_docs, pstep = nwaves;
  if (a.doc.offsets) {
    const int64_t t0 = uniform(a.doc.offsets[0]);
    const int64_t ntok = uniform(a.doc.offsets[a.doc.n_docs]) - t0;
    const int64_t lo = t0 + ntok * wave / nwaves, hi = t0 + ntok * (wave + 1) / nwaves;
    nearest_boundaries(a.doc.offsets, a.doc.n_docs, lo, hi, lane, pb, pend);
    if (wave == nwaves - 1) pend = a.doc.n_docs;
    if (wave == 0) pb = 0;
    pstep = 1;
  } else if (a.doc.contiguous) {
    pb = a.doc.n_docs * wave / nwaves;
    pend = a.doc.n_docs * (wave + 1) / nwaves;
    pstep = 1;
  }
  int64_t pfirst = 0, plen = 0, ptile = 0;
  if (pb < pend) doc_extent(a.doc, pb, pfirst, plen);

  struct Tile {
    int64_t doc;
    bool valid, doc_end, empty;
  };
  u32x4_t buf[P][KS];
  uint32_t sc[P][KS];
  Tile slot[P];
  auto issue = [&](u32x4_t(&dst)[KS], uint32_t(&ds)[KS], Tile &sl) {
    sl.valid = false;
    const char *base = a.Q;  // a dummy in range for empty or exhausted slots: the query's first row
    const uint8_t *sbase = a.q_scale;
    int last = 0;
    if (pb < pend) {
      sl.valid = true;
      sl.doc = pb;
      bool advance = true;
      if (plen <= 0) {
        sl.doc_end = sl.empty = true;
      } else {
        const int64_t t0 = ptile * ROWS, rem = plen - 1 - t0;
        last = rem < ROWS - 1 ? (int)rem : ROWS - 1;
        base = a.doc.D + (pfirst + t0) * RB;
        sbase = a.d_scale + (pfirst + t0) * a.blocks;
        sl.empty = false;
        sl.doc_end = rem < ROWS;
        advance = sl.doc_end;
        ptile++;
      }
      if (advance) {
        pb += pstep;
        ptile = 0;
        if (pb < pend) doc_extent(a.doc, pb, pfirst, plen);
      }
    }
    const uint32_t row = tile_row < last ? tile_row : last;
#pragma unroll
    for (int c = 0; c < KS; c++) {
      const uint32_t at = row * a.blocks + blk[c];
      dst[c] = load16_nt(base + at * 16);
      ds[c] = sbase[at];
    }
  };
#pragma unroll
  for (int p = 0; p < P; p++) issue(buf[p], sc[p], slot[p]);

  float m[QB];
#pragma unroll
  for (int qb = 0; qb < QB; qb++) m[qb] = -__builtin_inff();

  for (;;) {
#pragma unroll
    for (int p = 0; p < P; p++) {
      if (!slot[p].valid) goto done;
      // The operands are read anew for every tile: kept in registers, as the compiler would, they leave
      // room for one wave a SIMD (5000 documents of 180 tokens, d = 128: 300 query tokens 117 us so,
      // 46 read anew; 500 tokens, d = 256: 121 and 72). 64 blocks do not fit there anyway, and the
      // compiler's own choice is better (1024 tokens: 83 us, 133 read anew).
      int at = lane;
      if constexpr (QLDS && QB < 64) asm volatile("" : "+v"(at));
#pragma unroll
      for (int block = 0; block < QB * SUB; block++) {
        const int qb = block / SUB, sub = block % SUB;
        f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KS; c++) {
          if constexpr (QLDS) {
            const int i = qb * KS + c;
            const u32x4_t v = *(const u32x4_t *)(lds + i * OPERAND + at * 16);
            const uint32_t s = (uint8_t)lds[QB * KS * OPERAND + i * WAVE + at];
            acc = mfma_mx4(buf[p][c], sc[p][c], v, s, acc);
          } else {
            acc = mfma_mx4(buf[p][c], sc[p][c], qreg[qb][c * SUB + sub], qs[qb][c * SUB + sub], acc);
          }
        }
        m[qb] = __builtin_fmaxf(__builtin_fmaxf(m[qb], acc[0]), acc[1]);
        m[qb] = __builtin_fmaxf(__builtin_fmaxf(m[qb], acc[2]), acc[3]);
      }
      if (slot[p].doc_end) {
        float s = 0.f;
#pragma unroll
        for (int qb = 0; qb < QB; qb++) {
          const float v = max_row_groups(m[qb]);
          if (qb * 16 + r16 < q_len) s += v;
          m[qb] = -__builtin_inff();
        }
        s = sum_row16(s);
        if (slot[p].empty) s = -__builtin_inff();
        if (lane == 0) a.doc.out[slot[p].doc] = s;
      }
      issue(buf[p], sc[p], slot[p]);
    }
  }
done:
  return;
}

}  // namespace maxsim
