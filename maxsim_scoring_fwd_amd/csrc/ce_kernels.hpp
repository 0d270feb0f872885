// Softmax cross entropy of a linear layer over a vocabulary, without its logits (include/maxsim.h,
// maxsim_linear_cross_entropy). Rows that have a label are gathered first, so that the others cost
// nothing and what they hold is never used; their number stays on the device.
//   forward:  logits tile by tile on the matrix cores (z = scale * <w_v, h_i>, transposed, so that a
//             lane's registers hold one row's logits); a tile leaves its largest logit and its sum
//             of exponentials for every row; ce_join_kernel joins those.
//   backward: piece after piece of the vocabulary: the tile again, P = (exp(z - lse) - [label]) *
//             grad * scale, rounded to the storage type, into a workspace that holds one piece, then
//             dw = P^T h of the piece and dh += P w over it.
// Sums are 32 bits wide, every one has one owner and a fixed order. P is rounded because the matrix
// cores take 16-bit operands, after a scaling (ce_up) that fits fp16's short range and leaves a mean's
// gradients exact. Where they differ from row to row they are rounded as well, half a step of 16 bits
// each at most: relative errors of dh and dw against 64 bits (2048 rows, 8000 x 256 in bf16) 0.00168 with
// a mean's, 0.00235 with gradients uniform in [0, 1 / n], and 0.00166 from rounding dh and dw alone.
// The matrix cores bound the training step and the bytes of w the few rows of a query. Measured (one
// MI355X): 8192 rows, 30522 entries, d = 768 in bf16: gathering 11 us (twice), logits and their
// sums 374 to 390 (1.03 to 0.99 PFLOP/s; a library product of the shape takes 410 and writes the
// logits), join 8.5, P 389 to 412, both products 656 to 675 (1.15; the library 419 + 573), dh's join
// 19; the clock falls to 1.6 to 1.8 GHz meanwhile, and the matrix cores are busy half of the cycles
// (54, 51 and 65 in 100). 32 rows: 12 us and 4.4 for the join, of which 9.3 are w's 47 MB.
#pragma once

#include "tile_gemm.hpp"

namespace maxsim {

// Tiles: 128 registers of sums a lane, and a ring of three steps in 72 KB, so that two workgroups fit a
// CU and one multiplies while the other one waits or goes on with its logits. Tiles of 128 x 128
// read a third more (logits of 8192 x 30522 x 768: 424 us for 395, the panels' share included).
constexpr int CE_BM = 128, CE_BN = 256;   // vocabulary x rows of a tile of logits
constexpr int CE_PM = 256, CE_PN = 128;   // columns x vocabulary (dw) or rows (dh) of a product's
// Where there are no more rows than that, or few tiles (100 rows, 100000 x 896 in fp16: forward 48 us and backward
// 169, in tiles of 256 rows 62 and 187; 78 rows, 25314 x 712 in fp32 70 and 168 for 107 and 203).
constexpr int CE_HALF_BN = 128;
constexpr int CE_FEW = 32;                // most rows of the kernel for few rows: one tile's
constexpr int CE_GATHER = 16;             // rows of a workgroup of the gathering
constexpr int CE_COUNT = 1024;            // rows of a workgroup of the counting
// Up to so many rows the gathering counts the labels before its own by itself: at most 64 KB of them
// from L2, which hides behind the rows' copies, and a launch of some 5 us less.
constexpr int CE_DIRECT = 8192;

struct CeArgs {
  const char *h, *w;
  const int64_t *labels;
  const float *grad;      // backward: of the losses
  int64_t n, vocab;
  int d, row_bytes;
  float scale;
  float *loss, *lse;      // forward: written; backward: lse is read
  char *dh, *dw;
  // workspace
  int32_t *counted;       // [1]: rows that have a label
  int32_t *counts;        // [blocks of CE_COUNT rows]
  float *most;            // [the same]: the largest absolute gradient
  int4 *info;             // [n]: of gathered row i (CeRow)
  char *hc;               // gathered rows in panels of 64 bytes, n rows each, zeros past d
  float2 *part;           // [tiles of the vocabulary][n]: largest product, and sum (CeSum)
  float *picked;          // [n]: the label's product
  char *p;                // P in panels of 64 bytes, whole tiles of rows each
  float *dhp, *dwp;       // tiles of dh and, where they go in parts, of dw, in the kernels' register layout
  int32_t *queue;         // [8]: units of the products that are taken
  int64_t p_elements;     // that p has room for
  int64_t slots, w_slots; // tiles that dhp and dwp have room for
  int64_t piece;          // backward: number of this piece
};

// Whether the forward takes the kernel for few rows: two launches for three, and as many steps under
// way as LDS holds (32 rows, 30522 x 768 in bf16: 15.6 us for 22.4; 64 rows would take two rounds
// of its tiles, 27 us, and take 22 in tiles of 128).
inline bool ce_few(const CeArgs &a) { return a.n <= CE_FEW; }

// A gathered row: its label, its place among all rows, and for the backward its lse (16-bit types: in
// units of log 2) and its gradient times scale.
struct CeRow {
  int label, row;
  float lse, grad;
};

// The pieces of the vocabulary for m rows: as many whole tiles as P's room takes, of equal size.
struct CePieces {
  int64_t cols, n, rows;
  __device__ __host__ __forceinline__ CePieces(int64_t m, int64_t vocab, int64_t p_elements) {
    rows = blocks_of(m < 1 ? 1 : m, CE_BN) * CE_BN;
    const int64_t tiles = blocks_of(vocab, CE_BM);
    int64_t most = p_elements / (rows * CE_BM);
    most = most < 1 ? 1 : most;
    n = blocks_of(tiles, most);
    cols = blocks_of(tiles, n) * CE_BM;
    n = blocks_of(vocab, cols);
  }
};

// The products of one piece: tiles of dw, and of dh, whose sums over the piece go in several parts
// where a tile is more than a workgroup's share of it all, so that all workgroups end about together.
// dh's parts are a share at most, of 8 steps and more. Shorter ones, of a third, cost more to join
// than they even out, since the longer units go first and a workgroup that is left alone on its CU
// runs faster (backward of 3001 rows, 50021 x 512 in fp16: 559 us in thirds, 548; 2048 rows, 30522 x
// 768 in bf16: 321 and 306); fp32's products leave no such slack: half a share (2000 rows, 20000 x
// 512: 1114 us in shares, 986 in halves). dw's tiles are few where the rows are many and short, and
// need a launch more to be joined: parts of half a share, of 16 steps and more (whole and in parts:
// 32768 rows, 30522 x 256 in bf16 3135 and 2130 us; 16384 rows, 10000 x 384 in fp16 555 and 547, in
// shares 588; 8192 rows, 500 x 512 164 and 66).
constexpr int CE_LANES = 512;  // workgroups at once: two on each of 256 CUs
constexpr int CE_H_LEAST = 8, CE_W_LEAST = 16;  // steps of a part
struct CeUnits {
  uint32_t w_across, w_down, h_across, h_down;
  uint32_t w_splits, h_splits;  // parts along the rows, along the piece
  __device__ __host__ __forceinline__ CeUnits(const CeArgs &a, int64_t m, const CePieces &p, int eb) {
    w_across = h_across = (uint32_t)blocks_of(a.d, CE_PM);
    w_down = (uint32_t)blocks_of(p.cols, CE_PN);
    h_down = (uint32_t)blocks_of(m, CE_PN);
    const int64_t w = (int64_t)w_across * w_down, h = (int64_t)h_across * h_down;
    const int64_t w_steps = blocks_of(m * eb, 64), h_steps = p.cols * eb / 64;
    const int64_t all = (a.dw ? w * w_steps : 0) + (a.dh ? h * h_steps : 0);
    // powers of two: the parts are dealt to 8 XCDs in order, and one that has parts of two kinds
    // reads the columns of both (8192 rows, 30522 x 768: 729 us in 3 parts, 663 in 4, 710 in 6)
    auto parts = [&](int64_t tiles, int64_t steps, int64_t slots, int least, int fine) {
      uint32_t n = 1;
      if (all >= steps * CE_LANES) return n;  // a tile is within a share
      while (n * all < steps * CE_LANES * fine && 2 * n * tiles <= slots && 2 * least * n <= steps) n *= 2;
      return n;
    };
    w_splits = parts(w, w_steps, a.w_slots, CE_W_LEAST, 2);
    h_splits = parts(h, h_steps, a.slots, CE_H_LEAST, eb == 4 ? 2 : 1);
  }
};

// What P is multiplied by before it is rounded. Its entries at the labels are the gradients (times p -
// 1, which is -1 but for well known labels), and those of a mean are all alike: divided by the
// mantissa of one of them they are powers of two, and rounding does not move them all by the same
// amount. fp16: that of the largest, which becomes 2^14; bf16: that of the first row. Where the
// gradients are not alike it fits that row only, and the others are rounded as they come.
template <int DT> __device__ __forceinline__ float ce_up(const CeArgs &a) {
  if constexpr (DT == DT_FP32) return 1.0f;
  float most = 0.0f;
  if constexpr (DT == DT_BF16) {
    most = __builtin_bit_cast(CeRow, a.info[0]).grad;
  } else {
    const int64_t blocks = blocks_of(a.n, CE_COUNT);
    for (int64_t i = threadIdx.x & 63; i < blocks; i += 64) most = __builtin_fmaxf(most, a.most[i]);
    for (int o = 32; o > 0; o >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, o, 64));
    most *= a.scale;
  }
  const uint32_t bits = __float_as_uint(most), exponent = (bits >> 23) & 255;
  if (exponent == 0 || exponent == 255) return 1.0f;  // zero, or not a number
  const float up = __builtin_amdgcn_rcpf(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
  if constexpr (DT == DT_BF16) return up;
  int e = 14 - (int)exponent + 127;
  e = e > 120 ? 120 : (e < -120 ? -120 : e);
  return up * __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ bool ce_counts(const CeArgs &a, int64_t label) { return label >= 0 && label < a.vocab; }

// Sum over a workgroup of 256, in every thread.
__device__ __forceinline__ int ce_block_sum(int v) {
  __shared__ int part[4];
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return part[0] + part[1] + part[2] + part[3];
}

// Rows with a label, and the largest gradient among them, of every CE_COUNT rows.
template <int DT> __global__ void __launch_bounds__(GEMM_THREADS) ce_count_kernel(CeArgs a) {
  __shared__ float part[4];
  int c = 0;
  float most = 0.0f;
  for (int i = threadIdx.x; i < CE_COUNT; i += GEMM_THREADS) {
    const int64_t r = (int64_t)blockIdx.x * CE_COUNT + i;
    if (r < a.n && ce_counts(a, a.labels[r])) {
      c++;
      if (a.grad) most = __builtin_fmaxf(most, __builtin_fabsf(a.grad[r]));
    }
  }
  c = ce_block_sum(c);
  for (int o = 32; o > 0; o >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, o, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    a.counts[blockIdx.x] = c;
    a.most[blockIdx.x] = __builtin_fmaxf(__builtin_fmaxf(part[0], part[1]), __builtin_fmaxf(part[2], part[3]));
  }
}

// Copies the rows that have a label to their places, in order; the others get their results here.
template <int DT> __global__ void __launch_bounds__(GEMM_THREADS) ce_gather_kernel(CeArgs a) {
  __shared__ int place[CE_GATHER];
  const int64_t r0 = (int64_t)blockIdx.x * CE_GATHER, block = a.n > CE_DIRECT ? r0 / CE_COUNT : 0;
  int before = 0;
  for (int64_t i = threadIdx.x; i < block; i += GEMM_THREADS) before += a.counts[i];
#pragma unroll 4
  for (int64_t r = block * CE_COUNT + threadIdx.x; r < r0; r += GEMM_THREADS)
    before += ce_counts(a, a.labels[r]) ? 1 : 0;
  before = ce_block_sum(before);
  if (threadIdx.x < 64) {
    const int64_t r = r0 + threadIdx.x;
    const bool in = threadIdx.x < CE_GATHER && r < a.n;
    const int64_t label = in ? a.labels[r] : -1;
    const bool counts = in && ce_counts(a, label);
    const uint64_t all = __ballot(counts);
    const int at = before + __popcll(all & ((1ull << threadIdx.x) - 1));
    if (threadIdx.x < CE_GATHER) place[threadIdx.x] = counts ? at : -1;
    if (counts) {
      CeRow row{(int)label, (int)r, 0.0f, 0.0f};
      if (a.grad) {
        row.lse = DT == DT_FP32 ? a.lse[r] : a.lse[r] * LOG2E;
        row.grad = a.grad[r] * a.scale;
      }
      a.info[at] = __builtin_bit_cast(int4, row);
    } else if (in && a.loss) {
      a.loss[r] = 0.0f;
      a.lse[r] = -__builtin_inff();
    }
    if (threadIdx.x == 0 && r0 + CE_GATHER >= a.n) *a.counted = before + __popcll(all);
  }
  __syncthreads();
  // four panels at a time: 16 rows x 256 bytes, so that both sides move whole lines
  constexpr int BYTES = GEMM_THREADS / CE_GATHER * 16;
  const int i = threadIdx.x / (BYTES / 16), c0 = threadIdx.x % (BYTES / 16) * 16;
  if (r0 + i >= a.n) return;
  const int at = place[i];
  const char *from = a.h + (r0 + i) * a.row_bytes;
  const int padded = (a.row_bytes + PANEL - 1) / PANEL * PANEL;
  if (at >= 0) {
    char *to = a.hc + (int64_t)at * PANEL;
    constexpr int AHEAD = 4;
    for (int c = c0; c < padded; c += AHEAD * BYTES) {
      u32x4_t x[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; j++) {
        const int k = c + j * BYTES;
        x[j] = load16(from + (k < a.row_bytes ? k : a.row_bytes - 16));
      }
#pragma unroll
      for (int j = 0; j < AHEAD; j++) {
        const int k = c + j * BYTES;
        if (k >= a.row_bytes) x[j] = u32x4_t{0, 0, 0, 0};
        if (k < padded) *(u32x4_t *)(to + (int64_t)(k / PANEL) * a.n * PANEL + k % PANEL) = x[j];
      }
    }
  } else if (a.dh) {
    char *to = a.dh + (r0 + i) * a.row_bytes;
    for (int c = c0; c < a.row_bytes; c += BYTES) *(u32x4_t *)(to + c) = u32x4_t{0, 0, 0, 0};
  }
}

// A block of 32 x 32 of P, each lane's row times f, rounded, to a panel's 32 rows (fp32: two panels').
template <int DT> __device__ __forceinline__ void store_block(char *lds, const f32x16_t &x, float f, char *out, int64_t panel) {
  using L = RowLayout<DT, 32>;
  using T = typename AttnElem<DT>::type;
  typedef T v4 __attribute__((ext_vector_type(4)));
  const int l = threadIdx.x & 63, row = l & 31, h = l >> 5;
#pragma unroll
  for (int g = 0; g < 4; g++) {
    v4 y;
#pragma unroll
    for (int e = 0; e < 4; e++) y[e] = (T)(x[4 * g + e] * f);
    const int at = (8 * g + 4 * h) * L::eb;
    *(v4 *)(lds + row * L::bytes + ((at & ~15) ^ L::f(row)) + (at & 15)) = y;
  }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < (32 * L::chunks) / 64; i++) {
    const int p = i * 64 + l, r = p / L::chunks, c = p % L::chunks * 16;
    *(u32x4_t *)(out + c / PANEL * panel + r * PANEL + c % PANEL) = *(const u32x4_t *)(lds + r * L::bytes + (c ^ L::f(r)));
  }
  wave_lds_sync();
}

// Tile number i of `across` tiles along one side times `down` along the other, so that tiles beside
// each other in the order share both operands in an XCD's L2: 8 tiles down at a time.
__device__ __forceinline__ void ce_tile(uint32_t i, uint32_t across, uint32_t down, uint32_t &v, uint32_t &r) {
  const uint32_t group = i / (8 * across), in = i - group * 8 * across;
  const uint32_t wide = down - group * 8 < 8 ? down - group * 8 : 8;
  v = in / wide;
  r = group * 8 + in - v * wide;
}
// The same with an eighth of the vocabulary for each XCD: the vocabulary's rows are then read by one
// XCD alone, and 8 tiles of rows stay in its L2 while it goes through its eighth (8192 x 30522 x 768:
// logits 390 us for 395 with one order over all XCDs, P 404 for 418).
__device__ __forceinline__ void ce_tile_of_xcd(uint32_t i, uint32_t across, uint32_t down, uint32_t &v, uint32_t &r) {
  const uint32_t eighth = (across + 7) / 8, x = i / (eighth * down), v0 = x * eighth;
  ce_tile(i - x * eighth * down, across - v0 < eighth ? across - v0 : eighth, down, v, r);
  v += v0;
}

// Logits of a tile: acc[n][m] of lane l is row 32 n + l % 32 and vocabulary entry 32 m +
// acc_row(reg) + 4 (l / 32) of the wave's part, without scale. The rows' CeRow come to LDS with the
// first loads. A workgroup takes tiles one after the other; the first loads of the next one are
// under way while it goes on with the logits.
template <int DT, int BM, int BN, int WM, int STAGES> struct CeLogits {
  using G = TileGemm<DT, BM, BN, WM, SIDE_ROWS, SIDE_ROWS_P, STAGES>;
  static constexpr int ring = G::lds, info = (BN < 64 ? 64 : BN) * 16, lds = ring + 2 * info;
  static constexpr int scratch = (STAGES - 1) * G::stage;  // of the ring: free between tiles
  G g;
  uint32_t across, down, total, next;  // tiles; number of the next one
  int64_t v0, r0;                      // of the tile at hand
  int64_t v1, r1;                      // of the next
  int m, which;                        // place of the tile's CeRows

  __device__ __forceinline__ void start(const CeArgs &a, char *lds, int rows, int64_t vocab0, int64_t cols) {
    m = rows;
    across = (uint32_t)blocks_of(cols, BM);
    down = (uint32_t)blocks_of(m, BN);
    total = across * down;
    next = blockIdx.x;
    which = 1;
    begin(a, lds, vocab0);
  }
  __device__ __forceinline__ void begin(const CeArgs &a, char *lds, int64_t vocab0) {
    which ^= 1;
    if (next >= total) return;
    uint32_t tv, tr;
    ce_tile_of_xcd(xcd_order(next, total), across, down, tv, tr);
    v1 = vocab0 + (int64_t)tv * BM;
    r1 = (int64_t)tr * BN;
    const int exist = m - (int)r1 < BN ? m - (int)r1 : BN;
    const int wave = uniform((int)threadIdx.x >> 6);
    if (wave * 64 < BN) {
      const int r = (int)threadIdx.x < exist ? (int)threadIdx.x : exist - 1;
      const int to = lds_address(lds + ring + which * info) + wave * 1024;  // 64 rows a wave
      asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                   :
                   : "{m0}"(uniform(to)), "v"((uint32_t)r * 16u),
                     "s"(uniform((int64_t)(uintptr_t)(a.info + r1))));
    }
    const int64_t vs = a.vocab - v1;
    g.a.start(a.w + v1 * a.row_bytes, a.row_bytes, vs < BM ? (int)vs : BM);
    g.b.start(a.hc + r1 * PANEL, a.n * PANEL, exist);
    const int steps = (a.row_bytes + 63) / 64;
    g.begin(lds, steps, a.row_bytes - (steps - 1) * 64, 64);  // the panels hold zeros past d
  }
  // The next tile's logits; false after the last. row(i): CeRow i of the tile.
  __device__ __forceinline__ bool tile(const CeArgs &a, char *lds, int64_t vocab0) {
    if (next >= total) return false;
    v0 = v1;
    r0 = r1;
    g.clear();
    g.finish(lds);
    next += gridDim.x;
    begin(a, lds, vocab0);
    return true;
  }
  __device__ __forceinline__ CeRow row(const char *lds, int i) const {
    return *(const CeRow *)(lds + ring + (which ^ 1) * info + i * 16);
  }
};

// The exponentials of a row over a part of the vocabulary: the largest product x.most, unscaled, and the
// sum of 2^(x f - round(most f)), f = scale / log 2 rounded. What the rounding of most f takes away the
// exponentials hold, so that nothing of the size of the logits is rounded before the end (finish).
struct CeSum {
  float most, sum;
  __device__ __forceinline__ void add(const CeSum &o, float f) {
#pragma clang fp contract(off)  // most f is to be rounded before anything is taken from it
    const float m = __builtin_fmaxf(most, o.most), from = m == -__builtin_inff() ? 0.0f : m * f;
    sum = sum * __builtin_amdgcn_exp2f(most * f - from) + o.sum * __builtin_amdgcn_exp2f(o.most * f - from);
    most = m;
  }
  // lse and loss, each rounded once from 64 bits: the logarithm is of what is left beside the largest
  // logit, and the logit of a product is exact. (In 32 bits and units of log 2, rounded at each step,
  // losses of 1.3 to 29 from logits of 193 to 413 were off by up to 2.9e-5, here 5e-7.)
  __device__ __forceinline__ void finish(float scale, float f, float picked, float &lse, float &loss) const {
#pragma clang fp contract(off)
    // sum = m 2^e with m in [3/4, 3/2): the logarithm of a sum near 1 keeps its digits
    float m = __builtin_amdgcn_frexp_mantf(sum);
    int e = __builtin_amdgcn_frexp_expf(sum);
    if (m < 0.75f) {
      m *= 2.0f;
      e--;
    }
    const double product = (double)most, beside = (double)(most * f) - product * (double)f + e + (double)__builtin_log2f(m);
    constexpr double LN2_64 = 0.693147180559945309417;
    lse = (float)(scale * product + beside * LN2_64);
    loss = (float)(scale * (product - (double)picked) + beside * LN2_64);
  }
};

// What a tile of logits leaves: for every row its CeSum over the tile, and the label's product where the
// tile holds it. label(i): the label of row i of the tile;
// red: scratch of WM * BN pairs. The workgroup is together again afterwards.
template <typename G, int BM, int BN, int WM, typename Label>
__device__ __forceinline__ void ce_tile_sums(const CeArgs &a, G &g, int64_t v0, int64_t r0, int m, float2 *red, Label label) {
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  const int h4 = 4 * (lane >> 5);
  const float f = a.scale * LOG2E;
  // this wave's part of the vocabulary
  const int64_t first = v0 + wm * (BM / WM);
  const int exist = a.vocab - first < BM / WM ? (int)(a.vocab - first) : BM / WM;
#pragma unroll
  for (int n = 0; n < G::TN; n++) {
    f32x16_t(&x)[G::TM] = g.acc[n];
    const int i = (wn * G::TN + n) * 32 + (lane & 31);
    const int64_t r = r0 + i;
    const int at = r < m ? label(i) - (int)first : -1;
    if (__any(at >= 0 && at < BM / WM)) {
      float picked = 0.0f;
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int e = 0; e < 16; e++)
          if (k * 32 + acc_row(e) == at - h4) picked = x[k][e];
      if (at >= 0 && at < BM / WM && (at & 4) == h4) a.picked[r] = picked;
    }
    if (exist < BM / WM) {
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int e = 0; e < 16; e++)
          if (k * 32 + acc_row(e) + h4 >= exist) x[k][e] = -__builtin_inff();
    }
    float most = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < G::TM; k++)
#pragma unroll
      for (int e = 0; e < 16; e++) most = __builtin_fmaxf(most, x[k][e]);
    most = half_max(most);  // scale is positive
    const float from = most == -__builtin_inff() ? 0.0f : most * f;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < G::TM; k++)
#pragma unroll
      for (int e = 0; e < 16; e++) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(x[k][e], f, -from));
    sum = half_sum(sum);
    if (lane < 32) red[wm * BN + i] = make_float2(most, sum);
  }
  __syncthreads();
  if (threadIdx.x < BN && r0 + threadIdx.x < m) {
    CeSum s = __builtin_bit_cast(CeSum, red[threadIdx.x]);
#pragma unroll
    for (int k = 1; k < WM; k++) s.add(__builtin_bit_cast(CeSum, red[k * BN + threadIdx.x]), f);
    a.part[v0 / BM * a.n + r0 + threadIdx.x] = __builtin_bit_cast(float2, s);
  }
}

template <int DT, int BM, int BN, int WM, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_forward_kernel(CeArgs a) {
  using Z = CeLogits<DT, BM, BN, WM, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  Z z;
  z.start(a, lds, uniform(*a.counted), 0, a.vocab);
  while (z.tile(a, lds, 0))
    ce_tile_sums<typename Z::G, BM, BN, WM>(a, z.g, z.v0, z.r0, z.m, (float2 *)(lds + Z::scratch),
                                            [&](int i) { return z.row(lds, i).label; });
}

// Few rows (up to 32): every workgroup finds the ones with a label by itself and
// reads them where they are, which saves the launch that gathers them; one workgroup a tile. The
// vocabulary's bytes bound it: as many steps under way as LDS holds.
template <int DT, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS) ce_few_kernel(CeArgs a) {
  constexpr int BM = CE_BM, BN = CE_FEW, WM = 4;
  using G = TileGemm<DT, BM, BN, WM, SIDE_ROWS, SIDE_ROWS, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  CeRow *row = (CeRow *)(lds + G::lds);  // of the rows that count
  int m;
  {
    const int r = threadIdx.x & 63;  // in every wave, for m
    const int64_t label = r < a.n ? a.labels[r] : -1;
    const bool counts = r < a.n && ce_counts(a, label);
    const uint64_t all = __ballot(counts);
    m = __popcll(all);
    const CeRow mine{(int)label, r, 0.0f, 0.0f};
    const int at = __popcll(all & ((1ull << r) - 1));
    if (threadIdx.x < 64) {
      if (counts) row[at] = mine;
      if (blockIdx.x == 0) {  // for the joining
        if (counts) {
          a.info[at] = __builtin_bit_cast(int4, mine);
        } else if (r < a.n) {
          a.loss[r] = 0.0f;
          a.lse[r] = -__builtin_inff();
        }
        if (r == 0) *a.counted = m;
      }
    }
  }
  if (m == 0) return;
  const int64_t v0 = (int64_t)blockIdx.x * BM;
  __syncthreads();
  G g;
  const int64_t vs = a.vocab - v0;
  g.a.start(a.w + v0 * a.row_bytes, a.row_bytes, vs < BM ? (int)vs : BM);
  g.b.start(a.h, a.row_bytes, m, [&](int i) { return row[i].row; });
  g.clear();
  const int steps = (a.row_bytes + 63) / 64, last = a.row_bytes - (steps - 1) * 64;
  g.begin(lds, steps, last, last);
  g.template finish<true>(lds);
  ce_tile_sums<G, BM, BN, WM>(a, g, v0, 0, m, (float2 *)lds, [&](int i) { return row[i].label; });
}

// lse and loss of a row from its tiles' parts: 8 rows a workgroup, 32 threads to each.
template <int DT> __global__ void __launch_bounds__(GEMM_THREADS) ce_join_kernel(CeArgs a, int tiles) {
  const int m = *a.counted;
  const int row = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int64_t r = (int64_t)blockIdx.x * 8 + row;
  if ((int64_t)blockIdx.x * 8 >= m) return;
  __shared__ CeSum part[32][8];
  CeSum s{-__builtin_inff(), 0.0f};
  const float f = a.scale * LOG2E;
  if (r < m) {
#pragma unroll 4
    for (int t = slice; t < tiles; t += 32) s.add(__builtin_bit_cast(CeSum, a.part[(int64_t)t * a.n + r]), f);
  }
  part[slice][row] = s;
  __syncthreads();
  for (int o = 16; o > 0; o >>= 1) {
    if (slice < o) part[slice][row].add(part[slice + o][row], f);
    __syncthreads();
  }
  if (slice == 0 && r < m) {
    const int64_t to = __builtin_bit_cast(CeRow, a.info[r]).row;
    part[0][row].finish(a.scale, f, a.picked[r], a.lse[to], a.loss[to]);
  }
}

// dh, or a piece's dw, from its parts, rounded once, to the rows' own places, by the whole launch. The
// parts' bytes bound it; where there are few tiles of many parts, their loads' waits do: 8 under way
// (130 rows, 100000 x 128, 256 parts: the backward 158 us with one block a workgroup and a part at
// a time, 88 so).
template <int DT, bool DW>
__device__ __forceinline__ void ce_join_parts(const CeArgs &a, int m, const CePieces &pieces, int64_t piece) {
  constexpr int BM = CE_PM, BN = CE_PN, WM = 2;
  using G = TileGemm<DT, BM, BN, WM, SIDE_COLS, SIDE_ROWS_P, 3>;
  using T = typename AttnElem<DT>::type;
  typedef T v4 __attribute__((ext_vector_type(4)));
  const CeUnits units(a, m, pieces, Elem<DT>::bytes);
  const int64_t piece0 = piece * pieces.cols;
  if (DW && units.w_splits == 1) return;
  const int64_t rows = DW ? (a.vocab - piece0 < pieces.cols ? a.vocab - piece0 : pieces.cols) : m;
  const uint32_t across = DW ? units.w_across : units.h_across, splits = DW ? units.w_splits : units.h_splits;
  const uint32_t down = (uint32_t)blocks_of(rows, BN), tiles = across * down;
  const float back = 1.0f / ce_up<DT>(a);
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  // A quarter of a block of 32 x 32 of a tile for each wave and round, so that few tiles of many parts
  // spread over the chip; the quarters of a block on one XCD, whose L2 joins what they write.
  const uint32_t total = tiles * G::TN * G::TM * 4;
  static_assert(G::TN * G::TM % 8 == 0, "whole rounds of the XCDs");
  const int64_t part = (int64_t)tiles * (BM * BN / 4);
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    const uint32_t block = i / 32 * 8 + i % 8, q = i / 8 % 4;
    const uint32_t tile = block / (G::TN * G::TM), nk = block - tile * (G::TN * G::TM);
    const int n = nk / G::TM, k = nk - n * G::TM;
    uint32_t tc, tr;
    ce_tile(tile, across, down, tc, tr);
    const int64_t r = (int64_t)tr * BN + (wn * G::TN + n) * 32 + (lane & 31);
    const int c = (int)tc * BM + (wm * G::TM + k) * 32 + 4 * (lane >> 5) + 8 * q;
    const f32x4_t *p = (const f32x4_t *)(DW ? a.dwp : a.dhp) + (int64_t)tile * (BM * BN / 4) +
                       (nk * 4 + q) * GEMM_THREADS + threadIdx.x;
    constexpr int AHEAD = 8;
    f32x4_t x = {};
    uint32_t s = 0;
    for (; s + AHEAD <= splits; s += AHEAD) {
      f32x4_t y[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; j++) y[j] = p[(s + j) * part];
#pragma unroll
      for (int j = 0; j < AHEAD; j++) x += y[j];
    }
    for (; s < splits; s++) x += p[s * part];
    if (r >= rows || c >= a.d) continue;  // d is a multiple of 4 entries
    T *to = (T *)(DW ? a.dw + (piece0 + r) * a.row_bytes
                     : a.dh + (int64_t)__builtin_bit_cast(CeRow, a.info[r]).row * a.row_bytes);
    v4 o;
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = (T)(x[e] * back);
    *(v4 *)(to + c) = o;
  }
}

// P of one piece: [rows, whole tiles of them][cols], zeros past the rows and, in whole tiles, past
// the vocabulary.
// Where dw goes in parts, those of the piece before are joined first: a launch for it would also cost
// the pieces that are not there (3001 of 20011 rows count: 18 us of 746).
template <int DT, int BM, int BN, int WM, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_p_kernel(CeArgs a) {
  using Z = CeLogits<DT, BM, BN, WM, STAGES>;
  using G = typename Z::G;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if (blockIdx.x == 0 && threadIdx.x < 8) a.queue[threadIdx.x] = 0;
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  if (a.piece >= pieces.n) return;
  if (a.piece > 0 && a.dw && a.w_slots) ce_join_parts<DT, true>(a, m, pieces, a.piece - 1);
  const int64_t piece0 = a.piece * pieces.cols;
  const int64_t cols = a.vocab - piece0 < pieces.cols ? a.vocab - piece0 : pieces.cols;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  const int h4 = 4 * (lane >> 5);
  const float up = ce_up<DT>(a), f = a.scale * LOG2E;
  // a block of 32 x 32 leaves through LDS: a panel of 32 rows, which is one piece of memory
  constexpr int eb = Elem<DT>::bytes, part = BM / WM;
  static_assert(4 * 32 * 32 * eb <= G::stage, "within the place that is free");
  char *mine = lds + Z::scratch + wave * (32 * 32 * eb);
  const int64_t panel = pieces.rows * PANEL;
  Z z;
  z.start(a, lds, m, piece0, cols);
  while (z.tile(a, lds, piece0)) {
    const int64_t first = z.v0 + wm * part;
    const int exist = a.vocab - first < part ? (int)(a.vocab - first) : part;  // or negative
#pragma unroll
    for (int n = 0; n < G::TN; n++) {
      f32x16_t(&x)[G::TM] = z.g.acc[n];
      const int i = (wn * G::TN + n) * 32 + (lane & 31);
      const CeRow row = z.row(lds, i);  // past the last row: the last one's, with a gradient of 0
      const bool real = z.r0 + i < z.m;
      const float by = real ? row.grad * up : 0.0f;
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int e = 0; e < 16; e++)
          // fp32: the difference before the change of units, so that nothing is rounded at the size of the
          // logits (of 645 to 1745: dw off by 1.6e-5 of its size otherwise, 4e-8 so); 16 bits are rounded by
          // far more
          x[k][e] = DT == DT_FP32 ? __builtin_amdgcn_exp2f(__builtin_fmaf(x[k][e], a.scale, -row.lse) * LOG2E)
                                  : __builtin_amdgcn_exp2f(__builtin_fmaf(x[k][e], f, -row.lse));
      const int at = real ? row.label - (int)first : -1;
      if (__any(at >= 0 && at < part)) {
#pragma unroll
        for (int k = 0; k < G::TM; k++)
#pragma unroll
          for (int e = 0; e < 16; e++)
            if (k * 32 + acc_row(e) == at - h4) x[k][e] -= 1.0f;
      }
      if (exist < part) {
#pragma unroll
        for (int k = 0; k < G::TM; k++)
#pragma unroll
          for (int e = 0; e < 16; e++)
            if (k * 32 + acc_row(e) + h4 >= exist) x[k][e] = 0.0f;
      }
      char *out = a.p + (first - piece0) * eb / PANEL * panel + (z.r0 + (wn * G::TN + n) * 32) * PANEL;
#pragma unroll
      for (int k = 0; k < G::TM; k++) store_block<DT>(mine, x[k], by, out + k * 32 * eb / PANEL * panel, panel);
    }
  }
}

// A tile in the register layout, added to what is there or not.
template <typename G> __device__ __forceinline__ void ce_store_tile(const G &g, f32x4_t *out, bool add) {
#pragma unroll
  for (int n = 0; n < G::TN; n++)
#pragma unroll
    for (int k = 0; k < G::TM; k++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        f32x4_t y = {g.acc[n][k][4 * q], g.acc[n][k][4 * q + 1], g.acc[n][k][4 * q + 2], g.acc[n][k][4 * q + 3]};
        f32x4_t *at = out + ((n * G::TM + k) * 4 + q) * GEMM_THREADS + threadIdx.x;
        if (add) y += *at;
        *at = y;
      }
}

// The products of one piece: dw = P^T h over the gathered rows, tile by tile, in parts in the register
// layout or at once; and dh's sums over the piece, added to those of the pieces before, likewise. The units of each
// XCD's workgroups lie side by side, so that its L2 serves what they share; a workgroup takes the
// next one when it has ended one, the longer kind first. Who makes a unit does not change it.
template <int DT, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_products_kernel(CeArgs a) {
  constexpr int BM = CE_PM, BN = CE_PN, WM = 2;
  using GW = TileGemm<DT, BM, BN, WM, SIDE_COLS_P, SIDE_COLS_P, STAGES>;
  using GH = TileGemm<DT, BM, BN, WM, SIDE_COLS, SIDE_ROWS_P, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  __shared__ int taken;
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  if (a.piece >= pieces.n) return;
  const int64_t piece0 = a.piece * pieces.cols;
  const int64_t cols = a.vocab - piece0 < pieces.cols ? a.vocab - piece0 : pieces.cols;
  const CeUnits units(a, m, pieces, Elem<DT>::bytes);
  const uint32_t w_down = (uint32_t)blocks_of(cols, BN);
  const uint32_t w_tiles = units.w_across * w_down, h_tiles = units.h_across * units.h_down;
  const uint32_t w_units = a.dw ? w_tiles * units.w_splits : 0, h_units = a.dh ? h_tiles * units.h_splits : 0;
  const uint32_t x = blockIdx.x & 7;
  const uint32_t w_from = (uint64_t)w_units * x / 8, w_n = (uint64_t)w_units * (x + 1) / 8 - w_from;
  const uint32_t h_from = (uint64_t)h_units * x / 8, h_n = (uint64_t)h_units * (x + 1) / 8 - h_from;
  const bool h_first = cols * units.w_splits > (int64_t)m * units.h_splits;
  const uint32_t first_n = h_first ? h_n : w_n;
  const int wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  const float back = 1.0f / ce_up<DT>(a);
  constexpr int eb = Elem<DT>::bytes, part = BM / WM;
  const int64_t panel = pieces.rows * PANEL;
  for (;;) {
    __syncthreads();
    if (threadIdx.x == 0) taken = atomicAdd(a.queue + x, 1);
    __syncthreads();
    uint32_t unit = uniform(taken);
    if (unit >= w_n + h_n) break;
    const bool second = unit >= first_n;
    if (second) unit -= first_n;
    uint32_t tc, tr;
    if (second == h_first) {
      const uint32_t id = w_from + unit, split = id / w_tiles;
      ce_tile(id - split * w_tiles, units.w_across, w_down, tc, tr);
      const int c0 = (int)tc * BM;
      const int64_t v0 = (int64_t)tr * BN;
      const int steps = (int)blocks_of(m, GW::BK);
      const int from = (int)((int64_t)steps * split / units.w_splits);
      const int to = (int)((int64_t)steps * (split + 1) / units.w_splits);
      GW g;
      g.clear();
      if (to > from) {
        const int64_t k0 = (int64_t)from * GW::BK;
        g.a.start(a.hc + ((int64_t)(c0 * eb / PANEL) * a.n + k0) * PANEL, a.n * PANEL, a.row_bytes - c0 * eb);
        g.b.start(a.p + v0 * eb / PANEL * panel + k0 * PANEL, panel, BN * eb);
        // rows of P past the last are zeros, and whole tiles of rows are there
        const int left = m - (to - 1) * GW::BK;
        g.begin(lds, to - from, left < GW::BK ? left : GW::BK, GW::BK);
        g.finish(lds);
      }
      if (units.w_splits > 1) {
        ce_store_tile(g, (f32x4_t *)a.dwp + (int64_t)id * (BM * BN / 4), false);
        continue;
      }
      char *mine = lds + wave * (32 * part * eb);
      const int at = c0 + wm * part;
      const int row_bytes = (a.d - at < part ? a.d - at : part) * eb;
#pragma unroll
      for (int n = 0; n < GW::TN; n++) {
        const int64_t v = v0 + (wn * GW::TN + n) * 32, left = cols - v;
        if (row_bytes > 0 && left > 0)
          store_rows<DT, part, GW::TM>(mine, g.acc[n], back, a.dw + (piece0 + v) * a.row_bytes + (int64_t)at * eb,
                                       a.row_bytes, left < 32 ? (int)left : 32, row_bytes);
      }
    } else {
      const uint32_t id = h_from + unit, split = id / h_tiles;
      ce_tile(id - split * h_tiles, units.h_across, units.h_down, tc, tr);
      const int c0 = (int)tc * BM;
      const int64_t r0 = (int64_t)tr * BN;
      const int steps = (int)blocks_of(cols, GH::BK);
      const int from = (int)((int64_t)steps * split / units.h_splits);
      const int to = (int)((int64_t)steps * (split + 1) / units.h_splits);
      GH g;
      g.clear();
      if (to > from) {
        const int64_t k0 = (int64_t)from * GH::BK;
        g.a.start(a.w + (piece0 + k0) * a.row_bytes + (int64_t)c0 * eb, a.row_bytes, a.row_bytes - c0 * eb);
        g.b.start(a.p + k0 * eb / PANEL * panel + r0 * PANEL, panel, BN);
        // columns of P past the vocabulary are zeros
        const int64_t left = cols - (int64_t)(to - 1) * GH::BK;
        g.begin(lds, to - from, left < GH::BK ? (int)left : GH::BK, 64);
        g.finish(lds);
      }
      ce_store_tile(g, (f32x4_t *)a.dhp + (int64_t)id * (BM * BN / 4), a.piece > 0);
    }
  }
}

// dh, and the last piece's dw, from their parts.
template <int DT> __global__ void __launch_bounds__(GEMM_THREADS) ce_parts_kernel(CeArgs a) {
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  if (a.dw && a.w_slots) ce_join_parts<DT, true>(a, m, pieces, pieces.n - 1);
  if (a.dh) ce_join_parts<DT, false>(a, m, pieces, 0);
}

int ce_forward_bf16(const CeArgs &a, int cus, hipStream_t st);
int ce_forward_fp16(const CeArgs &a, int cus, hipStream_t st);
int ce_forward_fp32(const CeArgs &a, int cus, hipStream_t st);
int ce_backward_bf16(CeArgs &a, int64_t pieces, int cus, hipStream_t st);
int ce_backward_fp16(CeArgs &a, int64_t pieces, int cus, hipStream_t st);
int ce_backward_fp32(CeArgs &a, int64_t pieces, int cus, hipStream_t st);

}  // namespace maxsim
