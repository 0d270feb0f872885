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
// cores take 16-bit operands; in fp16, whose range is short, it is scaled by a power of two first,
// taken from the largest gradient of a row.
#pragma once

#include "tile_gemm.hpp"

namespace maxsim {

constexpr int CE_BM = 256, CE_BN = 128;              // vocabulary (or columns) x rows of a tile
constexpr int CE_SMALL_BM = 128, CE_SMALL_BN = 32;   // for few rows
constexpr int CE_GATHER = 32;                        // rows of a workgroup of the gathering
constexpr int CE_COUNT = 1024;                       // rows of a workgroup of the counting

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
  int32_t *row, *label;   // [n]: of gathered row i
  char *hc;               // [n][d]: gathered rows
  float2 *part;           // [tiles of the vocabulary][n]: largest logit (in units of log 2), sum
  float *picked;          // [n]: the label's logit, in units of log 2
  char *p;                // [rows][piece]: P
  float *dhp;             // tiles of dh in the kernels' register layout
  int64_t p_elements;     // that p has room for
  int64_t slots;          // tiles that dhp has room for
  int64_t piece;          // backward: number of this piece
};

// The pieces of the vocabulary for m rows: as many whole tiles as P's room takes, of equal size.
struct CePieces {
  int64_t cols, n;
  __device__ __host__ __forceinline__ CePieces(int64_t m, int64_t vocab, int64_t p_elements) {
    const int64_t rows = blocks_of(m < 1 ? 1 : m, CE_BN) * CE_BN;
    const int64_t tiles = blocks_of(vocab, CE_BM);
    int64_t most = p_elements / (rows * CE_BM);
    most = most < 1 ? 1 : most;
    n = blocks_of(tiles, most);
    cols = blocks_of(tiles, n) * CE_BM;
    n = blocks_of(vocab, cols);
  }
};

// How many parts dh's sums over a piece go in: as many as there is room for and steps enough.
__device__ __host__ __forceinline__ int64_t ce_splits(int64_t tiles, int64_t slots, int64_t cols, int bk) {
  const int64_t most = cols / (8 * bk);
  int64_t s = slots / (tiles < 1 ? 1 : tiles);
  s = s < most ? s : most;
  return s < 1 ? 1 : s;
}

// fp16: the power of two that P is scaled by.
template <int DT> __device__ __forceinline__ float ce_up(const CeArgs &a) {
  if constexpr (DT != DT_FP16) return 1.0f;
  float most = 0.0f;
  const int64_t blocks = blocks_of(a.n, CE_COUNT);
  for (int64_t i = threadIdx.x & 63; i < blocks; i += 64) most = __builtin_fmaxf(most, a.most[i]);
  for (int o = 32; o > 0; o >>= 1) most = __builtin_fmaxf(most, __shfl_xor(most, o, 64));
  most *= a.scale;
  if (!(most > 0.0f && most < __builtin_inff())) return 1.0f;
  int e = 14 - (int)((__float_as_uint(most) >> 23) & 255) + 127;
  e = e > 120 ? 120 : (e < -120 ? -120 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
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
  const int64_t r0 = (int64_t)blockIdx.x * CE_GATHER, block = r0 / CE_COUNT;
  int before = 0;
  for (int64_t i = threadIdx.x; i < block; i += GEMM_THREADS) before += a.counts[i];
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
      a.row[at] = (int32_t)r;
      a.label[at] = (int32_t)label;
    } else if (in && a.loss) {
      a.loss[r] = 0.0f;
      a.lse[r] = -__builtin_inff();
    }
    if (threadIdx.x == 0 && r0 + CE_GATHER >= a.n) *a.counted = before + __popcll(all);
  }
  __syncthreads();
  const int chunks = a.row_bytes / 16;
  for (int i = threadIdx.x >> 6; i < CE_GATHER && r0 + i < a.n; i += 4) {
    const int at = uniform(place[i]);
    const char *from = a.h + (r0 + i) * a.row_bytes;
    if (at >= 0) {
      char *to = a.hc + (int64_t)at * a.row_bytes;
      for (int c = threadIdx.x & 63; c < chunks; c += 64) *(u32x4_t *)(to + c * 16) = load16(from + c * 16);
    } else if (a.dh) {
      char *to = a.dh + (r0 + i) * a.row_bytes;
      for (int c = threadIdx.x & 63; c < chunks; c += 64) *(u32x4_t *)(to + c * 16) = u32x4_t{0, 0, 0, 0};
    }
  }
}

// Tile number i of `across` tiles of the vocabulary times `down` tiles of rows, so that tiles
// beside each other in the order share both operands in an XCD's L2: 8 tiles of rows at a time.
__device__ __forceinline__ void ce_tile(uint32_t i, uint32_t across, uint32_t down, uint32_t &v, uint32_t &r) {
  const uint32_t group = i / (8 * across), in = i - group * 8 * across;
  const uint32_t wide = down - group * 8 < 8 ? down - group * 8 : 8;
  v = in / wide;
  r = group * 8 + in - v * wide;
}

// Logits of a tile, z in units of log 2 less nothing: acc[n][m] of lane l is row 32 n + l % 32 and
// vocabulary entry 32 m + acc_row(reg) + 4 (l / 32) of the wave's part.
template <int DT, int BM, int BN, int WM, int STAGES> struct CeLogits {
  using G = TileGemm<DT, BM, BN, WM, false, false, STAGES>;
  static __device__ __forceinline__ void run(G &g, const CeArgs &a, char *ring, int64_t v0, int64_t r0, int m) {
    const int64_t vs = a.vocab - v0;
    g.a.start(a.w + v0 * a.row_bytes, a.row_bytes, vs < BM ? (int)vs : BM);
    g.b.start(a.hc + r0 * a.row_bytes, a.row_bytes, m - (int)r0 < BN ? m - (int)r0 : BN);
    g.clear();
    const int steps = (a.row_bytes + 63) / 64, left = a.row_bytes - (steps - 1) * 64;
    g.run(ring, steps, left, 0, 0, a.row_bytes, a.row_bytes);
  }
};

template <int DT, int BM, int BN, int WM, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_forward_kernel(CeArgs a) {
  using G = TileGemm<DT, BM, BN, WM, false, false, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char ring[];
  const int m = uniform(*a.counted);
  const uint32_t across = (uint32_t)blocks_of(a.vocab, BM), down = (uint32_t)blocks_of(m, BN);
  const uint32_t total = across * down;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    uint32_t tv, tr;
    ce_tile(xcd_order(i, total), across, down, tv, tr);
    const int64_t v0 = (int64_t)tv * BM, r0 = (int64_t)tr * BN;
    G g;
    CeLogits<DT, BM, BN, WM, STAGES>::run(g, a, ring, v0, r0, m);
    // largest logit and sum of exponentials of each row over this wave's part of the vocabulary
    const float f = a.scale * LOG2E;
    const int64_t first = v0 + wm * (BM / WM);
    const int exist = a.vocab - first < BM / WM ? (int)(a.vocab - first) : BM / WM;
    float2 *red = (float2 *)ring;
#pragma unroll
    for (int n = 0; n < G::TN; n++) {
      const int64_t r = r0 + (wn * G::TN + n) * 32 + (lane & 31);
      const int at = (r < m ? a.label[r] - (int)first : -1) - 4 * (lane >> 5);
      float most = -__builtin_inff(), z = 0.0f;
      bool mine = false;
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const int v = k * 32 + acc_row(e);
          float x = g.acc[n][k][e] * f;
          if (v == at) z = x, mine = true;
          if (v + 4 * (lane >> 5) >= exist) x = -__builtin_inff();
          most = __builtin_fmaxf(most, x);
          g.acc[n][k][e] = x;
        }
      most = half_max(most);
      const float from = most == -__builtin_inff() ? 0.0f : most;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int e = 0; e < 16; e++) sum += __builtin_amdgcn_exp2f(g.acc[n][k][e] - from);
      sum = half_sum(sum);
      if (lane < 32) red[wm * BN + (wn * G::TN + n) * 32 + lane] = make_float2(most, sum);
      if (mine && r < m) a.picked[r] = z;
    }
    __syncthreads();
    if (threadIdx.x < BN && r0 + threadIdx.x < m) {
      float2 s = red[threadIdx.x];
#pragma unroll
      for (int k = 1; k < WM; k++) {
        const float2 o = red[k * BN + threadIdx.x];
        const float most = __builtin_fmaxf(s.x, o.x), from = most == -__builtin_inff() ? 0.0f : most;
        s.y = s.y * __builtin_amdgcn_exp2f(s.x - from) + o.y * __builtin_amdgcn_exp2f(o.x - from);
        s.x = most;
      }
      a.part[(int64_t)tv * a.n + r0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// lse and loss of a row from its tiles' parts: 8 rows a workgroup, 32 threads to each.
template <int DT> __global__ void __launch_bounds__(GEMM_THREADS) ce_join_kernel(CeArgs a, int tiles) {
  const int m = *a.counted;
  const int row = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int64_t r = (int64_t)blockIdx.x * 8 + row;
  if ((int64_t)blockIdx.x * 8 >= m) return;
  __shared__ float2 part[32][8];
  float2 s = make_float2(-__builtin_inff(), 0.0f);
  auto add = [](float2 s, float2 o) {
    const float most = __builtin_fmaxf(s.x, o.x), from = most == -__builtin_inff() ? 0.0f : most;
    return make_float2(most, s.y * __builtin_amdgcn_exp2f(s.x - from) + o.y * __builtin_amdgcn_exp2f(o.x - from));
  };
  if (r < m) {
#pragma unroll 4
    for (int t = slice; t < tiles; t += 32) s = add(s, a.part[(int64_t)t * a.n + r]);
  }
  part[slice][row] = s;
  __syncthreads();
  for (int o = 16; o > 0; o >>= 1) {
    if (slice < o) part[slice][row] = add(part[slice][row], part[slice + o][row]);
    __syncthreads();
  }
  if (slice == 0 && r < m) {
    s = part[0][row];
    const float l = s.x + __builtin_log2f(s.y);
    const int64_t to = a.row[r];
    a.lse[to] = l * LN2;
    a.loss[to] = (l - a.picked[r]) * LN2;
  }
}

// P of one piece: [rows, whole tiles of them][cols], zeros past the rows and, in whole tiles, past
// the vocabulary.
template <int DT, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_p_kernel(CeArgs a) {
  constexpr int BM = CE_BM, BN = CE_BN, WM = 2;
  using G = TileGemm<DT, BM, BN, WM, false, false, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char ring[];
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  if (a.piece >= pieces.n) return;
  const int64_t piece0 = a.piece * pieces.cols;
  const int64_t cols = a.vocab - piece0 < pieces.cols ? a.vocab - piece0 : pieces.cols;
  const uint32_t across = (uint32_t)blocks_of(cols, BM), down = (uint32_t)blocks_of(m, BN), total = across * down;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  const float up = ce_up<DT>(a);
  constexpr int eb = Elem<DT>::bytes, part = BM / WM;
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    uint32_t tv, tr;
    ce_tile(xcd_order(i, total), across, down, tv, tr);
    const int64_t v0 = piece0 + (int64_t)tv * BM, r0 = (int64_t)tr * BN;
    const int64_t first = v0 + wm * part;
    const int exist = a.vocab - first < part ? (int)(a.vocab - first) : part;  // or negative
    G g;
    CeLogits<DT, BM, BN, WM, STAGES>::run(g, a, ring, v0, r0, m);
    const float f = a.scale * LOG2E;
    char *mine = ring + wave * (32 * part * eb);
#pragma unroll
    for (int n = 0; n < G::TN; n++) {
      const int64_t r = r0 + (wn * G::TN + n) * 32 + (lane & 31);
      const bool real = r < m;
      const int64_t source = real ? a.row[r] : 0;
      const float by = real ? a.grad[source] * a.scale * up : 0.0f;
      const float from = real ? a.lse[source] * LOG2E : 0.0f;
      const int at = (real ? a.label[r] - (int)first : -1) - 4 * (lane >> 5);
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const int v = k * 32 + acc_row(e);
          float x = __builtin_amdgcn_exp2f(g.acc[n][k][e] * f - from);
          if (v == at) x -= 1.0f;
          x *= by;
          g.acc[n][k][e] = real && v + 4 * (lane >> 5) < exist ? x : 0.0f;
        }
      const int64_t out = (r0 + (wn * G::TN + n) * 32) * pieces.cols + (first - piece0);
      store_rows<DT, part, G::TM>(mine, g.acc[n], 1.0f, a.p + out * eb, pieces.cols * eb, 32, part * eb);
    }
    __syncthreads();
  }
}

// dw of one piece: P^T h over the gathered rows.
template <int DT, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_dw_kernel(CeArgs a) {
  constexpr int BM = CE_BM, BN = CE_BN, WM = 2;
  using G = TileGemm<DT, BM, BN, WM, true, true, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char ring[];
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  if (a.piece >= pieces.n) return;
  const int64_t piece0 = a.piece * pieces.cols;
  const int64_t cols = a.vocab - piece0 < pieces.cols ? a.vocab - piece0 : pieces.cols;
  const uint32_t across = (uint32_t)blocks_of(a.d, BM), down = (uint32_t)blocks_of(cols, BN), total = across * down;
  const int wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  const float back = 1.0f / ce_up<DT>(a);
  constexpr int eb = Elem<DT>::bytes, part = BM / WM;
  const int steps = (int)blocks_of(m, G::BK);
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    uint32_t tc, tv;
    ce_tile(xcd_order(i, total), across, down, tc, tv);
    const int c0 = (int)tc * BM;
    const int64_t v0 = (int64_t)tv * BN;
    G g;
    g.clear();
    if (steps > 0) {
      g.a.start(a.hc + (int64_t)c0 * eb, a.row_bytes, a.row_bytes - c0 * eb);
      g.b.start(a.p + v0 * eb, pieces.cols * eb, BN * eb);
      // rows of P past the last are zeros, and whole tiles of rows are there
      g.run(ring, steps, 64, m - (steps - 1) * G::BK, G::BK, a.row_bytes, pieces.cols * eb);
    }
    char *mine = ring + wave * (32 * part * eb);
    const int at = c0 + wm * part;
    const int row_bytes = (a.d - at < part ? a.d - at : part) * eb;
#pragma unroll
    for (int n = 0; n < G::TN; n++) {
      const int64_t v = v0 + (wn * G::TN + n) * 32;
      const int64_t left = cols - v;
      if (row_bytes > 0 && left > 0)
        store_rows<DT, part, G::TM>(mine, g.acc[n], back, a.dw + (piece0 + v) * a.row_bytes + (int64_t)at * eb,
                                    a.row_bytes, left < 32 ? (int)left : 32, row_bytes);
    }
    __syncthreads();
  }
}

// dh's sums over one piece, added to those of the pieces before: tiles in register layout, the
// piece's steps in several parts where there are few tiles.
template <int DT, int STAGES>
__global__ void __launch_bounds__(GEMM_THREADS, 2) ce_dh_kernel(CeArgs a) {
  constexpr int BM = CE_BM, BN = CE_BN, WM = 2;
  using G = TileGemm<DT, BM, BN, WM, true, false, STAGES>;
  extern __shared__ __attribute__((aligned(1024))) char ring[];
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  if (a.piece >= pieces.n) return;
  const int64_t piece0 = a.piece * pieces.cols;
  const int64_t cols = a.vocab - piece0 < pieces.cols ? a.vocab - piece0 : pieces.cols;
  const uint32_t across = (uint32_t)blocks_of(a.d, BM), down = (uint32_t)blocks_of(m, BN), tiles = across * down;
  const uint32_t splits = (uint32_t)ce_splits(tiles, a.slots, pieces.cols, G::BK), total = tiles * splits;
  const int steps = (int)blocks_of(cols, G::BK);
  constexpr int eb = Elem<DT>::bytes;
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    const uint32_t id = xcd_order(i, total), split = id / tiles;
    uint32_t tc, tr;
    ce_tile(id - split * tiles, across, down, tc, tr);
    const int c0 = (int)tc * BM;
    const int64_t r0 = (int64_t)tr * BN;
    const int from = (int)((int64_t)steps * split / splits), to = (int)((int64_t)steps * (split + 1) / splits);
    G g;
    g.clear();
    if (to > from) {
      const int64_t k0 = (int64_t)from * G::BK;
      g.a.start(a.w + (piece0 + k0) * a.row_bytes + (int64_t)c0 * eb, a.row_bytes, a.row_bytes - c0 * eb);
      g.b.start(a.p + (r0 * pieces.cols + k0) * eb, pieces.cols * eb, BN);
      // columns of P past the vocabulary are zeros
      const int64_t left = cols - (int64_t)(to - 1) * G::BK;
      g.run(ring, to - from, 64, left < G::BK ? (int)left : G::BK, 0, a.row_bytes, pieces.cols * eb);
    }
    f32x4_t *out = (f32x4_t *)a.dhp + (int64_t)id * (BM * BN / 4) + threadIdx.x;
#pragma unroll
    for (int n = 0; n < G::TN; n++)
#pragma unroll
      for (int k = 0; k < G::TM; k++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          f32x4_t x = {g.acc[n][k][4 * q], g.acc[n][k][4 * q + 1], g.acc[n][k][4 * q + 2], g.acc[n][k][4 * q + 3]};
          f32x4_t *at = out + ((n * G::TM + k) * 4 + q) * GEMM_THREADS;
          if (a.piece > 0) x += *at;
          *at = x;
        }
  }
}

// dh from its parts, rounded once, to the rows' own places.
template <int DT> __global__ void __launch_bounds__(GEMM_THREADS) ce_dh_join_kernel(CeArgs a) {
  constexpr int BM = CE_BM, BN = CE_BN, WM = 2;
  using G = TileGemm<DT, BM, BN, WM, true, false, 3>;
  using T = typename AttnElem<DT>::type;
  typedef T v4 __attribute__((ext_vector_type(4)));
  const int m = uniform(*a.counted);
  const CePieces pieces(m, a.vocab, a.p_elements);
  const uint32_t across = (uint32_t)blocks_of(a.d, BM), down = (uint32_t)blocks_of(m, BN), tiles = across * down;
  const uint32_t splits = (uint32_t)ce_splits(tiles, a.slots, pieces.cols, G::BK);
  const float back = 1.0f / ce_up<DT>(a);
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), wm = wave % WM, wn = wave / WM;
  // a block of 32 x 32 of a tile for each round
  const uint32_t total = tiles * G::TN * G::TM;
  for (uint32_t i = blockIdx.x; i < total; i += gridDim.x) {
    const uint32_t tile = i / (G::TN * G::TM), nk = i - tile * (G::TN * G::TM);
    const int n = nk / G::TM, k = nk - n * G::TM;
    uint32_t tc, tr;
    ce_tile(tile, across, down, tc, tr);
    const int64_t r = (int64_t)tr * BN + (wn * G::TN + n) * 32 + (lane & 31);
    const int c = (int)tc * BM + (wm * G::TM + k) * 32 + 4 * (lane >> 5);
    const f32x4_t *p = (const f32x4_t *)a.dhp + (int64_t)tile * (BM * BN / 4) + nk * 4 * GEMM_THREADS + threadIdx.x;
    f32x4_t x[4] = {};
    for (uint32_t s = 0; s < splits; s++)
#pragma unroll
      for (int q = 0; q < 4; q++) x[q] += p[(int64_t)s * tiles * (BM * BN / 4) + q * GEMM_THREADS];
    if (r >= m) continue;
    T *to = (T *)(a.dh + (int64_t)a.row[r] * a.row_bytes);
#pragma unroll
    for (int q = 0; q < 4; q++) {
      if (c + 8 * q >= a.d) break;  // d is a multiple of 4 entries
      v4 o;
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] = (T)(x[q][e] * back);
      *(v4 *)(to + c + 8 * q) = o;
    }
  }
}

int ce_forward_bf16(const CeArgs &a, int cus, hipStream_t st);
int ce_forward_fp16(const CeArgs &a, int cus, hipStream_t st);
int ce_forward_fp32(const CeArgs &a, int cus, hipStream_t st);
int ce_backward_bf16(CeArgs &a, int64_t pieces, int cus, hipStream_t st);
int ce_backward_fp16(CeArgs &a, int64_t pieces, int cus, hipStream_t st);
int ce_backward_fp32(CeArgs &a, int64_t pieces, int cus, hipStream_t st);

}  // namespace maxsim
