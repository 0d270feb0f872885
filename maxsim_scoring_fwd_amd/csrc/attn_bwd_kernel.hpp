// Attention backward, after <dO, o> per row (attn_delta.hpp): dQ (keys in tiles, one wave on 32 queries) and
// dK / dV (queries in tiles, one wave on 32 keys, all heads that share them). The scores are
// computed again in both: 7 products instead of 5, but every sum has one owner, so there are no
// atomics and repeated calls give the same bits.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

template <int DT, int DP, int MODE>
__device__ __forceinline__ void attn_dq_tile(const AttnArgs &a, const AttnTile &t, char *lds) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = 32, OT = DP / 32, TILE = BN * L::bytes;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (int)(threadIdx.x >> 6) * 32;
  const int i = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  const int iq = i < t.len ? i : t.len - 1;
  Held<DT, DP> q, g;
  q.load(a.q + t.q + t.head * a.q_head, a.q_tok, iq, row_bytes);
  g.load(a.dO + (t.row0 * a.heads + t.head) * row_bytes, (int64_t)a.heads * row_bytes, iq, row_bytes);
  const int kv = t.head / a.group;
  const char *kp = a.k + t.k + kv * a.k_head, *vp = a.v + t.v + kv * a.v_head;
  const ScoreForm form = score_form<DT, MODE>(a, t.head);
  const int vis = visible(a, t, iq), wave_least = visible(a, t, wave0);
  const int last = t.first + ATTN_ROWS < t.len ? t.first + ATTN_ROWS - 1 : t.len - 1;
  const int n_keys = visible(a, t, last);
  const int64_t at = (int64_t)t.head * a.rows + t.row0 + iq;
  const float lse = a.lse[at] * LOG2E;
  const float gs = DT == DT_FP16 ? *a.grad_scale : 1.0f;
  const float delta = a.delta[at];

  const int tiles = (n_keys + BN - 1) / BN;
  const int wave_most = visible(a, t, wave0 + 31 < t.len ? wave0 + 31 : t.len - 1);
  const int wave_tiles = wave0 < t.len ? (wave_most + BN - 1) / BN : 0;

  // As in the forward, tile n + 1 is fetched in iteration n into the buffer that no wave reads any
  // more.
  const int wave = uniform((int)(threadIdx.x >> 6));
  Carry<DT, DP, BN> ck, cv;
  ck.init(a.k_tok, row_bytes);
  cv.init(a.v_tok, row_bytes);
  auto aim = [&](int n) {
    const int there = n < tiles ? n : tiles - 1, valid = n < tiles ? t.len - n * BN : 1;
    ck.aim(kp + (int64_t)there * BN * a.k_tok, a.k_tok, valid);
    cv.aim(vp + (int64_t)there * BN * a.v_tok, a.v_tok, valid);
  };
  constexpr int P = 2 * Carry<DT, DP, BN>::n;
  auto fetch = [&](int n, int from, int to) {  // pieces of tile n
    char *const next = lds + (n & 1) * 2 * TILE;
#pragma unroll
    for (int e = from; e < to; e++) {
      if (e & 1) cv.go(next + TILE, wave, e / 2);
      else ck.go(next, wave, e / 2);
    }
  };
  aim(0);
  fetch(0, 0, P);
  f32x16_t acc[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  const int row_lane = row_lane_offset<DT, DP>(), tr_lane = tr_lane_offset<DT, DP>();
  constexpr int A = L::steps, C = OT * 2;

  auto tile = [&](int n, bool masked) {
    const char *const ldsk = lds + (n & 1) * 2 * TILE, *const ldsv = ldsk + TILE;
    const float dist0 = (float)(i - n * BN - 4 * h);
    const int left = vis - n * BN - 4 * h;
    f32x16_t s, dp;
    Packed<DT> p;
    // products to weights, times the cap's slope where there is one
    auto weights = [&](int from, int to) {
#pragma unroll
      for (int r = from; r < to; r++) {
        float keep = 1.0f;
        float y = score<DT, MODE>(form, s[r], dist0 - (float)acc_row(r), &keep);
        if (masked) y = acc_row(r) < left ? y : -INFINITY;
        s[r] = __builtin_amdgcn_exp2f(y - lse) * (MODE == ATTN_CAP ? keep * gs : gs);
      }
    };
    auto grads = [&](int from, int to) {
#pragma unroll
      for (int r = from; r < to; r++) dp[r] = s[r] * (dp[r] - delta);
    };
    if constexpr (DT == DT_FP32) {
      s = mma_tile<DT, DP>(ldsk, q, zero16());
      dp = mma_tile<DT, DP>(ldsv, g, zero16());
      weights(0, 16);
      grads(0, 16);
      p.set(dp);
#pragma unroll
      for (int c = 0; c < OT; c++) acc[c] = mma_cols<DT, DP>(ldsk, tr_lane, 0, c * 32, p, acc[c]);
      fetch(n + 1, 0, P);
    } else {
      pipeline<2 * A + C, 4>(
          [&](int j) {
            return j < A       ? read_rows<DT, DP>(ldsk, row_lane, j)
                   : j < 2 * A ? read_rows<DT, DP>(ldsv, row_lane, j - A)
                               : read_cols<DT, DP>(ldsk, tr_lane, 0, (j - 2 * A) % OT * 32, (j - 2 * A) / OT);
          },
          [&](int j, u32x4_t x) {
            if (j < A) s = mma_rows<DT>(x, q.f[j % A], j ? s : zero16());
            else if (j < 2 * A) dp = mma_rows<DT>(x, g.f[j % A], j > A ? dp : zero16());
            else acc[(j - 2 * A) % OT] = mma_rows<DT>(x, p.f[(j - 2 * A) / OT], acc[(j - 2 * A) % OT]);
          },
          [&](int j) {
            if (j < A) fetch(n + 1, j * P / A, (j + 1) * P / A);
            else if (j < 2 * A) weights((j - A) * 16 / A, (j + 1 - A) * 16 / A);
            // the first 16 keys' share of dQ runs while the other 16 keys' gradients are made
            if (j == 2 * A - 1) {
              grads(0, 8);
              p.set_half(dp, 0);
            }
            if (j == 2 * A) {
              grads(8, 16);
              p.set_half(dp, 1);
            }
          });
    }
  };
  for (int n = 0; n < tiles; n++) {
    tile_barrier();
    aim(n + 1);
    if (n >= wave_tiles) {  // nothing for this wave's rows but to fetch
      fetch(n + 1, 0, P);
    } else if ((n + 1) * BN > wave_least) {
      asm volatile("; masked");  // see the forward
      tile(n, true);
    } else {
      asm volatile("; whole");
      tile(n, false);
    }
  }
  tile_barrier();  // the tiles' memory is free
  store_rows<DT, DP>(lds + (threadIdx.x >> 6) * TILE, acc, i < t.len ? a.scale / gs : 0.0f,
                     a.dq + ((t.row0 + wave0) * a.heads + t.head) * row_bytes,
                     (int64_t)a.heads * row_bytes, t.rows - wave0, row_bytes);
}

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS) attn_dq_kernel(const AttnArgs a) {
  __shared__ __align__(256) char lds[4 * 32 * RowLayout<DT, DP>::bytes];  // two buffers: one barrier a tile
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  if (t.first < t.len) attn_dq_tile<DT, DP, MODE>(a, t, lds);
  else zero_tile<DT>(a.dq, a.heads, t, ATTN_ROWS, a.d);
}

// WHAT: 1 for dK, 2 for dV, 3 for both. Heads wider than 128 take a launch for each: a wave has no
// registers for both sums, and computing the scores again costs less than spilling.
template <int DT, int DP, int MODE, int WHAT>
__device__ __forceinline__ void attn_dkv_tile(const AttnArgs &a, const AttnTile &t, char *lds, float (*stat)[64]) {
  using L = RowLayout<DT, DP>;
  constexpr int BM = 32, OT = DP / 32, TILE = BM * L::bytes;
  constexpr bool DK = WHAT & 1, DV = WHAT & 2;
  // fp16 P is rounded 2^8 times too large: rows over thousands of keys stay out of the subnormals
  constexpr float SHIFT = DT == DT_FP16 ? 8.0f : 0.0f;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (int)(threadIdx.x >> 6) * 32;
  const int j = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  const int jk = j < t.len ? j : t.len - 1;
  Held<DT, DP> k, v;
  k.load(a.k + t.k + t.head * a.k_head, a.k_tok, jk, row_bytes);
  if (DK) v.load(a.v + t.v + t.head * a.v_head, a.v_tok, jk, row_bytes);
  const int group = a.group;
  // with a causal mask only rows from the key on see it, unless it lies in the prefix
  const int from = t.first >= t.prefix ? t.first : 0;
  const int jmask = j < t.prefix ? -1 : j;
  const int total = (t.len - from + BM - 1) / BM * group;
  const float gs = DT == DT_FP16 ? *a.grad_scale : 1.0f;
  const float gs8 = gs * (DT == DT_FP16 ? 1.0f / 256.0f : 1.0f);

  // Tiles are fetched as in the other kernels, head by head; the rows' statistics pass through a
  // register, one tile further ahead.
  const int wave = uniform((int)(threadIdx.x >> 6));
  Carry<DT, DP, BM> cq, cg;
  float st = 0.0f;
  const int tok = a.heads * row_bytes;
  cq.init(a.q_tok, row_bytes);
  cg.init(tok, row_bytes);
  int next_head = t.head * group, next_row = from;  // of the tile to aim at
  const int end_head = next_head + group;
  auto aim = [&]() {
    const bool there = next_head < end_head;
    const int head = there ? next_head : end_head - 1, i0 = there ? next_row : from;
    const int valid = there ? t.len - i0 : 1;
    cq.aim(a.q + t.q + head * a.q_head + (int64_t)i0 * a.q_tok, a.q_tok, valid);
    cg.aim(a.dO + ((t.row0 + i0) * a.heads + head) * row_bytes, tok, valid);
    next_row += BM;
    if (next_row >= t.len) {
      next_row = from;
      next_head++;
    }
  };
  constexpr int P = 2 * Carry<DT, DP, BM>::n;
  auto fetch = [&](int n, int first, int to) {  // pieces of tile n
    char *const next = lds + (n & 1) * 2 * TILE;
#pragma unroll
    for (int e = first; e < to; e++) {
      if (e & 1) cg.go(next + TILE, wave, e / 2);
      else cq.go(next, wave, e / 2);
    }
  };
  // Statistics of the rows, where S and dP start: -lse in units of the product (of the score
  // behind a tanh), -inf for rows past the document, which weigh nothing; and -delta.
  const float unit = MODE == ATTN_CAP ? 1.0f : score_form<DT, MODE>(a, t.head * group).a;
  int stat_head = t.head * group, stat_row = from;  // of the tile whose statistics come next
  auto load_stat = [&]() {
    if (threadIdx.x < 2 * BM) {
      const int row = stat_row + (threadIdx.x & (BM - 1));
      const int head = stat_head < end_head ? stat_head : end_head - 1;
      const float x = (threadIdx.x < BM ? a.lse : a.delta)[(int64_t)head * a.rows + t.row0 +
                                                           (row < t.len ? row : t.len - 1)];
      st = threadIdx.x >= BM ? -x : row < t.len ? (SHIFT - x * LOG2E) / unit : -INFINITY;
    }
    stat_row += BM;
    if (stat_row >= t.len) {
      stat_row = from;
      stat_head++;
    }
  };
  auto store_stat = [&](int buf) {
    if (threadIdx.x < 2 * BM) stat[buf][threadIdx.x] = st;
  };
  aim();
  fetch(0, 0, P);
  load_stat();
  store_stat(0);
  load_stat();
  f32x16_t dk[OT], dv[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) {
    dk[c] = zero16();
    dv[c] = zero16();
  }
  const int row_lane = row_lane_offset<DT, DP>(), tr_lane = tr_lane_offset<DT, DP>();
  // matrix instructions of the four products, and pieces of a tile
  constexpr int A = L::steps, B = DK ? A : 0, C = DV ? OT * 2 : 0, D = DK ? OT * 2 : 0;

  auto tile = [&](const ScoreForm &form, int i0, int n, bool masked) {
    const char *const ldsq = lds + (n & 1) * 2 * TILE, *const ldsg = ldsq + TILE;
    const float *const stats = stat[n & 1];
    const float dist0 = (float)(i0 + 4 * h - j);
    const int hide = jmask - i0 - 4 * h;  // rows below it do not see key j
    f32x16_t s, dp;
    Packed<DT> pv, pk;
    // The sums start from the rows' statistics: dP from -delta, S from -lse / scale, so that
    // neither is subtracted (nor held) afterwards. The tanh wants S itself.
    auto rows_of = [&](const float *from) {
      f32x16_t x;
#pragma unroll
      for (int g4 = 0; g4 < 4; g4++) {
        const f32x4_t y = *(const f32x4_t *)(from + 8 * g4 + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; e++) x[4 * g4 + e] = y[e];
      }
      return x;
    };
    const f32x16_t lse = rows_of(stats);
    s = MODE == ATTN_CAP ? zero16() : lse;
    if constexpr (DK) dp = rows_of(stats + BM);
    f32x16_t slope;  // of the cap
    auto weights = [&](int first, int to) {
#pragma unroll
      for (int r = first; r < to; r++) {
        float keep = 1.0f;
        float y = score<DT, MODE>(form, s[r], dist0 + (float)acc_row(r), &keep);
        if (MODE == ATTN_CAP) y += lse[r];
        if (masked) y = acc_row(r) < hide ? -INFINITY : y;
        s[r] = __builtin_amdgcn_exp2f(y);
        if (MODE == ATTN_CAP) slope[r] = keep;
      }
    };
    auto grads = [&](int first, int to) {
#pragma unroll
      for (int r = first; r < to; r++) {
        dp[r] = s[r] * dp[r];
        if (MODE == ATTN_CAP) dp[r] *= slope[r];
        if (DT == DT_FP16) dp[r] *= gs8;
      }
    };
    if constexpr (DT == DT_FP32) {
      s = mma_tile<DT, DP>(ldsq, k, s);
      dp = mma_tile<DT, DP>(ldsg, v, dp);
      weights(0, 16);
      pv.set(s);
#pragma unroll
      for (int c = 0; c < OT; c++) dv[c] = mma_cols<DT, DP>(ldsg, tr_lane, 0, c * 32, pv, dv[c]);
      grads(0, 16);
      pk.set(dp);
#pragma unroll
      for (int c = 0; c < OT; c++) dk[c] = mma_cols<DT, DP>(ldsq, tr_lane, 0, c * 32, pk, dk[c]);
      fetch(n + 1, 0, P);
    } else {
      // S, then dP beside the weights, then dV beside dS, then dK; the next tile's fetch beside S
      pipeline<A + B + C + D, 4>(
          [&](int j) {
            if (j < A) return read_rows<DT, DP>(ldsq, row_lane, j);
            if (j < A + B) return read_rows<DT, DP>(ldsg, row_lane, j - A);
            const int x = j < A + B + C ? j - A - B : j - A - B - C;
            return read_cols<DT, DP>(j < A + B + C ? ldsg : ldsq, tr_lane, 0, x % OT * 32, x / OT);
          },
          [&](int j, u32x4_t x) {
            if (j < A) {
              s = mma_rows<DT>(x, k.f[j % A], s);
            } else if (j < A + B) {
              dp = mma_rows<DT>(x, v.f[(j - A) % A], dp);
            } else if (j < A + B + C) {
              const int y = j - A - B;
              dv[y % OT] = mma_rows<DT>(x, pv.f[y / OT], dv[y % OT]);
            } else {
              const int y = j - A - B - C;
              dk[y % OT] = mma_rows<DT>(x, pk.f[y / OT], dk[y % OT]);
            }
          },
          [&](int j) {
            if constexpr (DK) {
              if (j >= A && j < A + B) weights((j - A) * 16 / A, (j + 1 - A) * 16 / A);
            } else if (j == A - 1) {
              weights(0, 16);
            }
            if (DV && j == A + B - 1) pv.set(s);
            if constexpr (DK && DV) {
              if (j >= A + B && j < A + B + C) grads((j - A - B) * 16 / C, (j + 1 - A - B) * 16 / C);
              if (j == A + B + C - 1) pk.set(dp);
            } else {
              if (DK && j == A + B - 1) {
                grads(0, 16);
                pk.set(dp);
              }
            }
            if (j < A) fetch(n + 1, j * P / A, (j + 1) * P / A);
          });
    }
    store_stat((n + 1) & 1);
    load_stat();
  };
  int i0 = from, head = t.head * group;
  for (int n = 0; n < total; n++) {
    tile_barrier();
    aim();
    // nothing where this wave has no keys, or where the tile's rows see none of them
    if (wave0 >= t.len || (a.causal && wave0 >= t.prefix && wave0 > i0 + BM - 1)) {
      fetch(n + 1, 0, P);
      store_stat((n + 1) & 1);
      load_stat();
    } else {
      const ScoreForm form = score_form<DT, MODE>(a, head);
      if (a.causal && wave0 + 31 > i0) {
        asm volatile("; masked");
        tile(form, i0, n, true);
      } else {
        asm volatile("; whole");
        tile(form, i0, n, false);
      }
    }
    i0 += BM;
    if (i0 >= t.len) {
      i0 = from;
      head++;
    }
  }
  tile_barrier();  // the tiles' memory is free
  const int64_t first = ((t.row0 + wave0) * a.kv_heads + t.head) * row_bytes;
  const int64_t stride = (int64_t)a.kv_heads * row_bytes;
  char *const mine = lds + (threadIdx.x >> 6) * TILE;
  const bool real = j < t.len;
  if constexpr (DK)
    store_rows<DT, DP>(mine, dk, real ? a.scale / gs : 0.0f, a.dk + first, stride, t.rows - wave0, row_bytes);
  if constexpr (DV)
    store_rows<DT, DP>(mine, dv, real ? (DT == DT_FP16 ? 1.0f / 256.0f : 1.0f) : 0.0f, a.dv + first,
                     stride, t.rows - wave0, row_bytes);
}

template <int DT, int DP, int MODE, int WHAT>
__global__ void __launch_bounds__(ATTN_THREADS) attn_dkv_kernel(const AttnArgs a) {
  __shared__ __align__(256) char lds[4 * 32 * RowLayout<DT, DP>::bytes];  // two buffers: one barrier a tile
  __shared__ __align__(16) float stat[2][64];
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  if (t.first < t.len) {
    attn_dkv_tile<DT, DP, MODE, WHAT>(a, t, lds, stat);
    return;
  }
  if (WHAT & 1) zero_tile<DT>(a.dk, a.kv_heads, t, ATTN_ROWS, a.d);
  if (WHAT & 2) zero_tile<DT>(a.dv, a.kv_heads, t, ATTN_ROWS, a.d);
}

}  // namespace maxsim
