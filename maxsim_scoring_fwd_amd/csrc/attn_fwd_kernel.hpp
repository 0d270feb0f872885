// Attention forward: 4 waves of 32 queries each, keys in tiles through LDS. The softmax's vector
// work and the matrix products of a tile take about as long as each other, so a wave works on two
// tiles at once: the next tile's scores (matrix core) beside this tile's exponentials, and this
// tile's sum of values (matrix core) beside the next tile's scale, mask and maximum. K therefore
// arrives in LDS one tile ahead of V; each has two buffers, which makes one barrier a tile enough.
#pragma once

#include "attn_common.hpp"

#ifndef ATTN_FWD_KEYS
#define ATTN_FWD_KEYS 32
#endif

namespace maxsim {

template <int DT, int DP> struct FwdShape {
  static constexpr int keys = DT == DT_FP32 || DP >= 128 ? 32 : ATTN_FWD_KEYS;  // keys of a tile
  static constexpr int waves = DP >= 256 ? 1 : DP >= 96 ? 2 : 3;
};

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS)
__attribute__((amdgpu_waves_per_eu(FwdShape<DT, DP>::waves, FwdShape<DT, DP>::waves)))
attn_fwd_kernel(const AttnArgs a) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = FwdShape<DT, DP>::keys, NT = BN / 32, OT = DP / 32, TILE = BN * L::bytes;
  __shared__ __align__(256) char ldsk[2][TILE], ldsv[2][TILE];
  AttnTile t;
  if (!locate(a, ATTN_ROWS, a.group, t)) return;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (threadIdx.x >> 6) * 32;
  const int i = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  char *out = a.o + ((t.row0 + i) * a.heads + t.head) * row_bytes;
  float *lse = a.lse + (int64_t)t.head * a.rows + t.row0 + i;
  if (t.first >= t.len) {  // rows without a token
    if (i < t.rows) {
      zero_row<DT>(out, a.d);
      if (h == 0) *lse = -INFINITY;
    }
    return;
  }
  const int iq = i < t.len ? i : t.len - 1;
  Held<DT, DP> q;
  q.load(a.q + t.q + t.head * a.q_head, a.q_tok, iq, row_bytes);
  const int kv = t.head / a.group;
  const char *kp = a.k + t.k + kv * a.k_head, *vp = a.v + t.v + kv * a.v_head;
  const ScoreForm form = score_form<DT, MODE>(a, t.head);
  const float post = MODE == ATTN_PLAIN ? form.a : 1.0f;  // factor left to the exponentials
  const int vis = visible(a, t, iq);
  const int wave_least = visible(a, t, wave0);
  const int last = t.first + ATTN_ROWS < t.len ? t.first + ATTN_ROWS - 1 : t.len - 1;
  const int n_keys = visible(a, t, last);

  const int tr_lane = tr_lane_offset<DT, DP>();
  const int tiles = (n_keys + BN - 1) / BN;
  // tiles that some row of this wave sees; none where the wave has no rows
  const int wave_most = visible(a, t, wave0 + 31 < t.len ? wave0 + 31 : t.len - 1);
  const int wave_tiles = wave0 < t.len ? (wave_most + BN - 1) / BN : 0;

  Stage<DT, DP, BN> sk, sv;
  auto load = [&](auto &stage, const char *p, int tok, int n) {
    stage.load(p + (int64_t)n * BN * tok, tok, t.len - n * BN, row_bytes);
  };
  load(sk, kp, a.k_tok, 0);
  load(sv, vp, a.v_tok, 0);
  sk.store(ldsk[0]);
  __syncthreads();
  if (tiles > 1) load(sk, kp, a.k_tok, 1);

  f32x16_t acc[OT], s[NT];
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  float m = -1e30f, sum = 0.0f;  // a finite start: exp2(-inf - m) is 0 for rows that see nothing yet
  float top = -INFINITY;

  const int row_lane = row_lane_offset<DT, DP>();
  constexpr int N1 = NT * L::steps, N2 = NT * OT * 2, E = NT * 16;  // products; elements of a lane
  // Matrix work of a step, with share i of other vector work beside instruction i. 16-bit types
  // run it as a pipeline; fp32 is bound by its matrix instructions alone.
  auto products = [&](f32x16_t (&x)[NT], int n, auto work) {
    const char *tile = ldsk[n & 1];
    if constexpr (DT == DT_FP32) {
#pragma unroll
      for (int b = 0; b < NT; b++) x[b] = mma_tile<DT, DP>(tile + b * 32 * L::bytes, q);
#pragma unroll
      for (int i = 0; i < N1; i++) work(i);
    } else {
      pipeline<N1, 4>(
          [&](int i) { return read_rows<DT, DP>(tile + i / L::steps * 32 * L::bytes, row_lane, i % L::steps); },
          [&](int i, u32x4_t v) {
            f32x16_t &c = x[i / L::steps];
            c = mma_rows<DT>(v, q.f[i % L::steps], i % L::steps ? c : zero16());
          },
          work);
    }
  };
  auto values = [&](const Packed<DT> (&p)[NT], int n, auto work) {
    const char *tile = ldsv[n & 1];
    if constexpr (DT == DT_FP32) {
#pragma unroll
      for (int b = 0; b < NT; b++)
#pragma unroll
        for (int c = 0; c < OT; c++)
          acc[c] = mma_cols<DT, DP>(tile, tr_lane, b * 32, c * 32, p[b], acc[c]);
#pragma unroll
      for (int i = 0; i < N2; i++) work(i);
    } else {
      // 16 keys after 16, so that neighbours add to different accumulators
      pipeline<N2, 4>(
          [&](int i) { return read_cols<DT, DP>(tile, tr_lane, i / OT / 2 * 32, i % OT * 32, i / OT % 2); },
          [&](int i, u32x4_t v) { acc[i % OT] = mma_rows<DT>(v, p[i / OT / 2].f[i / OT % 2], acc[i % OT]); },
          work);
    }
  };
  // products of tile n to scores, and their maximum: elements from .. to - 1
  auto scores = [&](f32x16_t (&x)[NT], int n, bool masked, int from, int to) {
    const float dist0 = (float)(i - n * BN - 4 * h);
    const int left = vis - n * BN - 4 * h;
#pragma unroll
    for (int e = from; e < to; e++) {
      float y = x[e / 16][e % 16];
      const int key = e / 16 * 32 + acc_row(e % 16);
      if constexpr (MODE != ATTN_PLAIN) y = score<DT, MODE>(form, y, dist0 - (float)key, nullptr);
      if (masked) y = key < left ? y : -INFINITY;
      top = __builtin_fmaxf(top, y);
      x[e / 16][e % 16] = y;
    }
  };
  // scores to weights, not yet rounded
  auto weights = [&](f32x16_t (&x)[NT], int from, int to) {
#pragma unroll
    for (int e = from; e < to; e++) {
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e / 16][e % 16], post, -m));
      sum += w;
      x[e / 16][e % 16] = w;
    }
  };
  auto nothing = [](int) {};

  if (wave_tiles > 0) {
    products(s, 0, nothing);
    scores(s, 0, true, 0, E);
    top = half_max(top) * post;
  }
  for (int n = 0; n < tiles; n++) {
    if (n + 1 < tiles) sk.store(ldsk[(n + 1) & 1]);
    sv.store(ldsv[n & 1]);
    __syncthreads();
    if (n + 2 < tiles) load(sk, kp, a.k_tok, n + 2);
    if (n + 1 < tiles) load(sv, vp, a.v_tok, n + 1);
    if (n >= wave_tiles) continue;
    // The reference point of the exponentials follows the running maximum only once that is
    // 2^8 away: sums and weights up to 256 lose nothing, and most tiles leave the accumulator
    // as it is.
    if (__any(top > m + 8.0f)) {
      const float mn = __builtin_fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      sum *= f;
#pragma unroll
      for (int c = 0; c < OT; c++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[c][r] *= f;
    }
    Packed<DT> p[NT];
    if (n + 1 == wave_tiles) {
      weights(s, 0, E);
#pragma unroll
      for (int b = 0; b < NT; b++) p[b].set(s[b]);
      values(p, n, nothing);
      continue;
    }
    f32x16_t next[NT];
    products(next, n + 1, [&](int i) { weights(s, i * E / N1, (i + 1) * E / N1); });
#pragma unroll
    for (int b = 0; b < NT; b++) p[b].set(s[b]);
    top = -INFINITY;
    if ((n + 2) * BN > wave_least)
      values(p, n, [&](int i) { scores(next, n + 1, true, i * E / N2, (i + 1) * E / N2); });
    else
      values(p, n, [&](int i) { scores(next, n + 1, false, i * E / N2, (i + 1) * E / N2); });
    top = half_max(top) * post;
#pragma unroll
    for (int b = 0; b < NT; b++) s[b] = next[b];
  }
  sum = half_sum(sum);
  if (i < t.len) {
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int c = 0; c < OT; c++) store_cols<DT>(out, c * 32, a.d, acc[c], inv);
    if (h == 0) *lse = sum > 0.0f ? (m + __builtin_amdgcn_logf(sum)) * LN2 : -INFINITY;
  } else if (i < t.rows) {
    zero_row<DT>(out, a.d);
    if (h == 0) *lse = -INFINITY;
  }
}

}  // namespace maxsim
