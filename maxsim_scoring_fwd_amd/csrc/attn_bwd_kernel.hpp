// Attention backward, after <dO, o> per row (attn_delta.hpp): dQ (keys in tiles, one wave on 32 queries) and
// dK / dV (queries in tiles, one wave on 32 keys, all heads that share them). The scores are
// computed again in both: 7 products instead of 5, but every sum has one owner, so there are no
// atomics and repeated calls give the same bits.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS) attn_dq_kernel(const AttnArgs a) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = 32, OT = DP / 32, TILE = BN * L::bytes;
  __shared__ __align__(256) char lds[4 * TILE];  // two buffers: one barrier a tile
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (int)(threadIdx.x >> 6) * 32;
  const int i = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  char *out = a.dq + ((t.row0 + i) * a.heads + t.head) * row_bytes;
  if (t.first >= t.len) {
    if (i < t.rows) zero_row<DT>(out, a.d);
    return;
  }
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

  Stage<DT, DP, BN> sk, sv;
  sk.init(a.k_tok, row_bytes);
  sv.init(a.v_tok, row_bytes);
  sk.load(kp, a.k_tok, t.len);
  sv.load(vp, a.v_tok, t.len);
  f32x16_t acc[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  const int tr_lane = tr_lane_offset<DT, DP>();
  const int wave_most = visible(a, t, wave0 + 31 < t.len ? wave0 + 31 : t.len - 1);
  int buf = 0;
  for (int j0 = 0; j0 < n_keys; j0 += BN, buf ^= 2 * TILE) {
    const char *const ldsk = lds + buf, *const ldsv = ldsk + TILE;
    sk.store(lds + buf);
    sv.store(lds + buf + TILE);
    __syncthreads();
    if (j0 + BN < n_keys) {
      sk.load(kp + (int64_t)(j0 + BN) * a.k_tok, a.k_tok, t.len - j0 - BN);
      sv.load(vp + (int64_t)(j0 + BN) * a.v_tok, a.v_tok, t.len - j0 - BN);
    }
    if (wave0 >= t.len || j0 >= wave_most) continue;  // nothing for this wave's rows
    f32x16_t s = mma_tile<DT, DP>(ldsk, q);
    f32x16_t dp = mma_tile<DT, DP>(ldsv, g);
    const float dist0 = (float)(i - j0 - 4 * h);
    const int left = j0 + BN > wave_least ? vis - j0 - 4 * h : BN;
#pragma unroll
    for (int r = 0; r < 16; r++) {
      float keep = 1.0f;
      float y = score<DT, MODE>(form, s[r], dist0 - (float)acc_row(r), &keep);
      y = acc_row(r) < left ? y : -INFINITY;
      dp[r] = __builtin_amdgcn_exp2f(y - lse) * (dp[r] - delta) * (MODE == ATTN_CAP ? keep * gs : gs);
    }
    Packed<DT> p;
    p.set(dp);
#pragma unroll
    for (int c = 0; c < OT; c++) acc[c] = mma_cols<DT, DP>(ldsk, tr_lane, 0, c * 32, p, acc[c]);
  }
  __syncthreads();  // the tiles' memory is free
  store_rows<DT, DP>(lds + (threadIdx.x >> 6) * TILE, acc, i < t.len ? a.scale / gs : 0.0f,
                     a.dq + ((t.row0 + wave0) * a.heads + t.head) * row_bytes,
                     (int64_t)a.heads * row_bytes, t.rows - wave0, row_bytes);
}

// WHAT: 1 for dK, 2 for dV, 3 for both. Heads wider than 128 take a launch for each: a wave has no
// registers for both sums, and computing the scores again costs less than spilling.
template <int DT, int DP, int MODE, int WHAT>
__global__ void __launch_bounds__(ATTN_THREADS) attn_dkv_kernel(const AttnArgs a) {
  using L = RowLayout<DT, DP>;
  constexpr int BM = 32, OT = DP / 32, TILE = BM * L::bytes;
  constexpr bool DK = WHAT & 1, DV = WHAT & 2;
  // fp16 P is rounded 2^8 times too large: rows over thousands of keys stay out of the subnormals
  constexpr float SHIFT = DT == DT_FP16 ? 8.0f : 0.0f;
  __shared__ __align__(256) char lds[4 * TILE];  // two buffers: one barrier a tile
  __shared__ __align__(16) float stat[2][2 * BM];
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (int)(threadIdx.x >> 6) * 32;
  const int j = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  const int64_t out = ((t.row0 + j) * a.kv_heads + t.head) * row_bytes;
  if (t.first >= t.len) {
    if (j < t.rows) {
      if (DK) zero_row<DT>(a.dk + out, a.d);
      if (DV) zero_row<DT>(a.dv + out, a.d);
    }
    return;
  }
  const int jk = j < t.len ? j : t.len - 1;
  Held<DT, DP> k, v;
  k.load(a.k + t.k + t.head * a.k_head, a.k_tok, jk, row_bytes);
  if (DK) v.load(a.v + t.v + t.head * a.v_head, a.v_tok, jk, row_bytes);
  const int group = a.group;
  // with a causal mask only rows from the key on see it, unless it lies in the prefix
  const int from = t.first >= t.prefix ? t.first : 0;
  const int jmask = j < t.prefix ? -1 : j;
  const int n_tiles = (t.len - from + BM - 1) / BM, total = n_tiles * group;
  const float gs = DT == DT_FP16 ? *a.grad_scale : 1.0f;
  const float gs8 = gs * (DT == DT_FP16 ? 1.0f / 256.0f : 1.0f);

  Stage<DT, DP, BM> sq, sg;
  float st = 0.0f;
  const int tok = a.heads * row_bytes;
  sq.init(a.q_tok, row_bytes);
  sg.init(tok, row_bytes);
  auto load = [&](int n) {
    const int head = t.head * group + n / n_tiles, i0 = from + n % n_tiles * BM;
    sq.load(a.q + t.q + head * a.q_head + (int64_t)i0 * a.q_tok, a.q_tok, t.len - i0);
    sg.load(a.dO + ((t.row0 + i0) * a.heads + head) * row_bytes, tok, t.len - i0);
    if (threadIdx.x < 2 * BM) {
      const int r = threadIdx.x & (BM - 1);
      const bool is_lse = threadIdx.x < BM;
      // rows past the document weigh nothing: exp2(y - inf) = 0
      st = is_lse ? INFINITY : 0.0f;
      if (i0 + r < t.len) {
        const int64_t at = (int64_t)head * a.rows + t.row0 + i0 + r;
        st = is_lse ? a.lse[at] * LOG2E - SHIFT : a.delta[at];
      }
    }
  };
  load(0);
  f32x16_t dk[OT], dv[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) {
    dk[c] = zero16();
    dv[c] = zero16();
  }
  const int tr_lane = tr_lane_offset<DT, DP>();
  int buf = 0;
  for (int n = 0; n < total; n++, buf ^= 1) {
    char *const ldsq = lds + buf * 2 * TILE, *const ldsg = ldsq + TILE;
    const float *const stats = stat[buf];
    sq.store(ldsq);
    sg.store(ldsg);
    if (threadIdx.x < 2 * BM) stat[buf][threadIdx.x] = st;
    __syncthreads();
    if (n + 1 < total) load(n + 1);
    const int i0 = from + n % n_tiles * BM;
    // nothing where this wave has no keys, or where the tile's rows see none of them
    if (wave0 >= t.len || (a.causal && wave0 >= t.prefix && wave0 > i0 + BM - 1)) continue;
    const ScoreForm form = score_form<DT, MODE>(a, t.head * group + n / n_tiles);
    f32x16_t s = mma_tile<DT, DP>(ldsq, k);
    f32x16_t dp = DK ? mma_tile<DT, DP>(ldsg, v) : zero16();
    const float dist0 = (float)(i0 + 4 * h - j);
    const int hide = wave0 + 31 > i0 ? jmask - i0 - 4 * h : -1;  // rows below it do not see key j
#pragma unroll
    for (int g4 = 0; g4 < 4; g4++) {
      const f32x4_t ls = *(const f32x4_t *)(stats + 8 * g4 + 4 * h);
      const f32x4_t de = *(const f32x4_t *)(stats + BM + 8 * g4 + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int r = 4 * g4 + e;
        float keep = 1.0f;
        float y = score<DT, MODE>(form, s[r], dist0 + (float)acc_row(r), &keep);
        y = acc_row(r) < hide ? -INFINITY : y;
        s[r] = __builtin_amdgcn_exp2f(y - ls[e]);
        dp[r] = s[r] * (dp[r] - de[e]) * (MODE == ATTN_CAP ? keep * gs8 : gs8);
      }
    }
    Packed<DT> p;
    if constexpr (DV) {
      p.set(s);
#pragma unroll
      for (int c = 0; c < OT; c++) dv[c] = mma_cols<DT, DP>(ldsg, tr_lane, 0, c * 32, p, dv[c]);
    }
    if constexpr (DK) {
      p.set(dp);
#pragma unroll
      for (int c = 0; c < OT; c++) dk[c] = mma_cols<DT, DP>(ldsq, tr_lane, 0, c * 32, p, dk[c]);
    }
  }
  __syncthreads();  // the tiles' memory is free
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

}  // namespace maxsim
