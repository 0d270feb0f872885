// Attention forward: 4 waves of 32 queries each, keys in tiles through LDS.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

template <int DT, int DP> struct FwdShape {
  static constexpr int keys = DT == DT_FP32 ? 32 : 64;  // keys of a tile
  static constexpr int lds = keys * RowLayout<DT, DP>::bytes;
};

template <int N> struct Blocks { static constexpr int value = N; };

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS) attn_fwd_kernel(const AttnArgs a) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = FwdShape<DT, DP>::keys, NT = BN / 32, OT = (DP + 31) / 32;
  constexpr int TILE = FwdShape<DT, DP>::lds;
  // two buffers of a K and a V tile: one barrier a tile
  __shared__ __align__(16) char lds[4 * TILE];
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

  Stage<DT, DP, BN> sk, sv;
  sk.load(kp, a.k_tok, t.len, row_bytes);
  sv.load(vp, a.v_tok, t.len, row_bytes);
  f32x16_t acc[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  float m = -1e30f, sum = 0.0f;  // a finite start: exp2(-inf - m) is 0 for rows that see nothing yet
  const int tr_lane = TILE + tr_lane_offset<DT, L::bytes>();
  const int wave_most = visible(a, t, wave0 + 31 < t.len ? wave0 + 31 : t.len - 1);

  int buf = 0;
  for (int j0 = 0; j0 < n_keys; j0 += BN, buf ^= 2 * TILE) {
    const char *const ldsk = lds + buf, *const vt = ldsk + tr_lane;
    sk.store(lds + buf);
    sv.store(lds + buf + TILE);
    __syncthreads();
    if (j0 + BN < n_keys) {
      sk.load(kp + (int64_t)(j0 + BN) * a.k_tok, a.k_tok, t.len - j0 - BN, row_bytes);
      sv.load(vp + (int64_t)(j0 + BN) * a.v_tok, a.v_tok, t.len - j0 - BN, row_bytes);
    }
    // what one wave does with the tile's first 32 * blocks keys
    auto part = [&](auto blocks) {
      constexpr int N = decltype(blocks)::value;
      f32x16_t s[N];
#pragma unroll
      for (int n = 0; n < N; n++) s[n] = mma_tile<DT, DP>(ldsk + n * 32 * L::bytes, q);
      if constexpr (MODE != ATTN_PLAIN) {
        const float dist0 = (float)(i - j0 - 4 * h);
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
          for (int r = 0; r < 16; r++)
            s[n][r] = score<DT, MODE>(form, s[n][r], dist0 - (float)(n * 32 + acc_row(r)), nullptr);
      }
      if (j0 + BN > wave_least) {
        const int left = vis - j0 - 4 * h;
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
          for (int r = 0; r < 16; r++)
            s[n][r] = n * 32 + acc_row(r) < left ? s[n][r] : -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < N; n++)
#pragma unroll
        for (int r = 0; r < 16; r++) top = __builtin_fmaxf(top, s[n][r]);
      top = half_max(top) * post;
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
#pragma unroll
      for (int n = 0; n < N; n++) {
        Packed<DT> p;
#pragma unroll
        for (int r = 0; r < 16; r++) {
          s[n][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][r], post, -m));
          sum += s[n][r];
        }
        p.set(s[n]);
#pragma unroll
        for (int c = 0; c < OT; c++)
          acc[c] = mma_cols<DT, L::bytes>(vt, n * 32, c * 32, p, acc[c]);
      }
    };
    // 32-key blocks that no row of this wave sees (past the document or above the diagonal, or
    // all where the wave has no rows) are left out
    if (wave0 >= t.len || j0 >= wave_most) continue;
    if (NT == 1 || j0 + 32 < wave_most) part(Blocks<NT>{});
    else part(Blocks<1>{});
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
