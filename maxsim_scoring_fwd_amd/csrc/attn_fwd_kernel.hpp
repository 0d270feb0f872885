// Attention forward: 4 waves of 32 queries each, keys in tiles through LDS. The softmax's vector
// work and the matrix products of a tile take about as long as each other, so a wave works on two
// tiles at once: the next tile's scores (matrix core) beside this tile's exponentials, and this
// tile's sum of values (matrix core) beside the next tile's scale, mask and maximum. K therefore
// arrives in LDS one tile ahead of V; each has two buffers, which makes one barrier a tile enough.
#pragma once

#include "attn_common.hpp"

#ifndef ATTN_FWD_KEYS256
#define ATTN_FWD_KEYS256 32
#endif
#ifndef ATTN_FWD_KEYS
#define ATTN_FWD_KEYS 32
#endif

namespace maxsim {

template <int DT, int DP> struct FwdShape {
  static constexpr int keys = DT == DT_FP32 || DP == 128 ? 32 : DP == 256 ? ATTN_FWD_KEYS256 : ATTN_FWD_KEYS;  // keys of a tile
  static constexpr int waves = DP >= 256 ? 1 : DP >= 96 ? 2 : 3;
};

template <int N> struct From { static constexpr int value = N; };

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS)
__attribute__((amdgpu_waves_per_eu(FwdShape<DT, DP>::waves, FwdShape<DT, DP>::waves)))
attn_fwd_kernel(const AttnArgs a) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = FwdShape<DT, DP>::keys, NT = BN / 32, OT = DP / 32, TILE = BN * L::bytes;
  __shared__ __align__(256) char lds[4][TILE];  // two buffers of K, two of V
  static_assert(TILE >= 32 * L::bytes, "the result leaves through it, 32 rows a wave");
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (int)(threadIdx.x >> 6) * 32;
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

  // In iteration n, K's tile n + 2 and V's tile n + 1 are fetched into the buffers that no wave
  // reads any more. Past the last tile one row is fetched again, which keeps branches out.
  const int wave = uniform((int)(threadIdx.x >> 6));
  Carry<DT, DP, BN> ck, cv;
  ck.init(a.k_tok, row_bytes);
  cv.init(a.v_tok, row_bytes);
  auto aim = [&](auto &carry, const char *p, int tok, int n) {
    const int there = n < tiles ? n : tiles - 1;
    carry.aim(p + (int64_t)there * BN * tok, tok, n < tiles ? t.len - n * BN : 1);
  };
  aim(ck, kp, a.k_tok, 0);
  ck.all(lds[0], wave);
  aim(ck, kp, a.k_tok, 1);
  ck.all(lds[1], wave);
  aim(cv, vp, a.v_tok, 0);
  cv.all(lds[2], wave);
  tile_barrier();

  f32x16_t acc[OT], s[NT];
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  float m = -1e30f, sum = 0.0f;  // a finite start: exp2(-inf - m) is 0 for rows that see nothing yet
  float top = -INFINITY, base = 0.0f;  // of the tile at hand

  const int row_lane = row_lane_offset<DT, DP>();
  constexpr int N1 = NT * L::steps, N2 = NT * OT * 2, E = NT * 16;  // products; elements of a lane
  // Products of tile n with the keys alone, for the first tile.
  auto products = [&](f32x16_t (&x)[NT], int n) {
#pragma unroll
    for (int b = 0; b < NT; b++) x[b] = mma_tile<DT, DP>(lds[n & 1] + b * 32 * L::bytes, q, zero16());
  };
  // Tile n + 1's products and then, if VALUES, tile n's sum of values, as one run of matrix
  // instructions: work(i) beside each, i the number of the instruction. fp32 is bound by its
  // matrix instructions alone.
  auto run = [&](auto first, f32x16_t (&x)[NT], const Packed<DT> (&p)[NT], int n, auto work) {
    constexpr int F = decltype(first)::value;  // number of the first instruction: 0, or N1
    const char *kt = lds[(n + 1) & 1], *vt = lds[2 + (n & 1)];
    if constexpr (DT == DT_FP32) {
      if constexpr (F == 0) products(x, n + 1);
#pragma unroll
      for (int i = F; i < N1; i++) work(i);
#pragma unroll
      for (int b = 0; b < NT; b++)
#pragma unroll
        for (int c = 0; c < OT; c++)
          acc[c] = mma_cols<DT, DP>(vt, tr_lane, b * 32, c * 32, p[b], acc[c]);
#pragma unroll
      for (int i = N1; i < N1 + N2; i++) work(i);
    } else {
      pipeline<N1 + N2 - F, 4>(
          [&](int j) {
            const int i = j + F, y = i - N1;
            return i < N1 ? read_rows<DT, DP>(kt + i / L::steps * 32 * L::bytes, row_lane, i % L::steps)
                          // 16 keys after 16, so that neighbours add to different accumulators
                          : read_cols<DT, DP>(vt, tr_lane, y / OT / 2 * 32, y % OT * 32, y / OT % 2);
          },
          [&](int j, u32x4_t v) {
            const int i = j + F, y = i - N1;
            if (i < N1) {
              f32x16_t &c = x[i / L::steps % NT];
              c = mma_rows<DT>(v, q.f[i % L::steps], i % L::steps ? c : zero16());
            } else {
              acc[y % OT] = mma_rows<DT>(v, p[y / OT / 2].f[y / OT % 2], acc[y % OT]);
            }
          },
          [&](int j) { work(j + F); });
    }
  };
  // Products of tile n to scores, and their maximum, elements from .. to - 1. Where no key of the
  // tile is hidden and all lie on one side of the wave's rows, the distance bias is linear in the
  // key: a constant of the lane (`base`, left to the exponential) and one of the element, which
  // joins an FMA that is there anyway.
  f32x16_t slope_row;  // slope * key, and the cap's constant term
#pragma unroll
  for (int r = 0; r < 16; r++) slope_row[r] = __builtin_fmaf(form.slope, (float)acc_row(r), form.b);
  constexpr bool LINEAR = MODE == ATTN_BIAS || (MODE == ATTN_CAP && DT != DT_FP32);
  auto scores = [&](f32x16_t (&x)[NT], int n, bool linear, int from, int to) {
    const float dist0 = (float)(i - n * BN - 4 * h);
    const int left = vis - n * BN - 4 * h;
#pragma unroll
    for (int e = from; e < to; e++) {
      float y = x[e / 16][e % 16];
      const int b = e / 16 * 32, key = b + acc_row(e % 16);
      const float far = b ? slope_row[e % 16] + form.slope * (float)b : slope_row[e % 16];
      if (LINEAR && linear) {
        if (MODE == ATTN_CAP)
          y = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y * form.a)) * (-2.0f * form.b) + far;
        else
          y = __builtin_fmaf(y, form.a, far);
      } else if (MODE != ATTN_PLAIN) {
        y = score<DT, MODE>(form, y, dist0 - (float)key, nullptr);
      }
      if (!linear) y = key < left ? y : -INFINITY;
      top = __builtin_fmaxf(top, y);
      x[e / 16][e % 16] = y;
    }
  };
  // Tile n is linear: nothing hidden, and all keys at or before the wave's rows (the far side,
  // keys after the rows, would want the other sign: it takes the full form).
  auto linear_at = [&](int n) {
    const int end = (n + 1) * BN;
    return end <= wave_least && (!LINEAR || end <= wave0 + 1 || form.slope == 0.0f);
  };
  // scores to weights, not yet rounded
  auto weights = [&](f32x16_t (&x)[NT], float off, int from, int to) {
#pragma unroll
    for (int e = from; e < to; e++) {
      const float w = __builtin_amdgcn_exp2f(MODE == ATTN_PLAIN ? __builtin_fmaf(x[e / 16][e % 16], post, off)
                                                                : x[e / 16][e % 16] + off);
      sum += w;
      x[e / 16][e % 16] = w;
    }
  };
  if (wave_tiles > 0) {
    products(s, 0);
    scores(s, 0, false, 0, E);
    top = half_max(top) * post;
  }
  for (int n = 0; n < tiles; n++) {
    tile_barrier();
    aim(ck, kp, a.k_tok, n + 2);
    aim(cv, vp, a.v_tok, n + 1);
    constexpr int C = Carry<DT, DP, BN>::n;
    auto fetch = [&](int i) {
      if (i < C) ck.go(lds[n & 1], wave, i);
      else if (i < 2 * C) cv.go(lds[2 + ((n + 1) & 1)], wave, i - C);
    };
    if (n >= wave_tiles) {  // nothing for this wave's rows but to fetch
#pragma unroll
      for (int i = 0; i < 2 * C; i++) fetch(i);
      continue;
    }
    // The reference point of the exponentials follows the running maximum only once that is
    // 2^8 away: sums and weights up to 256 lose nothing, and most tiles leave the accumulator
    // as it is.
    if (__builtin_amdgcn_ballot_w64(top > m + 8.0f)) {
      const float mn = __builtin_fmaxf(m, top);
      const float f = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      sum *= f;
#pragma unroll
      for (int c = 0; c < OT; c++)
#pragma unroll
        for (int r = 0; r < 16; r++) acc[c][r] *= f;
    }
    const float off = base - m;
    Packed<DT> p[NT];
    f32x16_t next[NT];
    if (n + 1 == wave_tiles) {
      weights(s, off, 0, E);
#pragma unroll
      for (int b = 0; b < NT; b++) p[b].set(s[b]);
      run(From<N1>{}, next, p, n, [&](int i) { fetch(i - N1); });
      continue;
    }
    top = -INFINITY;
    auto step = [&](bool linear) {
      run(From<0>{}, next, p, n, [&](int i) {
        fetch(i);
        if (i < N1) weights(s, off, i * E / N1, (i + 1) * E / N1);
        if (i == N1 - 1) {
#pragma unroll
          for (int b = 0; b < NT; b++) p[b].set(s[b]);
        }
        if (i >= N1) scores(next, n + 1, linear, (i - N1) * E / N2, (i + 1 - N1) * E / N2);
      });
    };
    // (the marks keep the compiler from moving the two copies' common start, and with it the
    // vector work beside the first matrix instructions, before the branch)
    if (linear_at(n + 1)) {
      asm volatile("; linear");
      step(true);
      base = LINEAR ? -form.slope * (float)(i - (n + 1) * BN - 4 * h) : 0.0f;
    } else {
      asm volatile("; full");
      step(false);
      base = 0.0f;
    }
    top = half_max(__builtin_fmaf(top, post, base));  // the halves differ in base
#pragma unroll
    for (int b = 0; b < NT; b++) s[b] = next[b];
  }
  sum = half_sum(sum);
  const bool real = i < t.len && sum > 0.0f;
  tile_barrier();  // the tiles' memory is free
  if (h == 0 && i < t.rows) *lse = real ? (m + __builtin_amdgcn_logf(sum)) * LN2 : -INFINITY;
  store_rows<DT, DP>(lds[threadIdx.x >> 6], acc, real ? 1.0f / sum : 0.0f,
                     a.o + ((t.row0 + wave0) * a.heads + t.head) * row_bytes,
                     (int64_t)a.heads * row_bytes, t.rows - wave0, row_bytes);
}

}  // namespace maxsim
