// Attention forward: 4 waves of 32 queries each, keys in tiles of 32 through LDS. One pass over the
// keys with a running maximum m and sum of a query's weights:
//   y_j = score of key j,  w_j = exp2(y_j - m),  sum += w_j,  acc += w_j v_j,
//   o = acc / sum,  lse = (m + log2 sum) ln 2
// all in 32 bits; the weights are rounded to the inputs' 16 bits for the second product, which is
// the rounding that v has anyway (sum holds them unrounded).
//
// A wave works on two tiles at once: the next tile's scores (matrix core) beside this tile's
// exponentials, and this tile's sum of values (matrix core) beside the next tile's scale, mask and
// maximum. K is therefore used one tile ahead of V. Each has a ring of four tiles in LDS, which
// makes one barrier every two tiles enough.
//
// Measured (one MI355X): 1024 documents of 20 to 300 tokens, 12 heads of 64, bf16: 284 us, 1.0 GB in
// and out, 3.6 TB/s, 1.4 times a plain copy of it. 48 pages of about 1045 tokens, 8 heads of 256 on
// one shared, cap: 554 us, 760 TFLOP/s. Two causal documents of 5003 to 8191 tokens, 32 heads of 128
// on 8, fp16: 841 to 863 us by the GPU, 875 to 897 TFLOP/s, where a large library product reaches 1260. No single unit bounds
// the long ones: before the reads' addresses became constants, of 889 us 791 were left without LDS
// reads, 664 without the softmax, 808 without fetches. Matrix cores are busy 48% and vector units 62%
// of the cycles, at a clock that the load pulls to 1.7 GHz. Short documents spend half a wave's time
// waiting: to find its document, for the first tiles, and for the waves of its workgroup that have
// rows.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

// Waves a SIMD that the registers are divided for: as many as spill nothing, and no more than have
// room for their tiles in LDS (a workgroup's four waves are on four SIMDs), where fewer registers
// would buy nothing. The passages above take 282 us with four and 310 with three, the long documents
// 890 with two and 1095 with one. fp32 heads of 64, two by their LDS, take 514 to 524 us for 16 pages
// of 1045 tokens and 12 heads, held to the registers of three or not.
template <int DT, int DP, int MODE> struct FwdWaves {
  static constexpr int lds = 8 * 32 * RowLayout<DT, DP>::bytes;  // four tiles of K, four of V
  static constexpr int room = 160 * 1024 / lds;
  static constexpr int most = DP == 256 ? 1 : DP >= 96 ? 2 : DT != DT_FP32 && MODE == ATTN_PLAIN ? 4 : 3;
  static constexpr int value = room < most ? room : most;
  static_assert(value >= 1 && value * lds <= 160 * 1024, "waves without room for their tiles");
};

template <int DT, int DP, int MODE>
__device__ __forceinline__ void attn_fwd_tile(const AttnArgs &a, const AttnTile &t, char *lds) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = 32, OT = DP / 32, TILE = BN * L::bytes;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = uniform((int)(threadIdx.x >> 6));
  const int wave0 = t.first + wave * 32;
  const int i = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  const int iq = i < t.len ? i : t.len - 1;
  Held<DT, DP> q;
  q.load(a.q + t.q + t.head * a.q_head, a.q_tok, iq, row_bytes);
  const int kv = t.head / a.group;
  const char *kp = a.k + t.k + kv * a.k_head, *vp = a.v + t.v + kv * a.v_head;
  const ScoreForm form = score_form<DT, MODE>(a, t.head);
  // Without a bias the last factor of a score and its constant term are left to the exponentials.
  constexpr bool RAW = MODE == ATTN_PLAIN || (MODE == ATTN_CAP && staged<DT, MODE>);
  const float post = MODE == ATTN_PLAIN ? form.a : RAW ? 2.0f * form.b : 1.0f;
  const int vis = visible(a, t, iq);
  const int last = t.first + ATTN_ROWS < t.len ? t.first + ATTN_ROWS - 1 : t.len - 1;
  const int tiles = (visible(a, t, last) + BN - 1) / BN;
  // tiles that some row of this wave sees; none where the wave has no rows
  const int wave_most = visible(a, t, wave0 + 31 < t.len ? wave0 + 31 : t.len - 1);
  const int wave_tiles = wave0 < t.len ? (wave_most + BN - 1) / BN : 0;

  // Iteration n reads K's tile n + 1 and V's tile n, and fetches K's tile n + 3 and V's tile n + 2
  // into the places of K's n - 1 and V's n - 2, which no wave reads any more since the barrier
  // before iteration n (n even) or n - 1.
  const int lds_k = lds_address(lds), lds_v = lds_k + 4 * TILE;
  auto k_tile = [&](int n) { return lds + (n & 3) * TILE; };
  auto v_tile = [&](int n) { return lds + (4 + (n & 3)) * TILE; };
  // (`at` below: n, or a constant that is n modulo 4 where the rings' places shall be constants.)
  Carry<DT, DP> ck, cv;
  ck.init(a.k_tok, row_bytes);
  cv.init(a.v_tok, row_bytes);
  constexpr int C = Carry<DT, DP>::n;
  ck.start(kp, t.len);
  cv.start(vp, t.len);
  ck.all(lds_k, wave);
  ck.next();
  ck.all(lds_k + TILE, wave);
  cv.all(lds_v, wave);
  ck.next();
  ck.all(lds_k + 2 * TILE, wave);
  cv.next();
  cv.all(lds_v + TILE, wave);

  f32x16_t acc[OT], s;
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  float m = -1e30f, sum = 0.0f;  // a finite start: exp2(-inf - m) is 0 for rows that see nothing yet
  const float base0 = RAW ? form.c : 0.0f;
  float top = -INFINITY, base = base0;  // of the tile at hand
  const int row_lane = row_lane_offset<DT, DP>(), tr_lane = tr_lane_offset<DT, DP>();

  // Operands from LDS: N1 of a tile's products, N2 of its sum of values, a share of the keys after
  // the other, so that neighbours add to different accumulators.
  constexpr int N1 = L::steps, N2 = OT * Packed<DT>::n;
  auto values = [&](const Packed<DT> &p, int at, auto work) {
    const char *vt = v_tile(at);
    pipeline<N2, 4>([&](int e) { return read_cols<DT, DP>(vt, tr_lane, e % OT * 32, e / OT); },
                    [&](int e, u32x4_t v) { acc[e % OT] = mma_cols<DT>(v, p, e / OT, acc[e % OT]); }, work,
                    [](int) { return DT == DT_FP32 ? 0 : 2; });
  };
  // Tile n + 1's products and then tile n's values in one run, so that reads run ahead across.
  auto both = [&](f32x16_t &x, const Packed<DT> &p, int at, auto work) {
    const char *kt = k_tile(at + 1), *vt = v_tile(at);
    pipeline<N1 + N2, 4>(
        [&](int e) {
          return e < N1 ? read_rows<DT, DP>(kt, row_lane, e)
                        : read_cols<DT, DP>(vt, tr_lane, (e - N1) % OT * 32, (e - N1) / OT);
        },
        [&](int e, u32x4_t v) {
          const int y = e - N1;
          if (e < N1) x = mma_rows<DT>(v, q.f[e % N1], e ? x : zero16());
          else acc[y % OT] = mma_cols<DT>(v, p, y / OT, acc[y % OT]);
        },
        work, [](int e) { return DT == DT_FP32 ? 0 : e < N1 ? 1 : 2; });
  };

  // Products of tile n to scores, and their maximum, elements from .. to - 1. Where no key of the
  // tile is hidden and all lie at or before the wave's rows, the distance bias is linear in the
  // key: a constant of the lane (`base`, left to the exponential) and one of the element, which
  // joins an FMA that is there anyway.
  f32x16_t slope_row;  // slope * key, and the cap's constant term
#pragma unroll
  for (int r = 0; r < 16; r++) slope_row[r] = __builtin_fmaf(form.slope, (float)acc_row(r), form.c);
  constexpr bool LINEAR = has_bias(MODE) && (!has_cap(MODE) || staged<DT, MODE>);
  auto scores = [&](f32x16_t &x, int n, bool linear, int from, int to) {
    const float dist0 = (float)(i - n * BN - 4 * h);
    const int left = vis - n * BN - 4 * h;
    auto finish = [&](int r, float y) {
      if (!linear) y = acc_row(r) < left ? y : -INFINITY;
      top = __builtin_fmaxf(top, y);
      x[r] = y;
    };
    if constexpr (staged<DT, MODE>) {
      tanh_stages(form, x, from, to, [&](int r) {
        float y = x[r];
        if (has_bias(MODE) && linear) y = __builtin_fmaf(y, 2.0f * form.b, slope_row[r]);
        else if (has_bias(MODE)) y = score_of_tanh<MODE>(form, y, dist0 - (float)acc_row(r), form.c);
        finish(r, y);
      });
    } else {
#pragma unroll
      for (int r = from; r < to; r++) {
        float y = x[r];
        if (LINEAR && linear) y = __builtin_fmaf(y, form.a, slope_row[r]);
        else if (MODE != ATTN_PLAIN) y = score<DT, MODE>(form, y, dist0 - (float)acc_row(r), NOTHING, nullptr);
        finish(r, y);
      }
    }
  };
  // Tiles below this one are linear (keys after the rows would want the other sign of the slope;
  // they take the full form).
  const int seen_by_all = visible(a, t, wave0);
  const int linear_keys = LINEAR && form.slope != 0.0f && wave0 + 1 < seen_by_all ? wave0 + 1 : seen_by_all;
  const int linear_tiles = wave_tiles ? uniform(linear_keys / BN) : 0;
  // The tile's maximum over both halves, which differ in base.
  auto settle = [&]() { top = half_max(__builtin_fmaf(top, post, base)); };
  // The reference point of the exponentials follows the running maximum only once that is 2^8
  // away: sums and weights up to 256 lose nothing, and most tiles leave the accumulator as it is.
  auto follow = [&]() {
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
  };
  // scores to weights, not yet rounded
  auto weights = [&](f32x16_t &x, float off, int from, int to) {
#pragma unroll
    for (int r = from; r < to; r++) {
      const float w = __builtin_amdgcn_exp2f(RAW ? __builtin_fmaf(x[r], post, off) : x[r] + off);
      if (r > 0) sum += x[r - 1];  // one behind: the add does not wait for the exponential
      x[r] = w;
    }
    if (to == 16) sum += x[15];
  };
  // What iteration n begins with, and its fetches.
  int next_k = 0, next_v = 0;
  auto begin = [&](int at) {
    if ((at & 1) == 0) tile_barrier();
    ck.next();
    cv.next();
    next_k = lds_k + ((at + 3) & 3) * TILE;
    next_v = lds_v + ((at + 2) & 3) * TILE;
  };
  auto fetch = [&](int e) {
    if (e < C) ck.go(next_k, wave, e);
    else if (e < 2 * C) cv.go(next_v, wave, e - C);
  };
  auto step = [&](int n, int at, bool linear) {
    begin(at);
    follow();
    const float off = base - m;
    top = -INFINITY;
    Packed<DT> p;
    f32x16_t next;
    both(next, p, at, [&](int e) {
      fetch(e);
      if (e < N1) weights(s, off, e * 16 / N1, (e + 1) * 16 / N1);
      if (e == N1 - 1) p.set(s);
      if (e >= N1) scores(next, n + 1, linear, (e - N1) * 16 / N2, (e + 1 - N1) * 16 / N2);
    });
    base = LINEAR && linear ? -form.slope * (float)(i - (n + 1) * BN - 4 * h) : base0;
    settle();
    s = next;
  };

  tile_barrier();
  if (wave_tiles > 0) {
    s = mma_tile<DT, DP>(k_tile(0), q, zero16());
    scores(s, 0, false, 0, 16);
    settle();
  }
  // One loop for each kind of tile: merging the kinds in one would copy the accumulators.
  int n = 0;
  // Four at a time the rings' places are constants, and the reads' addresses need no additions: 844
  // in place of 891 us for the long documents. Heads of 256 gain nothing (their rings pass the 64 KB
  // that a read's offset reaches: 551 and 545 us for the pages), and with four waves it would spill.
  if constexpr (DP != 256 && FwdWaves<DT, DP, MODE>::value != 4) {
    for (; n + 4 < linear_tiles; n += 4) {
#pragma unroll
      for (int e = 0; e < 4; e++) step(n + e, e, true);
    }
  }
  for (; n + 1 < linear_tiles; n++) step(n, n, true);
  for (; n + 1 < wave_tiles; n++) step(n, n, false);
  if (wave_tiles > 0) {
    begin(n);
    follow();
    weights(s, base - m, 0, 16);
    Packed<DT> p;
    p.set(s);
    values(p, n, fetch);
    n++;
  }
  for (; n < tiles; n++) {  // nothing for this wave's rows but to fetch
    begin(n);
#pragma unroll
    for (int e = 0; e < 2 * C; e++) fetch(e);
  }
  tile_barrier();  // the tiles' memory is free
  sum = half_sum(sum);
  const bool real = i < t.len && sum > 0.0f;
  if (h == 0 && i < t.rows)
    a.lse[(int64_t)t.head * a.rows + t.row0 + i] = real ? (m + __builtin_amdgcn_logf(sum)) * LN2 : -INFINITY;
  store_rows<DT, DP>(lds + wave * TILE, acc, real ? 1.0f / sum : 0.0f,
                     a.o + ((t.row0 + wave0) * a.heads + t.head) * row_bytes,
                     (int64_t)a.heads * row_bytes, t.rows - wave0, row_bytes);
}

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS)
__attribute__((amdgpu_waves_per_eu(FwdWaves<DT, DP, MODE>::value, FwdWaves<DT, DP, MODE>::value)))
attn_fwd_kernel(const AttnArgs a) {
  __shared__ __align__(256) char lds[FwdWaves<DT, DP, MODE>::lds];
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  if (t.first < t.len) {
    attn_fwd_tile<DT, DP, MODE>(a, t, lds);
    return;
  }
  // rows without a token
  const int i = t.first + threadIdx.x;
  if (threadIdx.x < ATTN_ROWS && i < t.rows) a.lse[(int64_t)t.head * a.rows + t.row0 + i] = -INFINITY;
  zero_tile<DT>(a.o, a.heads, t, ATTN_ROWS, a.d);
}

}  // namespace maxsim
