// Attention backward, after <dO, o> per row (attn_delta.hpp): dQ (keys in tiles, one wave on 32 queries) and
// dK / dV (queries in tiles, one wave on 32 keys, all heads that share them). The scores are
// computed again in both: 7 products instead of 5, but every sum has one owner, so there are no
// atomics and repeated calls give the same bits. With P the weights exp(y - lse), recomputed:
//   dP = dO V^T,  dS = P (dP - delta) * (the cap's slope),  dQ = scale dS K,  dK = scale dS^T Q,
//   dV = P^T dO
// Sums are 32 bits wide; P and dS are rounded to the inputs' type as operands of the last three
// products (fp16 after a power of two that keeps dS in range).
//
// Measured (one MI355X): 512 documents of 20 to 300 tokens, 12 heads of 64, bf16: dQ 179 us, dK / dV
// 265 us, 0.63 and 0.76 GB, 3.5 and 2.9 TB/s; 16 pages of about 1045 tokens, 16 heads of 128 on 4,
// with cap: dQ 234 us, dK / dV 304 us, 900 and 920 TFLOP/s, 41 and 38% of what the matrix cores do
// at the clock of these passes. Instructions bound the pages (32 matrix instructions and 255 others a
// tile of dK / dV, one wave a SIMD), waits the short documents.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

template <int DT, int DP, int MODE>
__device__ __forceinline__ void attn_dq_tile(const AttnArgs &a, const AttnTile &t, char *lds) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = 32, OT = DP / 32, TILE = BN * L::bytes;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = uniform((int)(threadIdx.x >> 6));
  const int wave0 = t.first + wave * 32;
  const int i = wave0 + (lane & 31);
  const int row_bytes = a.d * L::eb;
  const int iq = i < t.len ? i : t.len - 1;
  Held<DT, DP> q, g;
  q.load(a.q + t.q + t.head * a.q_head, a.q_tok, iq, row_bytes);
  g.load(a.dO + (t.row0 * a.heads + t.head) * row_bytes, (int64_t)a.heads * row_bytes, iq, row_bytes);
  const int kv = t.head / a.group;
  const char *kp = a.k + t.k + kv * a.k_head, *vp = a.v + t.v + kv * a.v_head;
  const ScoreForm form = score_form<DT, MODE>(a, t.head);
  const int vis = visible(a, t, iq);
  const int last = t.first + ATTN_ROWS < t.len ? t.first + ATTN_ROWS - 1 : t.len - 1;
  const int tiles = (visible(a, t, last) + BN - 1) / BN;
  const int wave_most = visible(a, t, wave0 + 31 < t.len ? wave0 + 31 : t.len - 1);
  const int wave_tiles = wave0 < t.len ? (wave_most + BN - 1) / BN : 0;
  const int whole_tiles = wave0 < t.len ? visible(a, t, wave0) / BN : 0;  // nothing hidden in them
  const int64_t at = (int64_t)t.head * a.rows + t.row0 + iq;
  const float start = form.c - a.lse[at] * LOG2E, delta = -a.stats[at].y;
  constexpr float UNIT = slope_unit<DT, MODE>;
  const float gs = DT == DT_FP16 ? *a.grad_scale : 1.0f;

  // Rings of four tiles, as in the forward: tile n + 2 is fetched in iteration n.
  const int lds_k = lds_address(lds), lds_v = lds_k + 4 * TILE;
  Carry<DT, DP> ck, cv;
  ck.init(a.k_tok, row_bytes);
  cv.init(a.v_tok, row_bytes);
  constexpr int P = 2 * Carry<DT, DP>::n;
  auto fetch = [&](int n, int from, int to) {  // pieces of tile n
#pragma unroll
    for (int e = from; e < to; e++) {
      if (e & 1) cv.go(lds_v + (n & 3) * TILE, wave, e / 2);
      else ck.go(lds_k + (n & 3) * TILE, wave, e / 2);
    }
  };
  ck.start(kp, t.len);
  cv.start(vp, t.len);
  fetch(0, 0, P);
  ck.next();
  cv.next();
  fetch(1, 0, P);
  f32x16_t acc[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) acc[c] = zero16();
  const int row_lane = row_lane_offset<DT, DP>(), tr_lane = tr_lane_offset<DT, DP>();
  constexpr int A = L::steps, K = Packed<DT>::n, C = OT * K;

  auto begin = [&](int n, int at) {
    if (n > 0 && (at & 1) == 0) tile_barrier();
    ck.next();
    cv.next();
  };
  // at: n, or a constant that is n modulo 4
  auto tile = [&](int n, int at, bool masked) {
    begin(n, at);
    const char *const ldsk = lds + (at & 3) * TILE, *const ldsv = ldsk + 4 * TILE;
    const float dist0 = (float)(i - n * BN - 4 * h);
    const int left = vis - n * BN - 4 * h;
    f32x16_t s, dp;
    Packed<DT> p;
    // products to weights, times the cap's slope where there is one
    f32x16_t slope;  // of the cap
    auto weight = [&](int r, float y) {
      if (masked) y = acc_row(r) < left ? y : -INFINITY;
      s[r] = __builtin_amdgcn_exp2f(y);
    };
    auto scaled = [&](int r) {
      if (has_cap(MODE)) s[r] *= slope[r];
      if (DT == DT_FP16) s[r] *= gs * UNIT;
    };
    auto weights = [&](int from, int to) {
      if constexpr (staged<DT, MODE>) {
        tanh_stages(form, s, from, to, [&](int r) {
          if (r > 0) scaled(r - 1);
          slope[r] = slope_of_tanh(s[r]);
          weight(r, score_of_tanh<MODE>(form, s[r], dist0 - (float)acc_row(r), start));
          if (r == 15) scaled(15);
        });
      } else {
#pragma unroll
        for (int r = from; r < to; r++) {
          float keep = 1.0f;
          weight(r, score<DT, MODE>(form, s[r], dist0 - (float)acc_row(r), start, &keep));
          slope[r] = keep;
          scaled(r);
        }
      }
    };
    auto grads = [&](int from, int to) {
#pragma unroll
      for (int r = from; r < to; r++) dp[r] = s[r] * (dp[r] - delta);
    };
    auto read = [&](int j) {
      return j < A       ? read_rows<DT, DP>(ldsk, row_lane, j)
             : j < 2 * A ? read_rows<DT, DP>(ldsv, row_lane, j - A)
                         : read_cols<DT, DP>(ldsk, tr_lane, (j - 2 * A) % OT * 32, (j - 2 * A) / OT);
    };
    auto mma = [&](int j, u32x4_t x) {
      const int y = j - 2 * A;
      if (j < A) s = mma_rows<DT>(x, q.f[j % A], j ? s : zero16());
      else if (j < 2 * A) dp = mma_rows<DT>(x, g.f[j % A], j > A ? dp : zero16());
      else acc[y % OT] = mma_cols<DT>(x, p, y / OT, acc[y % OT]);
    };
    auto work = [&](int j) {
      if (j < A) fetch(at + 2, j * P / A, (j + 1) * P / A);
      else if (j < 2 * A) weights((j - A) * 16 / A, (j + 1 - A) * 16 / A);
      if (j == 2 * A - 1) {
        grads(0, 16);
        p.set(dp);
      }
    };
    auto reads = [](int j) { return DT == DT_FP32 ? 0 : j < 2 * A ? 1 : 2; };
    if constexpr (DP > 128) {  // in two, or it is too long for the compiler to unroll
      pipeline<2 * A, 4>(read, mma, work, reads);
      pipeline<C, 4>([&](int j) { return read(2 * A + j); }, [&](int j, u32x4_t x) { mma(2 * A + j, x); },
                     [](int) {}, [&](int j) { return reads(2 * A + j); });
    } else {
      pipeline<2 * A + C, 4>(read, mma, work, reads);
    }
  };
  tile_barrier();
  int n = 0;
  if constexpr (DP <= 128) {  // as in the forward: constant places, 136 vector instructions to 125
    for (; n + 4 <= whole_tiles; n += 4) {
#pragma unroll
      for (int e = 0; e < 4; e++) tile(n + e, e, false);
    }
  }
  for (; n < whole_tiles; n++) tile(n, n, false);
  for (; n < wave_tiles; n++) tile(n, n, true);
  for (; n < tiles; n++) {  // nothing for this wave's rows but to fetch
    begin(n, n);
    fetch(n + 2, 0, P);
  }
  tile_barrier();  // the tiles' memory is free
  store_rows<DT, DP>(lds + wave * TILE, acc, i < t.len ? (DT == DT_FP16 ? a.scale / gs : a.scale * UNIT) : 0.0f,
                     a.dq + ((t.row0 + wave0) * a.heads + t.head) * row_bytes,
                     (int64_t)a.heads * row_bytes, t.rows - wave0, row_bytes);
}

template <int DT, int DP, int MODE>
__global__ void __launch_bounds__(ATTN_THREADS) attn_dq_kernel(const AttnArgs a) {
  __shared__ __align__(256) char lds[8 * 32 * RowLayout<DT, DP>::bytes];  // two rings of four tiles
  AttnTile t;
  if (!locate(a, ATTN_ROWS, t)) return;
  if (t.first < t.len) attn_dq_tile<DT, DP, MODE>(a, t, lds);
  else zero_tile<DT>(a.dq, a.heads, t, ATTN_ROWS, a.d);
}

// WHAT: 1 for dK, 2 for dV, 3 for both. Heads wider than 128 take a launch for each: a wave has no
// registers for both sums, and computing the scores again costs less than spilling.
template <int DT, int DP, int MODE, int WHAT>
__device__ __forceinline__ void attn_dkv_tile(const AttnArgs &a, const AttnTile &t, char *lds, float *stat) {
  using L = RowLayout<DT, DP>;
  constexpr int BM = 32, OT = DP / 32, TILE = BM * L::bytes;
  constexpr bool DK = WHAT & 1, DV = WHAT & 2;
  constexpr float SHIFT = DT == DT_FP16 ? ATTN_WEIGHT_SHIFT : 0.0f;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave = uniform((int)(threadIdx.x >> 6));
  const int wave0 = t.first + wave * 32;
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
  const float gs = DT == DT_FP16 ? *a.grad_scale : 1.0f;
  constexpr float UNIT = slope_unit<DT, MODE>;
  const float gs8 = gs * __builtin_amdgcn_exp2f(-SHIFT) * UNIT;

  // Rings of four tiles as in the other kernels, the rows of one head after the other's, with the
  // rows' statistics beside them.
  const int lds_q = lds_address(lds), lds_g = lds_q + 4 * TILE, lds_s = lds_address((const char *)stat);
  Carry<DT, DP> cq, cg;
  const int tok = a.heads * row_bytes;
  cq.init(a.q_tok, row_bytes);
  cg.init(tok, row_bytes);
  const int end_head = (t.head + 1) * group;
  int next_head = t.head * group;  // of the tile that is fetched next
  uint64_t next_stats;
  auto start_head = [&]() {
    cq.start(a.q + t.q + next_head * a.q_head + (int64_t)from * a.q_tok, t.len - from);
    cg.start(a.dO + ((t.row0 + from) * a.heads + next_head) * row_bytes, t.len - from);
    next_stats = (uint64_t)(uintptr_t)(a.stats + (int64_t)next_head * a.rows + t.row0 + from);
  };
  auto next = [&]() {
    if (cq.left <= BM && next_head + 1 < end_head) {
      next_head++;
      start_head();
    } else {
      next_stats += cq.left > BM ? BM * sizeof(float2) : 0;
      cq.next();
      cg.next();
    }
  };
  constexpr int P = 2 * Carry<DT, DP>::n;
  auto fetch = [&](int n, int first, int to) {  // pieces of tile n
#pragma unroll
    for (int e = first; e < to; e++) {
      if (e & 1) cg.go(lds_g + (n & 3) * TILE, wave, e / 2);
      else cq.go(lds_q + (n & 3) * TILE, wave, e / 2);
    }
  };
  auto fetch_stats = [&](int n) {  // 32 pairs to 32 first and 32 second halves, a lane of wave 0 each
    if (wave == 0) {
      const int last = cq.left < BM ? cq.left - 1 : BM - 1, row = lane & 31;
      const uint32_t at = (uint32_t)(row < last ? row : last) * 8 + h * 4;
      asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, %2"
                   :
                   : "{m0}"(uniform(lds_s + (n & 3) * 256)), "v"(at), "s"(uniform((int64_t)next_stats)));
    }
  };
  start_head();
  fetch(0, 0, P);
  fetch_stats(0);
  next();
  fetch(1, 0, P);
  fetch_stats(1);
  f32x16_t dk[OT], dv[OT];
#pragma unroll
  for (int c = 0; c < OT; c++) {
    dk[c] = zero16();
    dv[c] = zero16();
  }
  const int row_lane = row_lane_offset<DT, DP>(), tr_lane = tr_lane_offset<DT, DP>();
  // operands of the four products
  constexpr int A = L::steps, B = DK ? A : 0, K = Packed<DT>::n, C = DV ? OT * K : 0, D = DK ? OT * K : 0;

  int n = 0;  // tiles done
  auto begin = [&](int at) {
    if (n > 0 && (at & 1) == 0) tile_barrier();
    next();
    fetch_stats(at + 2);
  };
  // at: n, or a constant that is n modulo 4
  auto tile = [&](const ScoreForm &form, int i0, int at, bool masked) {
    begin(at);
    const char *const ldsq = lds + (at & 3) * TILE, *const ldsg = ldsq + 4 * TILE;
    const f32x4_t *const stats = (const f32x4_t *)(stat + (at & 3) * 64 + 4 * h);
    const float dist0 = (float)(i0 + 4 * h - j);
    const int hide = jmask - i0 - 4 * h;   // rows below it do not see key j
    const int there = t.len - i0 - 4 * h;  // rows from it on do not exist
    f32x16_t s, dp;
    Packed<DT> pv, pk;
    // The sums start from the rows' statistics: dP from -delta, S from -lse / scale, so that
    // neither is subtracted (nor held) afterwards. The tanh wants S itself.
    f32x16_t lse;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const f32x4_t y = stats[2 * e], z = stats[2 * e + 8];  // rows 8 e + 4 h + 0 .. 3
#pragma unroll
      for (int g = 0; g < 4; g++) {
        lse[4 * e + g] = y[g];
        dp[4 * e + g] = z[g];
      }
    }
    s = has_cap(MODE) ? zero16() : lse;
    f32x16_t slope;  // of the cap
    auto weight = [&](int r, float y) {
      if (masked) y = acc_row(r) < hide || acc_row(r) >= there ? -INFINITY : y;
      s[r] = __builtin_amdgcn_exp2f(y);
    };
    auto weights = [&](int first, int to) {
      if constexpr (staged<DT, MODE>) {
        tanh_stages(form, s, first, to, [&](int r) {
          slope[r] = slope_of_tanh(s[r]);
          weight(r, score_of_tanh<MODE>(form, s[r], dist0 + (float)acc_row(r), lse[r]));
        });
      } else {
#pragma unroll
        for (int r = first; r < to; r++) {
          float keep = 1.0f;
          weight(r, score<DT, MODE>(form, s[r], dist0 + (float)acc_row(r), has_cap(MODE) ? lse[r] : NOTHING, &keep));
          slope[r] = keep;
        }
      }
    };
    auto grads = [&](int first, int to) {
#pragma unroll
      for (int r = first; r < to; r++) {
        dp[r] = s[r] * dp[r];
        if (has_cap(MODE)) dp[r] *= slope[r];
        if (DT == DT_FP16) dp[r] *= gs8;
      }
    };
    // S, then dP beside the weights, then dV beside dS, then dK; the next tile's fetch beside S
    auto read = [&](int e) {
      if (e < A) return read_rows<DT, DP>(ldsq, row_lane, e);
      if (e < A + B) return read_rows<DT, DP>(ldsg, row_lane, e - A);
      const int x = e < A + B + C ? e - A - B : e - A - B - C;
      return read_cols<DT, DP>(e < A + B + C ? ldsg : ldsq, tr_lane, x % OT * 32, x / OT);
    };
    auto mma = [&](int e, u32x4_t x) {
      if (e < A) {
        s = mma_rows<DT>(x, k.f[e % A], s);
      } else if (e < A + B) {
        dp = mma_rows<DT>(x, v.f[(e - A) % A], dp);
      } else if (e < A + B + C) {
        const int y = e - A - B;
        dv[y % OT] = mma_cols<DT>(x, pv, y / OT, dv[y % OT]);
      } else {
        const int y = e - A - B - C;
        dk[y % OT] = mma_cols<DT>(x, pk, y / OT, dk[y % OT]);
      }
    };
    auto work = [&](int e) {
      if constexpr (DK) {
        if (e >= A && e < A + B) weights((e - A) * 16 / A, (e + 1 - A) * 16 / A);
      } else if (e == A - 1) {
        weights(0, 16);
      }
      if (DV && e == A + B - 1) pv.set(s);
      if constexpr (DK && DV) {
        if (e >= A + B && e < A + B + C) grads((e - A - B) * 16 / C, (e + 1 - A - B) * 16 / C);
        if (e == A + B + C - 1) pk.set(dp);
      } else if (DK && e == A + B - 1) {
        grads(0, 16);
        pk.set(dp);
      }
      if (e < A) fetch(at + 2, e * P / A, (e + 1) * P / A);
    };
    auto reads = [](int e) { return DT == DT_FP32 ? 0 : e < A + B ? 1 : 2; };
    if constexpr (DT == DT_FP32 || DP > 128) {  // in two, or it is too long for the compiler to unroll
      pipeline<A + B, 4>(read, mma, work, reads);
      pipeline<C + D, 4>([&](int e) { return read(A + B + e); }, [&](int e, u32x4_t x) { mma(A + B + e, x); },
                         [&](int e) { work(A + B + e); }, [&](int e) { return reads(A + B + e); });
    } else {
      pipeline<A + B + C + D, 4>(read, mma, work, reads);
    }
    n++;
  };
  tile_barrier();
  // One loop for each kind of tile: merging the kinds in one would copy the accumulators. Rows that
  // see none of the wave's keys come first, then those that see some of them.
  const int hidden_rows = wave0 >= t.len ? t.len : a.causal && wave0 >= t.prefix ? wave0 : 0;
  const int some_rows = a.causal && wave0 + 31 >= t.prefix ? wave0 + 31 : 0;
  for (int head = t.head * group; head < end_head; head++) {
    const ScoreForm form = score_form<DT, MODE>(a, head);
    int i0 = from;
    for (; i0 < t.len && i0 + BM - 1 < hidden_rows; i0 += BM) {
      begin(n);
      fetch(n + 2, 0, P);
      n++;
    }
    if (wave0 >= t.len) {
      if (i0 < t.len) {
        begin(n);
        fetch(n + 2, 0, P);
        n++;
      }
      continue;
    }
    for (; i0 < t.len && i0 < some_rows; i0 += BM) tile(form, i0, n, true);
    // As in the forward: constant places, 145 vector instructions to 128 for heads of 128; with dQ's,
    // training on the pages takes 775 in place of 802 us, and the backward pass of 16 pages with heads
    // of 64 347 in place of 359. Heads of 96, and fp32's of 64, have no registers to spare.
    if constexpr (DP == 128 || (DP == 64 && DT != DT_FP32)) {
      for (; i0 + BM <= t.len && (n & 3); i0 += BM) tile(form, i0, n, false);
      for (; i0 + 4 * BM <= t.len; i0 += 4 * BM) {
#pragma unroll
        for (int e = 0; e < 4; e++) tile(form, i0 + e * BM, e, false);
      }
    }
    for (; i0 + BM <= t.len; i0 += BM) tile(form, i0, n, false);
    if (i0 < t.len) tile(form, i0, n, true);
  }
  tile_barrier();  // the tiles' memory is free
  const int64_t first = ((t.row0 + wave0) * a.kv_heads + t.head) * row_bytes;
  const int64_t stride = (int64_t)a.kv_heads * row_bytes;
  char *const mine = lds + wave * TILE;
  const bool real = j < t.len;
  if constexpr (DK)
    store_rows<DT, DP>(mine, dk, real ? (DT == DT_FP16 ? a.scale / gs : a.scale * UNIT) : 0.0f, a.dk + first, stride, t.rows - wave0, row_bytes);
  if constexpr (DV)
    store_rows<DT, DP>(mine, dv, real ? __builtin_amdgcn_exp2f(-SHIFT) : 0.0f, a.dv + first, stride,
                       t.rows - wave0, row_bytes);
}

// Waves a SIMD: left to itself the compiler takes a few registers more than the 256 of two waves for
// 16-bit heads of 96 with a cap. Held to them, fp16 with cap and bias spills one; dK / dV of 16 pages
// of 1060 tokens with 8 heads take 210 us so and 247 with one wave, of 256 documents of 300 with 12
// heads 575 and 818, of two of 4000 with 16 on 4 580 and 568. The other forms fit or miss by far
// (heads of 128 would spill 75 and more), and holding them costs 1 to 3%.
template <int DT, int DP, int MODE> struct DkvWaves {
  static constexpr int value = DT != DT_FP32 && DP == 96 && staged<DT, MODE> ? 2 : 1;
};

template <int DT, int DP, int MODE, int WHAT>
__global__ void __launch_bounds__(ATTN_THREADS) __attribute__((amdgpu_waves_per_eu(DkvWaves<DT, DP, MODE>::value)))
attn_dkv_kernel(const AttnArgs a) {
  __shared__ __align__(256) char lds[8 * 32 * RowLayout<DT, DP>::bytes];  // two rings of four tiles
  __shared__ __align__(256) float stat[4 * 64];
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
