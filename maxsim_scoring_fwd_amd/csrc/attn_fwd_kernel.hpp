// Attention forward: 4 waves of 32 * CB queries each, keys in tiles of 32 through LDS.
//
// The softmax's vector work and the matrix products of a tile take about as long as each other,
// so a wave works on two tiles at once: the next tile's scores (matrix core) beside this tile's
// exponentials, and this tile's sum of values (matrix core) beside the next tile's scale, mask and
// maximum. K therefore arrives in LDS one tile ahead of V; each has two buffers, which makes one
// barrier a tile enough.
//
// CB = 2 reads a key's or a value's operand from LDS once for 64 queries: the transposing reads
// leave LDS at 128 bytes a clock, four waves that use each for one matrix instruction want that.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

// Waves a SIMD that the registers are divided for.
template <int DP, int CB> struct FwdWaves {
  static constexpr int value = DP == 256 ? 1 : CB == 2 ? (DP >= 96 ? 1 : 2) : DP >= 96 ? 2 : 3;
};

template <int DT, int DP, int MODE, int CB>
__device__ __forceinline__ void attn_fwd_tile(const AttnArgs &a, const AttnTile &t,
                                              char (*lds)[32 * RowLayout<DT, DP>::bytes]) {
  using L = RowLayout<DT, DP>;
  constexpr int BN = 32, OT = DP / 32, TILE = BN * L::bytes, RB = 32 * CB;
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int wave0 = t.first + (int)(threadIdx.x >> 6) * RB;
  const int i = wave0 + (lane & 31);  // this lane's row of block 0; block b has i + 32 b
  const int row_bytes = a.d * L::eb;
  float *const lse = a.lse + (int64_t)t.head * a.rows + t.row0 + i;
  const char *const qp = a.q + t.q + t.head * a.q_head;
  Held<DT, DP> q[CB];
  int vis[CB];
#pragma unroll
  for (int b = 0; b < CB; b++) {
    const int iq = i + 32 * b < t.len ? i + 32 * b : t.len - 1;
    q[b].load(qp, a.q_tok, iq, row_bytes);
    vis[b] = visible(a, t, iq);
  }
  const int kv = t.head / a.group;
  const char *kp = a.k + t.k + kv * a.k_head, *vp = a.v + t.v + kv * a.v_head;
  const ScoreForm form = score_form<DT, MODE>(a, t.head);
  const float post = MODE == ATTN_PLAIN ? form.a : 1.0f;  // factor left to the exponentials
  const int wave_least = visible(a, t, wave0);
  const int last = t.first + 4 * RB < t.len ? t.first + 4 * RB - 1 : t.len - 1;
  const int tiles = (visible(a, t, last) + BN - 1) / BN;
  // tiles that some row of this wave sees; none where the wave has no rows
  const int wave_most = visible(a, t, wave0 + RB - 1 < t.len ? wave0 + RB - 1 : t.len - 1);
  const int wave_tiles = wave0 < t.len ? (wave_most + BN - 1) / BN : 0;

  // In iteration n, V's tile n + 1 and K's tile n + 2 are fetched into the buffers that no wave
  // reads any more. Past the last tile one row is fetched again, which keeps branches out.
  const int wave = uniform((int)(threadIdx.x >> 6));
  Carry<DT, DP, BN> ck, cv;
  ck.init(a.k_tok, row_bytes);
  cv.init(a.v_tok, row_bytes);
  constexpr int C = Carry<DT, DP, BN>::n;
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

  f32x16_t acc[CB][OT], s[CB];
  // a finite start of m: exp2(-inf - m) is 0 for rows that see nothing yet
  float m[CB], sum[CB], top[CB], base = 0.0f;  // top, base: of the tile at hand
#pragma unroll
  for (int b = 0; b < CB; b++) {
    m[b] = -1e30f;
    sum[b] = 0.0f;
    top[b] = -INFINITY;
#pragma unroll
    for (int c = 0; c < OT; c++) acc[b][c] = zero16();
  }
  const int row_lane = row_lane_offset<DT, DP>(), tr_lane = tr_lane_offset<DT, DP>();

  // Matrix instructions' operands from LDS: N1 of a tile's products, N2 of its sum of values, 16
  // keys after 16, so that neighbours add to different accumulators. fp32 is bound by its matrix
  // instructions alone and has none of this.
  constexpr int N1 = L::steps, N2 = OT * 2;
  auto product = [&](f32x16_t (&x)[CB], int e, u32x4_t v) {
#pragma unroll
    for (int b = 0; b < CB; b++) x[b] = mma_rows<DT>(v, q[b].f[e], e ? x[b] : zero16());
  };
  auto value = [&](const Packed<DT> (&p)[CB], int e, u32x4_t v) {
#pragma unroll
    for (int b = 0; b < CB; b++) acc[b][e % OT] = mma_rows<DT>(v, p[b].f[e / OT], acc[b][e % OT]);
  };
  auto products = [&](f32x16_t (&x)[CB], int n, auto work) {
    if constexpr (DT == DT_FP32) {
#pragma unroll
      for (int b = 0; b < CB; b++) x[b] = mma_tile<DT, DP>(lds[n & 1], q[b], zero16());
#pragma unroll
      for (int e = 0; e < N1; e++) work(e);
    } else {
      pipeline<N1, 4>([&](int e) { return read_rows<DT, DP>(lds[n & 1], row_lane, e); },
                      [&](int e, u32x4_t v) { product(x, e, v); }, work);
    }
  };
  auto values = [&](const Packed<DT> (&p)[CB], int n, auto work) {
    const char *vt = lds[2 + (n & 1)];
    if constexpr (DT == DT_FP32) {
#pragma unroll
      for (int b = 0; b < CB; b++)
#pragma unroll
        for (int c = 0; c < OT; c++) acc[b][c] = mma_cols<DT, DP>(vt, tr_lane, 0, c * 32, p[b], acc[b][c]);
#pragma unroll
      for (int e = 0; e < N2; e++) work(e);
    } else {
      pipeline<N2, 4>([&](int e) { return read_cols<DT, DP>(vt, tr_lane, 0, e % OT * 32, e / OT); },
                      [&](int e, u32x4_t v) { value(p, e, v); }, work);
    }
  };
  // Tile n + 1's products and then tile n's values in one run, so that reads run ahead across.
  auto both = [&](f32x16_t (&x)[CB], const Packed<DT> (&p)[CB], int n, auto work) {
    if constexpr (DT == DT_FP32) {
      products(x, n + 1, work);
      values(p, n, [&](int e) { work(N1 + e); });
    } else {
      const char *kt = lds[(n + 1) & 1], *vt = lds[2 + (n & 1)];
      pipeline<N1 + N2, 4>(
          [&](int e) {
            return e < N1 ? read_rows<DT, DP>(kt, row_lane, e)
                          : read_cols<DT, DP>(vt, tr_lane, 0, (e - N1) % OT * 32, (e - N1) / OT);
          },
          [&](int e, u32x4_t v) {
            if (e < N1) product(x, e, v);
            else value(p, e - N1, v);
          },
          work);
    }
  };

  // Products of tile n to scores, and their maximum, elements from .. to - 1 of every block. Where
  // no key of the tile is hidden and all lie at or before the wave's rows, the distance bias is
  // linear in the key: a constant of the lane (`base`, left to the exponential; the same for every
  // block but for 32 slope b) and one of the element, which joins an FMA that is there anyway.
  f32x16_t slope_row;  // slope * key, and the cap's constant term
#pragma unroll
  for (int r = 0; r < 16; r++) slope_row[r] = __builtin_fmaf(form.slope, (float)acc_row(r), form.b);
  constexpr bool LINEAR = MODE == ATTN_BIAS || (MODE == ATTN_CAP && DT != DT_FP32);
  auto scores = [&](f32x16_t (&x)[CB], int n, bool linear, int from, int to) {
#pragma unroll
    for (int b = 0; b < CB; b++) {
      const float dist0 = (float)(i + 32 * b - n * BN - 4 * h);
      const int left = vis[b] - n * BN - 4 * h;
#pragma unroll
      for (int r = from; r < to; r++) {
        float y = x[b][r];
        if (LINEAR && linear) {
          if (MODE == ATTN_CAP)
            y = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y * form.a)) * (-2.0f * form.b) + slope_row[r];
          else
            y = __builtin_fmaf(y, form.a, slope_row[r]);
        } else if (MODE != ATTN_PLAIN) {
          y = score<DT, MODE>(form, y, dist0 - (float)acc_row(r), nullptr);
        }
        if (!linear) y = acc_row(r) < left ? y : -INFINITY;
        top[b] = __builtin_fmaxf(top[b], y);
        x[b][r] = y;
      }
    }
  };
  // Keys after the rows would want the other sign of the slope: such tiles take the full form.
  auto linear_at = [&](int n) {
    const int end = (n + 1) * BN;
    return end <= wave_least && (!LINEAR || end <= wave0 + 1 || form.slope == 0.0f);
  };
  auto base_of = [&](int n) { return LINEAR ? -form.slope * (float)(i - n * BN - 4 * h) : 0.0f; };
  auto block_base = [&](int b) { return LINEAR && b && base != 0.0f ? base - form.slope * 32.0f * b : base; };
  auto settle = [&]() {  // the tile's maximum over both halves, which differ in base
#pragma unroll
    for (int b = 0; b < CB; b++) top[b] = half_max(__builtin_fmaf(top[b], post, block_base(b)));
  };
  // The reference point of the exponentials follows the running maximum only once that is 2^8
  // away: sums and weights up to 256 lose nothing, and most tiles leave the accumulator as it is.
  auto follow = [&]() {
    bool far = false;
#pragma unroll
    for (int b = 0; b < CB; b++) far |= top[b] > m[b] + 8.0f;
    if (__builtin_amdgcn_ballot_w64(far)) {
#pragma unroll
      for (int b = 0; b < CB; b++) {
        const float mn = __builtin_fmaxf(m[b], top[b]);
        const float f = __builtin_amdgcn_exp2f(m[b] - mn);
        m[b] = mn;
        sum[b] *= f;
#pragma unroll
        for (int c = 0; c < OT; c++)
#pragma unroll
          for (int r = 0; r < 16; r++) acc[b][c][r] *= f;
      }
    }
  };
  // scores to weights, not yet rounded
  auto weights = [&](f32x16_t (&x)[CB], const float (&off)[CB], int from, int to) {
#pragma unroll
    for (int b = 0; b < CB; b++)
#pragma unroll
      for (int r = from; r < to; r++) {
        const float w = __builtin_amdgcn_exp2f(MODE == ATTN_PLAIN ? __builtin_fmaf(x[b][r], post, off[b])
                                                                  : x[b][r] + off[b]);
        sum[b] += w;
        x[b][r] = w;
      }
  };

  tile_barrier();
  if (wave_tiles > 0) {
    products(s, 0, [](int) {});
    scores(s, 0, false, 0, 16);
    settle();
  }
  for (int n = 0; n < tiles; n++) {
    tile_barrier();
    aim(ck, kp, a.k_tok, n + 2);
    aim(cv, vp, a.v_tok, n + 1);
    auto fetch = [&](int e) {
      if (e < C) ck.go(lds[n & 1], wave, e);
      else if (e < 2 * C) cv.go(lds[2 + ((n + 1) & 1)], wave, e - C);
    };
    if (n >= wave_tiles) {  // nothing for this wave's rows but to fetch
#pragma unroll
      for (int e = 0; e < 2 * C; e++) fetch(e);
      continue;
    }
    follow();
    Packed<DT> p[CB];
    float off[CB];
#pragma unroll
    for (int b = 0; b < CB; b++) off[b] = block_base(b) - m[b];
    if (n + 1 == wave_tiles) {
      weights(s, off, 0, 16);
#pragma unroll
      for (int b = 0; b < CB; b++) p[b].set(s[b]);
      values(p, n, fetch);
      continue;
    }
    f32x16_t next[CB];
#pragma unroll
    for (int b = 0; b < CB; b++) top[b] = -INFINITY;
    auto step = [&](bool linear) {
      both(next, p, n, [&](int e) {
        fetch(e);
        if (e < N1) weights(s, off, e * 16 / N1, (e + 1) * 16 / N1);
        if (e == N1 - 1) {
#pragma unroll
          for (int b = 0; b < CB; b++) p[b].set(s[b]);
        }
        if (e >= N1) scores(next, n + 1, linear, (e - N1) * 16 / N2, (e + 1 - N1) * 16 / N2);
      });
    };
    // (the marks keep the compiler from moving the two copies' common start, and with it the
    // vector work beside the first matrix instructions, before the branch)
    if (linear_at(n + 1)) {
      asm volatile("; linear");
      step(true);
      base = base_of(n + 1);
    } else {
      asm volatile("; full");
      step(false);
      base = 0.0f;
    }
    settle();
#pragma unroll
    for (int b = 0; b < CB; b++) s[b] = next[b];
  }
  tile_barrier();  // the tiles' memory is free
#pragma unroll
  for (int b = 0; b < CB; b++) {
    sum[b] = half_sum(sum[b]);
    const bool real = i + 32 * b < t.len && sum[b] > 0.0f;
    if (h == 0 && i + 32 * b < t.rows)
      lse[32 * b] = real ? (m[b] + __builtin_amdgcn_logf(sum[b])) * LN2 : -INFINITY;
    store_rows<DT, DP>(lds[threadIdx.x >> 6], acc[b], real ? 1.0f / sum[b] : 0.0f,
                       a.o + ((t.row0 + wave0 + 32 * b) * a.heads + t.head) * row_bytes,
                       (int64_t)a.heads * row_bytes, t.rows - wave0 - 32 * b, row_bytes);
  }
}

template <int DT, int DP, int MODE, int CB>
__global__ void __launch_bounds__(ATTN_THREADS)
__attribute__((amdgpu_waves_per_eu(FwdWaves<DP, CB>::value, FwdWaves<DP, CB>::value)))
attn_fwd_kernel(const AttnArgs a) {
  using L = RowLayout<DT, DP>;
  __shared__ __align__(256) char lds[4][32 * L::bytes];  // two buffers of K, two of V
  AttnTile t;
  if (!locate(a, 128 * CB, t)) return;
  if (t.first < t.len) {
    attn_fwd_tile<DT, DP, MODE, CB>(a, t, lds);
    return;
  }
  // rows without a token
  const int i = t.first + threadIdx.x;
  if (threadIdx.x < 128 * CB && i < t.rows) a.lse[(int64_t)t.head * a.rows + t.row0 + i] = -INFINITY;
  zero_tile<DT>(a.o, a.heads, t, 128 * CB, a.d);
}

}  // namespace maxsim
