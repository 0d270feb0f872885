// Root-mean-square norm with the residual's addition (include/maxsim.h, maxsim_rms_norm):
//   h = residual + dropout(x),   y = h * rsqrt(mean h^2 + eps) * w,
// its 8-bit form, and its backward. Bytes bound all three: a group of lanes holds a whole row in
// registers, so that each tensor is read and written once. Measured (one MI355X): 81907 rows of 768
// in bf16 with a residual and dropout, 83 us (503 MB, 6.0 TB/s) forward, 112 us and 5 us for the
// weight's gradient (629 MB, 5.6 TB/s) backward; 163877 rows of 128 to 8 bits 17 us, of which the
// launch and one wait for memory are a third; 32 rows of 768 3 us.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.hpp"
#include "rms_norm_args.hpp"
#include "row_chunks.hpp"

namespace maxsim {

// Sum and maximum over the G lanes of a row, in every one of them; the order is fixed.
template <int G> __device__ __forceinline__ float group_sum(float v, float *lds) {
  v = sum_row16(v);
  uint32_t a, b;
  if constexpr (G >= 32) {
    row_pair<16>(__float_as_uint(v), a, b);
    v = __uint_as_float(a) + __uint_as_float(b);
  }
  if constexpr (G >= 64) {
    row_pair<32>(__float_as_uint(v), a, b);
    v = __uint_as_float(a) + __uint_as_float(b);
  }
  if constexpr (G == 256) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    __syncthreads();
  }
  return v;
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL> __device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max_u32(v, __builtin_amdgcn_update_dpp(0u, v, CTRL, 0xF, 0xF, true));
}
// Of the bit patterns of absolute values: a NaN is above all, infinity above all numbers.
template <int G> __device__ __forceinline__ uint32_t group_max(uint32_t v, float *lds) {
  v = dpp_max<DPP_XOR1>(v);
  v = dpp_max<DPP_XOR2>(v);
  v = dpp_max<DPP_HALF_MIRROR>(v);
  v = dpp_max<DPP_MIRROR>(v);
  uint32_t a, b;
  if constexpr (G >= 32) {
    row_pair<16>(v, a, b);
    v = max_u32(a, b);
  }
  if constexpr (G >= 64) {
    row_pair<32>(v, a, b);
    v = max_u32(a, b);
  }
  if constexpr (G == 256) {
    uint32_t *p = (uint32_t *)lds;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) p[wave] = v;
    __syncthreads();
    v = max_u32(max_u32(p[0], p[1]), max_u32(p[2], p[3]));
    __syncthreads();
  }
  return v;
}

// A row's entry e has bits e % 8 of block row * ceil(d / 8) + e / 8.
__device__ __forceinline__ uint64_t drop_block(int64_t row, int d, int chunk) {
  return (uint64_t)row * (uint32_t)((d + 7) / 8) + chunk;
}

// Rows of whole chunks, with a shorter one at the end, and of less than one.
enum { ROW_WHOLE, ROW_TAIL, ROW_TINY };

// What a lane holds of a row: C chunks, lane l of the row's G lanes chunks l, l + G, ... Loads need
// no branch, so that all of a lane's are under way at once: those past the row's end fetch its last 8
// entries again, and a shorter last chunk is moved into place afterwards (settle); has(c) tells
// which chunks count, in(c, e) which entries. TINY rows, of less than 8 entries, go one by one.
template <typename T, int G, int C, int KIND, bool ONCE> struct NormRow {
  int lane, d;
  __device__ __forceinline__ int at(int c) const { return (c * G + lane) * 8; }
  __device__ __forceinline__ bool has(int c) const { return at(c) < d; }
  __device__ __forceinline__ bool in(int c, int e) const { return KIND == ROW_WHOLE ? has(c) : at(c) + e < d; }
  template <typename V> __device__ __forceinline__ void load(const V *row, Chunk8<V> (&v)[C]) const { load<ONCE>(row, v); }
  template <bool PAST, typename V> __device__ __forceinline__ void load(const V *row, Chunk8<V> (&v)[C]) const {
#pragma unroll
    for (int c = 0; c < C; c++) {
      if constexpr (KIND != ROW_TINY) {
        v[c] = whole_chunk<PAST>(row + (at(c) + 8 <= d ? at(c) : d - 8));
      } else {
        float f[8] = {};
        if (has(c)) load_chunk(row, at(c), d, f);
        v[c] = rounded<V>(f);  // exact: they were of this type
      }
    }
  }
  template <typename V> __device__ __forceinline__ void settle(Chunk8<V> (&v)[C]) const {
    if constexpr (KIND == ROW_TAIL) {
#pragma unroll
      for (int c = 0; c < C; c++) {
        const int by = at(c) + 8 - d;  // entries that the load began too early
        if (by <= 0 || by >= 8) continue;
#pragma unroll
        for (int s = 4; s > 0; s /= 2)
          if (by & s) {
#pragma unroll
            for (int e = 0; e + s < 8; e++) v[c].e[e] = v[c].e[e + s];
          }
      }
    }
  }
  template <typename V> __device__ __forceinline__ void store(V *row, int c, const float (&f)[8]) const {
    if constexpr (KIND == ROW_WHOLE) store_whole<ONCE>(row + at(c), rounded<V>(f));
    else store_chunk(row, at(c), d, f);
  }
};

// T: storage type, G: lanes of a row, C: chunks of a lane, W32: weights in fp32, else in T. I8: 8-bit
// output. ONCE: past the caches.
template <typename T, int G, int C, int KIND, bool W32, bool I8, bool ONCE>
__global__ void __launch_bounds__(NORM_THREADS) norm_kernel(NormArgs a) {
  using W = std::conditional_t<W32, float, T>;
  constexpr int GROUPS = NORM_THREADS / G, R = norm_rows<C>;
  __shared__ float lds[4];
  const NormRow<T, G, C, KIND, ONCE> part{(int)threadIdx.x % G, a.d};
  const int64_t row0 = a.first + (int64_t)blockIdx.x * (GROUPS * R) + threadIdx.x / G;
  Chunk8<T> x[R][C], r[R][C];
  Chunk8<W> w[C];
  // every lane takes part in the reductions: past the last row it holds that one again
#pragma unroll
  for (int i = 0; i < R; i++) {
    const int64_t row = row0 + i * GROUPS < a.rows ? row0 + i * GROUPS : a.rows - 1;
    part.load((const T *)a.x + row * a.x_stride, x[i]);
    if (a.residual) part.load((const T *)a.residual + row * a.residual_stride, r[i]);
  }
  part.template load<false>((const W *)a.weight, w);
  DropKey key{};
  if (a.drop.rng) key.load(a.drop.rng);
  part.settle(w);
#pragma unroll
  for (int i = 0; i < R; i++) {
    part.settle(x[i]);
    if (a.residual) part.settle(r[i]);
    const int64_t row = row0 + i * GROUPS;
    const bool real = row < a.rows;
    float h[C][8], squares = 0.0f;
#pragma unroll
    for (int c = 0; c < C; c++) {
      DropBits bits;
      if (a.drop.rng) bits.make(key, a.drop, drop_block(row, a.d, part.at(c) / 8));
#pragma unroll
      for (int e = 0; e < 8; e++) {
        // the product and the sum are rounded apart: what is handed on does not depend on the compiler
        float v = (float)x[i][c].e[e];
        if (a.drop.rng) v = bits.apply(a.drop, e, v);
        if (a.residual) v = __fadd_rn(v, (float)r[i][c].e[e]);
        // The norm is of h as it is handed on, rounded: the backward, which reads that h, is the
        // derivative of just this function.
        h[c][e] = (float)(T)v;
      }
      if (a.h && real && part.has(c)) part.store((T *)a.h + row * a.d, c, h[c]);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        if (!part.in(c, e)) h[c][e] = 0.0f;
        squares = __builtin_fmaf(h[c][e], h[c][e], squares);
      }
    }
    squares = group_sum<G>(squares, lds);
    const float rstd = rsqrtf(__builtin_fmaf(squares, a.one_over_d, a.eps));
    if (!I8 && a.rstd && real && part.lane == 0) a.rstd[row] = rstd;
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < C; c++) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        h[c][e] = h[c][e] * rstd * (float)w[c].e[e];
        if (I8 && part.in(c, e)) most = max_u32(most, __float_as_uint(h[c][e]) & 0x7fffffffu);
      }
      if (!I8 && real && part.has(c)) part.store((T *)a.y + row * a.d, c, h[c]);
    }
    if constexpr (I8) {
      most = group_max<G>(most, lds);
      const float scale = __uint_as_float(most) * (1.0f / 127.0f);
      if (real && part.lane == 0) a.scale[row] = scale;
      // Rows of tiny entries are lifted by 2^100, so that the unit and its reciprocal are normal numbers; one
      // that holds an infinity or a NaN has that as its scale, and codes of 0. Few waves come here.
      float unit = scale;
      const bool none = most == 0 || most >= 0x7f800000u;
      if (__any(none || most < 0x0d800000u)) {
        const float lift = most < 0x0d800000u ? 0x1p100f : 1.0f;
        unit = none ? 1.0f : __uint_as_float(most) * lift * (1.0f / 127.0f);
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
          for (int e = 0; e < 8; e++) h[c][e] = none ? 0.0f : h[c][e] * lift;
      }
      const float to = __builtin_amdgcn_rcpf(unit);
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (!part.has(c) || !real) continue;
        Chunk8<int8_t> q;
        float far = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float v = h[c][e] * to, near = __builtin_rintf(v);
          far = __builtin_fmaxf(far, __builtin_fabsf(v - near));
          q.e[e] = (int8_t)(int)near;
        }
        // The reciprocal and the product put v off by up to 3 * 2^-24 of at most 128: next to a tie the
        // code may be the neighbour's. What the code leaves of the entry is exact and decides there; a
        // wave in 16 comes here (163877 x 128 in bf16, by events: 19.9 us, 25.2 with the remainder of
        // every entry).
        if (__any(far > 0.5f - 0x1p-14f)) {
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const float left = __builtin_fmaf(-(float)q.e[e], unit, h[c][e]), twice = 2.0f * __builtin_fabsf(left);
            if (twice > unit || (twice == unit && (q.e[e] & 1))) q.e[e] += left > 0.0f ? 1 : -1;
          }
        }
        int8_t *o = a.codes + row * a.d;
        if (KIND == ROW_WHOLE || part.at(c) + 8 <= a.d) {
          *(Chunk8<int8_t> *)(o + part.at(c)) = q;
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++)
            if (part.at(c) + e < a.d) o[part.at(c) + e] = q.e[e];
        }
      }
    }
  }
}

// Gradients. With n = h * rstd and g = grad_y * w: dh = rstd * (g - n * mean(g * n)) + grad_h, the
// residual's gradient as it is and x's through dropout; the weight's is the sum of grad_y * n over
// the rows: a group of lanes keeps the sums of the rows that it takes in registers, a workgroup
// leaves one row of sums, and norm_weight_kernel adds those up, all in a fixed order. The next row's
// loads are under way while a row is worked on.
template <typename T, int G, int C, int KIND, bool W32, bool ONCE>
__global__ void __launch_bounds__(NORM_THREADS) norm_backward_kernel(NormArgs a) {
  using W = std::conditional_t<W32, float, T>;
  constexpr int GROUPS = NORM_THREADS / G;
  __shared__ float lds[4];
  __shared__ float sums[NORM_THREADS * 8];
  const NormRow<T, G, C, KIND, ONCE> part{(int)threadIdx.x % G, a.d};
  const int group = threadIdx.x / G;
  DropKey key{};
  if (a.drop.rng) key.load(a.drop.rng);
  Chunk8<W> w[C];
  part.template load<false>((const W *)a.weight, w);
  part.settle(w);
  float dw[C][8];
#pragma unroll
  for (int c = 0; c < C; c++)
#pragma unroll
    for (int e = 0; e < 8; e++) dw[c][e] = 0.0f;
  Chunk8<T> hn[C], gn[C], kn[C];
  float rn = 0.0f;
  auto load = [&](int64_t asked) {
    const int64_t row = asked < a.rows ? asked : a.rows - 1;
    part.load((const T *)a.x + row * a.x_stride, hn);
    part.load((const T *)a.grad_y + row * a.d, gn);
    if (a.grad_h) part.load((const T *)a.grad_h + row * a.d, kn);
    rn = a.rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t base = (int64_t)blockIdx.x * GROUPS;
  load(base + group);
  // every group of a workgroup makes the same number of rounds: the reductions hold barriers
  for (; base < a.rows; base += step) {
    const int64_t row = base + group;
    const bool real = row < a.rows;
    Chunk8<T> k[C];
    float g[C][8], n[C][8], dot = 0.0f;
    const float rstd = real ? rn : 0.0f;
    part.settle(hn);
    part.settle(gn);
    if (a.grad_h) part.settle(kn);
#pragma unroll
    for (int c = 0; c < C; c++) {
      k[c] = kn[c];
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const bool in = real && part.in(c, e);
        n[c][e] = in ? (float)hn[c].e[e] * rstd : 0.0f;
        g[c][e] = in ? (float)gn[c].e[e] : 0.0f;
      }
    }
    if (base + step < a.rows) load(row + step);
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        dw[c][e] = __builtin_fmaf(g[c][e], n[c][e], dw[c][e]);
        g[c][e] *= (float)w[c].e[e];
        dot = __builtin_fmaf(g[c][e], n[c][e], dot);
      }
    if (!a.dx && !a.dresidual) continue;
    dot = group_sum<G>(dot, lds) * a.one_over_d;
    if (!real) continue;
#pragma unroll
    for (int c = 0; c < C; c++) {
      if (!part.has(c)) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; e++) {
        o[e] = rstd * (g[c][e] - n[c][e] * dot);
        if (a.grad_h) o[e] += (float)k[c].e[e];
      }
      if (a.dresidual) part.store((T *)a.dresidual + row * a.d, c, o);
      if (!a.dx) continue;
      if (a.drop.rng) {
        DropBits bits;
        bits.make(key, a.drop, drop_block(row, a.d, part.at(c) / 8));
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = bits.apply(a.drop, e, o[e]);
      }
      part.store((T *)a.dx + row * a.d, c, o);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int c = 0; c < C; c++) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; e++) sums[threadIdx.x * 8 + e] = dw[c][e];
    __syncthreads();
    for (int i = threadIdx.x; i < G * 8; i += NORM_THREADS) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < GROUPS; k++) s += sums[k * G * 8 + i];
      const int at = c * G * 8 + i;
      if (at < a.d) a.part[(int64_t)blockIdx.x * a.d + at] = s;
    }
  }
}

template <typename T, int G, int C, int KIND, int WHICH, bool W32, bool ONCE> const void *norm_kernel_of() {
  static_assert(W32 || sizeof(T) == 2, "fp32 rows have fp32 weights");
  if constexpr (WHICH == NORM_BACK) return (const void *)norm_backward_kernel<T, G, C, KIND, W32, ONCE>;
  else return (const void *)norm_kernel<T, G, C, KIND, W32, WHICH == NORM_I8, ONCE>;
}
template <typename T, int G, int C, int KIND, int WHICH, bool ONCE> const void *norm_kernel_of(bool w32) {
  if constexpr (sizeof(T) == 2)
    if (!w32) return norm_kernel_of<T, G, C, KIND, WHICH, false, ONCE>();
  return norm_kernel_of<T, G, C, KIND, WHICH, true, ONCE>();
}
template <typename T, int G, int C, int KIND, int WHICH> const void *norm_kernel_of(bool w32, bool once) {
  if constexpr (KIND == ROW_WHOLE && WHICH != NORM_I8 && sizeof(T) == 2)
    if (once) return norm_kernel_of<T, G, C, KIND, WHICH, true>(w32);
  return norm_kernel_of<T, G, C, KIND, WHICH, false>(w32);
}

template <typename T, int WHICH> const void *norm_pick(int d, bool w32, bool once) {
  const int of = norm_lanes(d) * 8 + norm_chunks(d);
  if (d < 8) return norm_kernel_of<T, 16, 1, ROW_TINY, WHICH>(w32, once);
  if (d % 8) {
    switch (of) {
    case 16 * 8 + 1: return norm_kernel_of<T, 16, 1, ROW_TAIL, WHICH>(w32, once);
    case 16 * 8 + 2: return norm_kernel_of<T, 16, 2, ROW_TAIL, WHICH>(w32, once);
    case 16 * 8 + 4: return norm_kernel_of<T, 16, 4, ROW_TAIL, WHICH>(w32, once);
    case 32 * 8 + 4: return norm_kernel_of<T, 32, 4, ROW_TAIL, WHICH>(w32, once);
    case 64 * 8 + 4: return norm_kernel_of<T, 64, 4, ROW_TAIL, WHICH>(w32, once);
    default: return norm_kernel_of<T, 256, 4, ROW_TAIL, WHICH>(w32, once);
    }
  }
  switch (of) {
  case 16 * 8 + 1: return norm_kernel_of<T, 16, 1, ROW_WHOLE, WHICH>(w32, once);
  case 16 * 8 + 2: return norm_kernel_of<T, 16, 2, ROW_WHOLE, WHICH>(w32, once);
  case 16 * 8 + 3: return norm_kernel_of<T, 16, 3, ROW_WHOLE, WHICH>(w32, once);
  case 16 * 8 + 4: return norm_kernel_of<T, 16, 4, ROW_WHOLE, WHICH>(w32, once);
  case 32 * 8 + 3: return norm_kernel_of<T, 32, 3, ROW_WHOLE, WHICH>(w32, once);
  case 32 * 8 + 4: return norm_kernel_of<T, 32, 4, ROW_WHOLE, WHICH>(w32, once);
  case 64 * 8 + 3: return norm_kernel_of<T, 64, 3, ROW_WHOLE, WHICH>(w32, once);
  case 64 * 8 + 4: return norm_kernel_of<T, 64, 4, ROW_WHOLE, WHICH>(w32, once);
  case 256 * 8 + 2: return norm_kernel_of<T, 256, 2, ROW_WHOLE, WHICH>(w32, once);
  case 256 * 8 + 3: return norm_kernel_of<T, 256, 3, ROW_WHOLE, WHICH>(w32, once);
  default: return norm_kernel_of<T, 256, 4, ROW_WHOLE, WHICH>(w32, once);
  }
}
template <typename T> const void *norm_kernel_for(int which, int d, bool w32, bool once) {
  return which == NORM_Y    ? norm_pick<T, NORM_Y>(d, w32, once)
         : which == NORM_I8 ? norm_pick<T, NORM_I8>(d, w32, once)
                            : norm_pick<T, NORM_BACK>(d, w32, once);
}

}  // namespace maxsim
