// Root-mean-square norm with the residual's addition (include/maxsim.h, maxsim_rms_norm):
//   h = residual + dropout(x),   y = h * rsqrt(mean h^2 + eps) * w,
// its 8-bit form, and its backward. Bytes bound all three: a group of lanes holds a whole row in
// registers, so that each tensor is read and written once.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.hpp"
#include "dropout_bits.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"
#include "row_chunks.hpp"

using namespace maxsim;

namespace {

constexpr int NORM_THREADS = 256;
constexpr int NORM_MOST_D = MAXSIM_MAX_NORM;

struct NormArgs {
  const void *x, *residual, *weight;
  int64_t x_stride, residual_stride;  // entries
  int64_t first, rows;                // first row of this launch, all rows
  int d;
  float eps, one_over_d;
  DropArgs drop;
  void *y, *h;
  int8_t *codes;
  float *scale, *rstd;
  // backward
  const void *grad_y, *grad_h;
  void *dx, *dresidual;
  float *part;  // [workgroups][d]: sums of the weight's gradient
};

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

// What a lane holds of a row: C chunks, lane l of the row's G lanes chunks l, l + G, ... WHOLE: d is a
// multiple of 8, and loads need no branch: those past the row's end fetch its last chunk again, so
// that all of a lane's loads are under way at once; has(c) tells which count. Otherwise the last
// chunk goes entry by entry.
template <typename T, int G, int C, bool WHOLE> struct NormRow {
  int lane, d;
  __device__ __forceinline__ int at(int c) const { return (c * G + lane) * 8; }
  __device__ __forceinline__ bool has(int c) const { return at(c) < d; }
  template <typename V> __device__ __forceinline__ void load(const V *row, Chunk8<V> (&v)[C]) const {
#pragma unroll
    for (int c = 0; c < C; c++) {
      if constexpr (WHOLE) {
        v[c] = whole_chunk(row + (has(c) ? at(c) : d - 8));
      } else {
        float f[8] = {};
        if (has(c)) load_chunk(row, at(c), d, f);
        v[c] = rounded<V>(f);  // exact: they were of this type
      }
    }
  }
  template <typename V> __device__ __forceinline__ void store(V *row, int c, const float (&f)[8]) const {
    if constexpr (WHOLE) *(Chunk8<V> *)(row + at(c)) = rounded<V>(f);
    else store_chunk(row, at(c), d, f);
  }
};

// Rows of a group of lanes: where a lane holds one chunk of a row it takes two rows at once (500000
// rows of 128 in bf16 to 8 bits: 50.2 us one at a time, 47.3 two, 49.9 four).
template <int C> constexpr int norm_rows = C == 1 ? 2 : 1;

// T: storage type, G: lanes of a row, C: chunks of a lane, W32: weights in fp32, else in T. I8: 8-bit
// output.
template <typename T, int G, int C, bool WHOLE, bool W32, bool I8>
__global__ void __launch_bounds__(NORM_THREADS) norm_kernel(NormArgs a) {
  using W = std::conditional_t<W32, float, T>;
  constexpr int GROUPS = NORM_THREADS / G, R = norm_rows<C>;
  __shared__ float lds[4];
  const NormRow<T, G, C, WHOLE> part{(int)threadIdx.x % G, a.d};
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
  part.load((const W *)a.weight, w);
  DropKey key{};
  if (a.drop.rng) key.load(a.drop.rng);
#pragma unroll
  for (int i = 0; i < R; i++) {
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
        if (!part.has(c) || (!WHOLE && part.at(c) + e >= a.d)) h[c][e] = 0.0f;
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
        if (I8 && part.has(c) && (WHOLE || part.at(c) + e < a.d)) most = max_u32(most, __float_as_uint(h[c][e]) & 0x7fffffffu);
      }
      if (!I8 && real && part.has(c)) part.store((T *)a.y + row * a.d, c, h[c]);
    }
    if constexpr (I8) {
      most = group_max<G>(most, lds);
      // A row that holds an infinity or a NaN has that as its scale, and codes of 0.
      const float scale = __uint_as_float(most) * (1.0f / 127.0f);
      // 127 / most stays finite: rows of tiny entries are lifted by 2^100 first
      const float lift = most < 0x0d800000u ? 0x1p100f : 1.0f;
      const float to = most > 0 && most < 0x7f800000u ? 127.0f * __builtin_amdgcn_rcpf(__uint_as_float(most) * lift) : 0.0f;
      if (real && part.lane == 0) a.scale[row] = scale;
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (!part.has(c) || !real) continue;
        Chunk8<int8_t> q;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float v = __builtin_rintf(h[c][e] * lift * to);  // an infinity times 0 is a NaN
          q.e[e] = (int8_t)(v == v ? (int)v : 0);
        }
        int8_t *o = a.codes + row * a.d;
        if (WHOLE || part.at(c) + 8 <= a.d) {
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
template <typename T, int G, int C, bool WHOLE, bool W32>
__global__ void __launch_bounds__(NORM_THREADS) norm_backward_kernel(NormArgs a) {
  using W = std::conditional_t<W32, float, T>;
  constexpr int GROUPS = NORM_THREADS / G;
  __shared__ float lds[4];
  __shared__ float sums[NORM_THREADS * 8];
  const NormRow<T, G, C, WHOLE> part{(int)threadIdx.x % G, a.d};
  const int group = threadIdx.x / G;
  DropKey key{};
  if (a.drop.rng) key.load(a.drop.rng);
  Chunk8<W> w[C];
  part.load((const W *)a.weight, w);
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
#pragma unroll
    for (int c = 0; c < C; c++) {
      k[c] = kn[c];
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const bool in = part.has(c) && real && (WHOLE || part.at(c) + e < a.d);
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

// The weight's gradient from the workgroups' sums: 16 entries a workgroup, 64 threads to each.
constexpr int NORM_JOIN = 1024;
template <typename W>
__global__ void __launch_bounds__(NORM_JOIN) norm_weight_kernel(const float *part, int n, int d, W *dw) {
  __shared__ float sums[64][17];
  const int col = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int at = blockIdx.x * 16 + col;
  float s = 0.0f;
  if (at < d) {
#pragma unroll 8
    for (int i = slice; i < n; i += 64) s += part[(int64_t)i * d + at];
  }
  sums[slice][col] = s;
  __syncthreads();
  for (int o = 32; o > 0; o >>= 1) {
    if (slice < o) sums[slice][col] += sums[slice + o][col];
    __syncthreads();
  }
  if (slice == 0 && at < d) dw[at] = (W)sums[0][col];
}

enum { NORM_Y, NORM_I8, NORM_BACK };

template <typename T, int G, int C, bool WHOLE, int WHICH> const void *norm_kernel_of(bool w32) {
  if constexpr (WHICH == NORM_BACK)
    return w32 ? (const void *)norm_backward_kernel<T, G, C, WHOLE, true>
               : (const void *)norm_backward_kernel<T, G, C, WHOLE, false>;
  else
    return w32 ? (const void *)norm_kernel<T, G, C, WHOLE, true, WHICH == NORM_I8>
               : (const void *)norm_kernel<T, G, C, WHOLE, false, WHICH == NORM_I8>;
}

// Lanes of a row and chunks of a lane: the fewest lanes whose registers hold the row, so that the
// fewest of them stand idle at its end (768 entries: 32 lanes of 3 chunks). Rows that are no multiple
// of 8 entries, which go slower anyway, have fewer forms.
int norm_lanes(int d) {
  const int n = (d + 7) / 8;
  if (d % 8) return n <= 16 ? 16 : n <= 256 ? 64 : 256;
  return n <= 64 ? 16 : n <= 128 ? 32 : n <= 256 ? 64 : 256;
}
int norm_chunks(int d) {
  const int g = norm_lanes(d), n = (d + 7) / 8;
  return d % 8 ? (g == 16 ? 1 : 4) : (n + g - 1) / g;
}
template <typename T, int WHICH> const void *norm_pick(int d, bool w32) {
  const int g = norm_lanes(d), c = norm_chunks(d);
  if (d % 8) {
    if (g == 16) return norm_kernel_of<T, 16, 1, false, WHICH>(w32);
    if (g == 64) return norm_kernel_of<T, 64, 4, false, WHICH>(w32);
    return norm_kernel_of<T, 256, 4, false, WHICH>(w32);
  }
  switch (g * 8 + c) {
  case 16 * 8 + 1: return norm_kernel_of<T, 16, 1, true, WHICH>(w32);
  case 16 * 8 + 2: return norm_kernel_of<T, 16, 2, true, WHICH>(w32);
  case 16 * 8 + 3: return norm_kernel_of<T, 16, 3, true, WHICH>(w32);
  case 16 * 8 + 4: return norm_kernel_of<T, 16, 4, true, WHICH>(w32);
  case 32 * 8 + 3: return norm_kernel_of<T, 32, 3, true, WHICH>(w32);
  case 32 * 8 + 4: return norm_kernel_of<T, 32, 4, true, WHICH>(w32);
  case 64 * 8 + 3: return norm_kernel_of<T, 64, 3, true, WHICH>(w32);
  case 64 * 8 + 4: return norm_kernel_of<T, 64, 4, true, WHICH>(w32);
  case 256 * 8 + 2: return norm_kernel_of<T, 256, 2, true, WHICH>(w32);
  case 256 * 8 + 3: return norm_kernel_of<T, 256, 3, true, WHICH>(w32);
  default: return norm_kernel_of<T, 256, 4, true, WHICH>(w32);
  }
}
template <int WHICH> const void *norm_pick(int dtype, int d, int weight_dtype) {
  const bool w32 = weight_dtype == MAXSIM_FP32;
  return dtype == MAXSIM_FP32   ? norm_pick<float, WHICH>(d, true)
         : dtype == MAXSIM_FP16 ? norm_pick<_Float16, WHICH>(d, w32)
                                : norm_pick<__bf16, WHICH>(d, w32);
}

int norm_sizes(int64_t rows, int d, int dtype, int weight_dtype) {
  if (elem_bytes(dtype) == 0) return MAXSIM_ERR_DTYPE;
  if (weight_dtype != dtype && weight_dtype != MAXSIM_FP32) return MAXSIM_ERR_DTYPE;
  if (rows < 0 || rows > ((int64_t)1 << 31) || d < 1) return MAXSIM_ERR_SHAPE;
  return d > NORM_MOST_D ? MAXSIM_ERR_UNSUPPORTED : MAXSIM_OK;
}

int norm_launch(const void *kernel, NormArgs &a, hipStream_t st) {
  const int g = norm_lanes(a.d), c = norm_chunks(a.d);
  const int64_t per = NORM_THREADS / g * (c == 1 ? norm_rows<1> : norm_rows<2>);
  void *kargs[] = {&a};
  for (a.first = 0; a.first < a.rows; a.first += (int64_t)LAUNCH_MOST * per) {
    const int64_t left = (a.rows - a.first + per - 1) / per;
    const unsigned grid = (unsigned)(left < (int64_t)LAUNCH_MOST ? left : LAUNCH_MOST);
    if (hipLaunchKernel(kernel, dim3(grid), dim3(NORM_THREADS), kargs, 0, st) != hipSuccess) {
      (void)hipGetLastError();
      return MAXSIM_ERR_LAUNCH;
    }
  }
  return MAXSIM_OK;
}

// Workgroups of the backward: as many as the chip holds at once, so that each has many rows and
// there are few sums to join; no more than there are rows for.
constexpr int NORM_BACK_MOST = 1024;
unsigned norm_back_grid(int64_t rows, int g) {
  const int64_t n = (rows + NORM_THREADS / g - 1) / (NORM_THREADS / g);
  return (unsigned)(n < NORM_BACK_MOST ? n : NORM_BACK_MOST);
}

}  // namespace

extern "C" {

int maxsim_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                    int64_t n_rows, int d, int dtype, const void *weight, int weight_dtype, float eps,
                    double dropout, const int64_t *rng, int call, void *y, void *h, float *rstd,
                    void *stream) {
  int rc = norm_sizes(n_rows, d, dtype, weight_dtype);
  if (rc != MAXSIM_OK) return rc;
  if (!(eps >= 0) || !(dropout >= 0 && dropout <= 1) || call < 0) return MAXSIM_ERR_SHAPE;
  if (n_rows == 0) return MAXSIM_OK;
  const int eb = elem_bytes(dtype);
  const DropArgs drop = drop_args(dropout, rng, call);
  if (!x || !weight || !y || (dropout > 0 && !rng) || ((residual || drop.rng) && !h)) return MAXSIM_ERR_NULL;
  if (!aligned(x, eb) || !aligned(residual, eb) || !aligned(weight, elem_bytes(weight_dtype)) ||
      !aligned(y, eb) || !aligned(h, eb) || !aligned(rstd, 4) || !aligned(rng, 8))
    return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.weight = weight;
  a.rows = n_rows;
  a.d = d;
  a.one_over_d = 1.0f / (float)d;
  a.eps = eps;
  a.drop = drop;
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  return norm_launch(norm_pick<NORM_Y>(dtype, d, weight_dtype), a, (hipStream_t)stream);
}

int maxsim_rms_norm_i8(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                       int64_t n_rows, int d, int dtype, const void *weight, int weight_dtype, float eps,
                       int8_t *codes, float *scale, void *h, void *stream) {
  int rc = norm_sizes(n_rows, d, dtype, weight_dtype);
  if (rc != MAXSIM_OK) return rc;
  if (!(eps >= 0)) return MAXSIM_ERR_SHAPE;
  if (n_rows == 0) return MAXSIM_OK;
  const int eb = elem_bytes(dtype);
  if (!x || !weight || !codes || !scale || (residual && !h)) return MAXSIM_ERR_NULL;
  if (!aligned(x, eb) || !aligned(residual, eb) || !aligned(weight, elem_bytes(weight_dtype)) ||
      !aligned(scale, 4) || !aligned(h, eb))
    return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  NormArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.residual = residual;
  a.residual_stride = residual_stride;
  a.weight = weight;
  a.rows = n_rows;
  a.d = d;
  a.one_over_d = 1.0f / (float)d;
  a.eps = eps;
  a.codes = codes;
  a.scale = scale;
  a.h = h;
  return norm_launch(norm_pick<NORM_I8>(dtype, d, weight_dtype), a, (hipStream_t)stream);
}

size_t maxsim_rms_norm_backward_workspace_size(int64_t n_rows, int d) {
  if (n_rows < 1 || d < 1 || d > NORM_MOST_D) return 0;
  return (size_t)norm_back_grid(n_rows, norm_lanes(d)) * d * sizeof(float);
}

int maxsim_rms_norm_backward(const void *grad_y, const void *grad_h, const void *h, int64_t h_stride,
                             int64_t n_rows, int d, int dtype, const void *weight, int weight_dtype,
                             const float *rstd, double dropout, const int64_t *rng, int call, void *dx,
                             void *dresidual, void *dweight, void *workspace, size_t workspace_bytes,
                             void *stream) {
  int rc = norm_sizes(n_rows, d, dtype, weight_dtype);
  if (rc != MAXSIM_OK) return rc;
  if (!(dropout >= 0 && dropout <= 1) || call < 0) return MAXSIM_ERR_SHAPE;
  const int eb = elem_bytes(dtype);
  if (n_rows > 0 && (!grad_y || !h || !weight || !rstd || (dropout > 0 && !rng))) return MAXSIM_ERR_NULL;
  if (dweight && n_rows > 0 && !workspace) return MAXSIM_ERR_NULL;
  if (!aligned(grad_y, eb) || !aligned(grad_h, eb) || !aligned(h, eb) ||
      !aligned(weight, elem_bytes(weight_dtype)) || !aligned(rstd, 4) || !aligned(rng, 8) ||
      !aligned(dx, eb) || !aligned(dresidual, eb) || !aligned(dweight, elem_bytes(weight_dtype)) ||
      !aligned(workspace, 4))
    return MAXSIM_ERR_ALIGN;
  if (dweight && workspace_bytes < maxsim_rms_norm_backward_workspace_size(n_rows, d)) return MAXSIM_ERR_SHAPE;
  if ((!dx && !dresidual && !dweight) || (n_rows == 0 && !dweight)) return MAXSIM_OK;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  unsigned grid = 0;
  if (n_rows > 0) {
    NormArgs a{};
    a.grad_y = grad_y;
    a.grad_h = grad_h;
    a.x = h;
    a.x_stride = h_stride;
    a.rows = n_rows;
    a.d = d;
    a.one_over_d = 1.0f / (float)d;
    a.weight = weight;
    a.rstd = const_cast<float *>(rstd);
    a.drop = drop_args(dropout, rng, call);
    a.dx = dx;
    a.dresidual = dresidual;
    a.part = dweight ? (float *)workspace : nullptr;
    const void *kernel = norm_pick<NORM_BACK>(dtype, d, weight_dtype);
    grid = norm_back_grid(n_rows, norm_lanes(d));
    void *kargs[] = {&a};
    if (hipLaunchKernel(kernel, dim3(grid), dim3(NORM_THREADS), kargs, 0, st) != hipSuccess) {
      (void)hipGetLastError();
      return MAXSIM_ERR_LAUNCH;
    }
  }
  if (!dweight) return MAXSIM_OK;
  const dim3 cols((d + 15) / 16);
  const float *part = (const float *)workspace;
  if (weight_dtype == MAXSIM_FP32)
    hipLaunchKernelGGL(norm_weight_kernel<float>, cols, dim3(NORM_JOIN), 0, st, part, (int)grid, d, (float *)dweight);
  else if (weight_dtype == MAXSIM_FP16)
    hipLaunchKernelGGL(norm_weight_kernel<_Float16>, cols, dim3(NORM_JOIN), 0, st, part, (int)grid, d, (_Float16 *)dweight);
  else
    hipLaunchKernelGGL(norm_weight_kernel<__bf16>, cols, dim3(NORM_JOIN), 0, st, part, (int)grid, d, (__bf16 *)dweight);
  return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
}

}  // extern "C"
