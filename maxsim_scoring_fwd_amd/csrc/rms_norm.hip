// Root-mean-square norm with the residual's addition (include/maxsim.h, maxsim_rms_norm):
//   h = residual + dropout(x),   y = h * rsqrt(mean h^2 + eps) * w,
// its 8-bit form, and its backward. Bytes bound all three: a group of lanes holds a whole row in
// registers, so that each tensor is read and written once.
#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "dropout_bits.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"
#include "row_chunks.hpp"

using namespace maxsim;

namespace {

constexpr int NORM_THREADS = 256;
constexpr int NORM_MOST_D = MAXSIM_MAX_NORM;
constexpr int NORM_CHUNKS = 4;  // most chunks of 8 entries that a lane holds

struct NormArgs {
  const void *x, *residual, *weight;
  int64_t x_stride, residual_stride;  // entries
  int64_t first, rows;                // first row of this launch, all rows
  int d, weight_fp32;
  float eps;
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

template <typename T>
__device__ __forceinline__ void load_weight(const NormArgs &a, int at, float (&w)[8]) {
  if (a.weight_fp32) load_chunk((const float *)a.weight, at, a.d, w);
  else load_chunk((const T *)a.weight, at, a.d, w);
}

// A row's 8 kept entries of dropout are in block row * ceil(d / 8) + column / 8.
__device__ __forceinline__ uint64_t drop_block(int64_t row, int d, int chunk) {
  return (uint64_t)row * (uint32_t)((d + 7) / 8) + chunk;
}

// T: storage type, G: lanes of a row, C: chunks of a lane (lane l of the group holds chunks l,
// l + G, ...). I8: 8-bit output.
template <typename T, int G, int C, bool I8>
__global__ void __launch_bounds__(NORM_THREADS) norm_kernel(NormArgs a) {
  __shared__ float lds[4];
  const int lane = threadIdx.x % G;
  const int64_t row = a.first + (int64_t)blockIdx.x * (NORM_THREADS / G) + threadIdx.x / G;
  const bool real = row < a.rows;  // every lane takes part in the reductions
  const T *x = (const T *)a.x + row * a.x_stride;
  const T *r = a.residual ? (const T *)a.residual + row * a.residual_stride : nullptr;
  DropKey key{};
  if (a.drop.rng) key.load(a.drop.rng);
  float h[C][8], res[C][8];
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int at = (c * G + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; e++) h[c][e] = 0.0f;
    if (real && at < a.d) {
      load_chunk(x, at, a.d, h[c]);
      if (r) load_chunk(r, at, a.d, res[c]);
    }
  }
  float squares = 0.0f;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int at = (c * G + lane) * 8;
    if (!real || at >= a.d) continue;
    if (a.drop.rng) {
      const uint32_t keep = drop_keep(key, a.drop, drop_block(row, a.d, at / 8));
      // the product and the sum are rounded apart: what is handed on does not depend on the compiler
#pragma unroll
      for (int e = 0; e < 8; e++) h[c][e] = keep >> e & 1 ? __fmul_rn(h[c][e], a.drop.up) : 0.0f;
    }
    if (r) {
#pragma unroll
      for (int e = 0; e < 8; e++) h[c][e] = __fadd_rn(h[c][e], res[c][e]);
    }
    // The norm is of h as it is handed on, rounded: the backward, which reads that h, is the
    // derivative of just this function.
#pragma unroll
    for (int e = 0; e < 8; e++) h[c][e] = (float)(T)h[c][e];
    if (a.h) store_chunk((T *)a.h + row * a.d, at, a.d, h[c]);
    if (a.d - at < 8) {
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (at + e >= a.d) h[c][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; e++) squares = __builtin_fmaf(h[c][e], h[c][e], squares);
  }
  squares = group_sum<G>(squares, lds);
  const float rstd = 1.0f / __builtin_sqrtf(squares / (float)a.d + a.eps);
  if (!I8 && a.rstd && real && lane == 0) a.rstd[row] = rstd;
  uint32_t most = 0;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int at = (c * G + lane) * 8;
    if (!real || at >= a.d) continue;
    float w[8];
    load_weight<T>(a, at, w);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      h[c][e] = h[c][e] * rstd * w[e];
      if (I8 && at + e < a.d) most = max_u32(most, __float_as_uint(h[c][e]) & 0x7fffffffu);
    }
    if (!I8) store_chunk((T *)a.y + row * a.d, at, a.d, h[c]);
  }
  if constexpr (I8) {
    most = group_max<G>(most, lds);
    // A row that holds an infinity or a NaN has that as its scale, and codes of 0.
    const float scale = __uint_as_float(most) / 127.0f;
    // 127 / most stays finite: rows of tiny entries are lifted by 2^100 first
    const float lift = most < 0x0d800000u ? 0x1p100f : 1.0f;
    const float to = most > 0 && most < 0x7f800000u ? 127.0f / (__uint_as_float(most) * lift) : 0.0f;
    if (real && lane == 0) a.scale[row] = scale;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int at = (c * G + lane) * 8;
      if (!real || at >= a.d) continue;
      Chunk8<int8_t> q;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float v = __builtin_rintf(h[c][e] * lift * to);  // an infinity times 0 is a NaN
        q.e[e] = (int8_t)(v == v ? (int)v : 0);
      }
      int8_t *o = a.codes + row * a.d;
      if (at + 8 <= a.d) {
        *(Chunk8<int8_t> *)(o + at) = q;
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (at + e < a.d) o[at + e] = q.e[e];
      }
    }
  }
}

// Gradients. With n = h * rstd and g = grad_y * w: dh = rstd * (g - n * mean(g * n)) + grad_h, the
// residual's gradient as it is and x's through dropout; the weight's is the sum of grad_y * n over
// the rows: a group of lanes keeps the sums of the rows that it takes in registers, a workgroup
// leaves one row of sums, and norm_weight_kernel adds those up, all in a fixed order.
template <typename T, int G, int C>
__global__ void __launch_bounds__(NORM_THREADS) norm_backward_kernel(NormArgs a) {
  constexpr int GROUPS = NORM_THREADS / G;
  __shared__ float lds[4];
  __shared__ float sums[NORM_THREADS * 8];
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  DropKey key{};
  if (a.drop.rng) key.load(a.drop.rng);
  float w[C][8], dw[C][8];
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int at = (c * G + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; e++) w[c][e] = dw[c][e] = 0.0f;
    if (at < a.d) load_weight<T>(a, at, w[c]);
  }
  // every group of a workgroup makes the same number of rounds: the reductions hold barriers
  for (int64_t base = (int64_t)blockIdx.x * GROUPS; base < a.rows; base += (int64_t)gridDim.x * GROUPS) {
    const int64_t row = base + group;
    const bool real = row < a.rows;
    const T *gy = (const T *)a.grad_y + row * a.d, *hp = (const T *)a.x + row * a.x_stride;
    const T *gh = a.grad_h ? (const T *)a.grad_h + row * a.d : nullptr;
    float g[C][8], n[C][8];
    const float rstd = real ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int at = (c * G + lane) * 8;
#pragma unroll
      for (int e = 0; e < 8; e++) g[c][e] = n[c][e] = 0.0f;
      if (real && at < a.d) {
        load_chunk(hp, at, a.d, n[c]);
        load_chunk(gy, at, a.d, g[c]);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        n[c][e] *= rstd;
        dw[c][e] = __builtin_fmaf(g[c][e], n[c][e], dw[c][e]);
        g[c][e] *= w[c][e];
        dot = __builtin_fmaf(g[c][e], n[c][e], dot);
      }
    if (!a.dx && !a.dresidual) continue;
    dot = group_sum<G>(dot, lds) / (float)a.d;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int at = (c * G + lane) * 8;
      if (!real || at >= a.d) continue;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; e++) o[e] = rstd * (g[c][e] - n[c][e] * dot);
      if (gh) {
        float k[8];
        load_chunk(gh, at, a.d, k);
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] += k[e];
      }
      if (a.dresidual) store_chunk((T *)a.dresidual + row * a.d, at, a.d, o);
      if (!a.dx) continue;
      if (a.drop.rng) {
        const uint32_t keep = drop_keep(key, a.drop, drop_block(row, a.d, at / 8));
#pragma unroll
        for (int e = 0; e < 8; e++) o[e] = keep >> e & 1 ? o[e] * a.drop.up : 0.0f;
      }
      store_chunk((T *)a.dx + row * a.d, at, a.d, o);
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

// The weight's gradient from the workgroups' sums: 32 entries a workgroup, 8 threads to each.
template <typename W>
__global__ void __launch_bounds__(NORM_THREADS) norm_weight_kernel(const float *part, int n, int d, W *dw) {
  __shared__ float sums[8][32];
  const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int at = blockIdx.x * 32 + col;
  float s = 0.0f;
  if (at < d)
    for (int i = slice; i < n; i += 8) s += part[(int64_t)i * d + at];
  sums[slice][col] = s;
  __syncthreads();
  if (slice == 0 && at < d) {
#pragma unroll
    for (int k = 1; k < 8; k++) s += sums[k][col];
    dw[at] = (W)s;
  }
}

// Lanes of a row and chunks of a lane: the fewest lanes whose registers hold the row, so that the
// fewest of them stand idle at its end (768 entries: 32 lanes of 3 chunks).
template <typename T, template <typename, int, int> class F> const void *norm_pick(int d, int &g) {
  const int n = (d + 7) / 8;
  g = n <= 16 * NORM_CHUNKS ? 16 : n <= 32 * NORM_CHUNKS ? 32 : n <= 64 * NORM_CHUNKS ? 64 : 256;
  const int c = (n + g - 1) / g;
  auto of = [&](auto lanes) -> const void * {
    constexpr int G = decltype(lanes)::value;
    switch (c) {
    case 1: return F<T, G, 1>::kernel();
    case 2: return F<T, G, 2>::kernel();
    case 3: return F<T, G, 3>::kernel();
    default: return F<T, G, 4>::kernel();
    }
  };
  switch (g) {
  case 16: return of(std::integral_constant<int, 16>());
  case 32: return of(std::integral_constant<int, 32>());
  case 64: return of(std::integral_constant<int, 64>());
  default: return of(std::integral_constant<int, 256>());
  }
}
template <typename T, int G, int C> struct Forward {
  static const void *kernel() { return (const void *)norm_kernel<T, G, C, false>; }
};
template <typename T, int G, int C> struct Forward8 {
  static const void *kernel() { return (const void *)norm_kernel<T, G, C, true>; }
};
template <typename T, int G, int C> struct Backward {
  static const void *kernel() { return (const void *)norm_backward_kernel<T, G, C>; }
};
template <template <typename, int, int> class F> const void *norm_pick(int dtype, int d, int &g) {
  return dtype == MAXSIM_FP32   ? norm_pick<float, F>(d, g)
         : dtype == MAXSIM_FP16 ? norm_pick<_Float16, F>(d, g)
                                : norm_pick<__bf16, F>(d, g);
}

int norm_sizes(int64_t rows, int d, int dtype, int weight_dtype) {
  if (elem_bytes(dtype) == 0) return MAXSIM_ERR_DTYPE;
  if (weight_dtype != dtype && weight_dtype != MAXSIM_FP32) return MAXSIM_ERR_DTYPE;
  if (rows < 0 || rows > ((int64_t)1 << 31) || d < 1) return MAXSIM_ERR_SHAPE;
  return d > NORM_MOST_D ? MAXSIM_ERR_UNSUPPORTED : MAXSIM_OK;
}

int norm_launch(const void *kernel, NormArgs &a, int g, hipStream_t st) {
  const int64_t per = NORM_THREADS / g;
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
  a.weight_fp32 = weight_dtype == MAXSIM_FP32;
  a.rows = n_rows;
  a.d = d;
  a.eps = eps;
  a.drop = drop;
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  int g;
  const void *kernel = norm_pick<Forward>(dtype, d, g);
  return norm_launch(kernel, a, g, (hipStream_t)stream);
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
  a.weight_fp32 = weight_dtype == MAXSIM_FP32;
  a.rows = n_rows;
  a.d = d;
  a.eps = eps;
  a.codes = codes;
  a.scale = scale;
  a.h = h;
  int g;
  const void *kernel = norm_pick<Forward8>(dtype, d, g);
  return norm_launch(kernel, a, g, (hipStream_t)stream);
}

size_t maxsim_rms_norm_backward_workspace_size(int64_t n_rows, int d) {
  if (n_rows < 1 || d < 1 || d > NORM_MOST_D) return 0;
  int g;
  (void)norm_pick<Backward>(MAXSIM_FP32, d, g);
  return (size_t)norm_back_grid(n_rows, g) * d * sizeof(float);
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
    a.weight = weight;
    a.weight_fp32 = weight_dtype == MAXSIM_FP32;
    a.rstd = const_cast<float *>(rstd);
    a.drop = drop_args(dropout, rng, call);
    a.dx = dx;
    a.dresidual = dresidual;
    a.part = dweight ? (float *)workspace : nullptr;
    int g;
    const void *kernel = norm_pick<Backward>(dtype, d, g);
    grid = norm_back_grid(n_rows, g);
    void *kargs[] = {&a};
    if (hipLaunchKernel(kernel, dim3(grid), dim3(NORM_THREADS), kargs, 0, st) != hipSuccess) {
      (void)hipGetLastError();
      return MAXSIM_ERR_LAUNCH;
    }
  }
  if (!dweight) return MAXSIM_OK;
  const dim3 cols((d + 31) / 32);
  const float *part = (const float *)workspace;
  if (weight_dtype == MAXSIM_FP32)
    hipLaunchKernelGGL(norm_weight_kernel<float>, cols, dim3(NORM_THREADS), 0, st, part, (int)grid, d, (float *)dweight);
  else if (weight_dtype == MAXSIM_FP16)
    hipLaunchKernelGGL(norm_weight_kernel<_Float16>, cols, dim3(NORM_THREADS), 0, st, part, (int)grid, d, (_Float16 *)dweight);
  else
    hipLaunchKernelGGL(norm_weight_kernel<__bf16>, cols, dim3(NORM_THREADS), 0, st, part, (int)grid, d, (__bf16 *)dweight);
  return hipGetLastError() == hipSuccess ? MAXSIM_OK : MAXSIM_ERR_LAUNCH;
}

}  // extern "C"
