// maxsim_rms_norm, its 8-bit form and its backward: checks, sizes and launches (the kernels are in
// rms_norm_kernel.hpp).
#include <hip/hip_runtime.h>

#include "host_common.hpp"
#include "launch_parts.hpp"
#include "rms_norm_args.hpp"
#include "row_chunks.hpp"

using namespace maxsim;

namespace {

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

// tensors: how many of n_rows x d the call moves.
const void *norm_kernel(int which, int dtype, int64_t n_rows, int d, int weight_dtype, int tensors) {
  const bool w32 = weight_dtype == MAXSIM_FP32;
  const bool once = past_caches(n_rows * d * elem_bytes(dtype) * tensors, elem_bytes(dtype));
  return dtype == MAXSIM_FP32   ? norm_kernel_fp32(which, d)
         : dtype == MAXSIM_FP16 ? norm_kernel_fp16(which, d, w32, once)
                                : norm_kernel_bf16(which, d, w32, once);
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
  return norm_launch(norm_kernel(NORM_Y, dtype, n_rows, d, weight_dtype, 2 + (residual != nullptr) + (h != nullptr)), a, (hipStream_t)stream);
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
  return norm_launch(norm_kernel(NORM_I8, dtype, n_rows, d, weight_dtype, 0), a, (hipStream_t)stream);
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
    const void *kernel = norm_kernel(NORM_BACK, dtype, n_rows, d, weight_dtype,
                                     2 + (grad_h != nullptr) + (dx != nullptr) + (dresidual != nullptr));
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
