// Microscaled 4-bit vectors (include/maxsim.h, maxsim_quantize_mx4): 32 entries share a power of
// two, 2^(floor(log2 of the largest) - 2), and each is the nearest of 0, 1/2, 1, 3/2, 2, 3, 4 and 6
// times that, ties to the even code, 6 where it is larger. The conversions are the hardware's, on
// entries that were multiplied by an exact power of two first. Bytes bound both directions (1638401
// rows of 128 in bf16 on one MI355X: 84 us to codes, 531 MB at 6.3 TB/s, and 87 us back).
#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"
#include "row_chunks.hpp"

using namespace maxsim;

namespace {

constexpr int MX4_THREADS = 256;
constexpr int MX4_PER = 4;  // chunks of 8 entries of a thread, MX4_THREADS apart

// 2^(byte - 127), for bytes 0 .. 254
__device__ __forceinline__ float power_of(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

// Chunks of 8 entries; four neighbouring lanes hold a block of 32. n: chunks, a multiple of 4, so
// that the lanes of a block are in or out together. A thread past the end takes the last chunks
// again and stores nothing: no branch before the loads, which are all under way at once.
template <typename T, bool ONCE>
__global__ void __launch_bounds__(MX4_THREADS) mx4_quantize_kernel(const T *x, uint32_t *codes, uint8_t *scales,
                                                                   int64_t n, int64_t first) {
  const int64_t base = first + (int64_t)blockIdx.x * (MX4_THREADS * MX4_PER) + threadIdx.x;
  const int64_t last = n - 4 + (threadIdx.x & 3);
  Chunk8<T> c[MX4_PER];
#pragma unroll
  for (int i = 0; i < MX4_PER; i++) {
    const int64_t at = base + i * MX4_THREADS;
    c[i] = whole_chunk<ONCE>(x + (at < n ? at : last) * 8);
  }
#pragma unroll
  for (int i = 0; i < MX4_PER; i++) {
    const int64_t at = base + i * MX4_THREADS;
    float v[8];
    // bit patterns of absolute values: a NaN is above infinity, infinity above all numbers
    uint32_t most = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      v[e] = (float)c[i].e[e];
      const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
      most = b > most ? b : most;
    }
    uint32_t o = __builtin_amdgcn_update_dpp(0u, most, DPP_XOR1, 0xF, 0xF, true);
    most = o > most ? o : most;
    o = __builtin_amdgcn_update_dpp(0u, most, DPP_XOR2, 0xF, 0xF, true);
    most = o > most ? o : most;
    const bool finite = most < 0x7f800000u;
    const uint32_t ex = most >> 23;
    const uint32_t byte = finite ? (ex > 2 ? ex - 2 : 0) : 255;
    const float to = finite ? power_of(254 - byte) : 0.0f;
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] * to, v[1] * to, 1.0f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] * to, v[3] * to, 1.0f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] * to, v[5] * to, 1.0f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] * to, v[7] * to, 1.0f, 3);
    if (at < n) {
      q = finite ? q : 0;
      if (ONCE) __builtin_nontemporal_store(q, codes + at);
      else codes[at] = q;
      if ((threadIdx.x & 3) == 0) scales[at >> 2] = (uint8_t)byte;
    }
  }
}

template <typename T, bool ONCE>
__global__ void __launch_bounds__(MX4_THREADS) mx4_values_kernel(const uint32_t *codes, const uint8_t *scales, T *x,
                                                                 int64_t n, int64_t first) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const int64_t base = first + (int64_t)blockIdx.x * (MX4_THREADS * MX4_PER) + threadIdx.x;
  uint32_t q[MX4_PER], byte[MX4_PER];
#pragma unroll
  for (int i = 0; i < MX4_PER; i++) {
    const int64_t at = base + i * MX4_THREADS, in = at < n ? at : n - 1;
    q[i] = codes[in];
    byte[i] = scales[in >> 2];
  }
#pragma unroll
  for (int i = 0; i < MX4_PER; i++) {
    const int64_t at = base + i * MX4_THREADS;
    const float by = byte[i] < 255 ? power_of(byte[i]) : __builtin_nanf("");
    const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 3)};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = p[e / 2][e & 1] * by;
    if (at < n) store_whole<ONCE>(x + at * 8, rounded<T>(v));
  }
}

int mx4_sizes(int64_t n_rows, int d) {
  if (n_rows < 0 || n_rows > ((int64_t)1 << 36) || d < MAXSIM_MIN_D || d > MAXSIM_MAX_D || d % 32)
    return MAXSIM_ERR_SHAPE;
  return MAXSIM_OK;
}

template <typename Launch> int mx4_parts(int64_t n, Launch launch) {
  constexpr int64_t per = MX4_THREADS * MX4_PER;
  for (int64_t first = 0; first < n; first += (int64_t)LAUNCH_MOST * per) {
    const int64_t left = (n - first + per - 1) / per;
    launch((unsigned)(left < (int64_t)LAUNCH_MOST ? left : LAUNCH_MOST), first);
    if (hipGetLastError() != hipSuccess) return MAXSIM_ERR_LAUNCH;
  }
  return MAXSIM_OK;
}

// Whether n chunks in both forms pass the caches by.
template <typename T> bool mx4_once(int64_t n) { return past_caches(n * (int64_t)(8 * sizeof(T) + 4), sizeof(T)); }

template <typename T>
int mx4_quantize_run(const T *x, uint8_t *codes, uint8_t *scales, int64_t n, hipStream_t st) {
  auto kernel = mx4_quantize_kernel<T, false>;
  if constexpr (sizeof(T) == 2)
    if (mx4_once<T>(n)) kernel = mx4_quantize_kernel<T, true>;
  return mx4_parts(n, [&](unsigned grid, int64_t first) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(MX4_THREADS), 0, st, x, (uint32_t *)codes, scales, n, first);
  });
}

template <typename T>
int mx4_values_run(const uint8_t *codes, const uint8_t *scales, T *x, int64_t n, hipStream_t st) {
  auto kernel = mx4_values_kernel<T, false>;
  if constexpr (sizeof(T) == 2)
    if (mx4_once<T>(n)) kernel = mx4_values_kernel<T, true>;
  return mx4_parts(n, [&](unsigned grid, int64_t first) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(MX4_THREADS), 0, st, (const uint32_t *)codes, scales, x, n, first);
  });
}

}  // namespace

extern "C" {

int maxsim_quantize_mx4(const void *x, int64_t n_rows, int d, int dtype, uint8_t *codes, uint8_t *scales,
                        void *stream) {
  if (elem_bytes(dtype) == 0) return MAXSIM_ERR_DTYPE;
  int rc = mx4_sizes(n_rows, d);
  if (rc != MAXSIM_OK) return rc;
  if (n_rows == 0) return MAXSIM_OK;
  if (!x || !codes || !scales) return MAXSIM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16)) return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  switch (dtype) {
  case MAXSIM_BF16: return mx4_quantize_run((const __bf16 *)x, codes, scales, n_rows * (d / 8), st);
  case MAXSIM_FP16: return mx4_quantize_run((const _Float16 *)x, codes, scales, n_rows * (d / 8), st);
  default: return mx4_quantize_run((const float *)x, codes, scales, n_rows * (d / 8), st);
  }
}

int maxsim_dequantize_mx4(const uint8_t *codes, const uint8_t *scales, int64_t n_rows, int d, int dtype, void *x,
                          void *stream) {
  if (elem_bytes(dtype) == 0) return MAXSIM_ERR_DTYPE;
  int rc = mx4_sizes(n_rows, d);
  if (rc != MAXSIM_OK) return rc;
  if (n_rows == 0) return MAXSIM_OK;
  if (!x || !codes || !scales) return MAXSIM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16)) return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  switch (dtype) {
  case MAXSIM_BF16: return mx4_values_run(codes, scales, (__bf16 *)x, n_rows * (d / 8), st);
  case MAXSIM_FP16: return mx4_values_run(codes, scales, (_Float16 *)x, n_rows * (d / 8), st);
  default: return mx4_values_run(codes, scales, (float *)x, n_rows * (d / 8), st);
  }
}

}  // extern "C"
