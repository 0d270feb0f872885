// Dropout (include/maxsim.h, maxsim_dropout): y = x / (1 - p) where an entry is kept, else 0. One
// read and one write of the tensor, or the generator's arithmetic, bounds it: a thread makes the
// bits of the 8 entries that it holds.
#include <hip/hip_runtime.h>

#include "dropout_bits.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"
#include "row_chunks.hpp"

using namespace maxsim;

namespace {

constexpr int DROP_THREADS = 256;
constexpr int DROP_PER = 4;  // chunks of a thread

template <typename T>
__global__ void __launch_bounds__(DROP_THREADS) dropout_kernel(const T *x, T *y, int64_t n, int64_t first,
                                                               DropArgs drop) {
  DropKey key;
  key.load(drop.rng);
  const int64_t base = first + (int64_t)blockIdx.x * (DROP_THREADS * DROP_PER * 8);
  const int left = (int)(n - base < DROP_THREADS * DROP_PER * 8 ? n - base : DROP_THREADS * DROP_PER * 8);
  float v[DROP_PER][8];
#pragma unroll
  for (int i = 0; i < DROP_PER; i++) {
    const int at = (i * DROP_THREADS + threadIdx.x) * 8;
    if (at < left) load_chunk(x + base, at, left, v[i]);
  }
#pragma unroll
  for (int i = 0; i < DROP_PER; i++) {
    const int at = (i * DROP_THREADS + threadIdx.x) * 8;
    if (at >= left) break;
    const uint32_t keep = drop_keep(key, drop, (uint64_t)(base + at) >> 3);
#pragma unroll
    for (int e = 0; e < 8; e++) v[i][e] = keep >> e & 1 ? v[i][e] * drop.up : 0.0f;
    store_chunk(y + base, at, left, v[i]);
  }
}

// p = 0, and p that rounds to it: a copy.
template <typename T>
__global__ void __launch_bounds__(DROP_THREADS) keep_kernel(const T *x, T *y, int64_t n, int64_t first) {
  const int64_t base = first + (int64_t)blockIdx.x * (DROP_THREADS * DROP_PER * 8);
  const int left = (int)(n - base < DROP_THREADS * DROP_PER * 8 ? n - base : DROP_THREADS * DROP_PER * 8);
#pragma unroll
  for (int i = 0; i < DROP_PER; i++) {
    const int at = (i * DROP_THREADS + threadIdx.x) * 8;
    if (at >= left) break;
    float v[8];
    load_chunk(x + base, at, left, v);
    store_chunk(y + base, at, left, v);
  }
}

template <typename T>
int dropout_run(const void *x, int64_t n, const DropArgs &drop, void *out, hipStream_t st) {
  constexpr int64_t per = DROP_THREADS * DROP_PER * 8;
  for (int64_t first = 0; first < n; first += (int64_t)LAUNCH_MOST * per) {
    const int64_t left = (n - first + per - 1) / per;
    const unsigned grid = (unsigned)(left < (int64_t)LAUNCH_MOST ? left : LAUNCH_MOST);
    if (drop.rng)
      hipLaunchKernelGGL(dropout_kernel<T>, dim3(grid), dim3(DROP_THREADS), 0, st, (const T *)x, (T *)out, n,
                         first, drop);
    else
      hipLaunchKernelGGL(keep_kernel<T>, dim3(grid), dim3(DROP_THREADS), 0, st, (const T *)x, (T *)out, n, first);
    if (hipGetLastError() != hipSuccess) return MAXSIM_ERR_LAUNCH;
  }
  return MAXSIM_OK;
}

}  // namespace

extern "C" int maxsim_dropout(const void *x, int64_t n, int dtype, double p, const int64_t *rng, int call,
                              void *out, void *stream) {
  const int eb = elem_bytes(dtype);
  if (eb == 0) return MAXSIM_ERR_DTYPE;
  if (n < 0 || n > ((int64_t)1 << 40) || !(p >= 0 && p <= 1) || call < 0) return MAXSIM_ERR_SHAPE;
  if (n == 0) return MAXSIM_OK;
  if (!x || !out || !rng) return MAXSIM_ERR_NULL;
  if (!aligned(x, eb) || !aligned(out, eb) || !aligned(rng, 8)) return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  const int rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  const DropArgs drop = drop_args(p, rng, call);
  hipStream_t st = (hipStream_t)stream;
  switch (dtype) {
  case MAXSIM_BF16: return dropout_run<__bf16>(x, n, drop, out, st);
  case MAXSIM_FP16: return dropout_run<_Float16>(x, n, drop, out, st);
  default: return dropout_run<float>(x, n, drop, out, st);
  }
}
