// Dropout (include/maxsim.h, maxsim_dropout): y = x / (1 - p) where an entry is kept, else 0. One
// read and one write of the tensor bound it, with the generator's arithmetic hidden behind them: a
// thread makes the bits of the 8 entries that it holds, for 4 chunks whose loads are under way
// together (81907 x 2048 in bf16 on one MI355X: 107 to 111 us, 671 MB at 6.2 TB/s, and 188 with loads
// that wait for each other; 101 x 513 3.1 us).
#include <hip/hip_runtime.h>

#include "dropout_bits.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"
#include "row_chunks.hpp"

using namespace maxsim;

namespace {

constexpr int DROP_THREADS = 256;
constexpr int DROP_PER = 4;  // chunks of a thread

// DROP: else a copy (p = 0, and p that rounds to it).
// ONCE: past the caches.
template <typename T, bool DROP, bool ONCE>
__global__ void __launch_bounds__(DROP_THREADS) dropout_kernel(const T *x, T *y, int64_t n, int64_t first,
                                                               DropArgs drop) {
  constexpr int PER = DROP_THREADS * DROP_PER * 8;
  DropKey key{};
  if (DROP) key.load(drop.rng);
  const int64_t base = first + (int64_t)blockIdx.x * PER;
  auto run = [&](int at, float (&v)[8]) {
    if (!DROP) return;
    DropBits bits;
    bits.make(key, drop, (uint64_t)(base + at) >> 3);
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = bits.apply(drop, e, v[e]);
  };
  if (n - base >= PER) {  // all of a thread's loads are under way at once
    Chunk8<T> c[DROP_PER];
#pragma unroll
    for (int i = 0; i < DROP_PER; i++) c[i] = whole_chunk<ONCE>(x + base + (i * DROP_THREADS + threadIdx.x) * 8);
#pragma unroll
    for (int i = 0; i < DROP_PER; i++) {
      const int at = (i * DROP_THREADS + threadIdx.x) * 8;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = (float)c[i].e[e];
      run(at, v);
      store_whole<ONCE>(y + base + at, rounded<T>(v));
    }
  } else {
    const int left = (int)(n - base);
    for (int at = threadIdx.x * 8; at < left; at += DROP_THREADS * 8) {
      float v[8];
      load_chunk(x + base, at, left, v);
      run(at, v);
      store_chunk(y + base, at, left, v);
    }
  }
}

template <typename T>
int dropout_run(const void *x, int64_t n, const DropArgs &drop, void *out, hipStream_t st) {
  constexpr int64_t per = DROP_THREADS * DROP_PER * 8;
  auto kernel = drop.rng ? dropout_kernel<T, true, false> : dropout_kernel<T, false, false>;
  if constexpr (sizeof(T) == 2)
    if (past_caches(2 * n * (int64_t)sizeof(T), sizeof(T)))
      kernel = drop.rng ? dropout_kernel<T, true, true> : dropout_kernel<T, false, true>;
  for (int64_t first = 0; first < n; first += (int64_t)LAUNCH_MOST * per) {
    const int64_t left = (n - first + per - 1) / per;
    const unsigned grid = (unsigned)(left < (int64_t)LAUNCH_MOST ? left : LAUNCH_MOST);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(DROP_THREADS), 0, st, (const T *)x, (T *)out, n, first, drop);
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
