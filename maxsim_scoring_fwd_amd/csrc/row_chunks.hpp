// Rows of any length in chunks of 8 entries: whole chunks as 16-byte accesses wherever they lie
// (the hardware takes them at any address that fits the type), the last, shorter one entry by
// entry.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace maxsim {

// A call that moves more than the chip's last cache holds passes it by (non-temporal loads and
// stores): its lines would be gone before anyone could use them, and writing them back costs the
// call itself or the next one. Dropout of a tensor, and of its result, and so on: 128 MiB (256 moved)
// 39.4 us through the caches and 43.7 past them, 192 MiB 69.5 and 65.2; a norm's forward and backward
// in turn, 64 MiB a tensor (256 moved by the forward) 85.0 and 90.1, 96 MiB 138.2 and 133.5. Only
// 16-bit types: a chunk of fp32 is two accesses, each of half of what its lanes' lines hold, which the
// caches have to put together (260416 x 768 in fp32 from 4 bits: 221 us through them, 346 past them;
// dropout of that tensor 285 and 307; the norm of 80000 x 768 with a residual 177 and 193).
constexpr int64_t CACHE_BYTES = (int64_t)256 << 20;
inline bool past_caches(int64_t bytes, int entry_bytes) { return entry_bytes == 2 && bytes > CACHE_BYTES; }

template <typename T> struct Chunk8 {
  T e[8];
} __attribute__((packed, aligned(sizeof(T))));

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // 16 bytes anywhere
template <bool ONCE = false, typename T> __device__ __forceinline__ Chunk8<T> whole_chunk(const T *p) {
  if constexpr (!ONCE) return *(const Chunk8<T> *)p;
  else return __builtin_bit_cast(Chunk8<T>, __builtin_nontemporal_load((const u32x4_any *)p));
}
template <bool ONCE = false, typename T> __device__ __forceinline__ void store_whole(T *p, const Chunk8<T> &c) {
  if constexpr (!ONCE) {
    *(Chunk8<T> *)p = c;
  } else {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4_any, c), (u32x4_any *)p);
  }
}

template <typename T> __device__ __forceinline__ Chunk8<T> rounded(const float (&v)[8]) {
  Chunk8<T> c;
#pragma unroll
  for (int e = 0; e < 8; e++) c.e[e] = (T)v[e];
  return c;
}

// Entries at .. at + 7 of a row of n; those past its end are 0.
template <typename T> __device__ __forceinline__ void load_chunk(const T *row, int at, int n, float (&v)[8]) {
  if (at + 8 <= n) {
    const Chunk8<T> c = *(const Chunk8<T> *)(row + at);
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = (float)c.e[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = at + e < n ? (float)row[at + e] : 0.0f;
  }
}

// Each value rounded once, to nearest even.
template <typename T> __device__ __forceinline__ void store_chunk(T *row, int at, int n, const float (&v)[8]) {
  if (at + 8 <= n) {
    Chunk8<T> c;
#pragma unroll
    for (int e = 0; e < 8; e++) c.e[e] = (T)v[e];
    *(Chunk8<T> *)(row + at) = c;
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (at + e < n) row[at + e] = (T)v[e];
  }
}

}  // namespace maxsim
