// Rows of any length in chunks of 8 entries: whole chunks as 16-byte accesses wherever they lie
// (the hardware takes them at any address that fits the type), the last, shorter one entry by
// entry.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace maxsim {

template <typename T> struct Chunk8 {
  T e[8];
} __attribute__((packed, aligned(sizeof(T))));

template <typename T> __device__ __forceinline__ Chunk8<T> whole_chunk(const T *p) { return *(const Chunk8<T> *)p; }
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
