// Rotary positions (include/maxsim.h, maxsim_rotary): each pair (a, b) of a head is turned by
// the angle position * freq. One read and one write of the tensor bound it: the angles of a
// token (rot / 2 of them) are computed once and shared by all its heads. Measured (one MI355X):
// 207 us for 1.08 GB of 40 fp16 heads of 128 (5.2 TB/s; a 2 GiB copy runs at 4.9), 84 us for 396 MB
// of 16 fp32 heads of 96 with positions given (4.7 TB/s); 3.5 us for one query's 24 heads.
#include <hip/hip_runtime.h>

#include "doc_lookup.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"

using namespace maxsim;

namespace {

constexpr int ROT_THREADS = 256;
constexpr int ROT_ANGLES = 1024;  // angles of a workgroup's tokens held in LDS (8 KiB)

struct RotaryArgs {
  const char *x;
  char *y;
  int64_t x_token, x_head, y_token, y_head;  // strides in bytes
  int64_t first, n_tokens;  // first token of this launch; all tokens
  const float *freq;
  const int64_t *offsets;
  int64_t n_docs;
  const int32_t *positions;
  float mscale, sign;
  int half, heads, tokens;  // pairs per head, heads, tokens per workgroup
  uint32_t per_token, per_head;      // units (two vectors) of a token and of a head
  uint32_t token_magic, head_magic;  // ceil(2^32 / per_token), ceil(2^32 / per_head)
};

// n / d for n, d < 2^16 and magic = ceil(2^32 / d): n * d < 2^32, so the product's high word is
// the exact quotient. d = 1 has no 32-bit magic.
__device__ __forceinline__ uint32_t div16(uint32_t n, uint32_t d, uint32_t magic) {
  return d == 1 ? n : __umulhi(n, magic);
}

template <typename T, int V> struct Vec {
  T e[V];
} __attribute__((packed, aligned(sizeof(T) * V)));

// T: storage type, V: elements per vector, INTER: pairs are neighbours (else half a rotated
// part apart). A unit is two vectors: the a's and the b's of V pairs, two neighbouring vectors
// that hold V whole pairs, or 2 V entries past the rotated part, which are copied.
// 2 GiB-long tensors and views: addresses are 64-bit, token by token.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(ROT_THREADS) rotary_kernel(RotaryArgs a) {
  __shared__ float2 turn[ROT_ANGLES];
  __shared__ int64_t place[64];
  const int64_t t0 = a.first + (int64_t)blockIdx.x * a.tokens;
  const int n = (int)(a.n_tokens - t0 < a.tokens ? a.n_tokens - t0 : a.tokens);
  const int tid = threadIdx.x;
  if (tid < n) {
    const int64_t t = t0 + tid;
    place[tid] = a.positions ? (int64_t)a.positions[t]
                 : a.offsets ? place_in_document(a.offsets, a.n_docs, t) : t;
  }
  __syncthreads();
  // 64-bit angles: a 32-bit product at position 30000 is off by 1e-3 radians. The turn count is
  // reduced to [-1/2, 1/2] before it is rounded to 32 bits, an error of at most 1e-7 radians.
  for (int i = tid; i < n * a.half; i += ROT_THREADS) {
    const int t = i / a.half, f = i - t * a.half;
    double turns = (double)place[t] * (double)a.freq[f] * 0.15915494309189533577;
    turns -= __builtin_rint(turns);
    float s, c;
    sincospif((float)(2.0 * turns), &s, &c);
    turn[i] = make_float2(c * a.mscale, s * a.mscale * a.sign);
  }
  __syncthreads();
  const bool copy = a.x != a.y || a.x_token != a.y_token || a.x_head != a.y_head;
  const uint32_t rot_units = (uint32_t)a.half / V;
  const uint32_t total = (uint32_t)n * a.per_token;
#pragma unroll 4
  for (uint32_t i = tid; i < total; i += ROT_THREADS) {
    const uint32_t t = div16(i, a.per_token, a.token_magic), r = i - t * a.per_token;
    const uint32_t h = div16(r, a.per_head, a.head_magic), u = r - h * a.per_head;
    const bool rot = u < rot_units;
    if (!rot && !copy) continue;
    const int first = rot && !INTER ? u * V : u * 2 * V;
    const int second = rot && !INTER ? first + a.half : first + V;
    const char *src = a.x + (t0 + t) * a.x_token + (int64_t)h * a.x_head;
    char *dst = a.y + (t0 + t) * a.y_token + (int64_t)h * a.y_head;
    Vec<T, V> p = *(const Vec<T, V> *)(src + first * sizeof(T));
    Vec<T, V> q = *(const Vec<T, V> *)(src + second * sizeof(T));
    if (rot) {
      const float2 *w = turn + t * a.half + u * V;
      if constexpr (INTER) {
        T z[2 * V];
#pragma unroll
        for (int e = 0; e < 2 * V; e++) z[e] = e < V ? p.e[e] : q.e[e - V];
#pragma unroll
        for (int e = 0; e < V; e++) {
          const float c = w[e].x, s = w[e].y, va = (float)z[2 * e], vb = (float)z[2 * e + 1];
          z[2 * e] = (T)(va * c - vb * s);
          z[2 * e + 1] = (T)(vb * c + va * s);
        }
#pragma unroll
        for (int e = 0; e < V; e++) {
          p.e[e] = z[e];
          q.e[e] = z[e + V];
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; e++) {
          const float c = w[e].x, s = w[e].y, va = (float)p.e[e], vb = (float)q.e[e];
          p.e[e] = (T)(va * c - vb * s);
          q.e[e] = (T)(vb * c + va * s);
        }
      }
    }
    *(Vec<T, V> *)(dst + first * sizeof(T)) = p;
    *(Vec<T, V> *)(dst + second * sizeof(T)) = q;
  }
}

template <typename T, int V>
const void *rotary_pick(bool inter) {
  return inter ? (const void *)rotary_kernel<T, V, true> : (const void *)rotary_kernel<T, V, false>;
}

template <typename T> const void *rotary_pick(int v, bool inter) {
  switch (v) {
  case 8:
    if constexpr (sizeof(T) == 2) return rotary_pick<T, 8>(inter);
    [[fallthrough]];
  case 4: return rotary_pick<T, 4>(inter);
  case 2: return rotary_pick<T, 2>(inter);
  default: return rotary_pick<T, 1>(inter);
  }
}

}  // namespace

extern "C" int maxsim_rotary(const void *x, int64_t n_tokens, int n_heads, int d,
                             int64_t x_token_stride, int64_t x_head_stride, int dtype,
                             const float *freq, int rot, int layout, float mscale, int inverse,
                             const int64_t *doc_offsets, int64_t n_docs, const int32_t *positions,
                             void *out, int64_t out_token_stride, int64_t out_head_stride,
                             void *stream) {
  const int eb = elem_bytes(dtype);
  if (eb == 0) return MAXSIM_ERR_DTYPE;
  if (n_tokens < 0 || n_heads < 1 || d < 2 || d > MAXSIM_MAX_D || d % 2 ||
      (int64_t)n_heads * d > 65536 || rot < 2 || rot > d || rot % 2 || n_docs < 0)
    return MAXSIM_ERR_SHAPE;
  if (layout != MAXSIM_ROTARY_HALF && layout != MAXSIM_ROTARY_INTERLEAVED)
    return MAXSIM_ERR_UNSUPPORTED;
  if (n_tokens == 0) return MAXSIM_OK;
  if (!x || !out || !freq) return MAXSIM_ERR_NULL;
  if (doc_offsets && positions) return MAXSIM_ERR_UNSUPPORTED;
  if (!aligned(x, eb) || !aligned(out, eb) || !aligned(freq, 4) ||
      (doc_offsets && !aligned(doc_offsets, 8)) || (positions && !aligned(positions, 4)))
    return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  int rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;

  // The widest vector that divides the rotated and the copied part, every stride and both
  // addresses: 16 bytes for whole rows of the usual head sizes.
  int v = 16 / eb;
  while (v > 1) {
    const int64_t b = (int64_t)v * eb;
    if (rot % (2 * v) == 0 && (d - rot) % (2 * v) == 0 && aligned(x, b) && aligned(out, b) &&
        x_token_stride % v == 0 && x_head_stride % v == 0 && out_token_stride % v == 0 &&
        out_head_stride % v == 0)
      break;
    v /= 2;
  }
  RotaryArgs a{};
  a.x = (const char *)x;
  a.y = (char *)out;
  a.x_token = x_token_stride * eb;
  a.x_head = x_head_stride * eb;
  a.y_token = out_token_stride * eb;
  a.y_head = out_head_stride * eb;
  a.n_tokens = n_tokens;
  a.freq = freq;
  a.offsets = doc_offsets;
  a.n_docs = n_docs;
  a.positions = positions;
  a.mscale = mscale;
  a.sign = inverse ? -1.0f : 1.0f;
  a.half = rot / 2;
  a.heads = n_heads;
  a.per_head = (uint32_t)(d / (2 * v));
  a.per_token = a.per_head * (uint32_t)n_heads;
  auto magic = [](uint32_t k) { return (uint32_t)(((uint64_t)1 << 32) / k + (((uint64_t)1 << 32) % k != 0)); };
  a.head_magic = magic(a.per_head);
  a.token_magic = magic(a.per_token);
  // Tokens per workgroup: about 8 units a thread, so that a token's angles cost little beside
  // its data, but one token where that leaves CUs without a workgroup.
  int64_t tokens = (ROT_THREADS * 8 + a.per_token - 1) / a.per_token;
  const int64_t share = (n_tokens + 2 * di.cus - 1) / (2 * di.cus);
  if (tokens > share) tokens = share;
  if (tokens > ROT_ANGLES / a.half) tokens = ROT_ANGLES / a.half;
  if (tokens > 64) tokens = 64;
  while (tokens > 1 && tokens * a.per_token > 65535) tokens--;
  a.tokens = (int)(tokens < 1 ? 1 : tokens);
  const bool inter = layout == MAXSIM_ROTARY_INTERLEAVED;
  const void *fn = dtype == MAXSIM_FP32   ? rotary_pick<float>(v, inter)
                   : dtype == MAXSIM_FP16 ? rotary_pick<_Float16>(v, inter)
                                          : rotary_pick<__bf16>(v, inter);
  void *kargs[] = {&a};
  const int64_t most = (int64_t)LAUNCH_MOST * a.tokens;
  for (a.first = 0; a.first < n_tokens; a.first += most) {
    const int64_t left = n_tokens - a.first < most ? n_tokens - a.first : most;
    const unsigned grid = (unsigned)((left + a.tokens - 1) / a.tokens);
    if (hipLaunchKernel(fn, dim3(grid), dim3(ROT_THREADS), kargs, 0, (hipStream_t)stream) != hipSuccess) {
      (void)hipGetLastError();
      return MAXSIM_ERR_LAUNCH;
    }
  }
  return MAXSIM_OK;
}
