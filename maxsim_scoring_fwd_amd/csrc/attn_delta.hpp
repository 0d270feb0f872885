// What the backward kernels take from dO before them: <dO, o> of every row, and for fp16 the
// scale of dS. One read of dO and o: 52 us for 252 MB (4.8 TB/s, a plain copy's rate) over 512
// documents of 20 to 300 tokens and 12 heads of 64 in bf16.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

constexpr int DELTA_GRID = 1024;

// For each row of a head where the sums of dK / dV's products start: S from -lse in units of the
// product (of the score behind a tanh; + shift, see ATTN_WEIGHT_SHIFT), dP from -delta, delta =
// <dO, o> in fp32. 8 lanes to a row. With maxima set (fp16) also the largest squared norm of the
// rows of dO and of v, one pair per workgroup.
template <int DT>
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnArgs a, float2 *stats, float2 *maxima, float unit, float shift) {
  using T = typename AttnElem<DT>::type;
  constexpr int V = 16 / Elem<DT>::bytes;
  typedef T vec __attribute__((ext_vector_type(V)));
  const int sub = threadIdx.x & 7;
  const int chunks = a.d / V;
  // Rows of no document hold anything: those past a fixed document's length, and those before the
  // first offset or after the last.
  const int64_t begin = DT == DT_FP16 && a.offsets ? a.offsets[0] : 0;
  const int64_t end = DT == DT_FP16 && a.offsets ? a.offsets[a.n_docs] : a.rows;
  auto exists = [&](uint32_t row) {
    if (!a.lens) return row >= begin && row < end;
    const uint32_t doc = row / (uint32_t)a.nd;
    return (int)(row - doc * (uint32_t)a.nd) < a.lens[doc];
  };
  auto sum8 = [](float s) {
    s += dpp_f32<DPP_XOR1>(s);
    s += dpp_f32<DPP_XOR2>(s);
    s += dpp_f32<DPP_HALF_MIRROR>(s);
    return s;
  };
  const int64_t per = gridDim.x * 32, n = a.rows * a.heads;
  float top_do = 0.0f, top_v = 0.0f;
  for (int64_t at = blockIdx.x * 32 + threadIdx.x / 8; at < n; at += per) {
    float s = 0.0f, w = 0.0f;
    for (int c = sub; c < chunks; c += 8) {
      const vec g = ((const vec *)a.dO)[at * chunks + c], o = ((const vec *)a.o)[at * chunks + c];
#pragma unroll
      for (int e = 0; e < V; e++) {
        s = __builtin_fmaf((float)g[e], (float)o[e], s);
        if (DT == DT_FP16) w = __builtin_fmaf((float)g[e], (float)g[e], w);
      }
    }
    s = sum8(s);
    const int64_t row = at / a.heads, head = at - row * a.heads;
    if (sub == 0) {
      const int64_t to = head * a.rows + row;
      stats[to] = make_float2((shift - a.lse[to] * LOG2E) / unit, -s);
    }
    if (DT == DT_FP16 && exists((uint32_t)row)) top_do = __builtin_fmaxf(top_do, sum8(w));
  }
  if constexpr (DT == DT_FP16) {
    const int64_t nv = a.rows * a.kv_heads;
    for (int64_t at = blockIdx.x * 32 + threadIdx.x / 8; at < nv; at += per) {
      const int64_t row = at / a.kv_heads, head = at - row * a.kv_heads;
      if (!exists((uint32_t)row)) continue;
      const int64_t doc = a.offsets ? 0 : row / a.nd, in = a.offsets ? row : row - doc * a.nd;
      const vec *p = (const vec *)(a.v + doc * a.v_doc + in * a.v_tok + head * a.v_head);
      float w = 0.0f;
      for (int c = sub; c < chunks; c += 8) {
        const vec x = p[c];
#pragma unroll
        for (int e = 0; e < V; e++) w = __builtin_fmaf((float)x[e], (float)x[e], w);
      }
      top_v = __builtin_fmaxf(top_v, sum8(w));
    }
    __shared__ float2 part[32];
    if (sub == 0) part[threadIdx.x / 8] = make_float2(top_do, top_v);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 32; i++) {
        top_do = __builtin_fmaxf(top_do, part[i].x);
        top_v = __builtin_fmaxf(top_v, part[i].y);
      }
      maxima[blockIdx.x] = make_float2(top_do, top_v);
    }
  }
}

// The power of two that fp16 dS is scaled by before its rounding. |dP - delta| is at most
// 2 |dO| |v| (o is a mean of v rows), so this keeps dS below 2^15 and uses the range below it:
// unscaled, a loss averaged over many tokens leaves dS in the subnormals.
__global__ void attn_grad_scale_kernel(const float2 *maxima, int n, float *out) {
  float x = 0.0f, y = 0.0f;
  for (int i = threadIdx.x; i < n; i += 64) {
    x = __builtin_fmaxf(x, maxima[i].x);
    y = __builtin_fmaxf(y, maxima[i].y);
  }
  for (int o = 32; o > 0; o >>= 1) {
    x = __builtin_fmaxf(x, __shfl_xor(x, o, 64));
    y = __builtin_fmaxf(y, __shfl_xor(y, o, 64));
  }
  if (threadIdx.x == 0) {
    const float both = __builtin_sqrtf(x) * __builtin_sqrtf(y);
    float s = 1.0f;
    if (both > 0.0f && both < 1e30f) {
      float e = __builtin_floorf(14.0f - __builtin_amdgcn_logf(both));
      e = e < -100.0f ? -100.0f : (e > 100.0f ? 100.0f : e);
      s = __builtin_ldexpf(1.0f, (int)e);
    }
    *out = s;
  }
}

}  // namespace maxsim
