// libmaxsim attention entry points (include/maxsim.h).
#include <hip/hip_runtime.h>

#include <cmath>

#include "attn_delta.hpp"
#include "attn_dispatch.hpp"
#include "host_common.hpp"
#include "launch_parts.hpp"

using namespace maxsim;

namespace {

constexpr int64_t MAX_TOKEN_BYTES = (int64_t)1 << 24;  // 64 rows of it stay within 31 bits

// A tensor's strides (in elements, all multiples of 16 bytes) as byte strides.
int strides(const maxsim_attention_tensor &x, int eb, int64_t &doc, int64_t &head, int &tok) {
  if (!x.data) return MAXSIM_ERR_NULL;
  if (!aligned(x.data, 16) || (x.doc_stride * eb) % 16 || (x.head_stride * eb) % 16 ||
      (x.token_stride * eb) % 16)
    return MAXSIM_ERR_ALIGN;
  if (x.token_stride < 0 || x.token_stride * eb > MAX_TOKEN_BYTES || x.head_stride < 0 || x.doc_stride < 0)
    return MAXSIM_ERR_SHAPE;
  doc = x.doc_stride * eb;
  head = x.head_stride * eb;
  tok = (int)(x.token_stride * eb);
  return MAXSIM_OK;
}

// Tiles of `rows` tokens.
int set_tiles(AttnArgs &a, int rows) {
  const int64_t per_doc = ((int64_t)a.nd + rows - 1) / rows;
  const int64_t slots = a.offsets ? a.n_tokens / rows + a.n_docs + 2 : a.n_docs * per_doc;
  a.tiles_per_doc.set(per_doc ? (uint32_t)per_doc : 1);
  if (slots > 0x7fffffff || slots * a.heads > 0x7fffffff) return MAXSIM_ERR_SHAPE;
  a.slots = (uint32_t)slots;
  return MAXSIM_OK;
}

int fill(const maxsim_attention_desc *s, AttnArgs &a) {
  if (!s) return MAXSIM_ERR_NULL;
  const int eb = elem_bytes(s->dtype);
  if (eb == 0) return MAXSIM_ERR_DTYPE;
  const bool packed = s->doc_offsets != nullptr;
  if (s->n_docs < 0 || s->n_docs > 0x7fffffff || s->n_tokens < 0 || s->n_heads < 1 || s->n_kv_heads < 1 ||
      s->n_heads % s->n_kv_heads || s->d < 8 || s->d > MAXSIM_MAX_HEAD || s->d % 8)
    return MAXSIM_ERR_SHAPE;
  if (!packed && (s->nd < 0 || s->n_tokens != s->n_docs * s->nd)) return MAXSIM_ERR_SHAPE;
  if (s->n_tokens >= ((int64_t)1 << 31) || s->n_heads > 65535 ||
      (int64_t)s->n_heads * s->d * eb > MAX_TOKEN_BYTES)
    return MAXSIM_ERR_SHAPE;
  if (!(s->scale > 0) || !std::isfinite(s->scale) || !(s->softcap >= 0) || !std::isfinite(s->softcap))
    return MAXSIM_ERR_SHAPE;
  if (packed && s->doc_lens) return MAXSIM_ERR_UNSUPPORTED;
  if (s->prefix_lens && !s->causal) return MAXSIM_ERR_UNSUPPORTED;
  if (s->dtype == MAXSIM_FP32 && s->d > MAXSIM_MAX_HEAD_FP32) return MAXSIM_ERR_UNSUPPORTED;
  if (!aligned(s->doc_offsets, 8) || !aligned(s->doc_lens, 4) || !aligned(s->prefix_lens, 4) ||
      !aligned(s->slopes, 4))
    return MAXSIM_ERR_ALIGN;
  if (s->n_tokens == 0) return MAXSIM_OK;
  int rc = strides(s->q, eb, a.q_doc, a.q_head, a.q_tok);
  if (rc == MAXSIM_OK) rc = strides(s->k, eb, a.k_doc, a.k_head, a.k_tok);
  if (rc == MAXSIM_OK) rc = strides(s->v, eb, a.v_doc, a.v_head, a.v_tok);
  if (rc != MAXSIM_OK) return rc;
  a.q = (const char *)s->q.data;
  a.k = (const char *)s->k.data;
  a.v = (const char *)s->v.data;
  a.offsets = s->doc_offsets;
  a.n_tokens = a.rows = s->n_tokens;
  a.n_docs = s->n_docs;
  a.nd = packed ? 0 : s->nd;
  a.lens = s->doc_lens;
  a.prefix = s->prefix_lens;
  a.heads = s->n_heads;
  a.kv_heads = s->n_kv_heads;
  a.group = s->n_heads / s->n_kv_heads;
  a.d = s->d;
  a.causal = s->causal != 0;
  a.softcap = s->softcap;
  a.scale = s->scale;
  a.slopes = s->slopes;
  return set_tiles(a, ATTN_ROWS);
}

int mode_of(const AttnArgs &a, int dtype) {
  const bool cap = a.softcap > 0 && a.softcap <= ATTN_NO_CAP;
  if (cap && dtype != MAXSIM_FP32 && a.softcap > ATTN_NEAR_CAP) return ATTN_FAR_CAP;
  return (cap ? ATTN_CAP : ATTN_PLAIN) + (a.slopes ? ATTN_BIAS : 0);
}

// One workgroup for every tile of tokens and each of n_heads heads.
int run(const void *fn, AttnArgs &a, int n_heads, hipStream_t st) {
  a.per_group.set((uint32_t)(n_heads / a.kv_heads));
  a.per_kv.set(a.slots * a.per_group.d);
  a.total = a.slots * (uint32_t)n_heads;
  void *kargs[] = {&a};
  for (a.base = 0; a.base < a.total; a.base += LAUNCH_MOST) {
    const uint32_t left = a.total - a.base, grid = left < LAUNCH_MOST ? left : LAUNCH_MOST;
    if (hipLaunchKernel(fn, dim3(grid), dim3(ATTN_THREADS), kargs, 0, st) != hipSuccess) {
      (void)hipGetLastError();
      return MAXSIM_ERR_LAUNCH;
    }
  }
  return MAXSIM_OK;
}

const void *pick(int dtype, int dp, int mode, const void *(*bf)(int, int),
                 const void *(*fp)(int, int), const void *(*f32)(int, int)) {
  return dtype == MAXSIM_BF16 ? bf(dp, mode) : dtype == MAXSIM_FP16 ? fp(dp, mode) : f32(dp, mode);
}

size_t stat_floats(int64_t n_tokens, int n_heads) {
  return ((size_t)n_tokens * (size_t)n_heads + 1) / 2 * 4;
}

}  // namespace

extern "C" {

int maxsim_attention(const maxsim_attention_desc *desc, void *o, float *lse, void *stream) {
  AttnArgs a{};
  int rc = fill(desc, a);
  if (rc != MAXSIM_OK) return rc;
  if (desc->n_tokens == 0) return MAXSIM_OK;
  if (!o || !lse) return MAXSIM_ERR_NULL;
  if (!aligned(o, 16) || !aligned(lse, 4)) return MAXSIM_ERR_ALIGN;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  a.o = (char *)o;
  a.lse = lse;
  return run(pick(desc->dtype, attn_width(a.d), mode_of(a, desc->dtype), attn_fwd_bf16, attn_fwd_fp16, attn_fwd_fp32),
             a, a.heads, (hipStream_t)stream);
}

size_t maxsim_attention_backward_workspace_size(int64_t n_tokens, int n_heads) {
  if (n_tokens < 0 || n_heads < 1) return 0;
  return (stat_floats(n_tokens, n_heads) + 2 * DELTA_GRID + 4) * sizeof(float);
}

int maxsim_attention_backward(const maxsim_attention_desc *desc, const void *o, const float *lse,
                              const void *grad_o, void *dq, void *dk, void *dv, void *workspace,
                              size_t workspace_bytes, void *stream) {
  AttnArgs a{};
  int rc = fill(desc, a);
  if (rc != MAXSIM_OK) return rc;
  if (desc->n_tokens == 0) return MAXSIM_OK;
  if (!o || !lse || !grad_o || !workspace) return MAXSIM_ERR_NULL;
  if (!aligned(o, 16) || !aligned(lse, 4) || !aligned(grad_o, 16) || !aligned(dq, 16) ||
      !aligned(dk, 16) || !aligned(dv, 16) || !aligned(workspace, 16))
    return MAXSIM_ERR_ALIGN;
  if ((dk == nullptr) != (dv == nullptr)) return MAXSIM_ERR_NULL;
  if (workspace_bytes < maxsim_attention_backward_workspace_size(desc->n_tokens, desc->n_heads))
    return MAXSIM_ERR_SHAPE;
  if (!dq && !dk) return MAXSIM_OK;
  DeviceInfo di;
  rc = current_device(di);
  if (rc != MAXSIM_OK) return rc;
  hipStream_t st = (hipStream_t)stream;
  a.o = (char *)const_cast<void *>(o);
  a.lse = const_cast<float *>(lse);
  a.dO = (const char *)grad_o;
  a.dq = (char *)dq;
  a.dk = (char *)dk;
  a.dv = (char *)dv;
  float2 *stats = (float2 *)workspace;
  float2 *maxima = (float2 *)((float *)workspace + stat_floats(a.rows, a.heads));
  float *gscale = (float *)(maxima + DELTA_GRID);
  a.stats = stats;
  a.grad_scale = gscale;
  // 32 rows of a head a workgroup; fp16 needs one pair of maxima from each, so there are few
  int64_t grid = (a.rows * a.heads + 31) / 32;
  const int64_t most = desc->dtype == MAXSIM_FP16 ? DELTA_GRID : 16 * di.cus;
  if (grid > most) grid = most;
  const void *fn = desc->dtype == MAXSIM_BF16   ? (const void *)attn_delta_kernel<DT_BF16>
                   : desc->dtype == MAXSIM_FP16 ? (const void *)attn_delta_kernel<DT_FP16>
                                                : (const void *)attn_delta_kernel<DT_FP32>;
  const int dp = attn_width(a.d), mode = mode_of(a, desc->dtype);
  float unit = has_cap(mode) ? 1.0f : a.scale * LOG2E;
  // what exponents of the weights have beside the product: see ATTN_WEIGHT_SHIFT, ScoreForm::c
  float shift = desc->dtype == MAXSIM_FP16 ? ATTN_WEIGHT_SHIFT : 0.0f;
  if ((mode == ATTN_CAP || mode == ATTN_CAP_BIAS) && desc->dtype != MAXSIM_FP32) shift += a.softcap * LOG2E;
  void *kargs[] = {&a, &stats, &maxima, &unit, &shift};
  if (hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), kargs, 0, st) != hipSuccess) {
    (void)hipGetLastError();
    return MAXSIM_ERR_LAUNCH;
  }
  if (desc->dtype == MAXSIM_FP16) {
    hipLaunchKernelGGL(attn_grad_scale_kernel, dim3(1), dim3(64), 0, st, maxima, (int)grid, gscale);
    if (hipGetLastError() != hipSuccess) return MAXSIM_ERR_LAUNCH;
  }
  if (dq) {
    rc = run(pick(desc->dtype, dp, mode, attn_dq_bf16, attn_dq_fp16, attn_dq_fp32), a, a.heads, st);
    if (rc != MAXSIM_OK) return rc;
  }
  for (int part = 0; dk && part < attn_dkv_launches(dp); part++) {
    const void *kernel = desc->dtype == MAXSIM_BF16   ? attn_dkv_bf16(dp, mode, part)
                         : desc->dtype == MAXSIM_FP16 ? attn_dkv_fp16(dp, mode, part)
                                                      : attn_dkv_fp32(dp, mode, part);
    rc = run(kernel, a, a.kv_heads, st);
    if (rc != MAXSIM_OK) return rc;
  }
  return MAXSIM_OK;
}

}  // extern "C"
