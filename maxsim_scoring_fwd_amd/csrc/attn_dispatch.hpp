// Kernels of the attention entry points by storage type: one translation unit each.
#pragma once

#include "attn_common.hpp"

namespace maxsim {

// The kernel for heads of up to dp columns (a width of attn_width) and a score form.
const void *attn_fwd_bf16(int dp, int mode);
const void *attn_fwd_fp16(int dp, int mode);
const void *attn_fwd_fp32(int dp, int mode);
const void *attn_dq_bf16(int dp, int mode);
const void *attn_dq_fp16(int dp, int mode);
const void *attn_dq_fp32(int dp, int mode);
const void *attn_dkv_bf16(int dp, int mode);
const void *attn_dkv_fp16(int dp, int mode);
const void *attn_dkv_fp32(int dp, int mode);

// Head sizes are rounded up to one of these widths; the columns past the size are zeros.
inline int attn_width(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : 256; }

#define MAXSIM_ATTN_MODES(KERNEL, DT, DP)                       \
  case DP:                                                      \
    return mode == ATTN_PLAIN  ? (const void *)KERNEL<DT, DP, ATTN_PLAIN> \
           : mode == ATTN_BIAS ? (const void *)KERNEL<DT, DP, ATTN_BIAS>  \
                               : (const void *)KERNEL<DT, DP, ATTN_CAP>;

// fp32 heads wider than 128 would need more registers than a wave has.
#define MAXSIM_ATTN_PICK(NAME, KERNEL, DT)          \
  namespace maxsim {                                \
  const void *NAME(int dp, int mode) {              \
    switch (dp) {                                   \
      MAXSIM_ATTN_MODES(KERNEL, DT, 32)             \
      MAXSIM_ATTN_MODES(KERNEL, DT, 64)             \
      MAXSIM_ATTN_MODES(KERNEL, DT, 96)             \
      MAXSIM_ATTN_MODES(KERNEL, DT, 128)            \
    }                                               \
    if constexpr (DT != DT_FP32)                    \
      switch (dp) { MAXSIM_ATTN_MODES(KERNEL, DT, 256) } \
    return nullptr;                                 \
  }                                                 \
  }

}  // namespace maxsim
