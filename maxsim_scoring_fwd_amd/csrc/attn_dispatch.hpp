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
// part: 0, or 1 where there are two launches (attn_dkv_launches).
const void *attn_dkv_bf16(int dp, int mode, int part);
const void *attn_dkv_fp16(int dp, int mode, int part);
const void *attn_dkv_fp32(int dp, int mode, int part);

// Head sizes are rounded up to one of these widths; the columns past the size are zeros. fp32
// heads wider than 128 have no kernel (nullptr): they would need more registers than a wave has.
inline int attn_width(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : 256; }

inline int attn_dkv_launches(int dp) { return dp > 128 ? 2 : 1; }

}  // namespace maxsim
