// Attention dkv kernels, fp16.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

MAXSIM_ATTN_PICK(attn_dkv_fp16, attn_dkv_kernel, DT_FP16)
