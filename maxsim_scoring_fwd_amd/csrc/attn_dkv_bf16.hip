// Attention dkv kernels, bf16.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

MAXSIM_ATTN_PICK(attn_dkv_bf16, attn_dkv_kernel, DT_BF16)
