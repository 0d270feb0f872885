// Attention dq kernels, bf16.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

MAXSIM_ATTN_PICK(attn_dq_bf16, attn_dq_kernel, DT_BF16)
