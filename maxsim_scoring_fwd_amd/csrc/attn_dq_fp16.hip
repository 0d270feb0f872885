// Attention dq kernels, fp16.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

MAXSIM_ATTN_PICK(attn_dq_fp16, attn_dq_kernel, DT_FP16)
