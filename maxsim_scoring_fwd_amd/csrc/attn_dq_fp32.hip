// Attention dq kernels, fp32.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

MAXSIM_ATTN_PICK(attn_dq_fp32, attn_dq_kernel, DT_FP32)
