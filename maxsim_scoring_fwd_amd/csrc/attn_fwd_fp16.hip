// Attention fwd kernels, fp16.
#include "attn_dispatch.hpp"
#include "attn_fwd_kernel.hpp"

MAXSIM_ATTN_PICK(attn_fwd_fp16, attn_fwd_kernel, DT_FP16)
