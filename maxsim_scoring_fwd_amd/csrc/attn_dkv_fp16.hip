// Attention dkv kernels, fp16.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

namespace maxsim {
namespace {
template <int DP, int WHAT> const void *pick(int mode) {
  switch (mode) {
  case ATTN_PLAIN: return (const void *)attn_dkv_kernel<DT_FP16, DP, ATTN_PLAIN, WHAT>;
  case ATTN_BIAS: return (const void *)attn_dkv_kernel<DT_FP16, DP, ATTN_BIAS, WHAT>;
  case ATTN_CAP: return (const void *)attn_dkv_kernel<DT_FP16, DP, ATTN_CAP, WHAT>;
  case ATTN_FAR_CAP: return (const void *)attn_dkv_kernel<DT_FP16, DP, ATTN_FAR_CAP, WHAT>;
  default: return (const void *)attn_dkv_kernel<DT_FP16, DP, ATTN_CAP_BIAS, WHAT>;
  }
}
}  // namespace

const void *attn_dkv_fp16(int dp, int mode, int part) {
  switch (dp) {
  case 32: return pick<32, 3>(mode);
  case 64: return pick<64, 3>(mode);
  case 96: return pick<96, 3>(mode);
  case 128: return pick<128, 3>(mode);
  case 256: return part ? pick<256, 2>(mode) : pick<256, 1>(mode);
  }
  return nullptr;
}

}  // namespace maxsim
