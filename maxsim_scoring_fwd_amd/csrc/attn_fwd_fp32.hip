// Attention fwd kernels, fp32.
#include "attn_dispatch.hpp"
#include "attn_fwd_kernel.hpp"

namespace maxsim {
namespace {
template <int DP, int CB> const void *pick(int mode) {
  return mode == ATTN_PLAIN  ? (const void *)attn_fwd_kernel<DT_FP32, DP, ATTN_PLAIN, CB>
         : mode == ATTN_BIAS ? (const void *)attn_fwd_kernel<DT_FP32, DP, ATTN_BIAS, CB>
                             : (const void *)attn_fwd_kernel<DT_FP32, DP, ATTN_CAP, CB>;
}
}  // namespace

const void *attn_fwd_fp32(int dp, int mode, int blocks) {
  switch (dp) {
  case 32: return pick<32, 1>(mode);
  case 64: return pick<64, 1>(mode);
  case 96: return pick<96, 1>(mode);
  case 128: return pick<128, 1>(mode);
  }
  return nullptr;
}

}  // namespace maxsim
