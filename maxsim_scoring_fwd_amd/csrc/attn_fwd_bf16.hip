// Attention fwd kernels, bf16.
#include "attn_dispatch.hpp"
#include "attn_fwd_kernel.hpp"

namespace maxsim {
namespace {
template <int DP, int CB> const void *pick(int mode) {
  return mode == ATTN_PLAIN  ? (const void *)attn_fwd_kernel<DT_BF16, DP, ATTN_PLAIN, CB>
         : mode == ATTN_BIAS ? (const void *)attn_fwd_kernel<DT_BF16, DP, ATTN_BIAS, CB>
                             : (const void *)attn_fwd_kernel<DT_BF16, DP, ATTN_CAP, CB>;
}
}  // namespace

const void *attn_fwd_bf16(int dp, int mode, int blocks) {
  switch (dp) {
  case 32: return blocks == 2 ? pick<32, 2>(mode) : pick<32, 1>(mode);
  case 64: return blocks == 2 ? pick<64, 2>(mode) : pick<64, 1>(mode);
  case 96: return blocks == 2 ? pick<96, 2>(mode) : pick<96, 1>(mode);
  case 128: return blocks == 2 ? pick<128, 2>(mode) : pick<128, 1>(mode);
  case 256: return pick<256, 1>(mode);
  }
  return nullptr;
}

}  // namespace maxsim
