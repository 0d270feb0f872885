// Attention fwd kernels, fp16.
#include "attn_dispatch.hpp"
#include "attn_fwd_kernel.hpp"

namespace maxsim {
namespace {
template <int DP> const void *pick(int mode) {
  return mode == ATTN_PLAIN  ? (const void *)attn_fwd_kernel<DT_FP16, DP, ATTN_PLAIN>
         : mode == ATTN_BIAS ? (const void *)attn_fwd_kernel<DT_FP16, DP, ATTN_BIAS>
                             : (const void *)attn_fwd_kernel<DT_FP16, DP, ATTN_CAP>;
}
}  // namespace

const void *attn_fwd_fp16(int dp, int mode) {
  switch (dp) {
  case 32: return pick<32>(mode);
  case 64: return pick<64>(mode);
  case 96: return pick<96>(mode);
  case 128: return pick<128>(mode);
  case 256: return pick<256>(mode);
  }
  return nullptr;
}

}  // namespace maxsim
