// Attention dq kernels, bf16.
#include "attn_dispatch.hpp"
#include "attn_bwd_kernel.hpp"

namespace maxsim {
namespace {
template <int DP> const void *pick(int mode) {
  switch (mode) {
  case ATTN_PLAIN: return (const void *)attn_dq_kernel<DT_BF16, DP, ATTN_PLAIN>;
  case ATTN_BIAS: return (const void *)attn_dq_kernel<DT_BF16, DP, ATTN_BIAS>;
  case ATTN_CAP: return (const void *)attn_dq_kernel<DT_BF16, DP, ATTN_CAP>;
  case ATTN_FAR_CAP: return (const void *)attn_dq_kernel<DT_BF16, DP, ATTN_FAR_CAP>;
  default: return (const void *)attn_dq_kernel<DT_BF16, DP, ATTN_CAP_BIAS>;
  }
}
}  // namespace

const void *attn_dq_bf16(int dp, int mode) {
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
