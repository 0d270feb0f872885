// The bf16 kernels of maxsim_linear_cross_entropy.
#include "ce_dispatch.hpp"

namespace maxsim {

int ce_forward_bf16(const CeArgs &a, int cus, hipStream_t st) { return ce_forward<DT_BF16>(a, cus, st); }
int ce_backward_bf16(CeArgs &a, int64_t pieces, int cus, hipStream_t st) {
  return ce_backward<DT_BF16>(a, pieces, cus, st);
}

}  // namespace maxsim
