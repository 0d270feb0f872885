// The fp16 kernels of maxsim_linear_cross_entropy.
#include "ce_dispatch.hpp"

namespace maxsim {

int ce_forward_fp16(const CeArgs &a, int cus, hipStream_t st) { return ce_forward<DT_FP16>(a, cus, st); }
int ce_backward_fp16(CeArgs &a, int64_t pieces, int cus, hipStream_t st) {
  return ce_backward<DT_FP16>(a, pieces, cus, st);
}

}  // namespace maxsim
