// The fp32 kernels of maxsim_rms_norm.
#include "rms_norm_kernel.hpp"

const void *maxsim::norm_kernel_fp32(int which, int d) {
  return norm_kernel_for<float>(which, d, true, false);
}
