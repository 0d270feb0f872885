// The fp32 kernels of maxsim_rms_norm.
#include "rms_norm_kernel.hpp"

const void *maxsim::norm_kernel_fp32(int which, int d, bool w32, bool once) {
  return norm_kernel_for<float>(which, d, w32, once);
}
