// The fp16 kernels of maxsim_rms_norm.
#include "rms_norm_kernel.hpp"

const void *maxsim::norm_kernel_fp16(int which, int d, bool w32, bool once) {
  return norm_kernel_for<_Float16>(which, d, w32, once);
}
