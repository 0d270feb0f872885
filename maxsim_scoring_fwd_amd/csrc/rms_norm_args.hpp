// What the norm's host side and kernels share (rms_norm_kernel.hpp).
#pragma once

#include "dropout_bits.hpp"
#include "host_common.hpp"

namespace maxsim {

constexpr int NORM_THREADS = 256;
constexpr int NORM_MOST_D = MAXSIM_MAX_NORM;

struct NormArgs {
  const void *x, *residual, *weight;
  int64_t x_stride, residual_stride;  // entries
  int64_t first, rows;                // first row of this launch, all rows
  int d;
  float eps, one_over_d;
  DropArgs drop;
  void *y, *h;
  int8_t *codes;
  float *scale, *rstd;
  // backward
  const void *grad_y, *grad_h;
  void *dx, *dresidual;
  float *part;  // [workgroups][d]: sums of the weight's gradient
};

enum { NORM_Y, NORM_I8, NORM_BACK };

// Rows of a group of lanes: where a lane holds one chunk of a row it takes two rows at once (500000
// rows of 128 in bf16 to 8 bits: 50.2 us one at a time, 47.3 two, 49.9 four).
template <int C> constexpr int norm_rows = C == 1 ? 2 : 1;

// Lanes of a row and chunks of a lane: the fewest lanes whose registers hold the row, so that the
// fewest of them stand idle at its end (768 entries: 32 lanes of 3 chunks). Rows that are no multiple
// of 8 entries have fewer forms.
inline int norm_lanes(int d) {
  const int n = (d + 7) / 8;
  return n <= 64 ? 16 : n <= 128 ? 32 : n <= 256 ? 64 : 256;
}
inline int norm_chunks(int d) {
  const int g = norm_lanes(d), c = ((d + 7) / 8 + g - 1) / g;
  return d % 8 == 0 || c <= 2 && g == 16 ? c : 4;
}

// The kernel (of the three above) for rows of d entries; weights in fp32 or in the rows' type; past the
// caches or not. fp32 rows have neither choice.
const void *norm_kernel_bf16(int which, int d, bool w32, bool once);
const void *norm_kernel_fp16(int which, int d, bool w32, bool once);
const void *norm_kernel_fp32(int which, int d);

}  // namespace maxsim
