// Grids that are larger than a launch may be.
#pragma once

#include <stdint.h>

namespace maxsim {

// Most workgroups of 256 threads in one launch: a grid has fewer than 2^32 threads along x. Larger
// grids go in several launches. A multiple of 8, so that each begins on the first XCD.
constexpr uint32_t LAUNCH_MOST = 1u << 23;

}  // namespace maxsim
