// group_launch.hpp -- launches whose work-groups are numbered over two grid
// dimensions (groups.hpp; internal).
#pragma once

#include <hip/hip_runtime.h>

#include "groups.hpp"

namespace lmhead {

// The grid of n numbered work-groups, and a work-group's number in it: n and
// above for the last ones, where n passes one dimension.
inline dim3 numbered_grid(int64_t n) {
  const GroupGrid g = group_grid(n);
  return dim3(g.x, g.y);
}
__device__ __forceinline__ int64_t group_number() {
  return ((int64_t)blockIdx.y << GROUPS_X_BITS) + blockIdx.x;
}

}  // namespace lmhead
