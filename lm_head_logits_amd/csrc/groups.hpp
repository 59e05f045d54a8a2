// groups.hpp -- work-groups of a launch numbered beyond what one dimension
// takes (internal; the numbering is host code of its own, so that it can be
// checked without a GPU).
#pragma once

#include <stdint.h>

namespace lmhead {

// HIP takes fewer than 2^32 threads per dimension. Launches whose work-groups
// can pass that within the shape contract number them over x and y: x whole
// rows of 2^21 (2^31 threads of at most 1024 each), y as many as it takes. The
// last row's groups past the end find no work.
constexpr int GROUPS_X_BITS = 21;

struct GroupGrid {
  uint32_t x, y;
};
inline GroupGrid group_grid(int64_t n) {
  const int64_t most = (int64_t)1 << GROUPS_X_BITS;
  return n <= most ? GroupGrid{(uint32_t)n, 1} : GroupGrid{(uint32_t)most, (uint32_t)((n + most - 1) >> GROUPS_X_BITS)};
}

}  // namespace lmhead
