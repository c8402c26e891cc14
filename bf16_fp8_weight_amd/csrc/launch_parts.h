// launch_parts.h -- grids of more threads than one launch takes. No GPU call.
#pragma once

#include <cstdint>

namespace wt {

// One launch takes fewer than 2^32 threads: a grid of more is launched in parts. Calls launch(first, count) for each, in order,
// until one does not return `ok`; a part begins at a multiple of 8 workgroups, so that they go round the 8 XCDs as in one grid.
constexpr int64_t max_groups(int64_t threads) { return (((int64_t)1 << 32) / threads - 1) / 8 * 8; }

template <class Status, class F>
Status launch_parts(int64_t groups, int64_t threads, Status ok, F launch) {
  const int64_t most = max_groups(threads);
  Status st = ok;
  for (int64_t first = 0; first < groups && st == ok; first += most)
    st = launch((uint32_t)first, (uint32_t)(groups - first < most ? groups - first : most));
  return st;
}

}  // namespace wt
