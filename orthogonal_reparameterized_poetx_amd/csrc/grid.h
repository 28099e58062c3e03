// Work of more workgroups than one launch takes, shared by the launchers and by
// a host-side check.  Plain C++ (no HIP types).
#pragma once

#include <stdint.h>

namespace poetx {

// A launch takes fewer than 2^32 threads along x.  `count` workgroups of 256
// threads go in launches of at most GRID_MOST: launch(first, number) for each.
// (One launch of rows, with the workgroup's number formed from two, cost every
// workgroup: AdamW of 134 M bf16 values with 8-bit moments 329.5 us against 327.6 us.)
constexpr int64_t GRID_MOST = 1 << 23;
template <typename Launch>
inline void launches(int64_t count, Launch launch) {
  for (int64_t at = 0; at < count; at += GRID_MOST)
    launch(at, (uint32_t)(count - at < GRID_MOST ? count - at : GRID_MOST));
}

}  // namespace poetx
