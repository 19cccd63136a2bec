// Host-side choices of the 8-bit and mixture-of-experts operators, free of HIP so that they can be compiled and checked alone.
#pragma once

#include <cstdint>

namespace fp4 {

// A grid of `groups` workgroups of `threads` threads. One dimension of a launch holds less than 2^32 work-items, so more than
// that continue in y; the kernel's workgroup is blockIdx.y * gridDim.x + blockIdx.x, and those from `groups` on leave.
// x is a multiple of 8 wherever y > 1: workgroups go to the 8 XCDs in turn by this number.
struct Grid {
  unsigned x, y;
};
inline Grid grid_of(int64_t groups, int threads) {
  const int64_t most = (int64_t)(0xFFFFFFFFu / (unsigned)threads) / 8 * 8;
  if (groups <= most) return {(unsigned)groups, 1};
  return {(unsigned)most, (unsigned)((groups + most - 1) / most)};
}

}  // namespace fp4
