// The lengths of pieces that the plan of chunk attention chooses from, for the kernel and for
// tests on the host.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#define DGT_BOTH __host__ __device__ __forceinline__
#else
#define DGT_BOTH inline
#endif

namespace dgt {
namespace serve {

constexpr uint32_t kChoices = 32;

// Choice i cuts the longest tile, of `units` times 64 keys (up to 2^25), into about 1.25^i pieces of at
// least two units; choice 0 leaves it whole.
DGT_BOTH uint32_t piece_units(uint32_t units, uint32_t choice) {
  if (choice == 0) return units;  // (above 2^24 fp32 would round an odd number down, and cut it)
  const uint32_t len = (uint32_t)ceilf((float)units * exp2f(-0.32192809f * (float)choice)), least = units < 2 ? units : 2;
  return len > least ? len : least;
}

}  // namespace serve
}  // namespace dgt
