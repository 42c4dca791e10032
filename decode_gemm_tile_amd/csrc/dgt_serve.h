// Shared pieces of the serving operators (page plan, cache store, tree
// attention, low-rank adapters): vector types, conversions between fp32 and the
// 16-bit types, wave and workgroup scans, searches over request offsets.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dgt.h"

namespace dgt {
namespace serve {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kCUs = 256;

// The two 16-bit element types.  pack2 rounds two fp32 values to nearest even
// (one v_cvt_pk instruction for bf16 on gfx950).
struct Bf16 {
  typedef __bf16 T;
  static __device__ __forceinline__ float up(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef __bf16 x2 __attribute__((ext_vector_type(2)));
    x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ float add2(uint32_t v, float c) {  // c + both halves
    typedef __bf16 x2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(x2, v), __builtin_bit_cast(x2, 0x3F803F80u), c, false);
  }
  static __device__ __forceinline__ bool finite2(uint32_t v) {  // both halves finite
    return (v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u;
  }
  static __device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};

struct F16 {
  typedef _Float16 T;
  static __device__ __forceinline__ float up(uint32_t bits) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef _Float16 x2 __attribute__((ext_vector_type(2)));
    x2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ float add2(uint32_t v, float c) {
    typedef _Float16 x2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(x2, v), __builtin_bit_cast(x2, 0x3C003C00u), c, false);
  }
  static __device__ __forceinline__ bool finite2(uint32_t v) {
    return (v & 0x7C00u) != 0x7C00u && (v & 0x7C000000u) != 0x7C000000u;
  }
  static __device__ __forceinline__ floatx4 mfma(u32x4 a, u32x4 b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

// Token range of request b, held inside [0, tokens] whatever cu holds.
__device__ __forceinline__ void request_rows(const int32_t* cu, uint32_t b, uint32_t tokens,
                                             uint32_t* first, uint32_t* count) {
  const uint32_t s = (uint32_t)min(max(cu[b], 0), (int)tokens);
  const uint32_t e = (uint32_t)min(max(cu[b + 1], 0), (int)tokens);
  *first = s;
  *count = e > s ? e - s : 0u;
}

// Chunks of at most `rows` tokens that never span two requests: chunk j of
// request b gets number cu[b] / rows + b + j.  Request b + 1 starts at least
// ceil(n_b / rows) numbers later, so no two chunks share one, and all lie below
// tokens / rows + requests + 1; numbers that no chunk has are idle.  Finds the
// last b in [0, count) with cu[b] / rows + b <= c, the whole wave probing 64
// places a round.
__device__ __forceinline__ uint32_t chunk_request(const int32_t* cu, uint32_t count, uint32_t rows,
                                                  uint32_t c) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, len = count;
  while (len > 1) {
    const uint32_t step = (len + 63) / 64, at = lane * step;
    bool before = lane == 0;
    if (lane > 0 && at < len) {
      const uint32_t b = lo + at;
      before = (uint32_t)max(cu[b], 0) / rows + b <= c;
    }
    const uint32_t hits = (uint32_t)__popcll(__ballot(before));
    const uint32_t skip = (hits - 1) * step;
    lo += skip;
    len = min(step, len - skip);
  }
  return lo;
}

// Keeps what is computed from v inside the loop it stands in: the rare paths'
// addresses would otherwise be formed ahead of all loops and hold registers there.
__device__ __forceinline__ void keep_here(uint32_t& v) { asm volatile("" : "+v"(v)); }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool power_of_two(uint32_t v) { return v && !(v & (v - 1)); }
inline int launched() { return hipGetLastError() == hipSuccess ? DGT_OK : DGT_E_HIP; }

// Page sizes that the operators take, and their bound on requests per call.
constexpr uint32_t kMinBlock = 8, kMaxBlock = 1024, kMaxRequests = 8192;
inline bool block_ok(uint32_t block) {
  return power_of_two(block) && block >= kMinBlock && block <= kMaxBlock;
}
// A pool's slots are numbered in 31 bits.
inline bool pool_ok(uint32_t blocks, uint32_t block) {
  return (uint64_t)blocks * block <= 0x7FFFFFFFull;
}

}  // namespace serve
}  // namespace dgt
