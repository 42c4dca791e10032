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

// ------------------------------------------------- new tokens into the cache's pages
constexpr uint32_t kStoreRows = 64, kStoreDims = 128;  // a workgroup's tile; longer heads take several
constexpr uint32_t kStoreLine = kStoreRows + 2;        // elements of a value row in LDS

// Eight elements of a source row in the cache's type.
template <typename E, typename S>
__device__ __forceinline__ u32x4 load8(const S* p, bool wide) {
  if constexpr (sizeof(S) == 2) {
    if (wide) return *reinterpret_cast<const u32x4*>(p);
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = p[2 * j] | (uint32_t)p[2 * j + 1] << 16;
    return o;
  } else {
    floatx4 a, b;
    if (wide) {
      a = *reinterpret_cast<const floatx4*>(p);
      b = *reinterpret_cast<const floatx4*>(p + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = p[j];
        b[j] = p[4 + j];
      }
    }
    return u32x4{E::pack2(a[0], a[1]), E::pack2(a[2], a[3]), E::pack2(b[0], b[1]), E::pack2(b[2], b[3])};
  }
}

// Tokens of a tile whose slots follow one another within 8 aligned slots make a group: the
// wave's lanes hold a slot each (~0: no token, or one that is skipped); s_head gets the
// tokens that begin a group.
__device__ __forceinline__ void slot_groups(uint32_t slot, uint32_t* s_slot, uint32_t* s_head, uint32_t* s_heads) {
  const uint32_t t = threadIdx.x;
  s_slot[t] = slot;
  const uint32_t last = (uint32_t)__shfl_up((int)slot, 1, 64);
  const bool begins = slot != ~0u && (t == 0 || slot != last + 1 || last == ~0u || slot % 8 == 0);
  const uint64_t all = __ballot(begins);
  if (begins) s_head[__popcll(all & ((1ull << t) - 1))] = t;
  if (t == 0) *s_heads = (uint32_t)__popcll(all);
}

// Writes a tile's values, turned in LDS (s_v: kStoreLine elements a value row), into the
// pages of one head; vc points at the head's first page.
__device__ __forceinline__ void write_values(uint16_t* vc, uint32_t page_heads, uint32_t dim, uint32_t d0, uint32_t dims,
                                             uint32_t log_block, const uint16_t* s_v, const uint32_t* s_slot,
                                             const uint32_t* s_head, uint32_t heads) {
  const uint32_t block = 1u << log_block;
  // Two groups side by side, then the next value row, so that neighbours in memory go
  // to neighbouring lanes.
  for (uint32_t i = threadIdx.x; i < dims * (heads + (heads & 1)); i += 256) {
    const uint32_t two = i / (2 * dims), d = i / 2 % dims, group = 2 * two + (i & 1);
    if (group >= heads) continue;
    const uint32_t r0 = s_head[group], slot = s_slot[r0];
    uint16_t* to = vc + ((uint64_t)(slot >> log_block) * page_heads * dim + d0 + d) * block + (slot & (block - 1));
    const uint16_t* from = s_v + d * kStoreLine + r0;
    uint32_t n = 1;  // tokens of the group
    while (n < 8 - slot % 8 && r0 + n < kStoreRows && s_slot[r0 + n] == slot + n) ++n;
    if (n == 8) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = from[2 * j] | (uint32_t)from[2 * j + 1] << 16;
      *reinterpret_cast<u32x4*>(to) = o;
    } else {
      for (uint32_t j = 0; j < n; ++j) to[j] = from[j];
    }
  }
}

// Keeps what is computed from v inside the loop it stands in: the rare paths'
// addresses would otherwise be formed ahead of all loops and hold registers there.
__device__ __forceinline__ void keep_here(uint32_t& v) { asm volatile("" : "+v"(v)); }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool power_of_two(uint32_t v) { return v && !(v & (v - 1)); }
constexpr uint32_t kMaxGroups = 0xFFFFFF;  // workgroups of 256 threads: a launch counts threads in 32 bits
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
