// Queries, keys and values of new tokens: norms of heads, rotation by position, and the
// store into the paged cache, in one pass over the projection's rows.
#include "dgt_serve.h"

#include <algorithm>
#include <cmath>

namespace dgt {
namespace serve {
namespace {

// Rows and values are two kinds of workgroup of one launch: values are turned in LDS for their
// pages, and a row of queries or keys is 8 elements a lane, so norms and partners stay in a
// wave.  6792 tokens, 32 heads over 8 of 128, fp32, norms: 65 us, 3.8 TB/s (a copy 4.7), the rows
// alone 62; about 270 vector instructions a step of four heads are as much of it as the loads.  One
// token: 3.5 us.  Eight tokens a workgroup share their cosines; more and smaller workgroups, loads
// one step further ahead and non-temporal accesses took as long or longer.
struct RopeArgs {
  const void *q, *k, *v;
  const int32_t *positions, *slots;
  const double* freqs;
  const float *q_weight, *k_weight;
  uint16_t *q_out, *kc, *vc;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;  // element strides
  uint32_t tokens, heads, kv_heads, dim, pairs, log_block, blocks;
  uint32_t run, runs;        // heads of a row workgroup, and such workgroups a tile of tokens
  uint32_t row_groups;       // workgroups of rows; those of values follow
  float eps;
  bool interleaved, wide;    // wide: rows of q, k and v are 16-byte aligned
};

constexpr uint32_t kTokens = 8;  // of a row workgroup: their cosines are shared by all its heads
constexpr uint32_t kMaxDim = 256;

// cos and sin of 2 pi x, x in revolutions: the nearest quarter turn is taken off in fp64
// (a far position is millions of revolutions), and the Taylor series of both on what is
// left, |a| <= pi / 4, end below 2^-28.
__device__ __forceinline__ void turn(double x, float* c, float* s) {
  const double quarters = 4.0 * (x - __builtin_rint(x));
  const double whole = __builtin_rint(quarters);
  const float a = (float)(quarters - whole) * 1.57079632679f, z = a * a;
  const float sine = a * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), 1.f);
  const float cosine = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const int n = (int)whole & 3;
  *c = n == 0 ? cosine : n == 1 ? -sine : n == 2 ? -cosine : sine;
  *s = n == 0 ? sine : n == 1 ? cosine : n == 2 ? -sine : -cosine;
}

template <typename S>
__device__ __forceinline__ void load8f(const S* p, bool wide, float (&x)[8]);
template <>
__device__ __forceinline__ void load8f<float>(const float* p, bool wide, float (&x)[8]) {
  if (wide) {
    const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      x[4 + j] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[j];
  }
}
template <class E>
__device__ __forceinline__ void load8h(const uint16_t* p, bool wide, float (&x)[8]) {
  if (wide) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = E::up(a[j] & 0xFFFFu);
      x[2 * j + 1] = E::up(a[j] >> 16);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = E::up(p[j]);
  }
}
template <class E, typename S>
__device__ __forceinline__ void load_row(const S* p, bool wide, float (&x)[8]) {
  if constexpr (sizeof(S) == 4) load8f<float>(p, wide, x);
  else load8h<E>(p, wide, x);
}

// LDS traffic between the lanes of one wave: no instruction, but nothing moves across it.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// LANES lanes, 8 elements each, hold a head of up to 8 * LANES elements; a wave has
// 64 / LANES heads in hand.  A head's elements pass through the wave's own LDS to meet
// the other element of their pair.
template <class E, typename S, int LANES>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, float* s_cos, float* s_sin, float* s_x) {
  constexpr uint32_t kRows = 64 / LANES;  // of a wave
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const uint32_t t0 = blockIdx.x / a.runs * kTokens, live = min(a.tokens - t0, kTokens);
  const uint32_t h0 = blockIdx.x % a.runs * a.run, count = min(a.heads + a.kv_heads - h0, a.run);
  const uint32_t pairs = a.pairs;
  for (uint32_t i = t; i < live * pairs; i += 256) {
    const uint32_t tok = i / pairs;
    const int32_t pos = a.positions[t0 + tok];
    turn((double)pos * (a.freqs[i - tok * pairs] * 0.15915494309189533577), s_cos + i, s_sin + i);
  }
  __syncthreads();

  const uint32_t piece = lane % LANES, d = 8 * piece;
  const bool holds = d < a.dim;
  float* x_mine = s_x + (wave * kRows + lane / LANES) * (8 * LANES);  // this head's elements
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wq[e] = holds && a.q_weight ? a.q_weight[d + e] : 1.f;
    wk[e] = holds && a.k_weight ? a.k_weight[d + e] : 1.f;
  }
  const float inv_dim = 1.f / (float)a.dim;

  struct Row {
    float x[8];
    uint32_t tok, head;  // head: queries first, then keys
    bool on;
  };
  auto fetch = [&](uint32_t r0, Row& row) {
    const uint32_t r = r0 + lane / LANES;
    row.tok = r / count;
    row.head = h0 + r - row.tok * count;
    row.on = row.tok < live && a.positions[t0 + min(row.tok, live - 1)] >= 0;
    if (row.on && holds) {
      const S* p = row.head < a.heads
                       ? static_cast<const S*>(a.q) + (int64_t)(t0 + row.tok) * a.q_row + (int64_t)row.head * a.q_head
                       : static_cast<const S*>(a.k) + (int64_t)(t0 + row.tok) * a.k_row + (int64_t)(row.head - a.heads) * a.k_head;
      load_row<E, S>(p + d, a.wide, row.x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) row.x[e] = 0.f;
    }
  };
  auto finish = [&](Row& row) {
    const bool key = row.head >= a.heads;
    float (&x)[8] = row.x;
    if (key ? a.k_weight != nullptr : a.q_weight != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
      for (int m = 1; m < LANES; m <<= 1) sum += __shfl_xor(sum, m, 64);
      const float scale = 1.f / sqrtf(fmaf(sum, inv_dim, a.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= scale * (key ? wk[e] : wq[e]);
    }
    const float *c = s_cos + row.tok * pairs, *s = s_sin + row.tok * pairs;
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint32_t i = (d + e) / 2;
        if (row.on && i < pairs) {
          const float u = x[e], v = x[e + 1];
          x[e] = fmaf(u, c[i], -v * s[i]);
          x[e + 1] = fmaf(v, c[i], u * s[i]);
        }
      }
    } else if (pairs) {
      *reinterpret_cast<floatx4*>(x_mine + d) = floatx4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<floatx4*>(x_mine + d + 4) = floatx4{x[4], x[5], x[6], x[7]};
      wave_order();
      if (row.on && holds) {
        if (pairs % 4 == 0) {
          // four elements are on one side of their pairs
#pragma unroll
          for (int h = 0; h < 8; h += 4) {
            const uint32_t at = d + h;
            if (at < 2 * pairs) {
              const bool low = at < pairs;
              const uint32_t i = low ? at : at - pairs;
              const floatx4 o = *reinterpret_cast<const floatx4*>(x_mine + (low ? at + pairs : i));
              const floatx4 cs = *reinterpret_cast<const floatx4*>(c + i), sn = *reinterpret_cast<const floatx4*>(s + i);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[h + e] = fmaf(x[h + e], cs[e], low ? -o[e] * sn[e] : o[e] * sn[e]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t at = d + e;
            if (at < 2 * pairs) {
              const bool low = at < pairs;
              const uint32_t i = low ? at : at - pairs;
              const float o = x_mine[low ? at + pairs : i];
              x[e] = fmaf(x[e], c[i], low ? -o * s[i] : o * s[i]);
            }
          }
        }
      }
      wave_order();
    }
    if (!row.on || !holds) return;
    const u32x4 bits = {E::pack2(x[0], x[1]), E::pack2(x[2], x[3]), E::pack2(x[4], x[5]), E::pack2(x[6], x[7])};
    if (!key) {
      *reinterpret_cast<u32x4*>(a.q_out + (int64_t)(t0 + row.tok) * a.out_row + (int64_t)row.head * a.out_head + d) = bits;
    } else {
      const uint32_t slot = (uint32_t)a.slots[t0 + row.tok], in = slot & ((1u << a.log_block) - 1);
      if (slot < a.blocks << a.log_block)
        *reinterpret_cast<u32x4*>(a.kc + ((((uint64_t)(slot >> a.log_block) * a.kv_heads + row.head - a.heads) << a.log_block) + in) * a.dim + d) = bits;
    }
  };

  // two steps in hand: the second's loads are under way while the first is turned
  constexpr uint32_t kStep = 4 * kRows;
  const uint32_t total = live * count;
  for (uint32_t r = wave * kRows; r < total; r += 2 * kStep) {
    Row one, two;
    fetch(r, one);
    fetch(r + kStep, two);
    finish(one);
    finish(two);
  }
}

// 64 tokens of one head's values (128 of its elements), turned in LDS.
template <class E, typename S>
__device__ __forceinline__ void rope_values(const RopeArgs& a, uint16_t* s_v, uint32_t* s_slot, uint32_t* s_head,
                                            uint32_t* s_heads) {
  const uint32_t t = threadIdx.x, parts = (a.dim + kStoreDims - 1) / kStoreDims, x = blockIdx.x - a.row_groups;
  const uint32_t h = x / parts % a.kv_heads, d0 = x % parts * kStoreDims, dims = min(a.dim - d0, kStoreDims);
  const uint32_t t0 = x / parts / a.kv_heads * kStoreRows, rows = min(a.tokens - t0, kStoreRows);
  if (t < 64) {
    const uint32_t slot = t < rows && a.positions[t0 + t] >= 0 ? (uint32_t)a.slots[t0 + t] : ~0u;
    slot_groups(slot < a.blocks << a.log_block ? slot : ~0u, s_slot, s_head, s_heads);
  }
  __syncthreads();
  const S* v = static_cast<const S*>(a.v) + (int64_t)h * a.v_head + d0;
  const uint32_t pieces = dims / 8;
  constexpr uint32_t kIter = kStoreRows * kStoreDims / 8 / 256;
  u32x4 vv[kIter];
#pragma unroll
  for (uint32_t j = 0; j < kIter; ++j) {  // everything is asked for before anything is written
    const uint32_t i = t + 256 * j, r = i / pieces;
    if (r < rows && s_slot[r] != ~0u) vv[j] = load8<E>(v + (int64_t)(t0 + r) * a.v_row + 8 * (i % pieces), a.wide);
  }
#pragma unroll
  for (uint32_t j = 0; j < kIter; ++j) {
    const uint32_t i = t + 256 * j, r = i / pieces, d = 8 * (i % pieces);
    if (r < rows && s_slot[r] != ~0u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s_v[(d + 2 * e) * kStoreLine + r] = (uint16_t)vv[j][e];
        s_v[(d + 2 * e + 1) * kStoreLine + r] = (uint16_t)(vv[j][e] >> 16);
      }
  }
  __syncthreads();
  write_values(a.vc + ((uint64_t)h * a.dim << a.log_block), a.kv_heads, a.dim, d0, dims, a.log_block, s_v, s_slot, s_head,
               *s_heads);
}

template <class E, typename S, int LANES>
__global__ __launch_bounds__(256) void k_rope_store(RopeArgs a) {
  constexpr uint32_t kRowBytes = 2 * kTokens * (4 * LANES) * 4 + 4 * 64 * 8 * 4;
  constexpr uint32_t kValueBytes = kStoreDims * kStoreLine * 2;
  __shared__ u32x4 lds[(kRowBytes > kValueBytes ? kRowBytes : kValueBytes) / 16];
  __shared__ uint32_t s_slot[kStoreRows], s_head[kStoreRows], s_heads;
  if (blockIdx.x < a.row_groups) {
    float* s_cos = reinterpret_cast<float*>(lds);
    float* s_sin = s_cos + kTokens * (4 * LANES);
    rope_rows<E, S, LANES>(a, s_cos, s_sin, s_sin + kTokens * (4 * LANES));
  } else {
    rope_values<E, S>(a, reinterpret_cast<uint16_t*>(lds), s_slot, s_head, &s_heads);
  }
}

template <class E, typename S>
int launch_rope(const RopeArgs& a, uint32_t grid, hipStream_t st) {
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, st, a);
    return launched();
  };
  if (a.dim <= 64) return run(k_rope_store<E, S, 8>);
  if (a.dim <= 128) return run(k_rope_store<E, S, 16>);
  return run(k_rope_store<E, S, 32>);
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" int dgt_rope_store(const void* d_q, const void* d_k, const void* d_v, uint32_t source, int64_t q_row,
                              int64_t q_head, int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                              const int32_t* d_positions, const int32_t* d_slots, uint32_t tokens, uint32_t heads,
                              uint32_t kv_heads, uint32_t dim, const double* d_freqs, uint32_t pairs,
                              uint32_t interleaved, const float* d_q_weight, const float* d_k_weight, float eps,
                              uint32_t type, void* d_q_out, int64_t out_row, int64_t out_head, void* d_k_cache,
                              void* d_v_cache, uint32_t blocks, uint32_t block, void* stream) {
  if (!block_ok(block) || !pool_ok(blocks, block) || heads == 0 || kv_heads == 0 || heads > 65535 ||
      kv_heads > 65535 || dim == 0 || dim % 8 || dim > kMaxDim || pairs > dim / 2 || tokens > (1u << 20) ||
      (uint64_t)tokens * std::max(heads, kv_heads) > (1u << 30))
    return DGT_E_SHAPE;
  if (type != DGT_ELT_BF16 && type != DGT_ELT_F16) return DGT_E_UNSUPPORTED;
  if (source != DGT_ELT_F32 && source != type) return DGT_E_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DGT_E_ARG;
  if (tokens == 0) return DGT_OK;
  if (!d_q || !d_k || !d_v || !d_positions || !d_slots || !d_q_out || (pairs && !d_freqs)) return DGT_E_ARG;
  if (blocks && (!d_k_cache || !d_v_cache)) return DGT_E_ARG;
  if (!aligned(d_k_cache, 16) || !aligned(d_v_cache, 16) || !aligned(d_q_out, 16)) return DGT_E_ARG;
  if (tokens == 1) q_row = k_row = v_row = out_row = 0;  // one row, or one head, has no stride
  if (heads == 1) q_head = out_head = 0;
  if (kv_heads == 1) k_head = v_head = 0;
  if (out_row % 8 || out_head % 8) return DGT_E_ARG;
  RopeArgs a;
  a.q = d_q;
  a.k = d_k;
  a.v = d_v;
  a.positions = d_positions;
  a.slots = d_slots;
  a.freqs = d_freqs;
  a.q_weight = d_q_weight;
  a.k_weight = d_k_weight;
  a.q_out = static_cast<uint16_t*>(d_q_out);
  a.kc = static_cast<uint16_t*>(d_k_cache);
  a.vc = static_cast<uint16_t*>(d_v_cache);
  a.q_row = q_row;
  a.q_head = q_head;
  a.k_row = k_row;
  a.k_head = k_head;
  a.v_row = v_row;
  a.v_head = v_head;
  a.out_row = out_row;
  a.out_head = out_head;
  a.tokens = tokens;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.dim = dim;
  a.pairs = pairs;
  a.log_block = (uint32_t)__builtin_ctz(block);
  a.blocks = blocks;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  const int64_t piece = source == DGT_ELT_F32 ? 4 : 8;  // elements of 16 bytes
  a.wide = aligned(d_q, 16) && aligned(d_k, 16) && aligned(d_v, 16) && q_row % piece == 0 && q_head % piece == 0 &&
           k_row % piece == 0 && k_head % piece == 0 && v_row % piece == 0 && v_head % piece == 0;
  // A workgroup of rows takes 8 tokens of as many heads as leave about four workgroups a
  // CU, but no fewer than its waves hold at a time.
  const uint32_t tiles = (tokens + kTokens - 1) / kTokens, all = heads + kv_heads;
  const uint32_t held = dim <= 64 ? 32 : dim <= 128 ? 16 : 8;  // heads in the waves' hands
  const uint32_t fewest = std::min(all, std::max(held / std::min(tokens, kTokens), 1u));
  const uint32_t wanted = (4 * kCUs + tiles - 1) / tiles;
  a.run = std::max((all + wanted - 1) / wanted, fewest);
  a.runs = (all + a.run - 1) / a.run;
  a.row_groups = tiles * a.runs;
  const uint64_t values = blocks == 0 ? 0 : (uint64_t)((tokens + kStoreRows - 1) / kStoreRows) * kv_heads *
                                                ((dim + kStoreDims - 1) / kStoreDims);
  const uint64_t grid = (uint64_t)tiles * a.runs + values;
  if (grid > kMaxGroups) return DGT_E_SHAPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (type == DGT_ELT_BF16)
    return source == DGT_ELT_F32 ? launch_rope<Bf16, float>(a, (uint32_t)grid, st)
                                 : launch_rope<Bf16, uint16_t>(a, (uint32_t)grid, st);
  return source == DGT_ELT_F32 ? launch_rope<F16, float>(a, (uint32_t)grid, st)
                               : launch_rope<F16, uint16_t>(a, (uint32_t)grid, st);
}
