// Attention of drafted tokens over a paged cache.
#include "dgt_serve.h"

#include <algorithm>
#include <cmath>

namespace dgt {
namespace serve {
namespace {

// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = exp(s q_i k_j - max), over the cached
// keys (j < ctx) and the drafted keys that token i may see.
//
// All query heads of a key head and all new tokens of a request are rows of one
// product: row r is token r / group, head r % group of its key head, so a key is
// read once for all of them.  A wave multiplies 32 keys by the rows as S^T = K Q^T
// (keys down, rows across the lanes): a lane then holds 8 keys of one row, which
// is the second operand of O^T = V^T P^T as it stands.  Keys are dealt to the
// rows of the first operand so that those 8 keys are consecutive, and the
// transposed value pages give V^T 16 bytes a lane.  Nothing but the sums
// between waves passes through LDS, and a row's maximum and sum need two lane
// exchanges.
//
// Work is cut into units of 128 keys (32 a wave) of one (request, key head, tile
// of rows); the units of the whole batch are numbered in that order and dealt to
// the workgroups in equal runs, whatever the lengths.  A run that holds only a
// part of a tile's keys leaves maximum, sum and unscaled output in the
// workspace, and the workgroup that comes last adds the parts up in the order of
// the keys.
struct AttnArgs {
  const uint16_t *q, *kc, *vc;
  const int32_t *table, *ctx, *cu;
  const uint64_t* mask;
  uint16_t* out;
  uint32_t* counters;
  float* parts;
  uint64_t q_row, q_head, out_row, out_head;  // element strides
  uint32_t requests, tokens, heads, group, dim, log_block, width, blocks, words;
  float scale;  // times log2(e)
};

constexpr uint32_t kWaves = 4, kTileKeys = 32, kUnitKeys = kWaves * kTileKeys;
constexpr uint32_t kMinUnits = 2;  // a workgroup's run is not cut below this

struct Shape {  // of one request
  uint32_t first, count, ctx, keys, tiles, chunks;
};

template <int RT>
__device__ __forceinline__ Shape request_shape(const AttnArgs& a, uint32_t b) {
  Shape s;
  request_rows(a.cu, b, a.tokens, &s.first, &s.count);
  const uint32_t room = a.width << a.log_block;
  s.ctx = min((uint32_t)max(a.ctx[b], 0), room);
  s.keys = min(s.ctx + s.count, room);
  s.tiles = (s.count * a.group + 16 * RT - 1) / (16 * RT);
  s.chunks = max((s.keys + kUnitKeys - 1) / kUnitKeys, 1u);
  return s;
}

template <int RT>
__device__ __forceinline__ uint64_t request_units(const AttnArgs& a, uint32_t b) {
  const Shape s = request_shape<RT>(a, b);
  return (uint64_t)s.tiles * s.chunks * a.heads;
}

__device__ __forceinline__ void agent_store(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float agent_load(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// What token `tok` of the request may see of the 8 keys from position kv on, one
// bit a key.  Cached keys are seen by every row.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs& a, const Shape& s, uint32_t tok, uint32_t kv) {
  const uint32_t real = kv < s.keys ? min(s.keys - kv, 8u) : 0u;
  const int j0 = (int)kv - (int)s.ctx;  // in drafted keys; both lie below 2^31
  uint32_t bits;
  if (!a.mask) {
    bits = (1u << min(max((int)tok + 1 - j0, 0), 8)) - 1;
  } else {
    const uint32_t old = (uint32_t)min(max(-j0, 0), 8), j = (uint32_t)max(j0, 0), w = j >> 6, sh = j & 63;
    const uint64_t* row = a.mask + (uint64_t)(s.first + tok) * a.words;
    uint64_t v = w < a.words ? row[w] >> sh : 0;
    if (sh > 56 && w + 1 < a.words) v |= row[w + 1] << (64 - sh);
    bits = ((uint32_t)v << old) | ((1u << old) - 1);
  }
  return bits & ((1u << real) - 1);
}

template <class E, int DP, int RT, bool PAD>
__global__ __launch_bounds__(256) void k_tree_attention(AttnArgs a) {
  constexpr int KS = DP / 32, DT = DP / 16, ROWS = 16 * RT;
  constexpr uint32_t kPart = ROWS * (DP + 2);  // floats of a part: m, l, o
  __shared__ float s_o[ROWS][DP + 4];
  __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS];
  __shared__ uint64_t s_sum[256];
  __shared__ uint32_t s_b, s_last;
  __shared__ uint64_t s_base;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6, g = lane >> 4, l16 = lane & 15;
  const uint32_t wg = blockIdx.x, grid = gridDim.x;

  // ------------------------------------------------ this workgroup's run of units
  const uint32_t per = (a.requests + 255) / 256;
  const uint32_t b_lo = min(t * per, a.requests), b_hi = min(b_lo + per, a.requests);
  uint64_t mine = 0;
  for (uint32_t b = b_lo; b < b_hi; ++b) mine += request_units<RT>(a, b);
  uint64_t scan = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up((unsigned long long)scan, d, 64);
    if (lane >= (uint32_t)d) scan += o;
  }
  if (lane == 63) s_sum[wave] = scan;
  __syncthreads();
  uint64_t units = 0;
  for (uint32_t w = 0; w < 4; ++w) {
    if (w < wave) scan += s_sum[w];
    units += s_sum[w];
  }
  if (units == 0) return;
  const uint64_t most = (units + kMinUnits - 1) / kMinUnits;
  const uint32_t wgs = (uint32_t)min((uint64_t)grid, most);
  if (wg >= wgs) return;
  const uint64_t u_end = units * (wg + 1) / wgs;
  uint64_t u = units * wg / wgs;
  const uint64_t before = scan - mine;
  if (before <= u && u < scan) {  // one thread holds the run's first unit
    uint64_t base = before;
    uint32_t b = b_lo;
    for (;; ++b) {
      const uint64_t n = request_units<RT>(a, b);
      if (u < base + n) break;
      base += n;
    }
    s_b = b;
    s_base = base;
  }
  __syncthreads();
  uint32_t b = __builtin_amdgcn_readfirstlane(s_b);
  uint64_t base = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(s_base >> 32)) << 32 |
                  __builtin_amdgcn_readfirstlane((uint32_t)s_base);
  Shape sh = request_shape<RT>(a, b);

  while (u < u_end) {
    while (u >= base + (uint64_t)sh.tiles * sh.chunks * a.heads) {  // on to the next request
      base += (uint64_t)sh.tiles * sh.chunks * a.heads;
      sh = request_shape<RT>(a, ++b);
    }
    const uint32_t in = (uint32_t)(u - base), item = in / sh.chunks, c0 = in % sh.chunks;
    const uint32_t head = item / sh.tiles, tile = item % sh.tiles;
    const uint64_t item0 = u - c0;  // the item's first unit
    const uint32_t c1 = (uint32_t)min((uint64_t)sh.chunks, u_end - item0);
    const uint32_t rows = sh.count * a.group, row0 = tile * ROWS;

    // queries, the product's second operand; rows past the end read the last one
    u32x4 q[RT][KS];
    uint32_t tok[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint32_t r = min(row0 + 16 * i + l16, rows - 1);
      tok[i] = r / a.group;
      const uint16_t* p = a.q + (uint64_t)(sh.first + tok[i]) * a.q_row +
                          (uint64_t)(head * a.group + r % a.group) * a.q_head;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t d = 32 * s + 8 * g;
        q[i][s] = (!PAD || d < a.dim) ? *reinterpret_cast<const u32x4*>(p + d) : u32x4{};
      }
    }
    floatx4 o[RT][DT];
    float m[RT], l[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[i][d] = floatx4{};
    }

    const int32_t* pages = a.table + (uint64_t)b * a.width;
    const uint32_t in_page = (1u << a.log_block) - 1;
    const uint64_t page_len = (uint64_t)a.dim << a.log_block;  // elements of a head's page
    for (uint32_t c = c0; c < c1; ++c) {
      const uint32_t kb = c * kUnitKeys + wave * kTileKeys;
      if (kb >= sh.keys) break;
      // the lane's group of 8 keys for masks and values, and for its key rows
      const uint32_t kv = kb + 8 * g, kk = kb + 8 * (l16 >> 2);
      uint32_t pv = kv < sh.keys ? (uint32_t)pages[kv >> a.log_block] : ~0u;
      uint32_t pk = kk < sh.keys ? (uint32_t)pages[kk >> a.log_block] : ~0u;
      const bool held = pv < a.blocks;
      pv = held ? pv : 0u;
      pk = pk < a.blocks ? pk : 0u;
      const uint16_t* kp = a.kc + ((uint64_t)pk * a.heads + head) * page_len +
                           (uint64_t)((kk & in_page) + (l16 & 3)) * a.dim;
      const uint16_t* vp = a.vc + ((uint64_t)pv * a.heads + head) * page_len + (kv & in_page);

      floatx4 s[RT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < RT; ++i) s[i][h] = floatx4{};
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          const uint32_t d = 32 * x + 8 * g;
          const u32x4 kf = (!PAD || d < a.dim)
                               ? *reinterpret_cast<const u32x4*>(kp + (uint64_t)4 * h * a.dim + d)
                               : u32x4{};
#pragma unroll
          for (int i = 0; i < RT; ++i) s[i][h] = E::mfma(kf, q[i][x], s[i][h]);
        }
      }
      u32x4 vf[DT];
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const uint32_t row = 16 * d + l16;
        vf[d] = (!PAD || row < a.dim)
                    ? *reinterpret_cast<const u32x4*>(vp + ((uint64_t)row << a.log_block))
                    : u32x4{};
      }

      // Past the cached keys, or where a page is missing, scores of unseen keys
      // become -inf and values of keys that do not exist become zero (0 * NaN
      // would not be).
      const bool edge = __any(kb + kTileKeys > sh.ctx || !held);
      bool odd_values = false;
      if (edge) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint32_t bits = held ? seen_bits(a, sh, tok[i], kv) : 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!((bits >> e) & 1)) s[i][e >> 2][e & 3] = -INFINITY;
        }
        const uint32_t real = !held || kv >= sh.keys ? 0u : min(sh.keys - kv, 8u);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t v = vf[d][w];
            if (real <= 2u * w) v = 0u;
            else if (real == 2u * w + 1) v &= 0xFFFFu;
            vf[d][w] = v;
            odd_values |= !E::finite2(v);
          }
        odd_values = __any(odd_values);
      }

#pragma unroll
      for (int i = 0; i < RT; ++i) {
        float top = fmaxf(fmaxf(fmaxf(s[i][0][0], s[i][0][1]), fmaxf(s[i][0][2], s[i][0][3])),
                          fmaxf(fmaxf(s[i][1][0], s[i][1][1]), fmaxf(s[i][1][2], s[i][1][3])));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float now = fmaxf(m[i], top);
        // a row that has seen nothing yet keeps -inf; its weights are exp2(-inf) = 0
        const float ref = now == -INFINITY ? 0.f : now * a.scale;
        const float keep = m[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[i] * a.scale - ref);
        m[i] = now;
        float sum = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[i][h][e], a.scale, -ref));
            s[i][h][e] = p;
            sum += p;
          }
        l[i] = fmaf(l[i], keep, sum);  // this lane's keys; the lanes are added at the end
#pragma unroll
        for (int d = 0; d < DT; ++d) o[i][d] *= keep;
      }

      if (!odd_values) {
        // The weights are rounded to the cache's type, as the matrix instruction
        // takes them; the sum that divides them is of the unrounded ones.
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const u32x4 p = {E::pack2(s[i][0][0], s[i][0][1]), E::pack2(s[i][0][2], s[i][0][3]),
                           E::pack2(s[i][1][0], s[i][1][1]), E::pack2(s[i][1][2], s[i][1][3])};
#pragma unroll
          for (int d = 0; d < DT; ++d) o[i][d] = E::mfma(vf[d], p, o[i][d]);
        }
      } else {
        // A drafted value is infinite or NaN: rows that do not see it must not
        // meet it, so keys of weight zero are left out one by one.
        const uint32_t real = min(sh.keys - kb, kTileKeys);
#pragma unroll 1
        for (uint32_t x = 0; x < real; ++x) {
          const uint32_t key = kb + x, page = (uint32_t)pages[key >> a.log_block];
          if (page >= a.blocks) continue;
          const uint16_t* vx = a.vc + ((uint64_t)page * a.heads + head) * page_len + (key & in_page);
          float p[RT];
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            float v = s[i][0][0];
#pragma unroll
            for (uint32_t e = 1; e < 8; ++e) v = (x & 7) == e ? s[i][e >> 2][e & 3] : v;
            p[i] = __shfl(v, (x >> 3) * 16 + l16, 64);
          }
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t row = 16 * d + 4 * g + j;
              if (PAD && row >= a.dim) continue;
              const float v = E::up(vx[(uint64_t)row << a.log_block]);
#pragma unroll
              for (int i = 0; i < RT; ++i)
                if (p[i] != 0.f) o[i][d][j] = fmaf(p[i], v, o[i][d][j]);
            }
        }
      }
    }

    // ------------------------------------------- the four waves' parts, added in order
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      l[i] += __shfl_xor(l[i], 16, 64);
      l[i] += __shfl_xor(l[i], 32, 64);
      if (g == 0) {
        s_m[wave][16 * i + l16] = m[i];
        s_l[wave][16 * i + l16] = l[i];
      }
    }
    __syncthreads();
    float top[RT], total[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint32_t r = 16 * i + l16;
      top[i] = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      const float ref = top[i] == -INFINITY ? 0.f : top[i];
      total[i] = 0.f;
#pragma unroll
      for (uint32_t w = 0; w < kWaves; ++w)
        total[i] += s_l[w][r] * __builtin_amdgcn_exp2f((s_m[w][r] - ref) * a.scale);
      const float f = __builtin_amdgcn_exp2f((m[i] - ref) * a.scale);
#pragma unroll
      for (int d = 0; d < DT; ++d) o[i][d] *= f;
    }
    for (uint32_t w = 0; w < kWaves; ++w) {
      if (w == wave) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            floatx4* p = reinterpret_cast<floatx4*>(&s_o[16 * i + l16][16 * d + 4 * g]);
            if (w == 0) *p = o[i][d];
            else *p += o[i][d];
          }
      }
      __syncthreads();
    }
    const uint32_t live = min(rows - row0, (uint32_t)ROWS);
    auto write = [&](uint32_t r, uint32_t d, float v0, float v1) {
      const uint32_t row = row0 + r, tk = row / a.group, hd = head * a.group + row % a.group;
      *reinterpret_cast<uint32_t*>(a.out + (uint64_t)(sh.first + tk) * a.out_row + (uint64_t)hd * a.out_head + d) =
          E::pack2(v0, v1);
    };
    if (wave == 0 && g == 0) {  // the joined statistics, for the threads that write
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        s_m[0][16 * i + l16] = top[i];
        s_l[0][16 * i + l16] = total[i];
      }
    }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == sh.chunks;
    if (whole) {
      for (uint32_t i = t; i < live * (DP / 2); i += 256) {
        const uint32_t r = i / (DP / 2), d = 2 * (i % (DP / 2));
        if (PAD && d >= a.dim) continue;
        const float inv = s_l[0][r] > 0.f || s_l[0][r] != s_l[0][r] ? 1.f / s_l[0][r] : 0.f;
        write(r, d, s_o[r][d] * inv, s_o[r][d + 1] * inv);
      }
    } else {
      // first and last workgroup of the item, from the runs' bounds
      const uint64_t end = item0 + sh.chunks - 1;
      auto owner = [&](uint64_t x) {
        uint32_t w = (uint32_t)(((x + 1) * wgs - 1) / units);  // the last w with units * w / wgs <= x
        return w;
      };
      const uint32_t w0 = owner(item0), w1 = owner(end);
      auto part_of = [&](uint32_t w) { return a.parts + ((uint64_t)2 * w + (w == w0)) * kPart; };
      float* part = part_of(wg);
      for (uint32_t i = t; i < live; i += 256) {
        agent_store(part + i, s_m[0][i]);
        agent_store(part + ROWS + i, s_l[0][i]);
      }
      for (uint32_t i = t; i < live * DP; i += 256)
        agent_store(part + 2 * ROWS + i, s_o[i / DP][i % DP]);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (t == 0) {
        const uint32_t old = __hip_atomic_fetch_add(a.counters + w0, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = old == w1 - w0;
      }
      __syncthreads();
      if (s_last) {
        if (t == 0) __hip_atomic_store(a.counters + w0, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        for (uint32_t i = t; i < live * (DP / 2); i += 256) {
          const uint32_t r = i / (DP / 2), d = 2 * (i % (DP / 2));
          if (PAD && d >= a.dim) continue;
          float mm = -INFINITY;
          for (uint32_t w = w0; w <= w1; ++w) mm = fmaxf(mm, agent_load(part_of(w) + r));
          const float ref = mm == -INFINITY ? 0.f : mm;
          float ll = 0.f, v0 = 0.f, v1 = 0.f;
          for (uint32_t w = w0; w <= w1; ++w) {
            const float* p = part_of(w);
            const float f = __builtin_amdgcn_exp2f((agent_load(p + r) - ref) * a.scale);
            ll = fmaf(agent_load(p + ROWS + r), f, ll);
            v0 = fmaf(agent_load(p + 2 * ROWS + r * DP + d), f, v0);
            v1 = fmaf(agent_load(p + 2 * ROWS + r * DP + d + 1), f, v1);
          }
          const float inv = ll > 0.f || ll != ll ? 1.f / ll : 0.f;
          write(r, d, v0 * inv, v1 * inv);
        }
      }
    }
    __syncthreads();  // the LDS is reused by the next item
    u = item0 + c1;
  }
}

struct AttnPlan {
  uint32_t dp, rt, grid;
  size_t part_off, ws_bytes;
};

AttnPlan plan_attention(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  AttnPlan p;
  p.dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  // rows of a request and key head, on the average
  const uint64_t rows = (uint64_t)tokens * (heads / kv_heads) / std::max(requests, 1u);
  p.rt = rows <= 16 ? 1 : rows <= 32 || p.dp == 256 ? 2 : 4;
  p.grid = kCUs * (p.rt == 1 ? 4 : p.rt == 2 ? 2 : 1);
  p.part_off = ((size_t)p.grid * 4 + 255) / 256 * 256;
  p.ws_bytes = p.part_off + (size_t)p.grid * 2 * (16 * p.rt) * (p.dp + 2) * 4;
  return p;
}

bool attn_shape_ok(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  return heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && heads <= 65536 && dim >= 8 &&
         dim <= 256 && dim % 8 == 0 && requests <= kMaxRequests && tokens <= (1u << 20) &&
         (uint64_t)tokens * heads <= (1u << 30);
}

template <class E, int DP, int RT>
int launch_attention(const AttnArgs& a, uint32_t grid, hipStream_t st) {
  if (a.dim == DP)
    hipLaunchKernelGGL((k_tree_attention<E, DP, RT, false>), dim3(grid), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_tree_attention<E, DP, RT, true>), dim3(grid), dim3(256), 0, st, a);
  return launched();
}

template <class E>
int launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  switch (p.dp * 8 + p.rt) {
    case 64 * 8 + 1: return launch_attention<E, 64, 1>(a, p.grid, st);
    case 64 * 8 + 2: return launch_attention<E, 64, 2>(a, p.grid, st);
    case 64 * 8 + 4: return launch_attention<E, 64, 4>(a, p.grid, st);
    case 128 * 8 + 1: return launch_attention<E, 128, 1>(a, p.grid, st);
    case 128 * 8 + 2: return launch_attention<E, 128, 2>(a, p.grid, st);
    case 128 * 8 + 4: return launch_attention<E, 128, 4>(a, p.grid, st);
    case 256 * 8 + 1: return launch_attention<E, 256, 1>(a, p.grid, st);
    case 256 * 8 + 2: return launch_attention<E, 256, 2>(a, p.grid, st);
  }
  return DGT_E_UNSUPPORTED;
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" {

size_t dgt_tree_attention_workspace(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim,
                                    uint32_t requests) {
  if (!attn_shape_ok(tokens, heads, kv_heads, dim, requests)) return 0;
  return plan_attention(tokens, heads, kv_heads, dim, requests).ws_bytes;
}

int dgt_tree_attention(uint32_t type, const void* d_q, uint64_t q_row, uint64_t q_head,
                       const void* d_k_cache, const void* d_v_cache, uint32_t blocks, uint32_t block,
                       const int32_t* d_table, uint32_t width, const int32_t* d_ctx, const int32_t* d_cu,
                       uint32_t requests, uint32_t tokens, uint32_t heads, uint32_t kv_heads,
                       uint32_t dim, const uint64_t* d_mask, uint32_t mask_words, float scale,
                       void* d_out, uint64_t out_row, uint64_t out_head, void* d_ws, size_t ws_bytes,
                       void* stream) {
  if (type != DGT_ELT_BF16 && type != DGT_ELT_F16) return DGT_E_UNSUPPORTED;
  if (!attn_shape_ok(tokens, heads, kv_heads, dim, requests) || !block_ok(block) ||
      !pool_ok(blocks, block) || (uint64_t)width * block > 0x7FFFFFFFull)
    return DGT_E_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return DGT_E_ARG;
  if (tokens == 0 || requests == 0) return DGT_OK;
  if (!d_q || !d_out || !d_cu || !d_ctx || !d_ws) return DGT_E_ARG;
  if ((width && !d_table) || (blocks && (!d_k_cache || !d_v_cache))) return DGT_E_ARG;
  if ((mask_words != 0) != (d_mask != nullptr) || mask_words > 1024) return DGT_E_ARG;
  if (!aligned(d_q, 16) || !aligned(d_k_cache, 16) || !aligned(d_v_cache, 16) || !aligned(d_out, 4) ||
      !aligned(d_ws, 256) || q_row % 8 || q_head % 8 || out_row % 2 || out_head % 2)
    return DGT_E_ARG;
  if (blocks == 0) return DGT_E_SHAPE;
  const AttnPlan p = plan_attention(tokens, heads, kv_heads, dim, requests);
  if (ws_bytes < p.ws_bytes) return DGT_E_BUFSIZE;
  AttnArgs a;
  a.q = static_cast<const uint16_t*>(d_q);
  a.kc = static_cast<const uint16_t*>(d_k_cache);
  a.vc = static_cast<const uint16_t*>(d_v_cache);
  a.table = d_table;
  a.ctx = d_ctx;
  a.cu = d_cu;
  a.mask = d_mask;
  a.out = static_cast<uint16_t*>(d_out);
  a.counters = static_cast<uint32_t*>(d_ws);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + p.part_off);
  a.q_row = q_row;
  a.q_head = q_head;
  a.out_row = out_row;
  a.out_head = out_head;
  a.requests = requests;
  a.tokens = tokens;
  a.heads = kv_heads;
  a.group = heads / kv_heads;
  a.dim = dim;
  a.log_block = (uint32_t)__builtin_ctz(block);
  a.width = width;
  a.blocks = blocks;
  a.words = mask_words;
  a.scale = scale * 1.4426950408889634f;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return type == DGT_ELT_BF16 ? launch_attention<Bf16>(a, p, st) : launch_attention<F16>(a, p, st);
}

}  // extern "C"
