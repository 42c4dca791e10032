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
// Work is cut into units of 128 keys of one (request, key head, tile of rows), and
// the units of the whole batch are numbered and dealt to the workgroups in equal
// runs, whatever the lengths.  The keys of a request fall into spans of a run's
// length; units are numbered request, head, span, tile of rows, key.  So the
// tiles of one span go to neighbouring workgroups, which read the same keys at the
// same time, from the cache of the die they share.  A run that holds only a part of
// a tile's keys leaves maximum, sum and unscaled output in the workspace, and the
// workgroup that comes last adds the parts up in the order of the keys.
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
// A workgroup's run is not cut below this (one token over 1000 keys: 11.2 us with two,
// 13.0 with four, 17.7 with six).
constexpr uint32_t kMinUnits = 2;
constexpr uint32_t kDies = 8;
constexpr uint32_t kNarrowPerCU = 3, kWidePerCU = 2;  // workgroups, as registers and LDS allow

struct Shape {  // of one request
  uint32_t first, count, ctx, keys, tiles, chunks;
};

template <int ROWS>
__device__ __forceinline__ Shape request_shape(const AttnArgs& a, uint32_t b) {
  Shape s;
  request_rows(a.cu, b, a.tokens, &s.first, &s.count);
  const uint32_t room = a.width << a.log_block;
  s.ctx = min((uint32_t)max(a.ctx[b], 0), room);
  s.keys = min(s.ctx + s.count, room);
  s.tiles = (s.count * a.group + ROWS - 1) / ROWS;
  s.chunks = max((s.keys + kUnitKeys - 1) / kUnitKeys, 1u);
  return s;
}

// The host has made sure that a batch whose offsets never fall has fewer units than
// this, and any one request too.  Offsets that fall can name the same rows again and
// again; sums stop growing here (min(a + b, most) is associative over numbers up to
// it), and a batch that reaches it is not computed.
constexpr uint32_t kMostUnits = 0x7FFFFFFF;
__device__ __forceinline__ uint32_t add_units(uint32_t a, uint32_t b) { return min(a + b, kMostUnits); }

template <int ROWS>
__device__ __forceinline__ uint32_t request_units(const AttnArgs& a, uint32_t b) {
  const Shape s = request_shape<ROWS>(a, b);
  return s.tiles * s.chunks * a.heads;
}

// n things dealt to `count` holders: the first n % count hold one more.
struct Deal {
  uint32_t n, count, each, more;
  __device__ __forceinline__ Deal(uint32_t n, uint32_t count)
      : n(n), count(count), each(n / count), more(n - each * count) {}
  __device__ __forceinline__ uint32_t begin(uint32_t i) const { return i * each + min(i, more); }
  __device__ __forceinline__ uint32_t owner(uint32_t x) const {
    const uint32_t longer = more * (each + 1);
    return x < longer ? x / (each + 1) : more + (x - longer) / each;
  }
  __device__ __forceinline__ uint32_t most() const { return each + (more != 0); }
};

// Parts pass between workgroups that may sit on different dies, so they are
// written through and read past the caches that the dies do not share (the sc1
// bit of a buffer access, as agent-scope atomics have it, but 16 bytes a lane).
constexpr int kAgent = 16;
__device__ __forceinline__ void part_store(__amdgpu_buffer_rsrc_t r, uint32_t at, floatx4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at * 4, 0, kAgent);
}
__device__ __forceinline__ void part_store(__amdgpu_buffer_rsrc_t r, uint32_t at, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at * 4, 0, kAgent);
}
__device__ __forceinline__ floatx4 part_load4(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, at * 4, 0, kAgent));
}
__device__ __forceinline__ float part_load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at * 4, 0, kAgent));
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

// A workgroup's run of units [u, end), and the request that holds unit u.
struct Run {
  Deal deal;         // of the batch's units to the runs
  uint32_t wg;       // this run's number
  uint32_t u, end;
  uint32_t b, base;  // the request and its first unit
};

// Every workgroup adds up the lengths for itself, which costs less than a launch;
// count 0: nothing is left for this one.
template <int ROWS>
__device__ __forceinline__ Run find_run(const AttnArgs& a, uint32_t* s_sum) {
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const uint32_t per = (a.requests + 255) / 256;
  const uint32_t b_lo = min(t * per, a.requests), b_hi = min(b_lo + per, a.requests);
  uint32_t mine = 0;
  for (uint32_t b = b_lo; b < b_hi; ++b) mine = add_units(mine, request_units<ROWS>(a, b));
  uint32_t scan = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(scan, d, 64);
    if (lane >= (uint32_t)d) scan = add_units(scan, o);
  }
  if (lane == 63) s_sum[wave] = scan;
  __syncthreads();
  uint32_t units = 0;
  for (uint32_t w = 0; w < 4; ++w) {
    if (w < wave) scan = add_units(scan, s_sum[w]);
    units = add_units(units, s_sum[w]);
  }
  units = __builtin_amdgcn_readfirstlane(units);
  Run run{Deal(units, min(gridDim.x, max((units + kMinUnits - 1) / kMinUnits, 1u))), 0, 0, 0, 0, 0};
  // Workgroups go round the dies; neighbouring runs, which read the same keys for
  // other rows, stay on one, so that its cache serves all but the first.
  const uint32_t runs = run.deal.count, die = blockIdx.x % kDies, nth = blockIdx.x / kDies;
  if (units == 0 || units == kMostUnits || nth >= runs / kDies + (die < runs % kDies)) return run;
  run.wg = die * (runs / kDies) + min(die, runs % kDies) + nth;
  run.u = run.deal.begin(run.wg);
  run.end = run.deal.begin(run.wg + 1);
  const uint32_t before = scan - mine;
  if (before <= run.u && run.u < scan) {  // one thread holds the run's first unit
    uint32_t base = before, b = b_lo;
    for (;; ++b) {
      const uint32_t n = request_units<ROWS>(a, b);
      if (run.u < base + n) break;
      base += n;
    }
    s_sum[4] = b;
    s_sum[5] = base;
  }
  __syncthreads();
  run.b = __builtin_amdgcn_readfirstlane(s_sum[4]);
  run.base = __builtin_amdgcn_readfirstlane(s_sum[5]);
  return run;
}

// The request's chunks in spans as long as the longest run, so that runs side by
// side are at the same key; the last one is from half to one and a half as long.
struct Spans {
  uint32_t chunks, len, count;
  __device__ __forceinline__ Spans(const Run& run, const Shape& sh)
      : chunks(sh.chunks), len(run.deal.most()), count(max((chunks + len / 2) / len, 1u)) {}
  __device__ __forceinline__ uint32_t begin(uint32_t i) const { return i < count ? i * len : chunks; }
  __device__ __forceinline__ uint32_t owner(uint32_t chunk) const { return min(chunk / len, count - 1); }
};

// What the run covers of one (request, key head, span, tile of rows).
struct Item {
  uint32_t head, tile, row0, rows;  // rows: of the request and head
  uint32_t c0, c1;                  // chunks of its keys
  uint32_t base;                    // first unit of the head
  uint32_t first;                   // unit of the span's first chunk for this tile
  bool whole;
};

template <int ROWS>
__device__ __forceinline__ Item next_item(const AttnArgs& a, Run* run, Shape* sh) {
  while (run->u - run->base >= sh->tiles * sh->chunks * a.heads) {
    run->base += sh->tiles * sh->chunks * a.heads;
    *sh = request_shape<ROWS>(a, ++run->b);
  }
  const Spans spans(*run, *sh);
  const uint32_t in = run->u - run->base, per = sh->tiles * sh->chunks, left = in % per;
  Item it;
  it.head = in / per;
  it.base = run->u - left;
  const uint32_t span = spans.owner(left / sh->tiles), begin = spans.begin(span), len = spans.begin(span + 1) - begin;
  const uint32_t within = left - sh->tiles * begin;
  it.tile = within / len;
  it.row0 = it.tile * ROWS;
  it.rows = sh->count * a.group;
  it.c0 = begin + within % len;
  it.first = run->u - within % len;
  it.c1 = min(begin + len, it.c0 + (run->end - run->u));
  it.whole = it.c0 == 0 && it.c1 == sh->chunks;
  run->u += it.c1 - it.c0;
  return it;
}

__device__ __forceinline__ uint16_t* out_at(const AttnArgs& a, const Shape& sh, const Item& it, uint32_t r) {
  const uint32_t row = it.row0 + r, tok = row / a.group, head = it.head * a.group + row % a.group;
  return a.out + (uint64_t)(sh.first + tok) * a.out_row + (uint64_t)head * a.out_head;
}

// 1 / the sum of weights; 0 where the row saw nothing (a NaN stays one).
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// Where the parts of a tile of rows lie.  Each of its spans is held by the runs from
// owner(span's first unit) to owner(its last); a run has room for three parts: one
// of a span that began before it, and one of a span that begins in either half of it
// (spans of a tile that is not whole are no shorter than half the longest run).  A part is ref[ROWS], l[ROWS] and
// the outputs, in floats.
constexpr uint32_t kRoom = 3;

template <int ROWS, int DP>
struct Parts {
  static constexpr uint32_t kFloats = ROWS * (DP + 2);
  const Deal runs;
  const Spans spans;
  uint32_t base;  // first unit of the head
  uint32_t tiles, tile;
  __amdgpu_buffer_rsrc_t at;
  __device__ __forceinline__ Parts(const AttnArgs& a, const Run& run, const Item& it, const Shape& sh)
      : runs(run.deal), spans(run, sh), base(it.base), tiles(sh.tiles), tile(it.tile) {
    // raw 32-bit data; accesses are checked against the length
    at = __builtin_amdgcn_make_buffer_rsrc(a.parts, 0, gridDim.x * kRoom * kFloats * 4, 0x00027000);
  }
  // number of the part that run w has of the span whose first unit is x
  __device__ __forceinline__ uint32_t number(uint32_t w, uint32_t x) const {
    const uint32_t begin = runs.begin(w);
    return kRoom * w + (x < begin ? 0u : 1u + (x - begin) / ((runs.most() + 1) / 2));
  }
  __device__ __forceinline__ uint32_t first(uint32_t span) const {
    const uint32_t b = spans.begin(span), e = spans.begin(span + 1);
    return base + tiles * b + tile * (e - b);
  }
  __device__ __forceinline__ uint32_t of(uint32_t w, uint32_t x) const { return number(w, x) * kFloats; }

  // The parts in the order of the keys: run w has one of span i.
  struct Place {
    uint32_t i, x, w, last;  // x: the span's first unit, last: its last run
  };
  __device__ __forceinline__ Place begin(uint32_t i) const {
    const uint32_t x = first(i);
    return Place{i, x, runs.owner(x), runs.owner(x + spans.begin(i + 1) - spans.begin(i) - 1)};
  }
  __device__ __forceinline__ void next(Place& p) const {
    if (p.w < p.last) ++p.w;
    else if (p.i + 1 < spans.count) p = begin(p.i + 1);
    else p.i = spans.count;
  }
  __device__ __forceinline__ uint32_t count() const {
    uint32_t n = 0;
    for (uint32_t i = 0; i < spans.count; ++i) {
      const Place p = begin(i);
      n += p.last - p.w + 1;
    }
    return n;
  }

  // Counts this workgroup's part in; true for the tile's last.  Waiting for the
  // stores before counting orders them without the cache writeback of a fence.
  __device__ __forceinline__ bool last(const AttnArgs& a, uint32_t* s_last) const {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t others = count() - 1;
      const uint32_t x = first(0);
      uint32_t* counter = a.counters + number(runs.owner(x), x);
      const uint32_t old = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *s_last = old == others;
      if (old == others)  // ready for the next call
        __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *s_last != 0;
  }

  // Joins row r of the parts in the order of the keys: N pieces of four outputs at
  // at0, at0 + step, ..., within a part.  Returns the sum of weights.  The parts come
  // from other dies' memory, microseconds away, so four are asked for at a time.
  template <int N>
  __device__ __forceinline__ float join(uint32_t r, uint32_t at0, uint32_t step, floatx4 (&o)[N]) const {
    constexpr int kBatch = 4;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = floatx4{};
    for (Place p = begin(0); p.i < spans.count;) {
      float mw[kBatch], lw[kBatch];
      floatx4 ow[kBatch][N];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        mw[k] = -INFINITY;
        lw[k] = 0.f;
        if (p.i < spans.count) {
          const uint32_t part = of(p.w, p.x);
          mw[k] = part_load(at, part + r);
          lw[k] = part_load(at, part + ROWS + r);
#pragma unroll
          for (int i = 0; i < N; ++i) ow[k][i] = part_load4(at, part + 2 * ROWS + at0 + i * step);
          next(p);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) ow[k][i] = floatx4{};
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float now = fmaxf(m, mw[k]), ref = now == -INFINITY ? 0.f : now;
        const float f = __builtin_amdgcn_exp2f(m - ref), fw = __builtin_amdgcn_exp2f(mw[k] - ref);
        m = now;
        l = fmaf(lw[k], fw, l * f);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = o[i] * f + ow[k][i] * fw;
      }
    }
    return l;
  }
};

template <class E>
__device__ __forceinline__ void write4(uint16_t* p, floatx4 v, float inv) {
  *reinterpret_cast<uint32_t*>(p) = E::pack2(v[0] * inv, v[1] * inv);
  *reinterpret_cast<uint32_t*>(p + 2) = E::pack2(v[2] * inv, v[3] * inv);
}

// Queries of 16 rows a lane group, the products' second operand; rows past the
// end read the last one.
template <int RT, int KS, bool PAD>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Shape& sh, const Item& it, uint32_t row,
                                             u32x4 (&q)[RT][KS], uint32_t (&tok)[RT]) {
  const uint32_t lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const uint32_t r = min(row + 16 * i + l16, it.rows - 1);
    tok[i] = r / a.group;
    const uint16_t* p = a.q + (uint64_t)(sh.first + tok[i]) * a.q_row +
                        (uint64_t)(it.head * a.group + r % a.group) * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t d = 32 * s + 8 * g;
      q[i][s] = (!PAD || d < a.dim) ? *reinterpret_cast<const u32x4*>(p + d) : u32x4{};
    }
  }
}

// Maximum and sum over the four lanes that hold one row (lanes l, l + 16, l + 32,
// l + 48): the swaps exchange half waves and neighbouring rows of 16 lanes.
__device__ __forceinline__ float row_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(fmaxf(v, __uint_as_float(a[0])), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(fmaxf(v, __uint_as_float(a[0])), __uint_as_float(a[1]));
}
__device__ __forceinline__ float row_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// The running softmax of one row.  Weights are 2^(score * scale - ref) against a
// reference that follows the maximum at a distance: it moves only when a score
// passes it by kSlack, so that the outputs are rarely multiplied (fp32 sums and
// 16-bit weights up to 2^kSlack lose nothing by it; following the maximum itself
// multiplied them in a third of the tiles).  ref is -inf until a key is seen.
constexpr float kSlack = 8.f;

struct Softmax {
  float ref = -INFINITY, l = 0.f;
};

// One step over the 4 N scores that a lane holds of its row: s becomes the weights;
// true, for the whole wave, if the outputs so far are to be multiplied by `keep`.  The
// weights are added to l where they are used (this lane's keys only; the lanes of a
// row are added at the end).
template <int N>
__device__ __forceinline__ bool softmax_step(floatx4 (&s)[N], Softmax& m, float& keep, float scale) {
  // (a maximum of three is one instruction; of two it is two more, to settle NaNs)
  float top = s[0][0];
#pragma unroll
  for (int h = 0; h < N; ++h) {
    top = fmaxf(fmaxf(top, s[h][0]), s[h][1]);
    top = fmaxf(fmaxf(top, s[h][2]), s[h][3]);
  }
  top = row_max(top) * scale;
  const bool moves = __any(top > m.ref + kSlack);
  if (moves) {
    const float now = fmaxf(m.ref, top);
    keep = m.ref == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m.ref - now);
    m.ref = now;
    m.l *= keep;
  }
  const float ref = m.ref == -INFINITY ? 0.f : m.ref;  // nothing seen: the weights are 2^-inf = 0
#pragma unroll
  for (int h = 0; h < N; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[h][e] = __builtin_amdgcn_exp2f(fmaf(s[h][e], scale, -ref));
  return moves;
}

// The weights of 8 keys, rounded to the cache's type: the matrix instruction has one
// type for both operands, and a second product for the bits that are lost would double
// half of the work.  It costs a bf16 result up to a third more error than its own
// rounding has (0.0019 to 0.0023 relative, 0.0017 with fp32 weights; fp16 0.00024 and
// 0.00021).  l, which divides the outputs, adds the rounded ones: where few keys hold
// most of the weight their rounding cancels.
template <class E>
__device__ __forceinline__ u32x4 weights(const floatx4& s0, const floatx4& s1, float& l) {
  const u32x4 p = {E::pack2(s0[0], s0[1]), E::pack2(s0[2], s0[3]), E::pack2(s1[0], s1[1]), E::pack2(s1[2], s1[3])};
#pragma unroll
  for (int w = 0; w < 4; ++w) l = E::add2(p[w], l);
  return p;
}

// The weights as they are, where they are used key by key.
template <int N>
__device__ __forceinline__ void add_weights(const floatx4 (&s)[N], float& l) {
#pragma unroll
  for (int h = 0; h < N; ++h) l += (s[h][0] + s[h][1]) + (s[h][2] + s[h][3]);
}

// Pages of the keys at hand, kept in LDS: table entries of up to kPageRoom pages.
constexpr uint32_t kPageRoom = 1024;

// ------------------------------------------------------------------ few rows
// Each wave streams its own 32 keys of a unit from memory straight into the
// operands; the waves meet once an item.  Bound by memory: 96 requests of up to 8100
// keys, one token on 8 key heads of 128, take 229 us for 1.29 GB, 5.6 TB/s (a large
// copy moves 5.1), three workgroups a CU keeping the loads in flight.  Small calls are
// a chain of latencies: lengths, table, keys, the waves' meeting, and where a tile's
// keys are split the parts (one token over 1000 keys: 11.2 us).
template <int DP>
struct Narrow {
  static constexpr uint32_t kRows = 16, kLine = DP + 4;  // floats of a row in LDS
  static constexpr uint32_t kBytes = kWaves * kRows * kLine * 4;
};

template <class E, int DP, bool PAD>
__global__ __launch_bounds__(256, 3) void k_attention_narrow(AttnArgs a) {
  constexpr int KS = DP / 32, DT = DP / 16, ROWS = 16;
  constexpr uint32_t kLine = Narrow<DP>::kLine;
  extern __shared__ u32x4 lds[];
  float* s_o = reinterpret_cast<float*>(lds);  // [waves][rows][kLine]
  __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS];
  __shared__ uint32_t s_sum[6];
  __shared__ uint32_t s_last;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6, g = lane >> 4, l16 = lane & 15;
  Run run = find_run<ROWS>(a, s_sum);
  if (run.u == run.end) return;
  Shape sh = request_shape<ROWS>(a, run.b);
  const uint32_t dim = PAD ? a.dim : (uint32_t)DP, in_page = (1u << a.log_block) - 1;
  const uint64_t page_len = (uint64_t)dim << a.log_block;  // elements of a head's page

  const uint32_t v_step = 16u << a.log_block;  // 16 value rows

  while (run.u < run.end) {
    const Item it = next_item<ROWS>(a, &run, &sh);
    u32x4 q[1][KS];
    uint32_t tok[1];
    load_queries<1, KS, PAD>(a, sh, it, it.row0, q, tok);
    floatx4 o[DT];
    Softmax m;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = floatx4{};

    const int32_t* pages = a.table + (uint64_t)run.b * a.width;
    // pages of the lane's group of 8 keys for masks and values, and for its key rows,
    // asked for a unit ahead
    auto page_of = [&](uint32_t key) { return key < sh.keys ? (uint32_t)pages[key >> a.log_block] : ~0u; };
    const uint32_t kb0 = it.c0 * kUnitKeys + wave * kTileKeys;
    uint32_t next_v = page_of(kb0 + 8 * g), next_k = page_of(kb0 + 8 * (l16 >> 2));
    for (uint32_t c = it.c0; c < it.c1; ++c) {
      const uint32_t kb = c * kUnitKeys + wave * kTileKeys;
      if (kb >= sh.keys) break;
      const uint32_t kv = kb + 8 * g, kk = kb + 8 * (l16 >> 2);
      uint32_t pv = next_v, pk = next_k;
      next_v = page_of(kv + kUnitKeys);
      next_k = page_of(kk + kUnitKeys);
      const bool held = pv < a.blocks;
      pv = held ? pv : 0u;
      pk = pk < a.blocks ? pk : 0u;
      const uint16_t* kp = a.kc + ((uint64_t)pk * a.heads + it.head) * page_len +
                           ((kk & in_page) + (l16 & 3)) * dim + 8 * g;
      const uint16_t* vp = a.vc + ((uint64_t)pv * a.heads + it.head) * page_len + (l16 << a.log_block) + (kv & in_page);

      u32x4 kf[2][KS], vf[DT];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          const uint32_t d = 32 * x + 8 * g;
          kf[h][x] = (!PAD || d < dim) ? *reinterpret_cast<const u32x4*>(kp + 4 * h * dim + 32 * x) : u32x4{};
        }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const uint32_t row = 16 * d + l16;
        vf[d] = (!PAD || row < dim) ? *reinterpret_cast<const u32x4*>(vp + d * v_step) : u32x4{};
      }
      floatx4 s[2] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < KS; ++x) s[h] = E::mfma(kf[h][x], q[0][x], s[h]);

      // Past the cached keys, or where a page is missing, scores of unseen keys
      // become -inf and values of keys that do not exist become zero (0 * NaN
      // would not be).
      const bool edge = __any(kb + kTileKeys > sh.ctx || !held);
      bool odd_values = false;
      if (edge) {
        const uint32_t bits = held ? seen_bits(a, sh, tok[0], kv) : 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((bits >> e) & 1)) s[e >> 2][e & 3] = -INFINITY;
        const uint32_t real = !held || kv >= sh.keys ? 0u : min(sh.keys - kv, 8u);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t v = vf[d][w];
            v = real <= 2u * w ? 0u : real == 2u * w + 1 ? v & 0xFFFFu : v;
            vf[d][w] = v;
            odd_values |= !E::finite2(v);
          }
        odd_values = __any(odd_values);
      }

      float keep;
      if (softmax_step<2>(s, m, keep, a.scale)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= keep;
      }
      if (!odd_values) {
        const u32x4 p = weights<E>(s[0], s[1], m.l);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = E::mfma(vf[d], p, o[d]);
      } else {
        // A drafted value is infinite or NaN: rows that do not see it must not
        // meet it, so keys of weight zero are left out one by one.
        const uint32_t real = min(sh.keys - kb, kTileKeys);
        add_weights(s, m.l);
#pragma unroll 1
        for (uint32_t x = 0; x < real; ++x) {
          const uint32_t key = kb + x, page = (uint32_t)pages[key >> a.log_block];
          if (page >= a.blocks) continue;
          const uint16_t* vx = a.vc + ((uint64_t)page * a.heads + it.head) * page_len + (key & in_page);
          uint32_t g_now = g;
          keep_here(g_now);
          float p = s[0][0];
#pragma unroll
          for (uint32_t e = 1; e < 8; ++e) p = (x & 7) == e ? s[e >> 2][e & 3] : p;
          p = __shfl(p, (x >> 3) * 16 + l16, 64);
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t row = 16 * d + 4 * g_now + j;
              if (PAD && row >= a.dim) continue;
              const float v = E::up(vx[(uint64_t)row << a.log_block]);
              if (p != 0.f) o[d][j] = fmaf(p, v, o[d][j]);
            }
        }
      }
    }

    // the four waves' parts meet in LDS and are added in order
    m.l = row_sum(m.l);
    if (g == 0) {
      s_m[wave][l16] = m.ref;
      s_l[wave][l16] = m.l;
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<floatx4*>(s_o + (wave * ROWS + l16) * kLine + 16 * d + 4 * g) = o[d];
    __syncthreads();
    constexpr uint32_t kFours = DP / 4;  // of a row
    const uint32_t live = min(it.rows - it.row0, (uint32_t)ROWS);
    const Parts<ROWS, DP> parts(a, run, it, sh);
    const uint32_t mine = it.whole ? 0u : parts.of(run.wg, it.first);
    for (uint32_t i = t; i < live * kFours; i += 256) {
      const uint32_t r = i / kFours, d = 4 * (i % kFours);
      const float top = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      const float ref = top == -INFINITY ? 0.f : top;
      float total = 0.f;
      floatx4 sum = {};
#pragma unroll
      for (uint32_t w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_m[w][r] - ref);
        total = fmaf(s_l[w][r], f, total);
        sum += *reinterpret_cast<floatx4*>(s_o + (w * ROWS + r) * kLine + d) * f;
      }
      if (it.whole) {
        if (!PAD || d < dim) write4<E>(out_at(a, sh, it, r) + d, sum, inverse(total));
      } else {
        part_store(parts.at, mine + 2 * ROWS + 4 * i, sum);
        if (d == 0) {
          part_store(parts.at, mine + r, top);
          part_store(parts.at, mine + ROWS + r, total);
        }
      }
    }
    if (!it.whole && parts.last(a, &s_last)) {
      for (uint32_t i = t; i < live * kFours; i += 256) {
        const uint32_t r = i / kFours, d = 4 * (i % kFours);
        floatx4 sum[1];
        const float all = parts.join(r, 4 * i, 0, sum);
        if (!PAD || d < dim) write4<E>(out_at(a, sh, it, r) + d, sum[0], inverse(all));
      }
    }
    __syncthreads();  // the LDS is reused by the next item
  }
}

// ----------------------------------------------------------------- more rows
// The waves take 16 RT rows each and share tiles of keys and values in LDS, two
// buffers deep: the next tile is loaded into registers while this one is
// multiplied.  16-byte pieces of a row are permuted by its number, which spreads the
// 16 rows of an operand read over 8 places; conflicts still take 24% of the LDS cycles.
//
// 64 rows are bound by memory (64 requests of 8000 keys, 8 key heads of 128: 5.7 TB/s
// with 16-token pages).  128 rows reach 560 TFLOP/s over keys in the caches (4 requests of
// 8000 keys, 32 tokens on 128 heads; 600 with 64-token pages): beside 64 matrix
// instructions a tile and wave has 216 vector ones, the exponentials among them, and the
// registers of two waves a SIMD leave no room to run one tile's products into another's
// softmax (tiles of 32 keys, the next tile's loads between the products, and wave
// priorities were measured and were no faster).
//
// A tile of rows runs over all keys of its request, also where there is no mask and the
// last of them lie behind all of its tokens, and treats every tile of keys past the cached
// ones as one that some row does not see.  Drafts are short beside what is cached, but a
// prompt pays twice: 4000 new tokens on 32 heads, nothing cached, take 498 us, 263 TFLOP/s
// of the products that are needed.
template <int DP>
struct Tile {
  static constexpr uint32_t kKeys = DP == 256 ? 32 : 64;
  static constexpr uint32_t kKPieces = DP / 8, kVPieces = kKeys / 8;  // of a row
  static constexpr uint32_t kPieces = kKeys * kKPieces;               // of a buffer, keys or values
  static constexpr uint32_t kEach = kPieces / 256;                    // a thread
  static constexpr uint32_t kBytes = 2 * 2 * kPieces * 16 + kPageRoom * 4;
  // rows of one operand read are r .. r + 3 and r + 8 .. r + 11 for keys, consecutive for values
  static __device__ __forceinline__ uint32_t k_at(uint32_t row, uint32_t piece) {
    return row * kKPieces + (piece ^ ((row & 3) | ((row >> 1) & 4)));
  }
  static __device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t piece) {
    return row * kVPieces + (piece ^ (row & (kVPieces - 1)));
  }
};

template <class E, int DP, int RT, bool PAD>
__global__ __launch_bounds__(256, 2) void k_attention_wide(AttnArgs a) {
  using T = Tile<DP>;
  constexpr int KS = DP / 32, DT = DP / 16, ROWS = 64 * RT, NS = T::kKeys / 16;
  extern __shared__ u32x4 lds[];
  u32x4* s_k = lds;                       // [2][kPieces]
  u32x4* s_v = lds + 2 * T::kPieces;      // [2][kPieces]
  uint32_t* s_page = reinterpret_cast<uint32_t*>(lds + 4 * T::kPieces);
  __shared__ uint32_t s_sum[6];
  __shared__ uint32_t s_last;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const uint32_t g = lane >> 4, l16 = lane & 15;
  Run run = find_run<ROWS>(a, s_sum);
  if (run.u == run.end) return;
  Shape sh = request_shape<ROWS>(a, run.b);
  const uint32_t dim = PAD ? a.dim : (uint32_t)DP, in_page = (1u << a.log_block) - 1;
  const uint64_t page_len = (uint64_t)dim << a.log_block;  // elements of a head's page
  // pieces of a page's value row that lie in one tile, as a power of two
  const uint32_t log_vp = min(a.log_block, (uint32_t)__builtin_ctz(T::kKeys)) - 3;

  // Piece x of a tile of values in the order of memory: page by page, value row by
  // row; which of the row's pieces it is.
  const uint32_t log_part = log_vp + (uint32_t)__builtin_ctz(DP);
  auto value_piece = [&](uint32_t x) { return (x >> log_part << log_vp) + (x & ((1u << log_vp) - 1)); };

  // a lane's place within its wave's pieces of a load, and a page of all heads, in bytes
  const uint32_t k_lane = 2 * ((lane / T::kKPieces) * dim + 8 * (lane % T::kKPieces));
  const uint32_t v_lane = 2 * (((lane >> log_vp) << a.log_block) + 8 * (lane & ((1u << log_vp) - 1)));
  const uint32_t page_bytes = (uint32_t)(2 * page_len) * a.heads;

  while (run.u < run.end) {
    const Item it = next_item<ROWS>(a, &run, &sh);
    const uint32_t row_w = it.row0 + wave * 16 * RT;  // the wave's first row
    const bool works = row_w < it.rows;
    u32x4 q[RT][KS];
    uint32_t tok[RT];
    load_queries<RT, KS, PAD>(a, sh, it, row_w, q, tok);
    floatx4 o[RT][DT];
    Softmax m[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int d = 0; d < DT; ++d) o[i][d] = floatx4{};
    const int32_t* pages = a.table + (uint64_t)run.b * a.width;
    const uint32_t k_end = min(it.c1 * kUnitKeys, sh.keys);
    const uint8_t* keys = reinterpret_cast<const uint8_t*>(a.kc + it.head * page_len);
    const uint8_t* values = reinterpret_cast<const uint8_t*>(a.vc + it.head * page_len);

    // in pieces of as many pages as the LDS has room for; a piece ends on a page's end
    for (uint32_t seg = it.c0 * kUnitKeys, seg_end; seg < k_end; seg = seg_end) {
      const uint32_t page0 = seg >> a.log_block;
      seg_end = min(k_end, (page0 + kPageRoom) << a.log_block);
      const uint32_t n_pages = ((seg_end - 1) >> a.log_block) - page0 + 1;
      for (uint32_t i = t; i < n_pages; i += 256) s_page[i] = (uint32_t)pages[page0 + i];
      __syncthreads();

      // Pages of a tile's groups of 8 keys, one a lane (repeating); ~0 where the group
      // does not exist.  `absent` has a bit for each such group.
      constexpr uint32_t kGroups = T::kKeys / 8;
      auto tile_pages = [&](uint32_t kb) {
        const uint32_t key = kb + 8 * (lane % kGroups);
        const uint32_t page = key < seg_end ? s_page[(key >> a.log_block) - page0] : ~0u;
        return page < a.blocks ? page : ~0u;
      };
      u32x4 rk[T::kEach], rv[T::kEach];
      uint32_t absent = 0, coming = tile_pages(seg);
      // A wave's pieces of one load lie in one page: key rows in a group of 8 keys,
      // values in the part of the tile that a page holds.  So the page is a scalar,
      // and nothing branches: where a group does not exist, page 0 is read instead.
      auto load = [&](uint32_t kb) {
        absent = (uint32_t)__ballot(coming == ~0u) & ((1u << kGroups) - 1);
        const uint32_t pages_now = coming == ~0u ? 0u : coming;
        coming = tile_pages(kb + T::kKeys);
        const uint32_t inside = kb & in_page;  // where the tile begins in a page longer than it
#pragma unroll
        for (uint32_t j = 0; j < T::kEach; ++j) {
          const uint32_t row_w = (64 * wave + 256 * j) / T::kKPieces;
          const uint8_t* from = keys + (uint64_t)__builtin_amdgcn_readlane(pages_now, row_w / 8) * page_bytes;
          const uint32_t at = (inside + (row_w & in_page)) * (2 * dim) + k_lane;
          rk[j] = !PAD || 8 * (t % T::kKPieces) < dim ? *reinterpret_cast<const u32x4*>(from + at) : u32x4{};
        }
#pragma unroll
        for (uint32_t j = 0; j < T::kEach; ++j) {
          const uint32_t x_w = 64 * wave + 256 * j, part = x_w >> log_part;
          const uint32_t y_w = x_w & ((1u << log_part) - 1);  // the wave's first piece within the part
          const uint8_t* from = values + (uint64_t)__builtin_amdgcn_readlane(pages_now, part << log_vp) * page_bytes;
          const uint32_t at = 2 * (((y_w >> log_vp) << a.log_block) + inside) + v_lane;
          rv[j] = !PAD || (y_w + lane) >> log_vp < dim ? *reinterpret_cast<const u32x4*>(from + at) : u32x4{};
        }
      };
      // Values of keys that do not exist become zero, and a drafted value that is
      // not finite is noted: a weight of zero times it is not zero.
      bool odd = false;
      auto store = [&](uint32_t kb, uint32_t buf) {
        const bool edge = kb + T::kKeys > sh.ctx || absent;
        odd = false;
#pragma unroll
        for (uint32_t j = 0; j < T::kEach; ++j) {
          const uint32_t x = t + 256 * j;
          s_k[buf * T::kPieces + T::k_at(x / T::kKPieces, x % T::kKPieces)] = rk[j];
        }
#pragma unroll
        for (uint32_t j = 0; j < T::kEach; ++j) {
          const uint32_t x = t + 256 * j, row = (x & ((DP << log_vp) - 1)) >> log_vp;
          const uint32_t piece = value_piece(x);
          if (edge) {
            const uint32_t key = kb + 8 * piece;
            const uint32_t real = (absent >> piece) & 1 || key >= sh.keys ? 0u : min(sh.keys - key, 8u);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t v = rv[j][w];
              v = real <= 2u * w ? 0u : real == 2u * w + 1 ? v & 0xFFFFu : v;
              rv[j][w] = v;
              odd |= !E::finite2(v);
            }
          }
          s_v[buf * T::kPieces + T::v_at(row, piece)] = rv[j];
        }
        // true where any thread noted one
        if (edge) odd = __syncthreads_or(odd);
        else __syncthreads();
      };

      load(seg);
      store(seg, 0);
      uint32_t buf = 0;
      for (uint32_t kb = seg; kb < seg_end; kb += T::kKeys, buf ^= 1) {
        const bool more = kb + T::kKeys < seg_end, odd_now = odd;
        const uint32_t absent_now = absent;
        if (more) load(kb + T::kKeys);
        if (works) {
          const u32x4* bk = s_k + buf * T::kPieces;
          const u32x4* bv = s_v + buf * T::kPieces;
          // Operands are read a step ahead of the products that take them (left to
          // itself the compiler reads each right before its use, 32 waits a tile).
          floatx4 s[RT][NS];
          u32x4 kf[2][KS];
          auto read_keys = [&](int h) {
            const uint32_t row = 32 * (h >> 1) + 8 * (l16 >> 2) + 4 * (h & 1) + (l16 & 3);
#pragma unroll
            for (int x = 0; x < KS; ++x) kf[h & 1][x] = bk[T::k_at(row, 4 * x + g)];
          };
          constexpr int kVf = 4, kVSteps = NS / 2 * DT / kVf;
          u32x4 vf[2][kVf];
          auto read_values = [&](int i) {
#pragma unroll
            for (int e = 0; e < kVf; ++e)
              vf[i & 1][e] = bv[T::v_at(16 * ((i * kVf + e) % DT) + l16, 4 * (i * kVf / DT) + g)];
          };
          read_keys(0);
#pragma unroll
          for (int h = 0; h < NS; ++h) {
            if (h + 1 < NS) read_keys(h + 1);
            else read_values(0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < RT; ++i) s[i][h] = floatx4{};
#pragma unroll
            for (int x = 0; x < KS; ++x)
#pragma unroll
              for (int i = 0; i < RT; ++i) s[i][h] = E::mfma(kf[h & 1][x], q[i][x], s[i][h]);
            __builtin_amdgcn_sched_barrier(0);
          }
          // scores of unseen keys become -inf: past the cached keys, and on missing pages
          if (kb + T::kKeys > sh.ctx || absent_now) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
              for (int h = 0; h < NS / 2; ++h) {
                const bool held = !((absent_now >> (4 * h + g)) & 1);
                const uint32_t bits = held ? seen_bits(a, sh, tok[i], kb + 32 * h + 8 * g) : 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (!((bits >> e) & 1)) s[i][2 * h + (e >> 2)][e & 3] = -INFINITY;
              }
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            float keep;
            if (softmax_step<NS>(s[i], m[i], keep, a.scale)) {
#pragma unroll
              for (int d = 0; d < DT; ++d) o[i][d] *= keep;
            }
          }
          if (!odd_now) {
            u32x4 p[NS / 2][RT];
#pragma unroll
            for (int h = 0; h < NS / 2; ++h)
#pragma unroll
              for (int i = 0; i < RT; ++i) p[h][i] = weights<E>(s[i][2 * h], s[i][2 * h + 1], m[i].l);
#pragma unroll
            for (int v = 0; v < kVSteps; ++v) {
              if (v + 1 < kVSteps) read_values(v + 1);
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int e = 0; e < kVf; ++e)
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                  const int d = (v * kVf + e) % DT;
                  o[i][d] = E::mfma(vf[v & 1][e], p[v * kVf / DT][i], o[i][d]);
                }
              __builtin_amdgcn_sched_barrier(0);
            }
          } else {
            // key by key, leaving out those of weight zero
            const uint16_t* values = reinterpret_cast<const uint16_t*>(bv);
#pragma unroll
            for (int i = 0; i < RT; ++i) add_weights(s[i], m[i].l);
#pragma unroll 1
            for (uint32_t x = 0; x < T::kKeys; ++x) {
              uint32_t g_now = g;
              keep_here(g_now);
              float p[RT];
#pragma unroll
              for (int i = 0; i < RT; ++i) {
                p[i] = 0.f;
#pragma unroll
                for (uint32_t e = 0; e < 2 * NS * 2; ++e)
                  p[i] = (x >> 5) * 8 + (x & 7) == e ? s[i][e >> 2][e & 3] : p[i];
                p[i] = __shfl(p[i], ((x >> 3) & 3) * 16 + l16, 64);
              }
#pragma unroll
              for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float v = E::up(values[T::v_at(16 * d + 4 * g_now + j, x >> 3) * 8 + (x & 7)]);
#pragma unroll
                  for (int i = 0; i < RT; ++i)
                    if (p[i] != 0.f) o[i][d][j] = fmaf(p[i], v, o[i][d][j]);
                }
            }
          }
        }
        if (more) store(kb + T::kKeys, buf ^ 1);
      }
      __syncthreads();  // the buffers and the pages are refilled
    }

#pragma unroll
    for (int i = 0; i < RT; ++i) m[i].l = row_sum(m[i].l);
    bool write = it.whole;
    if (!it.whole) {
      // outputs lie in the order of the lanes that hold them
      const Parts<ROWS, DP> parts(a, run, it, sh);
      const uint32_t mine = parts.of(run.wg, it.first), at0 = 4 * (wave * RT * DT * 64 + lane);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const uint32_t r = wave * 16 * RT + 16 * i + l16;
        if (it.row0 + r < it.rows) {
          if (g == 0) {
            part_store(parts.at, mine + r, m[i].ref);
            part_store(parts.at, mine + ROWS + r, m[i].l);
          }
#pragma unroll
          for (int d = 0; d < DT; ++d) part_store(parts.at, mine + 2 * ROWS + at0 + (i * DT + d) * 256, o[i][d]);
        }
      }
      write = parts.last(a, &s_last);
      if (write) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const uint32_t r = wave * 16 * RT + 16 * i + l16;
          if (it.row0 + r < it.rows) {
#pragma unroll
            for (int d = 0; d < DT; d += 4) {
              floatx4 four[4];
              m[i].l = parts.join(r, at0 + (i * DT + d) * 256, 256, four);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][d + e] = four[e];
            }
          }
        }
      }
    }
    if (write) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const uint32_t r = wave * 16 * RT + 16 * i + l16;
        if (it.row0 + r < it.rows) {
          const float inv = inverse(m[i].l);
          uint16_t* p = out_at(a, sh, it, r);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const uint32_t at = 16 * d + 4 * g;
            if (!PAD || at < dim) write4<E>(p + at, o[i][d], inv);
          }
        }
      }
    }
    __syncthreads();  // s_last is reused
  }
}

struct AttnPlan {
  uint32_t dp, rt, grid;  // rt: 0 the narrow kernel, else 16-row tiles a wave of the wide one
  size_t part_off, ws_bytes;
};

AttnPlan plan_attention(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  AttnPlan p;
  p.dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  // By the rows of a request and key head, on the average.  32 requests of 4000 keys, 8
  // key heads of 128, narrow against wide: 4 rows 103 and 98 us, 8 rows 105 and 97, 16
  // rows 112 and 98, 32 rows 196 and 100; but 8 requests of 1000 keys at 4 rows 12.5 and
  // 17.1, one of 4000 17 and 28: up to 8 rows the narrow kernel, whose workgroups need no
  // common tile, loses little where it loses.  64-row tiles against 128: 64 rows 107 and
  // 114 us, 80 rows 131 and 115.  Heads over 128 leave the narrow kernel too few
  // registers (16 requests of 4000 keys, 8 rows of 256: 286 and 110 us).
  // Uneven batches (4000 cached keys, 32 heads on 8; narrow, 64-row, 128-row tiles): one
  // request of 100 new tokens among 95 of one 280, 271, 286 us (the rule: narrow); 512
  // among 63 of one 360, 230, 240 (64-row); four of 512 among 60 of one 1067, 427, 366
  // (128-row); a prompt of 2000 among 31 of one 445, 293, 266 (128-row).
  const uint64_t rows = (uint64_t)tokens * (heads / kv_heads) / std::max(requests, 1u);
  p.rt = rows <= 8 && p.dp <= 128 ? 0 : rows <= 64 || p.dp == 256 ? 1 : 2;
  p.grid = kCUs * (p.rt == 0 ? kNarrowPerCU : kWidePerCU);
  // the counters' room is the same for every call, so that no call's parts lie where
  // another's counters are
  p.part_off = DGT_TREE_ATTENTION_ZEROED;
  p.ws_bytes = p.part_off + (size_t)p.grid * kRoom * (p.rt ? 64 * p.rt : 16) * (p.dp + 2) * 4;
  return p;
}

static_assert(DGT_TREE_ATTENTION_ZEROED % 256 == 0 &&
                  DGT_TREE_ATTENTION_ZEROED >= kCUs * std::max(kNarrowPerCU, kWidePerCU) * kRoom * 4,
              "a counter for each part");

bool attn_shape_ok(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  return heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && heads <= 65536 && dim >= 8 &&
         dim <= 256 && dim % 8 == 0 && requests <= kMaxRequests && tokens <= (1u << 20) &&
         (uint64_t)tokens * heads <= (1u << 30);
}

template <class E, int DP, int RT, bool PAD>
int launch_attention(const AttnArgs& a, uint32_t grid, hipStream_t st) {
  if constexpr (RT == 0) {
    hipLaunchKernelGGL((k_attention_narrow<E, DP, PAD>), dim3(grid), dim3(256), Narrow<DP>::kBytes, st, a);
  } else {
    const auto kernel = k_attention_wide<E, DP, RT, PAD>;
    if (Tile<DP>::kBytes > 64 * 1024 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)Tile<DP>::kBytes) != hipSuccess)
      return DGT_E_HIP;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), Tile<DP>::kBytes, st, a);
  }
  return launched();
}

template <class E, int DP, int RT>
int launch_attention(const AttnArgs& a, uint32_t grid, hipStream_t st) {
  return a.dim == DP ? launch_attention<E, DP, RT, false>(a, grid, st) : launch_attention<E, DP, RT, true>(a, grid, st);
}

template <class E>
int launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  switch (p.dp * 8 + p.rt) {
    case 64 * 8 + 0: return launch_attention<E, 64, 0>(a, p.grid, st);
    case 64 * 8 + 1: return launch_attention<E, 64, 1>(a, p.grid, st);
    case 64 * 8 + 2: return launch_attention<E, 64, 2>(a, p.grid, st);
    case 128 * 8 + 0: return launch_attention<E, 128, 0>(a, p.grid, st);
    case 128 * 8 + 1: return launch_attention<E, 128, 1>(a, p.grid, st);
    case 128 * 8 + 2: return launch_attention<E, 128, 2>(a, p.grid, st);
    case 256 * 8 + 1: return launch_attention<E, 256, 1>(a, p.grid, st);
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
  if (tokens == 1) q_row = out_row = 0;  // one row, or one head, has no stride
  if (heads == 1) q_head = out_head = 0;
  if (!aligned(d_q, 16) || !aligned(d_k_cache, 16) || !aligned(d_v_cache, 16) || !aligned(d_out, 4) ||
      !aligned(d_ws, 256) || q_row % 8 || q_head % 8 || out_row % 2 || out_head % 2)
    return DGT_E_ARG;
  // (a page's bytes are counted in 32 bits)
  if (blocks == 0 || (uint64_t)kv_heads * block * dim * 2 >= (1ull << 32)) return DGT_E_SHAPE;
  const AttnPlan p = plan_attention(tokens, heads, kv_heads, dim, requests);
  if (ws_bytes < p.ws_bytes) return DGT_E_BUFSIZE;
  // units of all requests, if each had its table full
  const uint64_t tile = p.rt ? 64 * p.rt : 16, tiles = (uint64_t)tokens * (heads / kv_heads) / tile + requests;
  if (tiles * ((uint64_t)width * block / kUnitKeys + 1) * kv_heads >= kMostUnits) return DGT_E_SHAPE;
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
