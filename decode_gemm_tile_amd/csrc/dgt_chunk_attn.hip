// Attention of a chunk of new tokens over a paged cache.
#include "dgt_serve.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace dgt {
namespace serve {
namespace {

// o_i = sum_j p_ij v_j / sum_j p_ij, p_ij = exp(s q_i k_j - max), over the keys j <= ctx + i.
//
// Rows of a request and key head are (token, query head of the group); a tile is as many
// whole tokens as fit kRows of them.  A workgroup runs over the keys of a tile, up to the
// last one that its last token sees, 64 at a time: tiles of keys and values are shared in
// LDS by four waves of 32 RT rows each.  S^T = K Q^T puts keys down and rows across the lanes;
// keys are dealt to the first operand so that a lane's scores are 8 consecutive keys of
// one row, the second operand of O^T = V^T P^T as it stands.
//
// Work is dealt in items: a piece of a tile's keys.  Whole tiles where there are enough of
// them; long tiles are cut where the card would be partly idle (k_chunk_plan weighs it),
// and k_chunk_join adds up their parts in the order of the keys.  Workgroups draw items
// from one queue a die, longest first; heads go round the dies, so a die's cache holds
// the keys of its heads.
struct ChunkArgs {
  const uint16_t *q, *kc, *vc;
  const int32_t *table, *ctx, *cu;
  uint16_t* out;
  uint32_t* plan;   // of the call, see Plan
  float* parts;
  uint64_t q_row, q_head, out_row, out_head;  // element strides
  uint32_t requests, tokens, heads, group, dim, log_block, width, blocks;
  uint32_t tile_tokens, splits;  // tokens of a tile; tiles a token's heads take (one of the two is 1)
  float scale;                   // times log2(e)
};

constexpr uint32_t kKeys = 64, kDies = 8;  // keys that pieces are counted in
constexpr uint32_t kMostParts = 1024;  // of all tiles together

// What k_chunk_plan leaves in the workspace, in words.
struct Plan {
  static constexpr uint32_t kQueue = 0;        // a counter a die, 64 bytes apart
  static constexpr uint32_t kPiece = 128;      // keys of a piece, a multiple of kKeys
  static constexpr uint32_t kItems = 129;      // in all
  static constexpr uint32_t kCut = 130;        // items among which those of cut tiles are
  static constexpr uint32_t kZeros = 144;      // 16 bytes
  static constexpr uint32_t kRecord = 160;     // [requests][kWords], the longest request first
  static constexpr uint32_t kWords = 8;        // item, part: the first ones; request, first row, rows, cached keys
  static __host__ __device__ constexpr uint32_t words(uint32_t requests) { return kRecord + kWords * requests; }
};

struct Chunk {  // one request
  uint32_t first, count, ctx, keys, tiles;
};

__device__ __forceinline__ void size_chunk(const ChunkArgs& a, Chunk& c) {
  c.keys = min(c.ctx + c.count, a.width << a.log_block);
  c.tiles = (c.count + a.tile_tokens - 1) / a.tile_tokens * a.splits;
}

__device__ __forceinline__ Chunk chunk_of(const ChunkArgs& a, uint32_t b) {
  Chunk c;
  request_rows(a.cu, b, a.tokens, &c.first, &c.count);
  c.ctx = min((uint32_t)max(a.ctx[b], 0), a.width << a.log_block);
  size_chunk(a, c);
  return c;
}

// One workgroup: how long pieces are, and the requests' items.  In units of a tile of 64
// keys, a call takes one piece where no CU gets two; else its work over the CUs, or a
// piece if that is more, and half an item, as the longest go first.  A part written and
// read again costs as much as kPart of them.
constexpr uint32_t kPlanThreads = 256, kMaxSorted = 1024, kChoices = 32;
constexpr float kPart = 6.f;

template <class T, class F>
__device__ __forceinline__ T reduce_all(T v, T* s, F f) {  // over the workgroup, to all threads
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = f(v, __shfl_xor(v, m, 64));
  if (lane == 0) s[wave] = v;
  __syncthreads();
  v = s[0];
  for (uint32_t w = 1; w < kPlanThreads / 64; ++w) v = f(v, s[w]);
  __syncthreads();
  return v;
}

__global__ __launch_bounds__(kPlanThreads) void k_chunk_plan(ChunkArgs a) {
  extern __shared__ uint32_t s_keys[];  // [requests] keys, [requests] tiles, [requests] the order
  uint32_t *s_tiles = s_keys + a.requests, *s_order = s_tiles + a.requests;
  __shared__ float s_f[kPlanThreads / 64], s_items[kPlanThreads], s_parts[kPlanThreads];
  __shared__ uint32_t s_u[kPlanThreads / 64], s_v[kPlanThreads / 64];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  float work = 0.f, rows = 0.f;
  uint32_t most = 0;
  for (uint32_t b = t; b < a.requests; b += kPlanThreads) {
    const Chunk c = chunk_of(a, b);
    s_keys[b] = c.tiles ? c.keys : 0;
    s_tiles[b] = c.tiles;
    // (their mean length: the first tiles see half of the new tokens less)
    work += (float)c.tiles * ((float)(c.keys + min(c.ctx, c.keys)) * (0.5f / kKeys) + 1.f);
    rows += (float)c.count;
    most = max(most, s_keys[b]);
  }
  auto add = [](float x, float y) { return x + y; };
  work = reduce_all(work, s_f, add) * (float)a.heads;
  // Offsets that fall name rows again and again, and no bound on items holds: such a batch
  // is not computed.  (Sums up to 2^24 are exact, and `tokens` is 2^20 at most.)
  const bool sound = reduce_all(rows, s_f, add) <= (float)a.tokens;
  most = reduce_all(most, s_u, [](uint32_t x, uint32_t y) { return max(x, y); });

  // Choice i cuts the longest tile into about 1.25^i pieces; 32 choices side by side, each
  // over the requests in eight strides.
  const uint32_t units = max((most + kKeys - 1) / kKeys, 1u), choice = t % kChoices;
  const uint32_t len = max((uint32_t)ceilf((float)units * exp2f(-0.32192809f * (float)choice)), min(units, 2u));
  float items = 0.f, parts = 0.f;
  for (uint32_t b = t / kChoices; b < a.requests; b += kPlanThreads / kChoices) {
    const uint32_t n = (uint32_t)(((uint64_t)s_keys[b] + len * kKeys - 1) / (len * kKeys));
    items += (float)s_tiles[b] * (float)max(n, 1u);
    if (n > 1) parts += (float)s_tiles[b] * (float)n;
  }
  s_items[t] = items;
  s_parts[t] = parts;
  __syncthreads();
  items = parts = 0.f;
  for (uint32_t i = choice; i < kPlanThreads; i += kChoices) {
    items += s_items[i];
    parts += s_parts[i];
  }
  items *= (float)a.heads;
  parts *= (float)a.heads;
  float time = items <= (float)kCUs ? (float)len : fmaxf(work / kCUs, (float)len) + 0.5f * work / items;
  if (parts > 0.f) time += kPart + parts * (kPart / kCUs);
  if (choice && parts > (float)kMostParts) time = 3.4e38f;
  uint32_t piece = len;
#pragma unroll
  for (int m = 1; m < (int)kChoices; m <<= 1) {
    const float ot = __shfl_xor(time, m, 64);
    const uint32_t ol = (uint32_t)__shfl_xor((int)piece, m, 64);
    if (ot < time || (ot == time && ol > piece)) {
      time = ot;
      piece = ol;
    }
  }
  piece *= kKeys;

  // requests by their longest tile, descending (of equals, the first first)
  for (uint32_t b = t; b < a.requests; b += kPlanThreads) {
    uint32_t rank = b;
    if (a.requests <= kMaxSorted) {
      rank = 0;
      const uint32_t mine = s_keys[b];
      for (uint32_t o = 0; o < a.requests; ++o) rank += s_keys[o] > mine || (s_keys[o] == mine && o < b);
    }
    s_order[rank] = b;
  }
  __syncthreads();
  uint32_t item = 0, part = 0;
  for (uint32_t i0 = 0; i0 < a.requests; i0 += kPlanThreads) {
    const uint32_t i = i0 + t;
    Chunk c = {};
    uint32_t n = 0, p = 0;
    if (i < a.requests) {
      c = chunk_of(a, s_order[i]);
      const uint32_t pieces = max((uint32_t)(((uint64_t)c.keys + piece - 1) / piece), 1u);
      n = c.tiles * pieces * a.heads;
      p = pieces > 1 ? n : 0;
    }
    uint32_t sn = n, sp = p;  // running sums of both
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t on = __shfl_up(sn, d, 64), op = __shfl_up(sp, d, 64);
      if (lane >= (uint32_t)d) {
        sn += on;
        sp += op;
      }
    }
    if (lane == 63) {
      s_u[wave] = sn;
      s_v[wave] = sp;
    }
    __syncthreads();
    uint32_t bn = item, bp = part;
    for (uint32_t w = 0; w < kPlanThreads / 64; ++w) {
      if (w == wave) {
        sn += bn;
        sp += bp;
      }
      bn += s_u[w];
      bp += s_v[w];
    }
    __syncthreads();
    if (i < a.requests) {
      u32x4* r = reinterpret_cast<u32x4*>(a.plan + Plan::kRecord + Plan::kWords * i);
      r[0] = u32x4{sn - n, sp - p, s_order[i], c.first};
      r[1] = u32x4{c.count, c.ctx, 0u, 0u};
    }
    item = bn;
    part = bp;
  }
  // every workgroup begins with the item of its own number
  if (t < kDies) a.plan[Plan::kQueue + 16 * t] = kCUs / kDies;
  if (t < 4) a.plan[Plan::kZeros + t] = 0;
  if (t == 0) {
    a.plan[Plan::kPiece] = piece;
    a.plan[Plan::kItems] = sound ? item : 0;
    // cut tiles come first where requests are sorted
    a.plan[Plan::kCut] = !sound || part == 0 ? 0 : a.requests <= kMaxSorted ? part : item;
  }
}

struct Item {
  Chunk c;
  uint32_t b, head, tile, piece, pieces;
  uint32_t token, tokens, member, members;  // its tokens, and the heads of the group that it holds
  uint32_t keys, k0, k1;                    // that its last token sees; of the piece
  uint32_t part;                            // where its part goes, if keys > piece
  __device__ __forceinline__ uint32_t rows() const { return tokens * members; }
};

// Item x of the call.  Of a request: tiles from the last, which sees most, pieces, heads.
__device__ __forceinline__ Item item_of(const ChunkArgs& a, uint32_t x, uint32_t piece, uint32_t rows) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t* records = a.plan + Plan::kRecord;
  uint32_t lo = 0, len = a.requests;
  while (len > 1) {
    const uint32_t step = (len + 63) / 64, at = lane * step;
    const bool before = lane == 0 || (at < len && records[Plan::kWords * (lo + at)] <= x);
    const uint32_t hits = (uint32_t)__popcll(__ballot(before));
    const uint32_t skip = (hits - 1) * step;
    lo += skip;
    len = min(step, len - skip);
  }
  const u32x4* record = reinterpret_cast<const u32x4*>(records + Plan::kWords * (uint32_t)__builtin_amdgcn_readfirstlane(lo));
  const u32x4 r0 = record[0], r1 = record[1];
  Item it;
  it.b = r0[2];
  it.c = Chunk{r0[3], r1[0], r1[1], 0, 0};
  size_chunk(a, it.c);
  it.pieces = max((uint32_t)(((uint64_t)it.c.keys + piece - 1) / piece), 1u);
  const uint32_t in = x - r0[0], rest = in / a.heads;
  it.head = in - rest * a.heads;
  it.piece = rest % it.pieces;
  it.tile = it.c.tiles - 1 - rest / it.pieces;
  it.part = r0[1] + in;
  const uint32_t split = it.tile % a.splits;
  it.token = it.tile / a.splits * a.tile_tokens;
  it.tokens = min(it.c.count - it.token, a.tile_tokens);
  it.member = split * rows;
  it.members = min(a.group - it.member, rows);
  it.keys = min(it.c.ctx + it.token + it.tokens, it.c.keys);
  it.k0 = it.piece * piece;
  it.k1 = min(it.keys, it.k0 + piece);
  return it;
}

// A tile of keys and values in LDS, in 16-byte pieces: rows of keys, then rows of values
// (a page holds them transposed).  Piece p of a row lies at p with some bits flipped by the
// row's number, so that 16 neighbouring rows of an operand read lie on different banks.
// Four tiles: one is multiplied by one half of the waves, the one before by the other,
// and two are on their way.
template <int DP, int WAVES>
struct Tile {
  static constexpr uint32_t kThreads = 64 * WAVES;
  static constexpr uint32_t kKeys = DP == 256 ? 32 : 64, kGroups = kKeys / 8;
  static constexpr uint32_t kKPieces = DP / 8, kVPieces = kKeys / 8;  // of a row
  static constexpr uint32_t kPieces = kKeys * kKPieces;               // keys or values
  static constexpr uint32_t kEach = kPieces / kThreads;               // a thread
  static constexpr uint32_t kBuffers = 4;
  static constexpr uint32_t kBytes = kBuffers * 2 * kPieces * 16;
  static __device__ __forceinline__ uint32_t k_flip(uint32_t row) { return kKPieces >= 16 ? row & 15 : (row >> 1) & 7; }
  static __device__ __forceinline__ uint32_t v_flip(uint32_t row) { return kVPieces == 8 ? (row >> 1) & 7 : (row >> 2) & 3; }
  static __device__ __forceinline__ uint32_t k_at(uint32_t row, uint32_t piece) { return row * kKPieces + (piece ^ k_flip(row)); }
  static __device__ __forceinline__ uint32_t v_at(uint32_t row, uint32_t piece) { return row * kVPieces + (piece ^ v_flip(row)); }
};

typedef float floatx16 __attribute__((ext_vector_type(16)));

template <class E>
__device__ __forceinline__ floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c);
template <>
__device__ __forceinline__ floatx16 mfma32<Bf16>(u32x4 a, u32x4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ floatx16 mfma32<F16>(u32x4 a, u32x4 b, floatx16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Maximum and sum over the two lanes that hold one row.
__device__ __forceinline__ float half_max(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Weights are 2^(score * scale - ref) against a reference that follows the row's maximum at
// a distance of at most 2^kSlack, so that outputs are rarely multiplied: fp32 sums and
// 16-bit weights up to 2^kSlack lose nothing by it.
constexpr float kSlack = 8.f;

template <int DP, int RT, int WAVES>
struct PartOf {  // ref[rows], l[rows], then the outputs in the order of the lanes that hold them
  static constexpr uint32_t kRows = WAVES * 32 * RT;
  static constexpr uint32_t kFloats = kRows * (DP + 2);
};

// 16 bytes a lane from memory into LDS, lane after lane from `to` (the same for all lanes of
// the wave) on.  The compiler does not know that it is under way: loads_wait<n> waits until no
// more than the last n of the wave's loads are.  (The compiler's own waits for its loads count
// these too, and so wait longer than they need.)
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory");
}
template <int N>
__device__ __forceinline__ void loads_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// What the threads of a workgroup have written to LDS is there for all of them; loads from
// memory stay under way (__syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <class E, int DP, int RT, int WAVES, bool PAD>
__global__ __launch_bounds__(64 * WAVES, 1) void k_chunk_attention(ChunkArgs a) {
  using T = Tile<DP, WAVES>;
  using P = PartOf<DP, RT, WAVES>;
  constexpr int KS = DP / 16, DT = DP / 32, NH = T::kKeys / 32;
  extern __shared__ u32x4 lds[];
  u32x4* s_k = lds;                               // [kBuffers][kPieces]
  u32x4* s_v = lds + T::kBuffers * T::kPieces;    // [kBuffers][kPieces]
  __shared__ uint32_t s_item;
  const uint32_t t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const uint32_t half = lane >> 5, l32 = lane & 31;
  const uint32_t group = wave >> 2;
  const uint32_t dim = PAD ? a.dim : (uint32_t)DP, in_page = (1u << a.log_block) - 1;
  const uint64_t page_len = (uint64_t)dim << a.log_block;  // elements of a head's page
  const uint32_t page_bytes = (uint32_t)(2 * page_len) * a.heads;
  const uint32_t piece = a.plan[Plan::kPiece], items = a.plan[Plan::kItems];

  // A wave's load fills 64 neighbouring pieces in LDS, so a lane asks for the piece that
  // belongs at its place.  Of the wave's first load: the lane's row and piece of it.  (Later
  // loads are some rows on; kinds of flips repeat with them, but for keys of 256 elements,
  // where bit 3 changes.)
  const uint32_t k_row = (64 * wave + lane) / T::kKPieces, k_piece = lane % T::kKPieces ^ T::k_flip(k_row);
  const uint32_t v_row = (64 * wave + lane) / T::kVPieces, v_piece = lane % T::kVPieces ^ T::v_flip(v_row);
  constexpr uint32_t kRowStep = T::kThreads / T::kKPieces, vRowStep = T::kThreads / T::kVPieces;
  static_assert(T::kVPieces == 8 ? vRowStep % 16 == 0 : vRowStep % 16 == 0, "values: the same flips in all loads");
  static_assert(T::kKPieces == 16 ? kRowStep % 16 == 0 : T::kKPieces == 8 ? kRowStep % 16 == 0 : kRowStep == 8, "keys");
  const uint32_t k_lane = 2 * (lane / T::kKPieces) * dim;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(a.plan + Plan::kZeros);  // what lies past dim

  uint32_t queue = blockIdx.x % kDies, tried = 0;
  auto draw = [&] { return __hip_atomic_fetch_add(a.plan + Plan::kQueue + 16 * queue, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  uint32_t drawn = blockIdx.x / kDies;
  for (;;) {
    if (t == 0) {
      uint32_t x = ~0u;
      while (tried < kDies) {
        if (drawn < (items + kDies - 1 - queue) / kDies) {
          x = drawn * kDies + queue;
          break;
        }
        queue = (queue + 1) % kDies;  // this die's is empty: help the next
        if (++tried < kDies) drawn = draw();
      }
      s_item = x;
    }
    __syncthreads();
    const uint32_t x = __builtin_amdgcn_readfirstlane(s_item);
    __syncthreads();
    if (x == ~0u) break;
    if (t == 0) drawn = draw();  // the next item's number is on its way while this one is worked on
    const Item it = item_of(a, x, piece, P::kRows);
    // (a piece past the tile's keys; a tile of no keys at all still has rows to write)
    if (it.k0 >= it.k1 && it.piece) continue;

    const uint32_t row_w = wave * 32 * RT;  // the wave's first row
    const uint32_t live = it.rows();
    const bool works = row_w < live;
    u32x4 q[RT][KS];
    uint32_t sees[RT];  // keys that a row sees
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const uint32_t r = min(row_w + 32 * i + l32, live - 1), tok = it.token + r / it.members;
      sees[i] = min(it.c.ctx + tok + 1, it.c.keys);
      const uint16_t* p = a.q + (uint64_t)(it.c.first + tok) * a.q_row +
                          (uint64_t)(it.head * a.group + it.member + r % it.members) * a.q_head;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const uint32_t d = 16 * s + 8 * half;
        q[i][s] = (!PAD || d < dim) ? *reinterpret_cast<const u32x4*>(p + d) : u32x4{};
      }
    }
    const uint32_t all_see = min(it.c.ctx + it.token + 1, it.c.keys);  // keys that every row sees
    floatx16 o[RT][DT];
    float ref[RT], l[RT];

    const int32_t* pages = a.table + (uint64_t)it.b * a.width;
    const uint8_t* keys = reinterpret_cast<const uint8_t*>(a.kc + it.head * page_len);
    const uint8_t* values = reinterpret_cast<const uint8_t*>(a.vc + it.head * page_len);
    // Pages of the groups of 8 keys of kSpan tiles, one a lane.  A table entry is looked at
    // kSpan tiles after it was asked for: waiting for it in each tile was a third of the
    // kernel's time.
    constexpr uint32_t kSpan = 64 / T::kGroups;
    auto key_of = [&](uint32_t n) { return it.k0 + n * T::kKeys + 8 * lane; };
    auto ask = [&](uint32_t n) { return (uint32_t)pages[min(key_of(n), it.k1 - 1) >> a.log_block]; };
    uint32_t coming = 0, have = 0;  // entries asked for, and pages in hand
    uint64_t gone = 0;              // a bit for each group in hand that does not exist
    // Sets tile n on its way into its buffer; where a group does not exist, page 0 is read
    // instead.  A wave's keys of one load lie in one group, so their page is a scalar.
    auto load = [&](uint32_t n) {
      const uint32_t in = n % kSpan * T::kGroups;
      if (in == 0) {
        const bool off = coming >= a.blocks || key_of(n) >= it.k1;
        gone = __ballot(off);
        have = off ? 0u : coming;
        coming = ask(n + kSpan);
      }
      const uint32_t inside = (it.k0 + n * T::kKeys) & in_page;  // where the tile begins in a page longer than it
      const uint32_t to = lds0 + (n % T::kBuffers) * T::kPieces * 16 + wave * 1024;
#pragma unroll
      for (uint32_t j = 0; j < T::kEach; ++j) {
        const uint32_t row = 64 * wave / T::kKPieces + kRowStep * j, p = k_piece ^ (T::kKPieces == 32 ? 8 * (j & 1) : 0);
        const uint8_t* from = keys + (uint64_t)__builtin_amdgcn_readlane(have, in + row / 8) * page_bytes +
                              (inside + (row & in_page)) * (2 * dim);
        // (every wave makes the same number of loads: waits count them)
        if constexpr (PAD) load_to_lds(8 * p < dim ? from + k_lane + 16 * p : zeros, to + T::kThreads * 16 * j);
        else load_to_lds(from, k_lane + 16 * p, to + T::kThreads * 16 * j);
      }
      const uint64_t page = (uint32_t)__shfl((int)have, in + v_piece, 64);
      const uint8_t* from = values + page * page_bytes + 2 * ((v_row << a.log_block) + inside + (8 * v_piece & in_page));
#pragma unroll
      for (uint32_t j = 0; j < T::kEach; ++j) {
        const uint8_t* row = from + j * ((uint64_t)(2 * vRowStep) << a.log_block);
        load_to_lds(!PAD || v_row + vRowStep * j < dim ? row : zeros, to + (T::kBuffers * T::kPieces + T::kThreads * j) * 16);
      }
      return (uint32_t)(gone >> in) & ((1u << T::kGroups) - 1);
    };
    constexpr int kLoads = 2 * T::kEach;  // of a wave and tile
    // Some row does not see all of tile n, or a page is missing.
    auto edge = [&](uint32_t n, uint32_t absent) { return it.k0 + (n + 1) * T::kKeys > all_see || absent; };
    // Such a tile, once it is there: values of keys that do not exist become zero, and one
    // that is not finite is noted, for a weight of zero times it is not zero.
    auto mend = [&](uint32_t n, uint32_t absent) {
      bool odd = false;
      for (uint32_t j = 0; j < T::kEach; ++j) {
        if (PAD && v_row + vRowStep * j >= dim) continue;
        u32x4* at = s_v + (n % T::kBuffers) * T::kPieces + t + T::kThreads * j;
        u32x4 v = *at;
        const uint32_t key = it.k0 + n * T::kKeys + 8 * v_piece;
        const uint32_t real = (absent >> v_piece) & 1 || key >= it.k1 ? 0u : min(it.k1 - key, 8u);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          v[w] = real <= 2u * w ? 0u : real == 2u * w + 1 ? v[w] & 0xFFFFu : v[w];
          odd |= !E::finite2(v[w]);
        }
        *at = v;
      }
      return __syncthreads_or(odd);
    };

    // The plain loop gives up at the first such value, and the slow one begins again.
    //
    // Waves w and w + 4 share a SIMD: while one is at its products, the other is at its
    // weights, and a barrier after each keeps it so.  (Left to themselves both did the same
    // at a time.)  In step 2 n the first half of the waves add the values of tile n - 1 and
    // multiply the keys of tile n, in step 2 n + 1 they turn scores into weights and set a
    // tile on its way; the second half is a step behind, and a tile ahead with its loads.
    // Tile n + 1 is there for all after step 2 n + 1.
    auto run = [&](auto slow) {
      constexpr bool kSlow = decltype(slow)::value;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        ref[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[i][d] = floatx16{};
      }
      const uint32_t tiles = it.k0 < it.k1 ? (it.k1 - it.k0 + T::kKeys - 1) / T::kKeys : 0;
      if (tiles == 0) return true;
      coming = ask(0);
      // bits of the missing groups of the tile at the products, and of those after it
      uint32_t absent = load(0), absent1 = 0, absent2 = 0, ahead = 1;
      if (ahead < tiles) absent1 = load(ahead++);
      if (group && ahead < tiles) absent2 = load(ahead++);
      if (ahead == 3) loads_wait<2 * kLoads>();
      else if (ahead == 2) loads_wait<kLoads>();
      else loads_wait<0>();
      lds_barrier();
      if (edge(0, absent) && mend(0, absent) && !kSlow) return false;

      floatx16 s[RT][NH];
      u32x4 p[RT][2 * NH];
      // Operands are read a step of four ahead of the products that take them.  Pieces 2 x on
      // from the first lie at its place with 2 x flipped, whatever the row: one register
      // addresses them all (with one each, some were kept in memory, and fetching those
      // waited for all loads of the next tile).  Row of the operand to key: bits 2 and 3
      // change places.
      const uint32_t k_first = T::k_at((l32 & 19) | ((l32 & 4) << 1) | ((l32 & 8) >> 1), half);
      const uint32_t v_first = T::v_at(l32, half);
      constexpr int kStep = 4, NK = NH * KS / kStep, NV = 2 * NH * DT / kStep;
      u32x4 kf[2][kStep], vf[2][kStep];
      auto read_keys = [&](uint32_t buf, int i) {
#pragma unroll
        for (int e = 0; e < kStep; ++e) {
          const int h = (kStep * i + e) / KS, x = (kStep * i + e) % KS;
          kf[i & 1][e] = s_k[((buf * T::kPieces + k_first) ^ 2 * x) + 32 * h * T::kKPieces];
        }
      };
      auto read_values = [&](uint32_t buf, int i) {
#pragma unroll
        for (int e = 0; e < kStep; ++e) {
          const int g = (kStep * i + e) / DT, d = (kStep * i + e) % DT;
          vf[i & 1][e] = s_v[((buf * T::kPieces + v_first) ^ 2 * g) + 32 * d * T::kVPieces];
        }
      };
      // o += the weighted values of the tile in buffer `buf`, whose first operands are in hand;
      // `then`: the buffer whose keys come next
      auto add_values = [&](uint32_t buf, uint32_t then) {
        if constexpr (!kSlow) {
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            if (n + 1 < NV) read_values(buf, n + 1);
            else read_keys(then, 0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < kStep; ++e) {
              const int g = (kStep * n + e) / DT, d = (kStep * n + e) % DT;
#pragma unroll
              for (int i = 0; i < RT; ++i) o[i][d] = mfma32<E>(vf[n & 1][e], p[i][g], o[i][d]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
          // key by key, leaving out those of weight zero
          const uint16_t* value = reinterpret_cast<const uint16_t*>(s_v + buf * T::kPieces);
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
              for (int e = 0; e < 16; ++e) l[i] += s[i][h][e];
#pragma unroll 1
          for (uint32_t x = 0; x < T::kKeys; ++x) {
            uint32_t h_now = half;
            keep_here(h_now);
            float w[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) {
              w[i] = 0.f;
#pragma unroll
              for (uint32_t e = 0; e < 16 * NH; ++e) w[i] = (x >> 4) * 8 + (x & 7) == e ? s[i][e >> 4][e & 15] : w[i];
              w[i] = __shfl(w[i], ((x >> 3) & 1) * 32 + l32, 64);
            }
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float v = E::up(value[T::v_at(32 * d + (e & 3) + 4 * h_now + 8 * (e >> 2), x >> 3) * 8 + (x & 7)]);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                  if (w[i] != 0.f) o[i][d][e] = fmaf(w[i], v, o[i][d][e]);
              }
          }
        }
      };

      if (group) lds_barrier();
      // after step 2 n + 1: waits for tile n + 1, all but the loads of the tile after it
      auto arrive = [&](uint32_t n, uint32_t absent) {
        if (ahead > n + 2) loads_wait<kLoads>();
        else loads_wait<0>();
        lds_barrier();
        return n + 1 < tiles && edge(n + 1, absent) && mend(n + 1, absent) && !kSlow;
      };
      // scores of the tile in buffer `buf`, whose first operands are in hand
      auto multiply = [&](uint32_t buf) {
#pragma unroll
        for (int m = 0; m < NK; ++m) {
          if (m + 1 < NK) read_keys(buf, m + 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int e = 0; e < kStep; ++e) {
            const int h = (kStep * m + e) / KS, x = (kStep * m + e) % KS;
#pragma unroll
            for (int i = 0; i < RT; ++i) s[i][h] = mfma32<E>(kf[m & 1][e], q[i][x], x ? s[i][h] : floatx16{});
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if (works) {
        read_keys(0, 0);
        multiply(0);
      }
      for (uint32_t n = 0;; ++n) {
        if (!group) lds_barrier();
        else if (arrive(n, absent1)) return false;

        const uint32_t kb = it.k0 + n * T::kKeys, buf = n % T::kBuffers, then = (n + 1) % T::kBuffers;
        const uint32_t absent_now = absent;
        absent = absent1;
        absent1 = absent2;
        if (ahead < tiles) {
          const uint32_t x = load(ahead++);
          (group ? absent2 : absent1) = x;
        }
        if (works) {
          // a lane's scores: keys kb + 16 g + 8 half + e are element 8 (g & 1) + e of s[g / 2]
          if (kb + T::kKeys > all_see || absent_now) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
              for (int g = 0; g < 2 * NH; ++g) {
                const uint32_t key = kb + 16 * g + 8 * half;
                const uint32_t seen = (absent_now >> (2 * g + half)) & 1 || key >= sees[i] ? 0u : min(sees[i] - key, 8u);
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e)
                  if (e >= seen) s[i][g >> 1][8 * (g & 1) + e] = -INFINITY;
              }
          }
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            float top = s[i][0][0];
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
              for (int e = 0; e < 16; e += 2) top = fmaxf(fmaxf(top, s[i][h][e]), s[i][h][e + 1]);
            top = half_max(top) * a.scale;
            if (__any(top > ref[i] + kSlack)) {
              const float now = fmaxf(ref[i], top);
              const float keep = ref[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref[i] - now);
              ref[i] = now;
              l[i] *= keep;
#pragma unroll
              for (int d = 0; d < DT; ++d) o[i][d] *= keep;
            }
            const float base = ref[i] == -INFINITY ? 0.f : ref[i];  // nothing seen: the weights are 2^-inf = 0
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
              for (int e = 0; e < 16; ++e) s[i][h][e] = __builtin_amdgcn_exp2f(fmaf(s[i][h][e], a.scale, -base));
            if constexpr (!kSlow) {
#pragma unroll
              for (int g = 0; g < 2 * NH; ++g)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  p[i][g][w] = E::pack2(s[i][g >> 1][8 * (g & 1) + 2 * w], s[i][g >> 1][8 * (g & 1) + 2 * w + 1]);
                  l[i] = E::add2(p[i][g][w], l[i]);
                }
            }
          }
          if (!kSlow) read_values(buf, 0);
        }
        if (group) lds_barrier();
        else if (arrive(n, absent)) return false;

        if (works) add_values(buf, then);
        if (n + 1 == tiles) break;
        if (works) {
          if (kSlow) read_keys(then, 0);
          multiply(then);
        }
      }
      if (!group) lds_barrier();
      return true;
    };
    if (!run(std::false_type{})) {
      loads_wait<0>();
      __syncthreads();  // the buffers are refilled
      run(std::true_type{});
    }

    const bool whole = it.keys <= piece;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      l[i] = half_sum(l[i]);
      const uint32_t r = row_w + 32 * i + l32;
      if (r >= live) continue;
      if (whole) {
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const uint32_t tok = it.token + r / it.members;
        uint16_t* p = a.out + (uint64_t)(it.c.first + tok) * a.out_row +
                      (uint64_t)(it.head * a.group + it.member + r % it.members) * a.out_head;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t at = 32 * d + 8 * g + 4 * half;
            if (!PAD || at < dim) {
              *reinterpret_cast<uint32_t*>(p + at) = E::pack2(o[i][d][4 * g] * inv, o[i][d][4 * g + 1] * inv);
              *reinterpret_cast<uint32_t*>(p + at + 2) = E::pack2(o[i][d][4 * g + 2] * inv, o[i][d][4 * g + 3] * inv);
            }
          }
      } else {
        float* part = a.parts + (uint64_t)it.part * P::kFloats;
        if (half == 0) {
          part[r] = ref[i];
          part[P::kRows + r] = l[i];
        }
        float* to = part + 2 * P::kRows + r * DP;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<floatx4*>(to + 32 * d + 8 * g + 4 * half) =
                floatx4{o[i][d][4 * g], o[i][d][4 * g + 1], o[i][d][4 * g + 2], o[i][d][4 * g + 3]};
      }
    }
    __syncthreads();  // the buffers are refilled
  }
}

// Adds up the parts of tiles that were cut, in the order of the keys: a workgroup takes
// some rows of a tile, a thread four outputs of a row.
template <class E, int DP, int RT, int WAVES>
__global__ __launch_bounds__(256) void k_chunk_join(ChunkArgs a) {
  using P = PartOf<DP, RT, WAVES>;
  constexpr uint32_t kFours = DP / 4, kRowsEach = 256 / kFours, kSteps = P::kRows / kRowsEach;
  const uint32_t piece = a.plan[Plan::kPiece], items = a.plan[Plan::kCut], t = threadIdx.x;
  for (uint64_t unit = blockIdx.x; unit < (uint64_t)items * kSteps; unit += gridDim.x) {
    const Item it = item_of(a, (uint32_t)(unit / kSteps), piece, P::kRows);
    if (it.piece || it.keys <= piece) continue;
    const uint32_t r = (uint32_t)(unit % kSteps) * kRowsEach + t / kFours, d = 4 * (t % kFours);
    if (r >= it.rows()) continue;
    // item numbers of a tile's pieces lie `heads` apart; four are asked for at a time
    float m = -INFINITY, l = 0.f;
    floatx4 o = {};
    const uint32_t count = (it.keys + piece - 1) / piece;
    const float* part = a.parts + (uint64_t)it.part * P::kFloats;
    const uint64_t step = (uint64_t)a.heads * P::kFloats;
    for (uint32_t k0 = 0; k0 < count; k0 += 4) {
      float mw[4], lw[4];
      floatx4 ow[4];
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        const float* from = part + min(k0 + k, count - 1) * step;
        mw[k] = from[r];
        lw[k] = from[P::kRows + r];
        ow[k] = *reinterpret_cast<const floatx4*>(from + 2 * P::kRows + r * DP + d);
      }
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) {
        if (k0 + k >= count) break;
        const float now = fmaxf(m, mw[k]), base = now == -INFINITY ? 0.f : now;
        const float f = __builtin_amdgcn_exp2f(m - base), fw = __builtin_amdgcn_exp2f(mw[k] - base);
        m = now;
        l = fmaf(lw[k], fw, l * f);
        o = o * f + ow[k] * fw;
      }
    }
    if (d >= a.dim) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const uint32_t tok = it.token + r / it.members;
    uint16_t* p = a.out + (uint64_t)(it.c.first + tok) * a.out_row +
                  (uint64_t)(it.head * a.group + it.member + r % it.members) * a.out_head + d;
    *reinterpret_cast<uint32_t*>(p) = E::pack2(o[0] * inv, o[1] * inv);
    *reinterpret_cast<uint32_t*>(p + 2) = E::pack2(o[2] * inv, o[3] * inv);
  }
}

struct ChunkPlan {
  uint32_t dp, rows, tile_tokens, splits;
  size_t part_off, ws_bytes;
};

ChunkPlan plan_chunk(uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  ChunkPlan p;
  p.dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
  p.rows = p.dp == 256 ? 128 : 256;
  const uint32_t group = heads / kv_heads;
  p.tile_tokens = std::max(p.rows / group, 1u);
  p.splits = (group + p.rows - 1) / p.rows;
  p.part_off = ((size_t)Plan::words(requests) * 4 + 255) / 256 * 256;
  p.ws_bytes = p.part_off + (size_t)kMostParts * p.rows * (p.dp + 2) * 4;
  return p;
}

bool chunk_shape_ok(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  return heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && heads <= 65536 && dim >= 8 &&
         dim <= 256 && dim % 8 == 0 && requests <= kMaxRequests && tokens <= (1u << 20) &&
         (uint64_t)tokens * heads <= (1u << 30);
}

template <class E, int DP, int RT, int WAVES, bool PAD>
int launch_chunk(const ChunkArgs& a, hipStream_t st) {
  using T = Tile<DP, WAVES>;
  const auto kernel = k_chunk_attention<E, DP, RT, WAVES, PAD>;
  if (T::kBytes > 64 * 1024 &&
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                          (int)T::kBytes) != hipSuccess)
    return DGT_E_HIP;
  hipLaunchKernelGGL(kernel, dim3(kCUs), dim3(64 * WAVES), T::kBytes, st, a);
  if (int rc = launched()) return rc;
  hipLaunchKernelGGL((k_chunk_join<E, DP, RT, WAVES>), dim3(4 * kCUs), dim3(256), 0, st, a);
  return launched();
}

template <class E>
int launch_chunk(const ChunkArgs& a, uint32_t dp, hipStream_t st) {
  const uint32_t lds = 3 * a.requests * 4;  // 96 KB at most
  if (lds > 60 * 1024 && hipFuncSetAttribute(reinterpret_cast<const void*>(k_chunk_plan),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
    return DGT_E_HIP;
  hipLaunchKernelGGL(k_chunk_plan, dim3(1), dim3(kPlanThreads), lds, st, a);
  if (int rc = launched()) return rc;
  const bool pad = a.dim != dp;
  switch (dp) {
    case 64: return pad ? launch_chunk<E, 64, 1, 8, true>(a, st) : launch_chunk<E, 64, 1, 8, false>(a, st);
    case 128: return pad ? launch_chunk<E, 128, 1, 8, true>(a, st) : launch_chunk<E, 128, 1, 8, false>(a, st);
  }
  return pad ? launch_chunk<E, 256, 1, 4, true>(a, st) : launch_chunk<E, 256, 1, 4, false>(a, st);
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" {

size_t dgt_chunk_attention_workspace(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim,
                                     uint32_t requests) {
  if (!chunk_shape_ok(tokens, heads, kv_heads, dim, requests)) return 0;
  return plan_chunk(heads, kv_heads, dim, requests).ws_bytes;
}

int dgt_chunk_attention(uint32_t type, const void* d_q, uint64_t q_row, uint64_t q_head,
                        const void* d_k_cache, const void* d_v_cache, uint32_t blocks, uint32_t block,
                        const int32_t* d_table, uint32_t width, const int32_t* d_ctx, const int32_t* d_cu,
                        uint32_t requests, uint32_t tokens, uint32_t heads, uint32_t kv_heads,
                        uint32_t dim, float scale, void* d_out, uint64_t out_row, uint64_t out_head,
                        void* d_ws, size_t ws_bytes, void* stream) {
  if (type != DGT_ELT_BF16 && type != DGT_ELT_F16) return DGT_E_UNSUPPORTED;
  if (!chunk_shape_ok(tokens, heads, kv_heads, dim, requests) || !block_ok(block) ||
      !pool_ok(blocks, block) || (uint64_t)width * block > 0x7FFFFFFFull)
    return DGT_E_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale)) return DGT_E_ARG;
  if (tokens == 0 || requests == 0) return DGT_OK;
  if (!d_q || !d_out || !d_cu || !d_ctx || !d_ws) return DGT_E_ARG;
  if ((width && !d_table) || (blocks && (!d_k_cache || !d_v_cache))) return DGT_E_ARG;
  if (tokens == 1) q_row = out_row = 0;  // one row, or one head, has no stride
  if (heads == 1) q_head = out_head = 0;
  if (!aligned(d_q, 16) || !aligned(d_k_cache, 16) || !aligned(d_v_cache, 16) || !aligned(d_out, 4) ||
      !aligned(d_ws, 256) || q_row % 8 || q_head % 8 || out_row % 2 || out_head % 2)
    return DGT_E_ARG;
  // (a page's bytes are counted in 32 bits)
  if (blocks == 0 || (uint64_t)kv_heads * block * dim * 2 >= (1ull << 32)) return DGT_E_SHAPE;
  const ChunkPlan p = plan_chunk(heads, kv_heads, dim, requests);
  if (ws_bytes < p.ws_bytes) return DGT_E_BUFSIZE;
  ChunkArgs a;
  a.q = static_cast<const uint16_t*>(d_q);
  a.kc = static_cast<const uint16_t*>(d_k_cache);
  a.vc = static_cast<const uint16_t*>(d_v_cache);
  a.table = d_table;
  a.ctx = d_ctx;
  a.cu = d_cu;
  a.out = static_cast<uint16_t*>(d_out);
  a.plan = static_cast<uint32_t*>(d_ws);
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
  a.tile_tokens = p.tile_tokens;
  a.splits = p.splits;
  a.scale = scale * 1.4426950408889634f;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return type == DGT_ELT_BF16 ? launch_chunk<Bf16>(a, p.dp, st) : launch_chunk<F16>(a, p.dp, st);
}

}  // extern "C"
