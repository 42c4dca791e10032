// Attention of a chunk of new tokens over a paged cache.
#include "dgt_chunk_plan.h"
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
// last one that its last token sees, 64 at a time (32 where heads are longer than 128): tiles of
// keys and values are shared in LDS by eight waves (four) of 32 rows each.  S^T = K Q^T puts
// keys down and rows across the lanes; keys are dealt to the first operand so that a lane's
// scores are 8 consecutive keys of one row, the second operand of O^T = V^T P^T as it stands.
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
  uint32_t rows, tile_tokens, splits;  // rows and tokens of a tile; tiles a token's heads take (one of the two is 1)
  float scale;                   // times log2(e)
};

constexpr uint32_t kKeys = 64, kDies = 8;  // keys that pieces are counted in
constexpr uint32_t kPartRows = 1 << 18;  // rows of all parts together

// What k_chunk_plan leaves in the workspace, in words.
struct Plan {
  static constexpr uint32_t kQueue = 0;        // a counter a die, 64 bytes apart
  static constexpr uint32_t kPiece = 128;      // keys of a piece, a multiple of kKeys
  static constexpr uint32_t kItems = 129;      // in all
  static constexpr uint32_t kCut = 130;        // cut tiles
  static constexpr uint32_t kMost = 131;       // pieces of the longest
  static constexpr uint32_t kZeros = 144;      // 16 bytes
  static constexpr uint32_t kRecord = 160;     // [requests][kWords], the longest request first
  // item, part: the first ones; request, first row, rows, cached keys, first cut tile
  static constexpr uint32_t kItem = 0, kTile = 6, kWords = 8;
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
constexpr uint32_t kPlanThreads = 256, kMaxSorted = 1024;
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
  __shared__ uint32_t s_u[kPlanThreads / 64], s_v[kPlanThreads / 64], s_w[kPlanThreads / 64];
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

  // 32 choices of lengths side by side, each over the requests in eight strides.
  const uint32_t units = max((most + kKeys - 1) / kKeys, 1u), choice = t % kChoices;
  const uint32_t len = piece_units(units, choice);
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
  if (choice && parts > (float)(kPartRows / a.rows)) time = 3.4e38f;
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
  uint32_t item = 0, part = 0, cut = 0;
  for (uint32_t i0 = 0; i0 < a.requests; i0 += kPlanThreads) {
    const uint32_t i = i0 + t;
    Chunk c = {};
    uint32_t n = 0, p = 0, c1 = 0;
    if (i < a.requests) {
      c = chunk_of(a, s_order[i]);
      const uint32_t pieces = max((uint32_t)(((uint64_t)c.keys + piece - 1) / piece), 1u);
      n = c.tiles * pieces * a.heads;
      p = pieces > 1 ? n : 0;
      c1 = pieces > 1 ? c.tiles * a.heads : 0;
    }
    uint32_t sn = n, sp = p, sc = c1;  // running sums of them
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t on = __shfl_up(sn, d, 64), op = __shfl_up(sp, d, 64), oc = __shfl_up(sc, d, 64);
      if (lane >= (uint32_t)d) {
        sn += on;
        sp += op;
        sc += oc;
      }
    }
    if (lane == 63) {
      s_u[wave] = sn;
      s_v[wave] = sp;
      s_w[wave] = sc;
    }
    __syncthreads();
    uint32_t bn = item, bp = part, bc = cut;
    for (uint32_t w = 0; w < kPlanThreads / 64; ++w) {
      if (w == wave) {
        sn += bn;
        sp += bp;
        sc += bc;
      }
      bn += s_u[w];
      bp += s_v[w];
      bc += s_w[w];
    }
    __syncthreads();
    if (i < a.requests) {
      u32x4* r = reinterpret_cast<u32x4*>(a.plan + Plan::kRecord + Plan::kWords * i);
      r[0] = u32x4{sn - n, sp - p, s_order[i], c.first};
      r[1] = u32x4{c.count, c.ctx, sc - c1, 0u};
    }
    item = bn;
    part = bp;
    cut = bc;
  }
  // every workgroup begins with the item of its own number
  if (t < kDies) a.plan[Plan::kQueue + 16 * t] = kCUs / kDies;
  if (t < 4) a.plan[Plan::kZeros + t] = 0;
  if (t == 0) {
    a.plan[Plan::kPiece] = piece;
    a.plan[Plan::kItems] = sound ? item : 0;
    a.plan[Plan::kCut] = sound ? cut : 0;
    a.plan[Plan::kMost] = (uint32_t)(((uint64_t)most + piece - 1) / piece);
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

// Item x of the call, or (BY = Plan::kTile) the first item of cut tile x.  Of a request: tiles
// from the last, which sees most, pieces, heads.
template <uint32_t BY>
__device__ __forceinline__ Item item_of(const ChunkArgs& a, uint32_t x, uint32_t piece, uint32_t rows) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t* records = a.plan + Plan::kRecord;
  uint32_t lo = 0, len = a.requests;
  while (len > 1) {
    const uint32_t step = (len + 63) / 64, at = lane * step;
    const bool before = lane == 0 || (at < len && records[Plan::kWords * (lo + at) + BY] <= x);
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
  uint32_t in = x - (BY == Plan::kItem ? r0[0] : r1[2]), rest = in / a.heads;
  it.head = in - rest * a.heads;
  if (BY == Plan::kTile) {
    rest *= it.pieces;
    in = rest * a.heads + it.head;
  }
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
// Four tiles: of the one whose values are multiplied, the next, whose keys are, and two that
// are on their way.
template <int DP, int WAVES>
struct Tile {
  static constexpr uint32_t kThreads = 64 * WAVES;
  static constexpr uint32_t kKeys = DP == 256 ? 32 : 64, kGroups = kKeys / 8;
  static constexpr uint32_t kKPieces = DP / 8, kVPieces = kKeys / 8;  // of a row
  static constexpr uint32_t kPieces = kKeys * kKPieces;               // keys or values
  static constexpr uint32_t kEach = kPieces / kThreads;               // a thread
  static constexpr uint32_t kBuffers = 4;
  static constexpr uint32_t kSpan = 64 / kGroups;                      // tiles that 64 table entries last for
  static constexpr uint32_t kTables = kBuffers * 2 * kPieces * 16;     // bytes in front of the tables
  static constexpr uint32_t kTable = 64 * 4 + 64 * 8;                  // a wave's: entries, addresses of values
  static constexpr uint32_t kBytes = kTables + WAVES * kTable;
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

// f(FROM), ..., f(TO - 1), each with a constant.
template <int FROM, int TO, class F>
__device__ __forceinline__ void steps(const F& f) {
  if constexpr (FROM < TO) {
    f(std::integral_constant<int, FROM>{});
    steps<FROM + 1, TO>(f);
  }
}

// Maximum and sum over the two lanes that hold one row.
template <class F>
__device__ __forceinline__ float over_row(float v, F f) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// Weights are 2^(score * scale - ref) against a reference that follows the row's maximum at
// a distance of at most 2^kSlack, so that outputs are rarely multiplied: fp32 sums and
// 16-bit weights up to 2^kSlack lose nothing by it.
constexpr float kSlack = 8.f;

template <int DP, int WAVES>
struct PartOf {  // ref[rows], l[rows], then the outputs in the order of the lanes that hold them
  static constexpr uint32_t kRows = WAVES * 32;
  static constexpr uint32_t kFloats = kRows * (DP + 2);
};

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved, and named so that nothing of the compiler's is kept in it
// 16 bytes a lane from memory into LDS, lane after lane from `to` (the same for all lanes of
// the wave) on.  The compiler does not know that it is under way: loads_wait<n> waits until no
// more than the last n of the wave's loads are.  (The compiler's own waits for its loads count
// these too, and so wait longer than they need.)
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, uint32_t to) {
  // (a base that a vector instruction has just written, as v_readlane does, may be read 5 steps on)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}
// The same with 4 bytes a lane.
__device__ __forceinline__ void load_word_to_lds(const void* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop
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

template <class E, int DP, int WAVES, bool PAD>
__global__ __launch_bounds__(64 * WAVES, 1) void k_chunk_attention(ChunkArgs a) {
  using T = Tile<DP, WAVES>;
  using P = PartOf<DP, WAVES>;
  constexpr int KS = DP / 16, DT = DP / 32, NH = T::kKeys / 32;
  extern __shared__ u32x4 lds[];
  u32x4* s_k = lds;                               // [kBuffers][kPieces]
  u32x4* s_v = lds + T::kBuffers * T::kPieces;    // [kBuffers][kPieces]
  __shared__ uint32_t s_item;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t dim = PAD ? a.dim : (uint32_t)DP, in_page = (1u << a.log_block) - 1;
  const uint64_t page_len = (uint64_t)dim << a.log_block;  // elements of a head's page
  const uint32_t page_bytes = (uint32_t)(2 * page_len) * a.heads;
  const uint32_t piece = a.plan[Plan::kPiece], items = a.plan[Plan::kItems];

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(a.plan + Plan::kZeros);  // what lies past dim

  uint32_t queue = blockIdx.x % kDies, tried = 0;
  auto draw = [&] { return __hip_atomic_fetch_add(a.plan + Plan::kQueue + 16 * queue, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  uint32_t drawn = blockIdx.x / kDies;
  for (;;) {
    // What follows from a thread's number is worked out anew for each item: kept over the loops
    // below it took 32 registers, for which operands had to go to memory.
    uint32_t t = threadIdx.x;
    keep_here(t);
    const uint32_t lane = t & 63, half = lane >> 5, l32 = lane & 31;
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
    const Item it = item_of<Plan::kItem>(a, x, piece, P::kRows);
    // (a piece past the tile's keys; a tile of no keys at all still has rows to write)
    if (it.k0 >= it.k1 && it.piece) continue;

    // A wave's load fills 64 neighbouring pieces in LDS, so a lane asks for the piece that
    // belongs at its place.  Of the wave's first load: the lane's row and piece of it.  (Later
    // loads are some rows on; flips repeat with them, but for keys of 256 elements, where bit 3
    // changes.)
    const uint32_t k_row = (64 * wave + lane) / T::kKPieces, k_piece = lane % T::kKPieces ^ T::k_flip(k_row);
    const uint32_t v_row = (64 * wave + lane) / T::kVPieces, v_piece = lane % T::kVPieces ^ T::v_flip(v_row);
    constexpr uint32_t kRowStep = T::kThreads / T::kKPieces, vRowStep = T::kThreads / T::kVPieces;
    static_assert(vRowStep % 16 == 0, "values: the same flips in all loads");
    static_assert(T::kKPieces == 32 ? kRowStep == 8 : kRowStep % 16 == 0, "keys");
    const uint32_t k_lane = 2 * (lane / T::kKPieces + 64 * wave / T::kKPieces % 8) * dim;

    const uint32_t row_w = wave * 32;  // the wave's first row
    const uint32_t live = it.rows();
    u32x4 q[KS];
    const uint32_t row = min(row_w + l32, live - 1), token = it.token + row / it.members;
    const uint32_t sees = min(it.c.ctx + token + 1, it.c.keys);  // keys that the row sees
    const uint16_t* from_q = a.q + (uint64_t)(it.c.first + token) * a.q_row +
                             (uint64_t)(it.head * a.group + it.member + row % it.members) * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uint32_t d = 16 * s + 8 * half;
      q[s] = (!PAD || d < dim) ? *reinterpret_cast<const u32x4*>(from_q + d) : u32x4{};
    }
    const uint32_t all_see = min(it.c.ctx + it.token + 1, it.c.keys);  // keys that every row sees
    floatx16 o[DT];
    float ref = -INFINITY, base = 0.f, l = 0.f;  // base: the reference, or 0 where there is none yet

    const int32_t* pages = a.table + (uint64_t)it.b * a.width;
    const uint8_t* keys = reinterpret_cast<const uint8_t*>(a.kc + it.head * page_len);
    const uint8_t* values = reinterpret_cast<const uint8_t*>(a.vc + it.head * page_len);
    // Table entries of the groups of 8 keys of kSpan tiles come into LDS, a copy a wave, kSpan
    // tiles ahead.  As the first of these tiles is loaded each lane turns an entry into addresses:
    // of the group's keys, which it keeps, and of its values, which go back into LDS.  What is
    // left to do in each tile is a few instructions: a wave gets one in about 5 cycles, and
    // addresses worked out in each tile (100 instructions) took as long as its weights.
    constexpr uint32_t kSpan = T::kSpan, kLoads = 2 * T::kEach;  // loads of a wave and tile
    uint32_t* entries = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(lds) + T::kTables + wave * T::kTable);
    uint64_t* places = reinterpret_cast<uint64_t*>(entries + 64);
    auto ask = [&](uint32_t n) {
      const uint32_t at = min(it.k0 + n * T::kKeys + 8 * lane, it.k1 - 1) >> a.log_block;
      load_word_to_lds(pages, 4 * at, lds0 + T::kTables + wave * T::kTable);
    };
    uint32_t keys_lo = 0, keys_hi = 0;  // where the keys of this lane's group are
    uint64_t gone = 0;                  // a bit for each group that does not exist; page 0 is read instead
    auto locate = [&](uint32_t n) {
      const uint32_t key = it.k0 + n * T::kKeys + 8 * lane;
      uint32_t id = entries[lane];
      keep_here(id);  // it is there before the next entries set out for its place
      const bool off = id >= a.blocks || key >= it.k1;
      gone = __ballot(off);
      const uint64_t page = (uint64_t)(off ? 0u : id) * page_bytes;
      const uint64_t k = (uint64_t)(uintptr_t)keys + page + (key & in_page) * (2 * dim);
      keys_lo = (uint32_t)k;
      keys_hi = (uint32_t)(k >> 32);
      places[lane] = (uint64_t)(uintptr_t)values + page + 2 * (key & in_page);
    };
    const uint32_t v_lane = (2 * v_row) << a.log_block, v_step = (2 * vRowStep) << a.log_block;
    // Before tile n's loads: bits of its groups that do not exist; `from`: of the lane's values.
    auto begin = [&](uint32_t n, uint64_t& from) {
      if (n % kSpan == 0) {
        locate(n);
        ask(n + kSpan);
      }
      const uint32_t in = n % kSpan * T::kGroups;
      from = places[in + v_piece];
      return (uint32_t)(gone >> in) & ((1u << T::kGroups) - 1);
    };
    // Sets a part of tile n on its way into its buffer: kEach parts of keys, kEach of values.  A
    // wave's keys of one part lie in one group.  (Every wave makes the same number of loads: waits
    // count them.)
    auto load_part = [&](uint32_t n, uint64_t from, uint32_t part) {
      const uint32_t j = part % T::kEach;
      const uint32_t to = lds0 + (n % T::kBuffers) * T::kPieces * 16 + wave * 1024 + T::kThreads * 16 * j;
      if (part < T::kEach) {
        const uint32_t at = n % kSpan * T::kGroups + (64 * wave / T::kKPieces + kRowStep * j) / 8;
        const uint8_t* k = reinterpret_cast<const uint8_t*>((uint64_t)__builtin_amdgcn_readlane(keys_hi, at) << 32 |
                                                            (uint32_t)__builtin_amdgcn_readlane(keys_lo, at));
        const uint32_t p = k_piece ^ (T::kKPieces == 32 ? 8 * (j & 1) : 0);
        if constexpr (PAD) load_to_lds(8 * p < dim ? k + k_lane + 16 * p : zeros, to);
        else load_to_lds(k, k_lane + 16 * p, to);
      } else {
        const uint8_t* v = reinterpret_cast<const uint8_t*>(from + v_lane + (uint64_t)v_step * j);
        load_to_lds(!PAD || v_row + vRowStep * j < dim ? v : zeros, to + T::kBuffers * T::kPieces * 16);
      }
    };
    auto load_keys = [&](uint32_t n) {
#pragma unroll
      for (uint32_t j = 0; j < T::kEach; ++j) load_part(n, 0, j);
    };
    auto load_values = [&](uint32_t n, uint64_t from) {
#pragma unroll
      for (uint32_t j = 0; j < T::kEach; ++j) load_part(n, from, T::kEach + j);
    };
    // Some row does not see all of tile n, or a page is missing.
    auto edge = [&](uint32_t n, uint32_t absent) { return it.k0 + (n + 1) * T::kKeys > all_see || absent; };
    // Such a tile, once it is there: values of keys that do not exist become zero, and so do those
    // that are not finite, for a weight of zero times them is not zero; they are added at the end.
    bool odd = false;
    uint32_t mended = ~0u;
    auto mend = [&](uint32_t n, uint32_t absent) {
      mended = min(mended, n);
#pragma unroll 1
      for (uint32_t j = 0; j < T::kEach; ++j) {
        if (PAD && v_row + vRowStep * j >= dim) continue;
        u32x4* at = s_v + (n % T::kBuffers) * T::kPieces + t + T::kThreads * j;
        u32x4 v = *at;
        const uint32_t key = it.k0 + n * T::kKeys + 8 * v_piece;
        const uint32_t real = (absent >> v_piece) & 1 || key >= it.k1 ? 0u : min(it.k1 - key, 8u);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          v[w] = real <= 2u * w ? 0u : real == 2u * w + 1 ? v[w] & 0xFFFFu : v[w];
          const uint32_t kept = (E::finite2(v[w] & 0xFFFFu) ? v[w] & 0xFFFFu : 0u) |
                                (E::finite2(v[w] & 0xFFFF0000u) ? v[w] & 0xFFFF0000u : 0u);
          odd |= kept != v[w];
          v[w] = kept;
        }
        *at = v;
      }
      lds_barrier();
    };

    // Two waves share a SIMD, whose matrix unit takes a product of 32 cycles while it issues four or
    // so other instructions, as long as they come from the same wave: products of the next tile's
    // keys and of this one's values alternate with this one's weights, a few instructions after
    // each product.  (Waves that took turns, one at its products and the other at its weights,
    // needed the sum of both: a product that waits for the unit keeps the other wave's
    // instructions back.)
    //
    // 3 prompts of 8190 tokens, 32 heads over 8 of 128, bf16: 795-855 us on several cards, 952-1024
    // TFLOP/s (in turns 861 where it is 820; the products alone 467).  The matrix units are busy for 46-49% of the cycles, at 1.8 to 2 GHz of 2.4:
    // the clock gives way to power (3 x 4096 tokens: 950 TFLOP/s, with zeros for keys and values 1125).
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = floatx16{};
    const uint32_t tiles = it.k0 < it.k1 ? (it.k1 - it.k0 + T::kKeys - 1) / T::kKeys : 0;
    if (tiles) {
      ask(0);
      loads_wait<0>();
      // Bits of the missing groups of a tile and of the next ones; where the next values are.  Keys
      // are a tile ahead of values with their loads as they are with their products.
      uint64_t from, from1 = 0, from2 = 0, from3 = 0;
      uint32_t absent = begin(0, from), absent1 = 0, absent2 = 0, absent3 = 0;
      load_keys(0);
      load_values(0, from);
      if (tiles > 1) {
        absent1 = begin(1, from1);
        load_keys(1);
      }
      if (tiles > 2) {
        absent2 = begin(2, from2);
        load_keys(2);
      }
      if (tiles > 1) load_values(1, from1);
      if (tiles > 3) {
        absent3 = begin(3, from3);
        load_keys(3);
      }
      if (tiles > 2) load_values(2, from2);
      // the first tile's and the second one's keys
      if (tiles > 3) loads_wait<4 * T::kEach>();
      else if (tiles > 2) loads_wait<3 * T::kEach>();
      else if (tiles > 1) loads_wait<T::kEach>();
      else loads_wait<0>();
      lds_barrier();
      if (edge(0, absent)) mend(0, absent);

      using Scores = floatx16[NH];
      u32x4 p[2 * NH];
      float top;
      // Steps of a tile: NA operands of keys, NB of values, read kAhead steps before the products
      // that take them, the next tile's first ones at the end of this one.  Pieces 2 x on from the
      // first lie at its place with 2 x flipped, whatever the row: one register addresses them all.
      // Row of the operand to key: bits 2 and 3 change places.
      constexpr int NA = NH * KS, NB = 2 * NH * DT, kAhead = 7;
      static_assert((NA + NB) % (kAhead + 1) == 0 && NB > kAhead, "the next tile's operands follow this one's");
      const uint32_t k_first = T::k_at((l32 & 19) | ((l32 & 4) << 1) | ((l32 & 8) >> 1), half);
      const uint32_t v_first = T::v_at(l32, half);
      u32x4 f[kAhead + 1];
      auto read = [&](uint32_t n, int step) {  // of the round of tile n: keys of the next, its own values
        if (step >= NA + NB) {
          step -= NA + NB;
          ++n;
        }
        if (step < NA) {
          const int h = step / KS, x = step % KS;
          f[step % (kAhead + 1)] = s_k[(((n + 1) % T::kBuffers * T::kPieces + k_first) ^ 2 * x) + 32 * h * T::kKPieces];
        } else {
          const int g = (step - NA) / DT, d = (step - NA) % DT;
          f[step % (kAhead + 1)] = s_v[((n % T::kBuffers * T::kPieces + v_first) ^ 2 * g) + 32 * d * T::kVPieces];
        }
      };
      // Weights of a tile come in pairs, in the order of the keys; those of 8 keys a lane have to be
      // there before their values' products.  kPairsA of them go beside the keys' products, the
      // rest beside the first kBy of the values', and the next tile's maximum beside the others.
      constexpr int kPairs = 8 * NH, kPairsA = (5 * kPairs + 4) / 8, kBy = (2 * NH - 1) * DT, kRefer = 2;
      constexpr auto pairs_after = [](int step) {
        return step < kRefer       ? 0
               : step < NA         ? (step - kRefer + 1) * kPairsA / (NA - kRefer)
               : step < NA + kBy   ? kPairsA + (step - NA + 1) * (kPairs - kPairsA) / kBy
                                   : kPairs;
      };
      // (the compiler would otherwise move them down to where they are used, away from the products)
      auto stay = [](float& v) { asm volatile("" : "+v"(v)); };
      auto weigh = [&](Scores& s, int pair) {
#pragma unroll
        for (int e = 2 * pair; e < 2 * pair + 2; ++e) {
          float w = __builtin_amdgcn_exp2f(fmaf(s[e >> 4][e & 15], a.scale, -base));
          stay(w);
          s[e >> 4][e & 15] = w;
        }
      };
      auto pack = [&](Scores& s, int pair) {
        const int e = 2 * pair;
        p[pair / 4][pair % 4] = E::pack2(s[e >> 4][e & 15], s[e >> 4][(e & 15) + 1]);
        l = E::add2(p[pair / 4][pair % 4], l);
        stay(l);
      };
      auto mask = [&](Scores& s, uint32_t n, uint32_t absent) {
        // a lane's scores: keys kb + 16 g + 8 half + e are element 8 (g & 1) + e of s[g / 2]
        const uint32_t kb = it.k0 + n * T::kKeys;
        if (kb + T::kKeys <= all_see && !absent) return;
#pragma unroll
        for (int g = 0; g < 2 * NH; ++g) {
          const uint32_t key = kb + 16 * g + 8 * half;
          const uint32_t seen = (absent >> (2 * g + half)) & 1 || key >= sees ? 0u : min(sees - key, 8u);
#pragma unroll
          for (uint32_t e = 0; e < 8; ++e)
            if (e >= seen) s[g >> 1][8 * (g & 1) + e] = -INFINITY;
        }
      };
      auto maximum = [&](Scores& s, int from, int to) {
        if (from == 0) top = s[0][0];
#pragma unroll
        for (int e = from; e < to; e += 2)
          top = fmaxf(fmaxf(top, s[e >> 4][e & 15]), s[e >> 4][(e & 15) + 1]);
        stay(top);
      };
      // (whether some score is far above its row's reference needs no maximum over the row's lanes)
      auto refer = [&] {
        top *= a.scale;
        if (!__any(top > ref + kSlack)) return;
        const float now = fmaxf(ref, over_row(top, [](float x, float y) { return fmaxf(x, y); }));
        const float keep = ref == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ref - now);
        ref = now;
        base = now == -INFINITY ? 0.f : now;  // nothing seen: the weights are 2^-inf = 0
        l *= keep;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= keep;
      };
      // Tile n: its scores are in `s`, and their maximum is known.  kNext: there is a next one, whose
      // scores go to `t`; kFull: there are at least four.  In the midst of the values' products
      // all waves are through with the keys of tile n + 1 and with tile n - 1, and the keys of tile
      // n + 2 and the values of tile n + 1 have arrived; the keys of tile n + 4 and the values of
      // tile n + 3 set out.
      constexpr int kMid = NA + NB - kAhead - 1, kEvery = (NA + NB - kMid) / kLoads;
      static_assert(kEvery >= 1, "a load in a step");
      auto round = [&](uint32_t n, Scores& s, Scores& t, auto next, auto full) {
        constexpr bool kNext = decltype(next)::value, kFull = decltype(full)::value;
        if constexpr (!kNext) {
          refer();
          steps<NA, NA + kAhead>([&](auto step) { read(n, step); });
          steps<0, kPairs>([&](auto pair) { weigh(s, pair); });
          steps<0, kPairs>([&](auto pair) { pack(s, pair); });
        }
        __builtin_amdgcn_sched_barrier(0);
        steps<kNext ? 0 : NA, NA + NB>([&](auto at) {
          constexpr int step = decltype(at)::value;
          if constexpr (kNext && step == kMid) {
            if (kFull || n + 3 < tiles) loads_wait<2 * T::kEach>();
            else if (n + 2 < tiles) loads_wait<T::kEach>();
            else loads_wait<0>();
            lds_barrier();
            if (edge(n + 1, absent1)) mend(n + 1, absent1);
            from = from3;
            if (kFull || n + 4 < tiles) absent = begin(n + 4, from3);
          }
          if constexpr (kNext || step + kAhead < NA + NB) read(n, step + kAhead);
          if constexpr (kNext) {
            if constexpr (step == kRefer) refer();
            steps<pairs_after(step - 2), pairs_after(step - 1)>([&](auto pair) { pack(s, pair); });
            if constexpr (step == NA + kBy) mask(t, n + 1, absent1);
          }
          if constexpr (step < NA) {
            constexpr int h = step / KS, x = step % KS;
            t[h] = mfma32<E>(f[step % (kAhead + 1)], q[x], x ? t[h] : floatx16{});
          } else {
            constexpr int g = (step - NA) / DT, d = (step - NA) % DT;
            static_assert(!kNext || pairs_after(step - 1) >= 4 * (g + 1), "weights before their products");
            o[d] = mfma32<E>(f[step % (kAhead + 1)], p[g], o[d]);
          }
          if constexpr (kNext) {
            steps<pairs_after(step - 1), pairs_after(step)>([&](auto pair) { weigh(s, pair); });
            constexpr int in = step - NA - kBy, kEach = 16 * NH / (NB - kBy);
            if constexpr (in >= 0) maximum(t, in * kEach, (in + 1) * kEach);
            constexpr int part = (step - kMid) / kEvery;
            if constexpr (step >= kMid && (step - kMid) % kEvery == 0 && part < (int)kLoads) {
              if constexpr (part < (int)T::kEach) {
                if (kFull || n + 4 < tiles) load_part(n + 4, 0, part);
              } else {
                if (kFull || n + 3 < tiles) load_part(n + 3, from, part);
              }
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        const uint32_t last = absent;  // of tile n + 4
        absent = absent1;
        absent1 = absent2;
        absent2 = absent3;
        absent3 = last;
      };
      Scores s, t;
      steps<0, NA>([&](auto step) {
        constexpr int h = step / KS, x = step % KS;
        read(~0u, step);
        s[h] = mfma32<E>(f[step % (kAhead + 1)], q[x], x ? s[h] : floatx16{});
      });
      mask(s, 0, absent);
      maximum(s, 0, 16 * NH);
      if (tiles > 1) steps<0, kAhead>([&](auto step) { read(0, step); });
      uint32_t n = 0;
      for (; n + 5 < tiles; n += 2) {
        round(n, s, t, std::true_type{}, std::true_type{});
        round(n + 1, t, s, std::true_type{}, std::true_type{});
      }
      for (; n + 1 < tiles; ++n) {
        round(n, s, t, std::true_type{}, std::false_type{});
#pragma unroll
        for (int h = 0; h < NH; ++h) s[h] = t[h];
      }
      round(n, s, t, std::false_type{}, std::false_type{});
    }

    const bool whole = it.keys <= piece;
    uint32_t t_end = threadIdx.x;
    keep_here(t_end);
    const uint32_t row32 = t_end & 31, dim4 = 4 * (t_end >> 5 & 1);
    if (__syncthreads_or(odd)) {
      // values that are not finite and were left out: whatever the weight of a key that a row sees
      for (uint32_t key = it.k0 + mended * T::kKeys; key < it.k1; ++key) {
        const uint32_t page = pages[key >> a.log_block];
        if (page >= a.blocks) continue;
        const uint8_t* from = values + (uint64_t)page * page_bytes + 2 * (key & in_page);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (uint32_t e = 0; e < 16; ++e) {
            const uint32_t at = 32 * d + 8 * (e >> 2) + dim4 + (e & 3);
            if (PAD && at >= dim) continue;
            const uint32_t v = *reinterpret_cast<const uint16_t*>(from + ((uint64_t)(2 * at) << a.log_block));
            if (E::finite2(v)) continue;
            if (key < sees) o[d][e] += E::up((uint16_t)v);
          }
      }
    }
    l = over_row(l, [](float x, float y) { return x + y; });
    const uint32_t r = row_w + row32;
    if (r < live && whole) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const uint32_t tok = it.token + r / it.members;
      uint16_t* p = a.out + (uint64_t)(it.c.first + tok) * a.out_row +
                    (uint64_t)(it.head * a.group + it.member + r % it.members) * a.out_head;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t at = 32 * d + 8 * g + dim4;
          if (!PAD || at < dim) {
            *reinterpret_cast<uint32_t*>(p + at) = E::pack2(o[d][4 * g] * inv, o[d][4 * g + 1] * inv);
            *reinterpret_cast<uint32_t*>(p + at + 2) = E::pack2(o[d][4 * g + 2] * inv, o[d][4 * g + 3] * inv);
          }
        }
    } else if (r < live) {
      float* part = a.parts + (uint64_t)it.part * P::kFloats;
      if (dim4 == 0) {
        part[r] = ref;
        part[P::kRows + r] = l;
      }
      float* to = part + 2 * P::kRows + r * DP;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<floatx4*>(to + 32 * d + 8 * g + dim4) =
              floatx4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
    }
    __syncthreads();  // the buffers are refilled
  }
}

// Adds up the parts of tiles that were cut, in the order of the keys: a workgroup takes some
// rows of a tile, a thread four outputs of a row in all parts, eight of which are asked for at a
// time.  Where the call's longest tile has more than kWhole, a workgroup takes a quarter as many rows,
// a thread a quarter of the parts, and the quarters meet in LDS.  (In quarters and without, by the
// longest tile's parts: 2 parts 46 and 16 us, 10 8.5 and 6.2, 14 to 16 9.2 and 7.6, 18 9.4 and 8.9, 21
// 5.9 and 6.8, 23 9.0 and 9.1, 28 8.4 and 9.9, 126 7.4 and 22.)
struct Joined {
  float m = -INFINITY, l = 0.f;
  floatx4 o = {};
  __device__ __forceinline__ void add(float om, float ol, floatx4 oo) {
    const float now = fmaxf(m, om), base = now == -INFINITY ? 0.f : now;
    const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(om - base);
    m = now;
    l = fmaf(ol, g, l * f);
    o = o * f + oo * g;
  }
};

template <class E, int DP, int WAVES>
__global__ __launch_bounds__(256) void k_chunk_join(ChunkArgs a) {
  using P = PartOf<DP, WAVES>;
  constexpr uint32_t kFours = DP / 4, kQuarters = 4, kAtOnce = 8, kWhole = 20;
  __shared__ floatx4 s_o[256];
  __shared__ float s_m[256], s_l[256];
  const uint32_t piece = a.plan[Plan::kPiece], cut = a.plan[Plan::kCut], t = threadIdx.x;
  const uint32_t quarters = a.plan[Plan::kMost] > kWhole ? kQuarters : 1;
  const uint32_t rows = 256 / kFours / quarters, steps = P::kRows / rows;  // of a workgroup, of a tile
  const uint32_t d = 4 * (t % kFours), row = t / kFours % rows, quarter = t / kFours / rows;
  for (uint64_t unit = blockIdx.x; unit < (uint64_t)cut * steps; unit += gridDim.x) {
    const Item it = item_of<Plan::kTile>(a, (uint32_t)(unit / steps), piece, P::kRows);
    const uint32_t r = (uint32_t)(unit % steps) * rows + row;
    // (a tile that sees fewer keys is one piece)
    if (it.keys <= piece || r - row >= it.rows()) continue;
    // item numbers of a tile's pieces lie `heads` apart
    const uint32_t count = (it.keys + piece - 1) / piece, each = (count + quarters - 1) / quarters;
    const uint32_t first = min(quarter * each, count), last = min(first + each, count);
    const float* part = a.parts + (uint64_t)it.part * P::kFloats;
    const uint64_t step = (uint64_t)a.heads * P::kFloats;
    Joined sum;
    for (uint32_t k0 = first; k0 < last; k0 += kAtOnce) {
      float m[kAtOnce], l[kAtOnce];
      floatx4 o[kAtOnce];
#pragma unroll
      for (uint32_t k = 0; k < kAtOnce; ++k) {
        const float* from = part + min(k0 + k, last - 1) * step;
        m[k] = from[r];
        l[k] = from[P::kRows + r];
        o[k] = *reinterpret_cast<const floatx4*>(from + 2 * P::kRows + r * DP + d);
      }
#pragma unroll
      for (uint32_t k = 0; k < kAtOnce; ++k)
        if (k0 + k < last) sum.add(m[k], l[k], o[k]);
    }
    if (quarters > 1) {
      s_m[t] = sum.m;
      s_l[t] = sum.l;
      s_o[t] = sum.o;
      __syncthreads();
    }
    if (quarter == 0 && r < it.rows() && d < a.dim) {
      if (quarters > 1)
        for (uint32_t x = t + 256 / kQuarters; x < 256; x += 256 / kQuarters) sum.add(s_m[x], s_l[x], s_o[x]);
      const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
      const uint32_t tok = it.token + r / it.members;
      uint16_t* p = a.out + (uint64_t)(it.c.first + tok) * a.out_row +
                    (uint64_t)(it.head * a.group + it.member + r % it.members) * a.out_head + d;
      *reinterpret_cast<uint32_t*>(p) = E::pack2(sum.o[0] * inv, sum.o[1] * inv);
      *reinterpret_cast<uint32_t*>(p + 2) = E::pack2(sum.o[2] * inv, sum.o[3] * inv);
    }
    if (quarters > 1) __syncthreads();  // the LDS is free again
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
  p.ws_bytes = p.part_off + (size_t)kPartRows * (p.dp + 2) * 4;
  return p;
}

bool chunk_shape_ok(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim, uint32_t requests) {
  return heads >= 1 && kv_heads >= 1 && heads % kv_heads == 0 && heads <= 65536 && dim >= 8 &&
         dim <= 256 && dim % 8 == 0 && requests <= kMaxRequests && tokens <= (1u << 20) &&
         (uint64_t)tokens * heads <= (1u << 30);
}

template <class E, int DP, int WAVES, bool PAD>
int launch_chunk(const ChunkArgs& a, hipStream_t st) {
  using T = Tile<DP, WAVES>;
  const auto kernel = k_chunk_attention<E, DP, WAVES, PAD>;
  if (T::kBytes > 64 * 1024 &&
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                          (int)T::kBytes) != hipSuccess)
    return DGT_E_HIP;
  hipLaunchKernelGGL(kernel, dim3(kCUs), dim3(64 * WAVES), T::kBytes, st, a);
  if (int rc = launched()) return rc;
  hipLaunchKernelGGL((k_chunk_join<E, DP, WAVES>), dim3(8 * kCUs), dim3(256), 0, st, a);
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
    case 64: return pad ? launch_chunk<E, 64, 8, true>(a, st) : launch_chunk<E, 64, 8, false>(a, st);
    case 128: return pad ? launch_chunk<E, 128, 8, true>(a, st) : launch_chunk<E, 128, 8, false>(a, st);
  }
  return pad ? launch_chunk<E, 256, 4, true>(a, st) : launch_chunk<E, 256, 4, false>(a, st);
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
  a.rows = p.rows;
  a.tile_tokens = p.tile_tokens;
  a.splits = p.splits;
  a.scale = scale * 1.4426950408889634f;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return type == DGT_ELT_BF16 ? launch_chunk<Bf16>(a, p.dp, st) : launch_chunk<F16>(a, p.dp, st);
}

}  // extern "C"
