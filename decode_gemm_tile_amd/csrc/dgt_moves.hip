// Pages after a step: what is kept of the drafts moves up and the rest goes back, requests
// that share pages, requests that end.
#include "dgt_serve.h"

#include <algorithm>

namespace dgt {
namespace serve {
namespace {

struct Pool {  // caches of all layers, in 16-bit elements
  uint16_t *kc, *vc;
  uint32_t layers, heads, dim, log_block, blocks;
  __device__ __forceinline__ uint64_t page(uint32_t layer, uint32_t id, uint32_t head) const {
    return ((((uint64_t)layer * blocks + id) * heads + head) * dim) << log_block;
  }
  __device__ __forceinline__ uint32_t block() const { return 1u << log_block; }
  __device__ __forceinline__ bool holds(uint32_t slot) const { return slot < blocks << log_block; }
};

// Exclusive sum over a workgroup's threads, in their order; s_sum holds one word a wave.
template <int THREADS>
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* s_sum, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t scan = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(scan, d, 64);
    if (lane >= (uint32_t)d) scan += o;
  }
  if (lane == 63) s_sum[wave] = scan;
  __syncthreads();
  uint32_t before = scan - v, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += s_sum[w];
    all += s_sum[w];
  }
  __syncthreads();  // s_sum is free again
  *total = all;
  return before;
}

// ----------------------------------------------------------------------- keep
// One launch: a workgroup for lengths and pages, the others move rows.  A workgroup goes through
// the chain of latencies (offsets, path, slots, rows) once for several layers and heads, so that
// all of them are on the card at a time.
// 128 trees of up to 61 in 4 layers of 8 heads of 128: 15-18 us, with a workgroup a layer and head 36.
// A token's values are 2 bytes of a row of each value page, so what moves is not the 21 MB of the
// elements (4.4 us) but their lines: 18 MB read and 24 written, 9 us at a copy's rate.  The rest is
// the chain, as in 4 requests in one layer: 4.6.
struct KeepArgs {
  const int32_t *path, *kept, *ctx, *cu, *slots, *free_head;
  int32_t *free_list, *table, *lens, *counts;
  uint32_t requests, tokens, free_len, width;
  uint32_t parts, each;  // workgroups a request, and the layers' heads that one takes
  Pool pool;
};

constexpr uint32_t kKeepRows = 16;  // tokens that a workgroup moves at a time

// How many rows a request keeps; the first new token of one that the plan refused has no
// slot.  (The loads do not wait for each other.)
__device__ __forceinline__ uint32_t kept_of(const KeepArgs& a, uint32_t b, uint32_t first, uint32_t count, bool* held) {
  const int32_t kept = a.kept[b];
  const uint32_t slot = count ? (uint32_t)a.slots[first] : ~0u;
  *held = a.pool.holds(slot);
  return *held ? min((uint32_t)max(kept, 0), count) : 0u;
}

// The kept rows that stay, of a request a thread (kept: how many at most, its rows are `count`
// from `first` on).  Row j of a path stays if its own place has a slot, and so has the row that
// moves there: a token that the plan gave no slot was never stored.  Of the first it and all
// behind it go.  16 lanes look at the first 16 rows of a request side by side; what longer ones
// have besides goes round the waves.
struct Kept {
  uint32_t first, count, rows;
};
__device__ __forceinline__ uint32_t rows_that_stay(const KeepArgs& a, uint32_t first, uint32_t count, uint32_t kept,
                                                   uint32_t left, Kept* s_kept) {
  const uint32_t t = threadIdx.x, lane = t & 63, n = t % 16;
  // Four rows a thread at a time, their loads beside one another (row 0's where there is none).
  auto look = [&](const Kept (&it)[4], const uint32_t (&j)[4], bool (&gone)[4]) {
    uint32_t place[4], from[4], slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = j[i] < it[i].rows ? it[i].first + j[i] : 0;
      place[i] = (uint32_t)a.slots[at];
      from[i] = a.path ? (uint32_t)a.path[at] : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool moves = j[i] < it[i].rows && from[i] > j[i] && from[i] < it[i].count;
      slot[i] = (uint32_t)a.slots[moves ? it[i].first + from[i] : 0];
      if (!moves) slot[i] = place[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) gone[i] = j[i] < it[i].rows && !(a.pool.holds(place[i]) && a.pool.holds(slot[i]));
  };
  s_kept[t] = Kept{first, count, kept};
  __syncthreads();
  for (uint32_t x0 = t / 16; x0 - t / 16 < min(left, 256u); x0 += 64) {
    Kept it[4];
    uint32_t j[4];
    bool gone[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      it[i] = s_kept[x0 + 16 * i];
      j[i] = n;
    }
    look(it, j, gone);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t all = __ballot(gone[i]) >> (lane & 48) & 0xFFFFu;
      if (n == 0 && all) s_kept[x0 + 16 * i].rows = (uint32_t)__builtin_ctzll(all);
    }
  }
  __syncthreads();
  if (__syncthreads_or(s_kept[t].rows > 16)) {
    const uint32_t wave = t >> 6;
    for (uint64_t todo = __ballot(s_kept[4 * lane + wave].rows > 16); todo; todo &= todo - 1) {
      const uint32_t x = 4 * (uint32_t)__builtin_ctzll(todo) + wave;
      const Kept one = s_kept[x];
      uint32_t least = one.rows;
      for (uint32_t j0 = 16; j0 < least; j0 += 256) {
        Kept it[4];
        uint32_t j[4];
        bool gone[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          it[i] = one;
          j[i] = j0 + 64 * i + lane;
        }
        look(it, j, gone);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (gone[i]) least = min(least, j[i]);
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) least = min(least, (uint32_t)__shfl_xor((int)least, m, 64));
      }
      if (lane == 0) s_kept[x].rows = least;
    }
    __syncthreads();
  }
  return s_kept[t].rows;  // (the next round's write is of the same thread)
}

// Some row of the step has no slot: only then may a path have to be cut, so a step without one (the
// rule) pays for one look at its slots, 16 bytes a thread.  (8 prompts of 8000 tokens: 10 us with it, 43
// with rows_that_stay; 1000 requests of 8: 10.5 and 34.)
__device__ __forceinline__ bool slots_missing(const KeepArgs& a) {
  const uint32_t t = threadIdx.x;
  const uint32_t own = t < a.tokens ? (uint32_t)a.slots[t] : 0;
  const uint32_t end = a.requests ? (uint32_t)min(max(a.cu[a.requests], 0), (int)a.tokens) : 0;
  bool missing = t < end && !a.pool.holds(own);
  uint32_t from = 256;
  if (reinterpret_cast<uintptr_t>(a.slots) % 16 == 0) {
    for (; from + 4 <= end; from += 4 * 256 * 8) {
      u32x4 v[8];
#pragma unroll
      for (uint32_t n = 0; n < 8; ++n) {
        const uint32_t i = from + 4 * (256 * n + t);
        v[n] = reinterpret_cast<const u32x4*>(a.slots)[i + 4 <= end ? i / 4 : 0];
      }
#pragma unroll
      for (uint32_t n = 0; n < 8; ++n)
        if (from + 4 * (256 * n + t) + 4 <= end)
#pragma unroll
          for (int e = 0; e < 4; ++e) missing |= !a.pool.holds(v[n][e]);
    }
    from = end > 256 ? end / 4 * 4 : 256;  // the last few
  }
  for (uint32_t i = from + t; i < end; i += 256) missing |= !a.pool.holds((uint32_t)a.slots[i]);
  return __syncthreads_or(missing);
}

// Lengths, and the pages past them, by one workgroup: the list's order is the requests'.
// A column past the kept tokens begins at or behind the cached ones' end, so a new token
// lies first in it and its slot names the page.  One that the plan gave no slot (a bad link,
// an index past the mask) has taken its page all the same: then the table names it.
__device__ __forceinline__ void keep_pages(const KeepArgs& a, uint32_t* s_sum, Kept* s_kept) {
  const uint32_t log = a.pool.log_block, round = a.pool.block() - 1;
  const uint32_t head = min((uint32_t)max(*a.free_head, 0), a.free_len);
  uint32_t total = 0;
  // rounds of 256 requests in which a path may be cut
  uint32_t cuts = slots_missing(a) ? ~0u : 0u;
  static_assert(kMaxRequests <= 32 * 256, "a bit a round");
  // where 256 threads do not hold all requests, twice over them: how many pages, then which
  for (int pass = a.requests <= 256; pass < 2; ++pass) {
    uint32_t done = 0;
    for (uint32_t b0 = 0; b0 < a.requests; b0 += 256) {
      const uint32_t b = b0 + threadIdx.x;
      uint32_t first = 0, count = 0, ctx = 0, kept = 0, now = 0, from = 0, to = 0;
      bool held = false;
      if (b < a.requests) {
        request_rows(a.cu, b, a.tokens, &first, &count);
        ctx = (uint32_t)max(a.ctx[b], 0);
        kept = kept_of(a, b, first, count, &held);
      }
      if (cuts >> b0 / 256 & 1) {
        const uint32_t most = kept;
        kept = rows_that_stay(a, first, count, kept, a.requests - b0, s_kept);
        if (pass == 0 && !__syncthreads_or(kept < most)) cuts &= ~(1u << b0 / 256);
      }
      if (b < a.requests) {
        now = (uint32_t)min((uint64_t)ctx + kept, (uint64_t)0x7FFFFFFF);
        from = min((uint32_t)(((uint64_t)now + round) >> log), a.width);
        to = held ? min((uint32_t)(((uint64_t)ctx + count + round) >> log), a.width) : from;
      }
      auto page = [&](uint32_t c) {  // of column c
        const uint32_t at = max(c << log, ctx) - ctx;
        if (at >= count) return ~0u;
        const uint32_t slot = (uint32_t)a.slots[first + at];
        const uint32_t id = a.pool.holds(slot) ? slot >> log : (uint32_t)a.table[(uint64_t)b * a.width + c];
        return id < a.pool.blocks ? id : ~0u;
      };
      uint32_t mine = 0;
      for (uint32_t c = from; c < to; ++c) mine += page(c) != ~0u;
      uint32_t all;
      uint32_t at = done + sum_before<256>(mine, s_sum, &all);
      done += all;
      if (pass == 0) continue;
      if (a.requests <= 256) total = all;
      for (uint32_t c = from; c < to; ++c) {
        const uint32_t id = page(c);
        if (id == ~0u) continue;
        // (there is room for all of them unless the list is not what they came from)
        if (head + at >= total) a.free_list[head + at - total] = (int32_t)id;
        a.table[(uint64_t)b * a.width + c] = -1;
        ++at;
      }
      if (b < a.requests) a.lens[b] = (int32_t)now;
    }
    total = done;
  }
  if (threadIdx.x == 0) {
    a.counts[0] = (int32_t)(head - min(total, head));
    a.counts[1] = (int32_t)total;
  }
}

// A workgroup moves the kept rows of one request in some heads of the layers, 16 at a
// time: all of them are read before any is written.  Index i_j >= j rises with j, so a
// row that a later step reads lies behind every place that this one writes.  Slots are
// looked up in the plan's list and not in the table, whose columns change at the same time,
// 64 rows at a time; of them wave 0 leaves the slots and a bit for each 16 that something of
// moves (kEnds: a row does not stay), in one of two sets of LDS in turn.
constexpr uint32_t kLook = 64, kEnds = 1u << 4;
struct Moves {
  uint32_t src[kLook], dst[kLook], what;
};
__device__ __forceinline__ void keep_rows(const KeepArgs& a, uint32_t unit, Moves* s_moves) {
  const uint32_t t = threadIdx.x, dim = a.pool.dim, log = a.pool.log_block, in_page = a.pool.block() - 1;
  const uint32_t b = unit / a.parts, part = unit - b * a.parts;
  const uint32_t lh0 = part * a.each, lh1 = min(lh0 + a.each, a.pool.layers * a.pool.heads);
  uint32_t first, count;
  request_rows(a.cu, b, a.tokens, &first, &count);
  int32_t ahead = t < min(count, kLook) ? a.path[first + t] : 0;
  bool held;
  const uint32_t kept = kept_of(a, b, first, count, &held);
  uint32_t what = 0;
  for (uint32_t j0 = 0; j0 < kept && !(what & kEnds); j0 += kLook) {
    Moves& s = s_moves[j0 / kLook % 2];
    if (t < kLook) {
      const uint32_t j = j0 + t;
      uint32_t src = ~0u, dst = ~0u;
      bool moves = false, stays = true;
      if (j < kept) {
        const uint32_t i = (uint32_t)(j0 ? a.path[first + j] : ahead);
        moves = i > j && i < count;
        dst = (uint32_t)a.slots[first + j];
        if (moves) src = (uint32_t)a.slots[first + i];
        stays = a.pool.holds(dst) && (!moves || a.pool.holds(src));
      }
      const uint64_t gone = __ballot(!stays);
      moves = moves && !(gone & ((2ull << t) - 1));  // neither the row nor one before it is gone
      const uint64_t all = __ballot(moves);
      s.src[t] = moves ? src : ~0u;
      s.dst[t] = dst;
      if (t == 0) {
        uint32_t bits = gone ? kEnds : 0;
#pragma unroll
        for (uint32_t g = 0; g < kLook / kKeepRows; ++g) bits |= (all >> (kKeepRows * g) & 0xFFFFu) ? 1u << g : 0u;
        s.what = bits;
      }
    }
    __syncthreads();
    what = __builtin_amdgcn_readfirstlane(s.what);
    for (uint32_t g = 0; g < kLook / kKeepRows; ++g) {
      if (!(what >> g & 1)) continue;
      const uint32_t *s_src = s.src + kKeepRows * g, *s_dst = s.dst + kKeepRows * g;
      const uint32_t vr = t % kKeepRows, v_src = s_src[vr], v_dst = v_src != ~0u ? s_dst[vr] : 0;
      for (uint32_t lh = lh0; lh < lh1; ++lh) {
        const uint32_t layer = lh / a.pool.heads, head = lh - layer * a.pool.heads;
        // value elements, a value row's side by side; 16-byte pieces of key rows, a row's side by side
        const uint16_t* vs = a.pool.vc + a.pool.page(layer, v_src != ~0u ? v_src >> log : 0, head) + (v_src & in_page);
        uint16_t* vd = a.pool.vc + a.pool.page(layer, v_dst >> log, head) + (v_dst & in_page);
        for (uint32_t d0 = 0; d0 < dim; d0 += 128) {
          const uint32_t dims = min(dim - d0, 128u);
          u32x4 k;
          uint16_t v[8];
          const uint32_t r = t / (dims / 8), d = d0 + 8 * (t % (dims / 8));
          const bool k_on = r < kKeepRows && s_src[r] != ~0u;
          if (k_on)
            k = *reinterpret_cast<const u32x4*>(a.pool.kc + a.pool.page(layer, s_src[r] >> log, head) + (s_src[r] & in_page) * dim + d);
#pragma unroll
          for (uint32_t n = 0; n < 8; ++n) {
            const uint32_t e = d0 + t / kKeepRows + 16 * n;
            if (v_src != ~0u && e < d0 + dims) v[n] = vs[(uint64_t)e << log];
          }
          __syncthreads();
          if (k_on)
            *reinterpret_cast<u32x4*>(a.pool.kc + a.pool.page(layer, s_dst[r] >> log, head) + (s_dst[r] & in_page) * dim + d) = k;
#pragma unroll
          for (uint32_t n = 0; n < 8; ++n) {
            const uint32_t e = d0 + t / kKeepRows + 16 * n;
            if (v_src != ~0u && e < d0 + dims) vd[(uint64_t)e << log] = v[n];
          }
        }
      }
      __syncthreads();  // what was written is behind what the next step reads
    }
  }
}

// (eight workgroups a CU, 64 registers: with 123 registers and four of them the trees take 20.6 us)
__global__ __launch_bounds__(256, 8) void k_page_keep(KeepArgs a) {
  __shared__ uint32_t s_sum[4];
  __shared__ Kept s_kept[256];
  __shared__ Moves s_moves[2];
  if (blockIdx.x == 0) keep_pages(a, s_sum, s_kept);
  else keep_rows(a, blockIdx.x - 1, s_moves);
}

// ----------------------------------------------------------------------- fork
// The copies bound it: 192 forks of up to 63 tokens in 4 layers of 8 heads of 128, 204 MB read and
// written: 64-71 us, 3 TB/s.
struct ForkArgs {
  const int32_t *src, *dst, *free_list, *free_head;
  int32_t *lens, *table, *shares, *counts;
  uint32_t forks, requests, width, free_len, parts;
  Pool pool;
};

// Every workgroup goes through the list of forks for itself (one is a few loads): s_first
// gets the first fork of each row, s_rank how many pages the forks before need, or ~0 for
// a refused one.  Returns the pages taken in all.
__device__ __forceinline__ uint32_t plan_forks(const ForkArgs& a, uint32_t* s_first, uint32_t* s_rank, uint32_t* s_sum) {
  const uint32_t t = threadIdx.x, in_page = a.pool.block() - 1;
  for (uint32_t i = t; i < a.requests; i += 256) s_first[i] = ~0u;
  __syncthreads();
  for (uint32_t i = t; i < a.forks; i += 256) {
    const uint32_t dst = (uint32_t)a.dst[i];
    if (dst < a.requests) atomicMin(&s_first[dst], i);  // the least of them, in any order
  }
  __syncthreads();
  const uint32_t head = min((uint32_t)max(*a.free_head, 0), a.free_len), left = a.free_len - head;
  uint32_t taken = 0;
  for (uint32_t i0 = 0; i0 < a.forks; i0 += 256) {
    const uint32_t i = i0 + t;
    bool sound = false, need = false;
    if (i < a.forks) {
      const uint32_t src = (uint32_t)a.src[i], dst = (uint32_t)a.dst[i];
      if (src < a.requests && dst < a.requests && s_first[dst] == i) {
        const int32_t len = a.lens[src];
        sound = len > 0 && a.lens[dst] <= 0 && ((uint64_t)len + in_page) >> a.pool.log_block <= a.width;
        need = sound && (len & in_page);
      }
    }
    uint32_t all;
    const uint32_t rank = taken + sum_before<256>(need, s_sum, &all);
    taken += all;
    if (i < a.forks) s_rank[i] = sound && (!need || rank < left) ? rank : ~0u;
  }
  __syncthreads();
  return min(taken, left);
}

// Part 0 of a fork writes the row of the table and counts the shares; every part copies its
// share of the last page's pieces in all layers and heads: key rows up to the length,
// values in pieces of 8 tokens.
__global__ __launch_bounds__(256) void k_page_fork(ForkArgs a) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t s_sum[4];
  uint32_t *s_first = lds, *s_rank = lds + a.requests;
  plan_forks(a, s_first, s_rank, s_sum);
  const uint32_t t = threadIdx.x, log = a.pool.log_block, dim = a.pool.dim;
  const uint32_t head = min((uint32_t)max(*a.free_head, 0), a.free_len);
  for (uint32_t unit = blockIdx.x; unit < a.forks * a.parts; unit += gridDim.x) {
    const uint32_t i = unit / a.parts, part = unit % a.parts, rank = s_rank[i];
    if (rank == ~0u) continue;
    const uint32_t src = (uint32_t)a.src[i], dst = (uint32_t)a.dst[i], len = (uint32_t)a.lens[src];
    const uint32_t full = len >> log, rest = len & (a.pool.block() - 1);
    const int32_t* from = a.table + (uint64_t)src * a.width;
    const uint32_t fresh = rest ? (uint32_t)a.free_list[head + rank] : ~0u;
    if (part == 0) {
      int32_t* to = a.table + (uint64_t)dst * a.width;
      for (uint32_t c = t; c < full; c += 256) {
        const uint32_t id = (uint32_t)from[c];
        to[c] = (int32_t)id;
        if (id < a.pool.blocks) atomicAdd(a.shares + id, 1);
      }
      if (t == 0 && rest) to[full] = (int32_t)fresh;
    }
    if (!rest) continue;
    const uint32_t old = (uint32_t)from[full];
    if (old >= a.pool.blocks || fresh >= a.pool.blocks || old == fresh) continue;
    const uint32_t k_pieces = rest * dim / 8, v_row = (rest + 7) / 8, each = k_pieces + v_row * dim;
    const uint32_t in_row = a.pool.block() / 8, heads = a.pool.layers * a.pool.heads;
    const float inv_row = 1.f / (float)v_row;
    for (uint32_t lh = part; lh < heads; lh += a.parts) {
      const uint64_t x = a.pool.page(lh / a.pool.heads, old, lh % a.pool.heads);
      const uint64_t y = a.pool.page(lh / a.pool.heads, fresh, lh % a.pool.heads);
      const u32x4 *kx = reinterpret_cast<const u32x4*>(a.pool.kc + x), *vx = reinterpret_cast<const u32x4*>(a.pool.vc + x);
      u32x4 *ky = reinterpret_cast<u32x4*>(a.pool.kc + y), *vy = reinterpret_cast<u32x4*>(a.pool.vc + y);
      for (uint32_t p0 = t; p0 < each; p0 += 256 * 4) {
        u32x4 v[4], was[4];
        uint32_t at[4], tokens[4];
#pragma unroll
        for (uint32_t n = 0; n < 4; ++n) {
          const uint32_t p = p0 + 256 * n;
          at[n] = p;
          tokens[n] = 8;
          if (p < k_pieces) {
            v[n] = kx[p];
          } else if (p < each) {
            // (exact: the quotients are below 2^17, a half off every border)
            const uint32_t row = (uint32_t)(((float)(p - k_pieces) + 0.5f) * inv_row), in = p - k_pieces - row * v_row;
            at[n] = row * in_row + in;
            tokens[n] = rest - 8 * in;
            v[n] = vx[at[n]];
            if (tokens[n] < 8) was[n] = vy[at[n]];
          }
        }
#pragma unroll
        for (uint32_t n = 0; n < 4; ++n) {
          const uint32_t p = p0 + 256 * n;
          if (p < k_pieces) {
            ky[p] = v[n];
          } else if (p < each) {
            // cells past the length stay as they are
#pragma unroll
            for (uint32_t w = 0; w < 4; ++w)
              if (tokens[n] <= 2 * w) v[n][w] = was[n][w];
              else if (tokens[n] == 2 * w + 1) v[n][w] = (v[n][w] & 0xFFFFu) | (was[n][w] & 0xFFFF0000u);
            vy[at[n]] = v[n];
          }
        }
      }
    }
  }
}

// Lengths and the head change in a launch of their own, after every workgroup of the first
// has read them.
__global__ __launch_bounds__(256) void k_fork_counts(ForkArgs a) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t s_sum[4], s_refused;
  uint32_t *s_first = lds, *s_rank = lds + a.requests;
  if (threadIdx.x == 0) s_refused = 0;
  const uint32_t taken = plan_forks(a, s_first, s_rank, s_sum);
  const uint32_t head = min((uint32_t)max(*a.free_head, 0), a.free_len);
  uint32_t refused = 0;
  for (uint32_t i = threadIdx.x; i < a.forks; i += 256) {
    // (a source is not empty and a destination is, so none of these is read here again)
    if (s_rank[i] != ~0u) a.lens[a.dst[i]] = a.lens[a.src[i]];
    else ++refused;
  }
  if (refused) atomicAdd(&s_refused, refused);  // whole numbers: any order gives the same
  __syncthreads();
  if (threadIdx.x == 0) {
    a.counts[0] = (int32_t)(head + taken);
    a.counts[1] = (int32_t)s_refused;
  }
}

// ----------------------------------------------------------------------- free
struct FreeArgs {
  const int32_t *rows, *free_head;
  int32_t *lens, *table, *free_list, *shares, *counts;
  uint32_t* bits;  // of the pages that go back
  uint32_t count, requests, width, free_len, log_block, blocks, words, parts;
};

// A page loses a holder for each row that ends; the one that finds none left marks it.
__global__ __launch_bounds__(256) void k_page_free(FreeArgs a) {
  const uint32_t t = threadIdx.x;
  for (uint32_t unit = blockIdx.x; unit < a.count * a.parts; unit += gridDim.x) {
    const uint32_t i = unit / a.parts, part = unit % a.parts, row = (uint32_t)a.rows[i];
    if (row >= a.requests) continue;
    bool again = false;  // a row that was named before
    for (uint32_t j = t; j < i; j += 256) again |= (uint32_t)a.rows[j] == row;
    if (__syncthreads_or(again)) continue;
    const uint32_t len = (uint32_t)max(a.lens[row], 0);
    const uint32_t pages = min((uint32_t)(((uint64_t)len + (1u << a.log_block) - 1) >> a.log_block), a.width);
    for (uint32_t c = t + 256 * part; c < pages; c += 256 * a.parts) {
      int32_t* at = a.table + (uint64_t)row * a.width + c;
      const uint32_t id = (uint32_t)*at;
      *at = -1;
      if (id < a.blocks && atomicSub(a.shares + id, 1) <= 0) atomicOr(a.bits + id / 32, 1u << id % 32);
    }
  }
}

// One workgroup writes the marked pages into the list, in the order of their ids, and
// clears the marks.
constexpr uint32_t kCollect = 1024;
__global__ __launch_bounds__(kCollect) void k_free_collect(FreeArgs a) {
  __shared__ uint32_t s_sum[kCollect / 64];
  const uint32_t t = threadIdx.x;
  const uint32_t head = min((uint32_t)max(*a.free_head, 0), a.free_len);
  uint32_t total = 0;
  for (uint32_t w = t; w < a.words; w += kCollect) total += __popc(a.bits[w]);
  sum_before<kCollect>(total, s_sum, &total);
  uint32_t done = 0;
  for (uint32_t w0 = 0; w0 < a.words; w0 += kCollect) {
    const uint32_t w = w0 + t;
    uint32_t bits = w < a.words ? a.bits[w] : 0, all;
    uint32_t at = done + sum_before<kCollect>(__popc(bits), s_sum, &all);
    done += all;
    if (bits) a.bits[w] = 0;
    for (; bits; bits &= bits - 1, ++at) {
      const uint32_t id = 32 * w + (uint32_t)__builtin_ctz(bits);
      a.shares[id] = 0;
      if (head + at >= total) a.free_list[head + at - total] = (int32_t)id;
    }
  }
  for (uint32_t i = t; i < a.count; i += kCollect)
    if ((uint32_t)a.rows[i] < a.requests) a.lens[a.rows[i]] = 0;
  __syncthreads();
  if (t == 0) {
    a.counts[0] = (int32_t)(head - min(total, head));
    a.counts[1] = (int32_t)total;
  }
}

bool caches_ok(uint32_t layers, uint32_t heads, uint32_t dim, uint32_t blocks, uint32_t block) {
  return block_ok(block) && pool_ok(blocks, block) && layers >= 1 && layers <= 4096 && heads >= 1 && heads <= 65535 &&
         dim >= 8 && dim % 8 == 0 && dim <= 1024;
}

bool table_ok(uint32_t requests, uint32_t width, uint32_t free_len, uint32_t block) {
  return requests <= kMaxRequests && free_len <= (1u << 30) && (uint64_t)width * block <= 0x7FFFFFFFull;
}

Pool make_pool(void* k, void* v, uint32_t layers, uint32_t heads, uint32_t dim, uint32_t blocks, uint32_t block) {
  return Pool{static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), layers, heads, dim, (uint32_t)__builtin_ctz(block),
              blocks};
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" {

int dgt_page_keep(const int32_t* d_path, const int32_t* d_kept, const int32_t* d_ctx, const int32_t* d_cu,
                  const int32_t* d_slots, uint32_t requests, uint32_t tokens, int32_t* d_free,
                  uint32_t free_len, const int32_t* d_free_head, int32_t* d_table, uint32_t width,
                  uint32_t layers, uint32_t heads, uint32_t dim, uint32_t blocks, uint32_t block,
                  void* d_k_cache, void* d_v_cache, int32_t* d_lens, int32_t* d_counts, void* stream) {
  if (!caches_ok(layers, heads, dim, blocks, block) || !table_ok(requests, width, free_len, block) || tokens > (1u << 28))
    return DGT_E_SHAPE;
  if (!d_free_head || !d_counts || (free_len && !d_free)) return DGT_E_ARG;
  if (requests && (!d_kept || !d_ctx || !d_cu || !d_lens || (width && !d_table))) return DGT_E_ARG;
  if (tokens && !d_slots) return DGT_E_ARG;
  if (blocks && (!d_k_cache || !d_v_cache)) return DGT_E_ARG;
  if (!aligned(d_k_cache, 16) || !aligned(d_v_cache, 16)) return DGT_E_ARG;
  KeepArgs a;
  a.path = d_path;
  a.kept = d_kept;
  a.ctx = d_ctx;
  a.cu = d_cu;
  a.slots = d_slots;
  a.free_head = d_free_head;
  a.free_list = d_free;
  a.table = d_table;
  a.lens = d_lens;
  a.counts = d_counts;
  a.requests = requests;
  a.tokens = tokens;
  a.free_len = free_len;
  a.width = width;
  a.pool = make_pool(d_k_cache, d_v_cache, layers, heads, dim, blocks, block);
  // as many workgroups a request as the card holds at a time, if it is not one each anyway
  const uint32_t all = layers * heads;
  a.parts = d_path && tokens && blocks && requests ? std::min(all, std::max(8 * kCUs / requests, 1u)) : 0;
  a.each = a.parts ? (all + a.parts - 1) / a.parts : 0;
  a.parts = a.parts ? (all + a.each - 1) / a.each : 0;
  hipLaunchKernelGGL(k_page_keep, dim3(1 + requests * a.parts), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return launched();
}

int dgt_page_fork(const int32_t* d_src, const int32_t* d_dst, uint32_t forks, int32_t* d_lens,
                  int32_t* d_table, uint32_t requests, uint32_t width, const int32_t* d_free,
                  uint32_t free_len, const int32_t* d_free_head, int32_t* d_shares, uint32_t layers,
                  uint32_t heads, uint32_t dim, uint32_t blocks, uint32_t block, void* d_k_cache,
                  void* d_v_cache, int32_t* d_counts, void* stream) {
  if (!caches_ok(layers, heads, dim, blocks, block) || !table_ok(requests, width, free_len, block) || forks > kMaxRequests)
    return DGT_E_SHAPE;
  if (!d_free_head || !d_counts || (free_len && !d_free)) return DGT_E_ARG;
  if (forks && (!d_src || !d_dst)) return DGT_E_ARG;
  if (requests && (!d_lens || (width && !d_table))) return DGT_E_ARG;
  if (blocks && (!d_k_cache || !d_v_cache || !d_shares)) return DGT_E_ARG;
  if (!aligned(d_k_cache, 16) || !aligned(d_v_cache, 16)) return DGT_E_ARG;
  ForkArgs a;
  a.src = d_src;
  a.dst = d_dst;
  a.free_list = d_free;
  a.free_head = d_free_head;
  a.lens = d_lens;
  a.table = d_table;
  a.shares = d_shares;
  a.counts = d_counts;
  a.forks = forks;
  a.requests = requests;
  a.width = width;
  a.free_len = free_len;
  a.pool = make_pool(d_k_cache, d_v_cache, layers, heads, dim, blocks, block);
  // parts of a fork, so that a few forks fill the card; a part is at least a head of a layer
  // (twice what is on the card at a time: 67-70 us, once: 70-75, for the 192 forks above)
  a.parts = std::min(layers * heads, std::max(16 * kCUs / std::max(forks, 1u), 1u));
  const uint32_t lds = 4 * (requests + forks);
  if (lds > 63 * 1024 &&  // with what the kernels have besides, more than the 64 KB of a plain launch
      (hipFuncSetAttribute(reinterpret_cast<const void*>(k_page_fork), hipFuncAttributeMaxDynamicSharedMemorySize,
                           (int)lds) != hipSuccess ||
       hipFuncSetAttribute(reinterpret_cast<const void*>(k_fork_counts), hipFuncAttributeMaxDynamicSharedMemorySize,
                           (int)lds) != hipSuccess))
    return DGT_E_HIP;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (forks) {
    hipLaunchKernelGGL(k_page_fork, dim3(std::min(forks * a.parts, 16 * kCUs)), dim3(256), lds, st, a);
    if (int rc = launched()) return rc;
  }
  hipLaunchKernelGGL(k_fork_counts, dim3(1), dim3(256), lds, st, a);
  return launched();
}

size_t dgt_page_free_workspace(uint32_t blocks) { return ((size_t)blocks + 31) / 32 * 4 + 4; }

int dgt_page_free(const int32_t* d_rows, uint32_t count, int32_t* d_lens, int32_t* d_table,
                  uint32_t requests, uint32_t width, int32_t* d_free, uint32_t free_len,
                  const int32_t* d_free_head, int32_t* d_shares, uint32_t blocks, uint32_t block,
                  int32_t* d_counts, void* d_ws, size_t ws_bytes, void* stream) {
  if (!block_ok(block) || !pool_ok(blocks, block) || !table_ok(requests, width, free_len, block) || count > kMaxRequests)
    return DGT_E_SHAPE;
  if (!d_free_head || !d_counts || (free_len && !d_free) || (count && !d_rows)) return DGT_E_ARG;
  if (requests && (!d_lens || (width && !d_table))) return DGT_E_ARG;
  if ((blocks && !d_shares) || !d_ws || !aligned(d_ws, 4)) return DGT_E_ARG;
  if (ws_bytes < dgt_page_free_workspace(blocks)) return DGT_E_BUFSIZE;
  FreeArgs a;
  a.rows = d_rows;
  a.free_head = d_free_head;
  a.lens = d_lens;
  a.table = d_table;
  a.free_list = d_free;
  a.shares = d_shares;
  a.counts = d_counts;
  a.bits = static_cast<uint32_t*>(d_ws);
  a.count = count;
  a.requests = requests;
  a.width = width;
  a.free_len = free_len;
  a.log_block = (uint32_t)__builtin_ctz(block);
  a.blocks = blocks;
  a.words = (blocks + 31) / 32;
  a.parts = std::max(1u, std::min((width + 255) / 256, 2 * kCUs / std::max(count, 1u)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (count) {
    hipLaunchKernelGGL(k_page_free, dim3(std::min(count * a.parts, 8 * kCUs)), dim3(256), 0, st, a);
    if (int rc = launched()) return rc;
  }
  hipLaunchKernelGGL(k_free_collect, dim3(1), dim3(kCollect), 0, st, a);
  return launched();
}

}  // extern "C"
