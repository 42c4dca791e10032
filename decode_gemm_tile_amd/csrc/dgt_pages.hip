// Page plan of a serving step and the store of new keys and values into the
// paged cache.
#include "dgt_serve.h"

#include <algorithm>

namespace dgt {
namespace serve {
namespace {

// ------------------------------------------------------------------ page plan
// Two exclusive sums over the requests (their new tokens, and the pages they
// still need) and then one independent computation per new token.  The sums are
// a few microseconds of latency and no work, so every workgroup forms them for
// itself in LDS and goes on to its own tokens: one launch, no hand-off.  Bound by its
// chain of latencies (8 tokens of 8 requests 3.2 us, 12750 tokens of 509 requests with
// trees of up to 61 8.3 us).
struct PlanArgs {
  const int32_t *ctx, *fresh_tokens, *free_list, *free_head, *parents;
  int32_t *table, *cu, *slots, *positions, *counts;
  uint64_t* mask;
  uint32_t requests, free_len, width, log_block, blocks, tokens, words;
  bool rows, sums;  // write what belongs to tokens and pages; write cu and counts
};

constexpr uint32_t kPlanThreads = 256;
// Parents kept in LDS: those of the workgroup's tokens and of this many before them.
constexpr uint32_t kPlanBefore = 768;

struct Request {
  uint32_t ctx, have;  // tokens and pages in the cache
  uint32_t need;       // pages to take from the free list
  bool wide;           // the table has a column for every page
};

// A request of c cached and n new tokens, both below 2^31.
__device__ __forceinline__ Request plan_request(const PlanArgs& p, uint32_t c, uint32_t n) {
  Request r;
  r.ctx = c;
  const uint32_t round = (1u << p.log_block) - 1;
  r.have = (c + round) >> p.log_block;
  const uint32_t after = (uint32_t)(((uint64_t)c + n + round) >> p.log_block);
  r.wide = after <= p.width;
  r.need = r.wide ? after - r.have : 0u;
  return r;
}

__global__ __launch_bounds__(kPlanThreads) void k_page_plan(PlanArgs p) {
  extern __shared__ uint32_t lds[];
  uint32_t* s_cu = lds;                        // [requests + 1] token offsets
  uint32_t* s_end = s_cu + p.requests + 1;     // [requests] pages needed up to and with b
  uint32_t* s_ctx = s_end + p.requests;        // [requests]
  __shared__ uint32_t s_tok[kPlanThreads / 64], s_page[kPlanThreads / 64], s_out[2];
  __shared__ int32_t s_par[kPlanBefore + kPlanThreads];
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6;
  // The launch is a chain of memory latencies and little else, so what does not
  // hang on the sums is asked for ahead of them.
  const int32_t head_in = *p.free_head;
  uint32_t kept = 0;  // parents from this row on are in LDS
  auto keep_parents = [&](uint32_t tile) {
    kept = tile - min(tile, kPlanBefore);
    for (uint32_t i = kept + t; i < min(tile + kPlanThreads, p.tokens); i += kPlanThreads) s_par[i - kept] = p.parents[i];
  };
  if (p.parents) keep_parents(blockIdx.x * kPlanThreads);
  // Sums stop growing one past what fits, so that no input overflows them:
  // min(a + b, cap) over non-negative numbers is associative.
  const uint32_t tok_cap = p.tokens + 1, page_cap = p.free_len + 1;
  uint32_t tok_base = 0, page_base = 0;
  for (uint32_t b0 = 0; b0 < p.requests; b0 += kPlanThreads) {
    const uint32_t b = b0 + t;
    uint32_t tok = 0, page = 0;
    if (b < p.requests) {
      const uint32_t c = (uint32_t)max(p.ctx[b], 0), n = (uint32_t)max(p.fresh_tokens[b], 0);
      tok = min(n, tok_cap);
      page = min(plan_request(p, c, n).need, page_cap);
      s_ctx[b] = c;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t to = __shfl_up(tok, d, 64), po = __shfl_up(page, d, 64);
      if (lane >= (uint32_t)d) {
        tok = min(tok + to, tok_cap);
        page = min(page + po, page_cap);
      }
    }
    if (lane == 63) {
      s_tok[wave] = tok;
      s_page[wave] = page;
    }
    __syncthreads();
    uint32_t tb = tok_base, pb = page_base;
    for (uint32_t w = 0; w < kPlanThreads / 64; ++w) {
      if (w == wave) {
        tok = min(tok + tb, tok_cap);
        page = min(page + pb, page_cap);
      }
      tb = min(tb + s_tok[w], tok_cap);
      pb = min(pb + s_page[w], page_cap);
    }
    tok_base = tb;
    page_base = pb;
    if (b < p.requests) {
      s_cu[b + 1] = tok;
      s_end[b] = page;
    }
    __syncthreads();  // s_tok and s_page are rewritten by the next round
  }
  if (t == 0) s_cu[0] = 0;
  if (t < 2) s_out[t] = 0;
  __syncthreads();

  const uint32_t head = (uint32_t)max(head_in, 0);
  const uint32_t left = head < p.free_len ? p.free_len - head : 0u;
  // (Where the offsets were cut, n is too small, but b does not fit anyway.)
  auto request = [&](uint32_t b) { return plan_request(p, s_ctx[b], s_cu[b + 1] - s_cu[b]); };
  // b keeps its tokens if its pages have columns, its rows exist and, where it
  // needs pages, the list still holds them.
  auto fits = [&](uint32_t b, const Request& r) {
    return r.wide && s_cu[b + 1] <= p.tokens && (r.need == 0 || s_end[b] <= left);
  };
  if (p.sums && blockIdx.x == 0) {
    uint32_t refused = 0, taken = 0;
    for (uint32_t b = t; b < p.requests; b += kPlanThreads) {
      const Request r = request(b);
      const bool ok = fits(b, r);
      if (!ok) refused += 1;
      if (ok && r.need) taken = max(taken, s_end[b]);
    }
    if (refused) atomicAdd(&s_out[0], refused);  // whole numbers: any order gives the same
    if (taken) atomicMax(&s_out[1], taken);
    for (uint32_t b = t; b <= p.requests; b += kPlanThreads)
      p.cu[b] = (int32_t)min(s_cu[b], p.tokens);
    __syncthreads();
    if (t == 0) {
      p.counts[0] = (int32_t)s_cu[p.requests];
      p.counts[1] = (int32_t)(head + s_out[1]);
      p.counts[2] = (int32_t)s_out[0];
    }
  }
  if (!p.rows) return;

  const uint32_t total = min(s_cu[p.requests], p.tokens), block = 1u << p.log_block;
  for (uint32_t tile = blockIdx.x * kPlanThreads; tile < p.tokens; tile += gridDim.x * kPlanThreads) {
    if (p.parents && tile != blockIdx.x * kPlanThreads) {
      __syncthreads();
      keep_parents(tile);
      __syncthreads();
    }
    const uint32_t tok = tile + t;
    // the last request whose first row is at or before tok
    uint32_t b = 0;
    if (tok < total) {
      uint32_t hi = p.requests;  // s_cu[b] <= tok < s_cu[hi]
      while (hi - b > 1) {
        const uint32_t mid = (b + hi) >> 1;
        if (s_cu[mid] <= tok) b = mid; else hi = mid;
      }
    }
    if (tok >= p.tokens) continue;  // (to the loop's end, as all of its workgroup's tiles but the last are whole)
    uint64_t* row = p.mask ? p.mask + (uint64_t)tok * p.words : nullptr;
    int32_t slot = -1, position = -1;
    uint32_t lowest = p.words;  // mask words from here on are written
    if (tok < total) {
      const uint32_t at = tok - s_cu[b];
      const Request r = request(b);
      const uint32_t pos = r.ctx + at;
      bool sound = true;
      uint32_t depth = at;
      if (p.parents) {
        // Walk to the root.  Parents lie before their children, so the walk ends
        // and meets mask words from the last to the first.
        auto parent = [&](uint32_t node) {
          const uint32_t i = s_cu[b] + node;
          return i >= kept ? s_par[i - kept] : p.parents[i];
        };
        depth = 0;
        sound = at < p.words * 64u;
        int32_t node = (int32_t)at;
        uint64_t bits = 0;
        uint32_t word = at >> 6;
        lowest = sound ? word + 1 : p.words;
        if (row) for (uint32_t w = lowest; w < p.words; ++w) row[w] = 0;
        while (sound) {
          if ((uint32_t)node >> 6 != word) {
            row[word] = bits;
            lowest = word;
            bits = 0;
            while (--word > (uint32_t)node >> 6) row[lowest = word] = 0;
          }
          bits |= 1ull << (node & 63);
          const int32_t up = parent((uint32_t)node);
          if (up == -1) break;
          sound = up >= 0 && up < node;
          node = up;
          ++depth;
        }
        if (sound) {
          row[word] = bits;
          lowest = word;
        } else {
          lowest = p.words;  // a bad link: the row sees nothing
        }
      }
      if (sound) position = (int32_t)(r.ctx + depth);
      if (fits(b, r)) {
        const uint32_t page = pos >> p.log_block;
        const uint64_t at_table = (uint64_t)b * p.width + page;
        const bool taken = page >= r.have;
        const int32_t* from = taken ? p.free_list + (head + s_end[b] - r.need + (page - r.have)) : p.table + at_table;
        const uint32_t id = (uint32_t)*from;
        if (taken && (pos & (block - 1)) == 0) p.table[at_table] = (int32_t)id;
        if (sound && id < p.blocks) slot = (int32_t)((id << p.log_block) + (pos & (block - 1)));
      }
    }
    p.slots[tok] = slot;
    p.positions[tok] = position;
    if (row) for (uint32_t w = 0; w < lowest; ++w) row[w] = 0;
  }
}

// ---------------------------------------------------------------- cache store
// A workgroup takes 64 tokens of one head.  Key rows are copied into their pages as
// they are, 16 bytes a thread.  Value pages are transposed: the values turn in LDS,
// and tokens whose slots follow one another within 8 aligned slots are written
// together, 16 bytes where all 8 are there.  6792 tokens of 8 heads of 128 from fp32
// rows take 22.6 us, 3.7 TB/s (35 us with one element a thread straight to its place),
// and 27.6 where no cache holds anything of them; a plain cast of as many values takes
// 16.6.  Bytes do not bound it alone: the 856 equal workgroups are 3.3 a CU, so the last
// round is partly empty.
struct StoreArgs {
  const void *k, *v;
  const int32_t* slots;
  uint16_t *kc, *vc;
  int64_t k_row, k_head, v_row, v_head;  // element strides of k and v
  uint32_t tokens, heads, dim, log_block, blocks;
  bool wide;  // rows of k and v are 16-byte aligned
};

template <typename E, typename S>
__global__ __launch_bounds__(256) void k_kv_store(StoreArgs a) {
  __shared__ uint32_t s_slot[kStoreRows], s_head[kStoreRows], s_heads;
  __shared__ uint16_t s_v[kStoreDims * kStoreLine];
  const uint32_t t = threadIdx.x, t0 = blockIdx.x * kStoreRows, h = blockIdx.y;
  const uint32_t d0 = blockIdx.z * kStoreDims, dims = min(a.dim - d0, kStoreDims);
  const uint32_t rows = min(a.tokens - t0, kStoreRows), block = 1u << a.log_block;
  if (t < 64) {
    const uint32_t slot = t < rows ? (uint32_t)a.slots[t0 + t] : ~0u;
    slot_groups(slot < a.blocks << a.log_block ? slot : ~0u, s_slot, s_head, &s_heads);
  }
  __syncthreads();
  const S* k = static_cast<const S*>(a.k) + (int64_t)h * a.k_head + d0;
  const S* v = static_cast<const S*>(a.v) + (int64_t)h * a.v_head + d0;
  const uint32_t pieces = dims / 8;
  constexpr uint32_t kIter = kStoreRows * kStoreDims / 8 / 256;
  u32x4 kv[kIter], vv[kIter];
#pragma unroll
  for (uint32_t j = 0; j < kIter; ++j) {  // everything is asked for before anything is written
    const uint32_t i = t + 256 * j, r = i / pieces, d = 8 * (i % pieces);
    if (r < rows && s_slot[r] != ~0u) {
      kv[j] = load8<E>(k + (int64_t)(t0 + r) * a.k_row + d, a.wide);
      vv[j] = load8<E>(v + (int64_t)(t0 + r) * a.v_row + d, a.wide);
    }
  }
#pragma unroll
  for (uint32_t j = 0; j < kIter; ++j) {
    const uint32_t i = t + 256 * j, r = i / pieces, d = 8 * (i % pieces);
    if (r < rows && s_slot[r] != ~0u) {
      const uint32_t slot = s_slot[r];
      const uint64_t base = ((uint64_t)(slot >> a.log_block) * a.heads + h) * block + (slot & (block - 1));
      *reinterpret_cast<u32x4*>(a.kc + base * a.dim + d0 + d) = kv[j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s_v[(d + 2 * e) * kStoreLine + r] = (uint16_t)vv[j][e];
        s_v[(d + 2 * e + 1) * kStoreLine + r] = (uint16_t)(vv[j][e] >> 16);
      }
    }
  }
  __syncthreads();
  write_values(a.vc + (uint64_t)h * a.dim * block, a.heads, a.dim, d0, dims, a.log_block, s_v, s_slot, s_head, s_heads);
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" {

int dgt_page_plan(const int32_t* d_ctx, const int32_t* d_new, uint32_t requests,
                  const int32_t* d_free, uint32_t free_len, const int32_t* d_free_head,
                  int32_t* d_table, uint32_t width, uint32_t block, uint32_t blocks,
                  uint32_t tokens, const int32_t* d_parents, uint32_t mask_words, int32_t* d_cu,
                  int32_t* d_slots, int32_t* d_positions, uint64_t* d_mask, int32_t* d_counts,
                  void* stream) {
  if (!block_ok(block) || !pool_ok(blocks, block)) return DGT_E_SHAPE;
  if (requests > kMaxRequests || tokens > (1u << 28) || free_len > (1u << 30) ||
      (uint64_t)width * block > 0x7FFFFFFFull || mask_words > 1024)
    return DGT_E_SHAPE;
  if (!d_cu || !d_counts || !d_free_head || (free_len && !d_free)) return DGT_E_ARG;
  if (requests && (!d_ctx || !d_new || (width && !d_table))) return DGT_E_ARG;
  if (tokens && (!d_slots || !d_positions)) return DGT_E_ARG;
  // a tree comes with its masks and masks with their tree
  if ((mask_words != 0) != (d_parents != nullptr) || (mask_words && tokens && !d_mask)) return DGT_E_ARG;
  PlanArgs p;
  p.ctx = d_ctx;
  p.fresh_tokens = d_new;
  p.free_list = d_free;
  p.free_head = d_free_head;
  p.parents = d_parents;
  p.table = d_table;
  p.cu = d_cu;
  p.slots = d_slots;
  p.positions = d_positions;
  p.counts = d_counts;
  p.mask = mask_words ? d_mask : nullptr;
  p.requests = requests;
  p.free_len = free_len;
  p.width = width;
  p.log_block = (uint32_t)__builtin_ctz(block);
  p.blocks = blocks;
  p.tokens = tokens;
  p.words = mask_words;
  const uint32_t lds = (3 * requests + 1) * 4;
  if (lds > 56 * 1024 &&  // with what the kernel has besides, more than the 64 KB of a plain launch
      hipFuncSetAttribute(reinterpret_cast<const void*>(k_page_plan),
                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
    return DGT_E_HIP;
  const uint32_t grid = std::min(std::max((tokens + kPlanThreads - 1) / kPlanThreads, 1u), 4 * kCUs);
  hipStream_t st = static_cast<hipStream_t>(stream);
  auto run = [&](uint32_t workgroups, bool rows, bool sums) {
    p.rows = rows;
    p.sums = sums;
    hipLaunchKernelGGL(k_page_plan, dim3(workgroups), dim3(kPlanThreads), lds, st, p);
    return launched();
  };
  // Every workgroup reads the list's head.  Where it lies in the counts (a step that
  // goes on from its own last result), the new one may be written only after the last
  // of them has read the old one, which the order of two launches gives (12750 tokens:
  // 13.8 us a pass, 10.0 with one); a single workgroup has its barriers.
  const uintptr_t head = reinterpret_cast<uintptr_t>(d_free_head), counts = reinterpret_cast<uintptr_t>(d_counts);
  if (grid > 1 && head + 4 > counts && head < counts + 12) {
    const int rc = run(grid, true, false);
    return rc ? rc : run(1, false, true);
  }
  return run(grid, true, true);
}

int dgt_kv_store(const void* d_k, const void* d_v, uint32_t source, int64_t k_row, int64_t k_head,
                 int64_t v_row, int64_t v_head, const int32_t* d_slots, uint32_t tokens,
                 uint32_t heads, uint32_t dim, uint32_t cache, void* d_k_cache, void* d_v_cache,
                 uint32_t blocks, uint32_t block, void* stream) {
  if (!block_ok(block) || !pool_ok(blocks, block) || heads == 0 || dim == 0 || dim % 8 ||
      dim > 1024 || heads > 65535 || tokens > (1u << 28))
    return DGT_E_SHAPE;
  if (cache != DGT_ELT_BF16 && cache != DGT_ELT_F16) return DGT_E_UNSUPPORTED;
  if (source != DGT_ELT_F32 && source != cache) return DGT_E_UNSUPPORTED;
  if (tokens == 0 || blocks == 0) return DGT_OK;
  if (!d_k || !d_v || !d_slots || !d_k_cache || !d_v_cache) return DGT_E_ARG;
  if (!aligned(d_k_cache, 16) || !aligned(d_v_cache, 16)) return DGT_E_ARG;
  StoreArgs a;
  a.k = d_k;
  a.v = d_v;
  a.slots = d_slots;
  a.kc = static_cast<uint16_t*>(d_k_cache);
  a.vc = static_cast<uint16_t*>(d_v_cache);
  a.k_row = k_row;
  a.k_head = k_head;
  a.v_row = v_row;
  a.v_head = v_head;
  a.tokens = tokens;
  a.heads = heads;
  a.dim = dim;
  a.log_block = (uint32_t)__builtin_ctz(block);
  a.blocks = blocks;
  const int64_t lane = source == DGT_ELT_F32 ? 4 : 8;  // elements of 16 bytes
  a.wide = aligned(d_k, 16) && aligned(d_v, 16) && k_row % lane == 0 && k_head % lane == 0 && v_row % lane == 0 &&
           v_head % lane == 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const dim3 grid((tokens + kStoreRows - 1) / kStoreRows, heads, (dim + kStoreDims - 1) / kStoreDims);
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a);
    return launched();
  };
  if (cache == DGT_ELT_BF16)
    return source == DGT_ELT_F32 ? run(k_kv_store<Bf16, float>) : run(k_kv_store<Bf16, uint16_t>);
  return source == DGT_ELT_F32 ? run(k_kv_store<F16, float>) : run(k_kv_store<F16, uint16_t>);
}

}  // extern "C"
