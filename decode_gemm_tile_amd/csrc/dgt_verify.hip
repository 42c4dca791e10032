// Verification of drafted tokens against the target's logits.
#include "dgt_serve.h"

#include <algorithm>

namespace dgt {
namespace serve {
namespace {

// A request's path starts at row 0 and goes down its tree or chain; an end's largest logit
// and sum of exponentials decide about the drafted tokens that follow it.  The sum is formed
// in fp32; where a draft's number lies nearer to its border than that can tell (kNear), about once
// in 50000 drafts, the path waits there for the launch of the last rows, which goes on with fp64
// sums.  A workgroup looks at one segment of one row.  The last to come for a row that is the path's
// end decides, and goes on if the row after it is complete too; else whoever completes
// that one does.  Nobody waits.  Rows come in the order of their index within the request,
// so a row's turn is mostly after the decisions above it, and one that the path has
// passed by is not read: of 64 trees of up to 27 nodes, less than half of them are.
//
// Then the next token out of the last row: a uniform number falls between two of a
// vocabulary's running sums, which lie 1 / vocab apart on the average; sums of fp32
// exponentials, off by 2^-24, would give another token in one of a hundred calls, so
// this row's weights are formed in fp64, a workgroup a segment, and the request's last
// workgroup chooses.  Where a chain was refused the weights are max(p - q, 0), p needs
// the whole row's sum first, and one more launch forms them.
//
// Measured: 96 chains of up to 7, 128000 tokens, bf16: 106 us (order 5, rows 45, last rows 28,
// refused ones 30); 64 trees of up to 27, fp32: 72-86 (5, 67, 21); 5 chains of up to 5, 32000, fp32:
// 37 (4, 15, 21).  Chains of latencies bound all of them (in the trees 160 MB of 380 are read,
// and the paths' rows are 77).  fp64 exponentials stand eight side by side, as one alone waits
// for itself.
struct VerifyArgs {
  const void* logits;
  const float *probs, *temperature, *accept, *sample;
  const int32_t *draft, *parents, *cu;
  int32_t *path, *accepted, *next;
  uint64_t* parts;          // [tokens][segs][2], see Part
  uint32_t* order;          // [tokens][2]: rows in their turn, and their requests
  uint32_t* counters;       // [tokens]: parts that are there, and one for a row on the path
  struct State* states;     // [requests]
  double* sums;             // [requests][segs]: of a last row's weights, then of max(p - q, 0)
  double* rest;
  struct End* ends;         // [2][requests]: of the paths; of those that were left open, once they are not
  uint64_t logits_row, probs_row;
  uint32_t requests, tokens, vocab, segs;
  bool wide, probs_wide;    // rows are 16-byte aligned
};

// A row's vocabulary in segments; a segment of a row is what one workgroup looks at.
constexpr uint32_t kSeg = 4096, kThreads = 256, kEach = kSeg / kThreads;

// What is known of a segment: sum of exp((l - top) / T), top (NaN if there is a NaN), the
// largest logit's place (the first of equals, within the vocabulary).  Parts, counters and
// states pass between workgroups that may sit on different dies: agent-scope accesses, and a
// wait for the stores before whatever tells of them.
struct Part {
  float sum, top;
  uint32_t at;
};
__device__ __forceinline__ void put(uint64_t* p, uint64_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t get(const uint64_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint32_t count_in(uint32_t* p) { return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// A request's path so far: its end's index in the low half (kOver: it is decided), its length.
struct State {
  uint64_t path;
};
constexpr uint32_t kOver = 0x7FFFFFFF;

enum Mode : uint32_t { kDone, kFromTarget, kFromRest, kOpen };
struct End {  // of a path
  uint32_t mode, row, counter, rest_counter;
  float top;     // of the row
  uint32_t at;   // the largest logit's place
  uint32_t end;  // the row within its request
  uint32_t lost; // children of it were refused; of an open one: the path's length
};

// 2^z for z <= 0 in fp64, off by 2^-39: the polynomial of degree 8 that meets 2^f in the nine
// Chebyshev points of |f| <= 1/2.  z is cut at -1000, whose power is as good as zero; the
// whole number is read out of the low bits of z + 1.5 * 2^52.
// (Eight side by side: one after another, each step waits for the one before.)
__device__ constexpr double kPowers[9] = {1.3255224878668817e-06, 1.5310079402249296e-05, 0.00015403455852453838,
                                          0.0013333450568000645,  0.009618129159402558,   0.05550410941205933,
                                          0.2402265069581299,     0.6931471805459335,     1.0};
template <int N>
__device__ __forceinline__ void exp2_64(double (&z)[N], const double* kC = kPowers) {
  constexpr double kRound = 6755399441055744.0;
  double f[N], p[N];
  uint32_t n[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const double cut = fmax(z[e], -1000.0), whole = cut + kRound;
    n[e] = (uint32_t)__builtin_bit_cast(uint64_t, whole);
    f[e] = cut - (whole - kRound);
    p[e] = kC[0];
  }
#pragma unroll
  for (int k = 1; k < 9; ++k)
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = fma(p[e], f[e], kC[k]);
#pragma unroll
  for (int e = 0; e < N; ++e) z[e] = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, p[e]) + ((uint64_t)n[e] << 52));
}
__device__ __forceinline__ double exp2_64(double z, const double* powers = kPowers) {
  double one[1] = {z};
  exp2_64<1>(one, powers);
  return one[0];
}

constexpr double kLog2e = 1.44269504088896340736;
// What logits are multiplied by: 1 / T in powers of two, or 0 for the largest logit's token.  (Of an
// infinite T so little is left that all tokens weigh the same, whatever their logits.)
__device__ __forceinline__ double heat(const VerifyArgs& a, uint32_t b) {
  const float t = a.temperature ? a.temperature[b] : 1.f;
  return !(t > 0.f) ? 0.0 : t < INFINITY ? kLog2e / (double)t : 1e-60;
}
// Twice that in fp32, where halves of logits are taken from each other: a mask of the type's lowest
// value and a large logit lie further apart than fp32 reaches.
__device__ __forceinline__ float heat32(double c) { return c > 0.0 ? fmaxf((float)fmin(2.0 * c, 3e38), 1.4e-45f) : 0.f; }
__device__ __forceinline__ float weight32(float x, float top, float c) {
  return __builtin_amdgcn_exp2f(fmaf(x, 0.5f, -0.5f * top) * c);
}

template <class E>
struct Logit {
  typedef uint16_t T;
  static constexpr uint32_t kPiece = 8;  // in 16 bytes
  static __device__ __forceinline__ float one(const void* p, uint64_t i) { return E::up(static_cast<const uint16_t*>(p)[i]); }
  static __device__ __forceinline__ void piece(const uint16_t* p, float* x) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = E::up(v[j] & 0xFFFFu);
      x[2 * j + 1] = E::up(v[j] >> 16);
    }
  }
};
struct F32 {};
template <>
struct Logit<F32> {
  typedef float T;
  static constexpr uint32_t kPiece = 4;
  static __device__ __forceinline__ float one(const void* p, uint64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void piece(const float* p, float* x) {
    const floatx4 v = *reinterpret_cast<const floatx4*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = v[j];
  }
};

// Place within a segment of a thread's element e: pieces of 16 bytes go round the threads.
template <class L>
__device__ __forceinline__ uint32_t place(uint32_t e) {
  return (e / L::kPiece * kThreads + threadIdx.x) * L::kPiece + e % L::kPiece;
}

// A segment's elements at the thread's places; past the vocabulary's end `none`.
template <class L, class F>
__device__ __forceinline__ void load_places(const void* base, uint64_t row, uint32_t seg, uint32_t vocab, bool wide, float none,
                                            F at, float (&x)[kEach]) {
  const typename L::T* p = static_cast<const typename L::T*>(base) + row + (uint64_t)seg * kSeg;
  const uint32_t left = vocab - seg * kSeg;
  if (wide && left >= kSeg) {
#pragma unroll
    for (uint32_t e = 0; e < kEach; e += L::kPiece) L::piece(p + at(e), x + e);
  } else {
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e) x[e] = at(e) < left ? L::one(p, at(e)) : none;
  }
}

// The order of candidates for the largest: greater first, then the lower place.
__device__ __forceinline__ void better(float& v, uint32_t& at, float ov, uint32_t oat) {
  const bool take = ov > v || (ov == v && oat < at);
  v = take ? ov : v;
  at = take ? oat : at;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// A thread's, a wave's or a workgroup's share of a row.
struct RowSum {
  float sum, top;  // sum of exp((l - top) / T)
  uint32_t at;     // the largest logit's place
  bool odd;        // a NaN
  static __device__ __forceinline__ RowSum none() { return RowSum{0.f, -INFINITY, 0xFFFFFFFFu, false}; }
  __device__ __forceinline__ void join(float osum, float otop, uint32_t oat, bool oodd, float c) {
    const float now = fmaxf(top, otop);
    if (now > -INFINITY)
      sum = sum * weight32(top, now, c) + osum * weight32(otop, now, c);
    better(top, at, otop, oat);
    odd |= oodd;
  }
  __device__ __forceinline__ void across_wave(float c) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
      join(__shfl_xor(sum, m, 64), __shfl_xor(top, m, 64), __shfl_xor(at, m, 64), __shfl_xor((int)odd, m, 64), c);
  }
  // a softmax exists
  __device__ __forceinline__ bool sound() const { return !odd && top > -INFINITY && top < INFINITY; }
};

// N elements at places that rise: their largest first, then the sum against it.  (Infinities
// make sums that are not numbers, but then the row is not sound.)
template <int N, class F>
__device__ __forceinline__ void add_elements(RowSum& r, const float (&x)[N], F place, float c) {
  float top = x[0];
  uint32_t at = place(0);
  bool odd = x[0] != x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) {
    odd |= x[e] != x[e];
    const bool take = x[e] > top;
    top = take ? x[e] : top;
    at = take ? place(e) : at;
  }
  float sum = 0.f;
  if (c > 0.f && top > -INFINITY)
#pragma unroll
    for (int e = 0; e < N; ++e) sum += weight32(x[e], top, c);
  r.join(sum, top, at, odd, c);
}

// How far the fp32 sum may be off, relative to it.  A weight is e^-y, y >= 0.  On its way into the
// sum it is multiplied by powers whose arguments add up to -y, each off by 3 * 2^-24 of itself (the
// difference, 1 / T, their product), at most 33 of them, each off by 2^-23; and 48 additions, 2^-24
// each, follow.  The weighted mean of y is at most ln(vocabulary) < 15.3 (the weights sum to at least
// 1).  Together less than (46 + 66 + 48) * 2^-24 < 2^-16.  (1 / T has fewer bits above T = 2^126, but
// y is less than 8 there.)
constexpr float kNear = 1.f / 65536;

// Before all: rows in the order of their index within the request, no counts, paths of row
// 0 alone.  Offsets that fall have no such order; their rows come as they are.
__global__ __launch_bounds__(kThreads) void k_verify_begin(VerifyArgs a) {
  extern __shared__ uint32_t s_cu[];  // [requests + 1]
  const uint32_t t = threadIdx.x, row = blockIdx.x * kThreads + t;
  bool falls = false;
  for (uint32_t b = t; b <= a.requests; b += kThreads) {
    s_cu[b] = (uint32_t)min(max(a.cu[b], 0), (int)a.tokens);
    falls |= b < a.requests && a.cu[b] > a.cu[b + 1];
  }
  falls = __syncthreads_or(falls);
  if (row < a.requests) {
    a.states[row].path = 1ull << 32;
    a.ends[row].mode = kDone;
    a.accepted[row] = 0;
    a.next[row] = -1;
  }
  if (row >= a.tokens) return;
  uint32_t b = 0, hi = a.requests;  // the last request that begins at or before the row
  while (hi - b > 1) {
    const uint32_t mid = (b + hi) >> 1;
    if (s_cu[mid] <= row) b = mid; else hi = mid;
  }
  const uint32_t first = s_cu[b], count = max(s_cu[b + 1], first) - first, j = row - first;
  const bool live = row >= first && j < count;
  uint32_t turn = row;
  if (!falls) {
    if (live) {
      turn = 0;
      for (uint32_t o = 0; o < a.requests; ++o) {
        const uint32_t n = s_cu[o + 1] - s_cu[o];
        turn += min(n, j) + (o < b && n > j);
      }
    } else {  // behind all of them
      turn = s_cu[a.requests] - s_cu[0] + (row < s_cu[0] ? row : s_cu[0] + row - s_cu[a.requests]);
    }
  }
  reinterpret_cast<uint64_t*>(a.order)[turn] = row | (uint64_t)(live ? b : 0xFFFFFFFFu) << 32;
  a.counters[row] = live && j == 0;
  if (live) a.path[row] = j ? -1 : 0;
}

// Up to 64 candidates for children of a path's end, a lane each: their tokens, and what is asked
// about them.
template <class L>
struct Children {
  float l = 0.f, u = 0.f, q = 1.f;
  uint32_t x = 0xFFFFFFFFu;
  static __device__ __forceinline__ uint32_t last(const VerifyArgs& a, uint32_t count, uint32_t end) {
    return a.parents ? count : min(count, end + 2);  // a chain has one child
  }
  static __device__ __forceinline__ bool is_child(const VerifyArgs& a, uint32_t first, uint32_t end, uint32_t j) {
    return a.parents ? a.parents[first + j] == (int32_t)end : j == end + 1;
  }
  // those from row j0 on; returns the lanes that are children
  __device__ __forceinline__ uint64_t load(const VerifyArgs& a, uint32_t first, uint32_t count, uint32_t end, uint32_t j0) {
    const uint64_t at = (uint64_t)first + end;
    const uint32_t j = j0 + (threadIdx.x & 63);
    const bool child = j < last(a, count, end) && is_child(a, first, end, j);
    x = child ? (uint32_t)a.draft[first + j] : 0xFFFFFFFFu;
    if (child) u = a.accept[first + j];
    if (x < a.vocab) {
      l = L::one(a.logits, at * a.logits_row + x);
      if (a.probs) q = fmaxf(a.probs[at * a.probs_row + x], 0.f);  // (a NaN counts as 0)
    }
    return __ballot(child);
  }
};

// The row's parts joined, by a wave; top, place and NaN are the same in all lanes.
__device__ __forceinline__ RowSum join_parts(const VerifyArgs& a, uint64_t at, float c) {
  RowSum row = RowSum::none();
  for (uint32_t s = threadIdx.x & 63; s < a.segs; s += 64) {
    const uint64_t* p = a.parts + 2 * (at * a.segs + s);
    const uint64_t v = get(p), w = get(p + 1);
    const float top = __uint_as_float((uint32_t)(v >> 32));
    row.join(__uint_as_float((uint32_t)v), top, (uint32_t)w, top != top, c);
  }
  row.across_wave(c);
  return row;
}

// Which child of `end` the wave's request goes to (0: none), against `left`, the row's sum, or none
// while a number lies within `near` of it (*open).  *lost: a child was refused.
template <class L>
__device__ __forceinline__ uint32_t choose_child(const VerifyArgs& a, uint32_t first, uint32_t count, uint32_t end, double c64,
                                                 const RowSum& row, Children<L>& child, uint64_t todo, double left, float near,
                                                 bool* open, bool* lost, const double* powers = kPowers) {
  const uint32_t lane = threadIdx.x & 63, last = Children<L>::last(a, count, end);
  // children in the order of their rows, 64 candidates at a time
  for (uint32_t j0 = end + 1; j0 < last && row.sound(); j0 += 64) {
    if (j0 != end + 1) todo = child.load(a, first, count, end, j0);
    const double e = child.x < a.vocab && child.l > -INFINITY ? exp2_64(((double)child.l - (double)row.top) * c64, powers) : 0.0;
    while (todo) {
      const int n = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      const uint32_t token = __shfl(child.x, n, 64), node = j0 + (uint32_t)n;
      const double weight = __shfl(e, n, 64), draw = (double)__shfl(child.u, n, 64) * (double)__shfl(child.q, n, 64);
      if (c64 > 0.0) {
        // a token that an earlier sibling had is refused already
        bool before = false;
        if (a.parents && *lost && token < a.vocab)
          for (uint32_t i = end + 1 + lane; i < node; i += 64)
            before |= Children<L>::is_child(a, first, end, i) && (uint32_t)a.draft[first + i] == token;
        if (token < a.vocab && !__any(before)) {
          // (left is without the refused tokens; with draft probabilities there is one child)
          if (fabs(draw * left - weight) < draw * near) {
            *open = true;
            return 0;
          }
          if (draw * left < weight) return node;
          left -= weight;
        }
      } else if (token == row.at) {
        return node;
      }
      *lost = true;
    }
  }
  return 0;
}

// A path's end; its next token if no more than the largest logit is asked for, or -1 if there is none.
__device__ __forceinline__ End end_path(const VerifyArgs& a, uint32_t b, uint32_t first, uint32_t end, uint32_t length, double c64,
                                        const RowSum& row, bool lost, bool writes) {
  const bool more = row.sound() && c64 > 0.0;  // the next token is still to be chosen
  if (writes) {
    a.accepted[b] = (int32_t)length;
    if (!more) a.next[b] = row.sound() ? (int32_t)row.at : -1;
  }
  return End{!more ? kDone : a.probs && lost ? kFromRest : kFromTarget, first + end, 0, 0, row.top, row.at, end, lost};
}

// The wave decides about row `end` of request b, all parts of which are there, and about
// those after it as far as theirs are.
template <class L>
__device__ __forceinline__ void decide(const VerifyArgs& a, uint32_t b, uint32_t first, uint32_t count, uint32_t end, double c64) {
  const uint32_t lane = threadIdx.x & 63;
  const float c = heat32(c64);
  uint32_t length = (uint32_t)(get(&a.states[b].path) >> 32);
  for (;;) {
    Children<L> child;
    const uint64_t todo = child.load(a, first, count, end, end + 1);  // (ahead of the sum)
    const RowSum row = join_parts(a, (uint64_t)first + end, c);
    // (the lanes' own fp32 sums differ in their last bits, as the terms come in another order)
    const float total = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(row.sum)));
    bool open = false, lost = false;
    const uint32_t go = choose_child<L>(a, first, count, end, c64, row, child, todo, total,
                                        c < 3e38f ? total * kNear : INFINITY, &open, &lost);
    if (!go) {
      if (lane == 0) {
        if (!open) {
          put(&a.states[b].path, kOver);
          a.ends[b] = end_path(a, b, first, end, length, c64, row, lost, true);
        } else {  // the state stays, so the rows below are all looked at
          a.ends[b] = End{kOpen, first + end, 0, 0, row.top, row.at, end, length};
        }
      }
      return;
    }
    end = go;
    uint32_t old = 0;
    if (lane == 0) {
      a.path[first + length] = (int32_t)end;
      put(&a.states[b].path, end | (uint64_t)(length + 1) << 32);
      __builtin_amdgcn_s_waitcnt(0);
      old = count_in(a.counters + first + end);
    }
    ++length;
    if (__builtin_amdgcn_readfirstlane(old) != a.segs) return;  // parts of it are still to come
  }
}

// One segment of one row.
template <class L>
__global__ __launch_bounds__(kThreads) void k_verify_rows(VerifyArgs a) {
  __shared__ RowSum s_part[kThreads / 64];
  __shared__ uint32_t s_passed[kThreads / 64];
  const uint32_t turn = blockIdx.x / a.segs, seg = blockIdx.x - turn * a.segs, t = threadIdx.x;
  const uint32_t row = a.order[2 * turn], b = a.order[2 * turn + 1];
  if (b >= a.requests) return;
  uint32_t first, count;
  request_rows(a.cu, b, a.tokens, &first, &count);
  const uint32_t j = row - first;
  if (j >= count) return;
  // On the way down from the path's end?  (An end that is not the latest only means that
  // less is passed by.  Each wave asks for itself while the path goes on, so some may find the
  // row passed by and others not: what one has found holds for good, and no part is left then.)
  const uint32_t end = __builtin_amdgcn_readfirstlane((uint32_t)get(&a.states[b].path));
  bool passed = j < end;
  if (end && a.parents && !passed) {
    uint32_t x = j;
    while (x > end) {
      const uint32_t up = (uint32_t)a.parents[first + x];
      x = up < x ? up : 0;  // (a link that is no tree's leads nowhere, and 0 is above the end)
    }
    passed = x < end;
  }
  const double c64 = heat(a, b);
  const float c = heat32(c64);
  RowSum r = RowSum::none();
  if (!passed) {
    float x[kEach];
    load_places<L>(a.logits, row * a.logits_row, seg, a.vocab, a.wide, -INFINITY, place<L>, x);
    add_elements(r, x, [&](uint32_t e) { return seg * kSeg + place<L>(e); }, c);
    r.across_wave(c);
  }
  if ((t & 63) == 0) {
    s_part[t >> 6] = r;
    s_passed[t >> 6] = passed;
  }
  __syncthreads();
  if (t >= 64) return;
  uint32_t old = 0;
  if (t == 0 && !(s_passed[0] | s_passed[1] | s_passed[2] | s_passed[3])) {
    for (uint32_t w = 1; w < kThreads / 64; ++w) r.join(s_part[w].sum, s_part[w].top, s_part[w].at, s_part[w].odd, c);
    uint64_t* p = a.parts + 2 * ((uint64_t)row * a.segs + seg);
    put(p, __float_as_uint(r.sum) | (uint64_t)__float_as_uint(r.odd ? NAN : r.top) << 32);
    put(p + 1, r.at);
    __builtin_amdgcn_s_waitcnt(0);
    old = count_in(a.counters + row);
  }
  if (__builtin_amdgcn_readfirstlane(old) == a.segs) decide<L>(a, b, first, count, j, c64);
}

// Exclusive running sum over the workgroup's threads in fp64.
__device__ __forceinline__ double run_before(double v, double* s_sum, double* total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double scan = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(scan, d, 64);
    if (lane >= (uint32_t)d) scan += o;
  }
  if (lane == 63) s_sum[wave] = scan;
  __syncthreads();
  double before = scan - v, all = 0.0;
#pragma unroll
  for (uint32_t w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before += s_sum[w];
    all += s_sum[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

// The first place of a segment whose running sum passes `border`, where `before` is the
// sum of all places before it; a thread holds the weights of kEach neighbours.  If rounding
// leaves none, the last place that has a weight; ~0 if no place has one.
__device__ __forceinline__ uint32_t choose(const double (&w)[kEach], double before, double border, double* s_sum, uint32_t* s_pick) {
  const uint32_t t = threadIdx.x;
  if (t == 0) s_pick[0] = 0xFFFFFFFFu, s_pick[1] = 0;
  double mine = 0.0, all;
  uint32_t last = 0;  // one past the last place with a weight
#pragma unroll
  for (uint32_t e = 0; e < kEach; ++e) {
    mine += w[e];
    if (w[e] > 0.0) last = kEach * t + e + 1;
  }
  double run = before + run_before(mine, s_sum, &all);
  if (last) atomicMax(&s_pick[1], last);
  uint32_t pick = 0xFFFFFFFFu;
#pragma unroll
  for (uint32_t e = 0; e < kEach; ++e) {
    run += w[e];
    if (w[e] > 0.0 && run > border) pick = min(pick, kEach * t + e);
  }
  if (pick != 0xFFFFFFFFu) atomicMin(&s_pick[0], pick);
  __syncthreads();
  return s_pick[0] != 0xFFFFFFFFu ? s_pick[0] : s_pick[1] - 1;
}

__device__ __forceinline__ double get_sum(const double* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The sum of all segments; v: the lane's first.
__device__ __forceinline__ double all_sums(const double* sums, uint32_t segs, double* v) {
  const uint32_t lane = threadIdx.x & 63;
  *v = lane < segs ? get_sum(sums + lane) : 0.0;
  double total = *v;
  for (uint32_t s = lane + 64; s < segs; s += 64) total += get_sum(sums + s);
  return wave_sum(total);
}

// The first segment in which the running sum passes border, by every wave for itself; v: the
// lane's first sum.  *before: the sum of those in front.  If rounding leaves none, the last
// segment that has a sum; ~0 if none has.
__device__ __forceinline__ uint32_t choose_segment(const double* sums, uint32_t segs, double v, double border, double* before) {
  const uint32_t lane = threadIdx.x & 63;
  double run = 0.0, last_before = 0.0;
  uint32_t last = 0xFFFFFFFFu;
  for (uint32_t s0 = 0; s0 < segs; s0 += 64) {
    if (s0) v = s0 + lane < segs ? get_sum(sums + s0 + lane) : 0.0;
    double scan = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(scan, d, 64);
      if (lane >= (uint32_t)d) scan += o;
    }
    scan += run;
    const uint64_t hit = __ballot(v > 0.0 && scan > border), some = __ballot(v > 0.0);
    const int at = hit ? __ffsll((unsigned long long)hit) - 1 : some ? 63 - __clzll((long long)some) : -1;
    if (at >= 0) {
      last = s0 + (uint32_t)at;
      const double up = __shfl(scan, at > 0 ? at - 1 : 0, 64);
      last_before = at > 0 ? up : run;
    }
    if (hit) break;
    run = __shfl(scan, 63, 64);
  }
  *before = last_before;
  return last;
}

// A segment's sum for the request's last workgroup: true, for all threads, in that one.
__device__ __forceinline__ bool put_sum(double* sums, uint32_t own, uint32_t segs, double v, uint32_t* counter, uint32_t* s_last) {
  if (threadIdx.x == 0) {
    __hip_atomic_store(sums + own, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);
    *s_last = count_in(counter) == segs - 1;
  }
  __syncthreads();
  return *s_last != 0;
}

// The next token by the segments' sums and the weights of one of them.  Where rounding has
// left nothing, the target's most likely token.
template <class F>
__device__ __forceinline__ void choose_next(const VerifyArgs& a, uint32_t b, const End& end, const double* sums, F weights,
                                            double* s_sum, uint32_t* s_pick) {
  double first, before;
  const double border = all_sums(sums, a.segs, &first) * (double)a.sample[b];
  const uint32_t seg = choose_segment(sums, a.segs, first, border, &before);
  uint32_t next = end.at;
  if (seg != 0xFFFFFFFFu) {
    double w[kEach];
    weights(seg, [](uint32_t e) { return kEach * threadIdx.x + e; }, w);
    const uint32_t pick = choose(w, before, border, s_sum, s_pick);
    if (pick != 0xFFFFFFFFu) next = seg * kSeg + pick;
  }
  if (threadIdx.x == 0) a.next[b] = (int32_t)next;
}

// exp((l - top) / T) at the thread's places of a segment of a path's last row.
template <class L, class F>
__device__ __forceinline__ void exponentials(const VerifyArgs& a, const End& end, double c, uint32_t seg, F at, double (&w)[kEach]) {
  float x[kEach];
  load_places<L>(a.logits, end.row * a.logits_row, seg, a.vocab, a.wide, -INFINITY, at, x);
#pragma unroll
  for (uint32_t e = 0; e < kEach; e += 8) {
    double z[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) z[i] = ((double)x[e + i] - (double)end.top) * c;
    exp2_64<8>(z);
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) w[e + i] = x[e + i] > -INFINITY ? z[i] : 0.0;
  }
}

__device__ __forceinline__ double sum_of(const double (&w)[kEach], double* s_sum) {  // to all threads
  double mine = 0.0, all;
#pragma unroll
  for (uint32_t e = 0; e < kEach; ++e) mine += w[e];
  run_before(mine, s_sum, &all);
  return all;
}

// max(p - q, 0): a workgroup a segment, and the last chooses.  inv: 1 / the row's sum.
template <class L>
__device__ __forceinline__ void choose_rest(const VerifyArgs& a, uint32_t b, uint32_t own, const End& end, double c, double inv,
                                            double* s_sum, uint32_t* s_pick, uint32_t* s_last) {
  auto weights = [&](uint32_t seg, auto at, double (&w)[kEach]) {
    float q[kEach];
    exponentials<L>(a, end, c, seg, at, w);
    load_places<Logit<F32>>(a.probs, end.row * a.probs_row, seg, a.vocab, a.probs_wide, 0.f, at, q);
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e) w[e] = fmax(w[e] * inv - (double)fmaxf(q[e], 0.f), 0.0);
  };
  double w[kEach];
  weights(own, place<L>, w);
  double* rest = a.rest + (uint64_t)b * a.segs;
  if (put_sum(rest, own, a.segs, sum_of(w, s_sum), &a.ends[b].rest_counter, s_last))
    choose_next(a, b, end, rest, weights, s_sum, s_pick);
}

// A path that was left open, to its end, by every workgroup of its request for itself (one writes):
// all rows that it may come to have their parts by now.  (Here and not on the spot: the fp64 sum
// in k_verify_rows takes 101 registers where 71 do, and of 96 chains 114.8 us for 109.6, of 64 trees
// 102.5 for 97.)
template <class L>
__device__ __forceinline__ End finish_path(const VerifyArgs& a, uint32_t b, const End& open, double c64, bool writes, double* s_sum) {
  uint32_t first, count, end = open.end, length = open.lost;
  request_rows(a.cu, b, a.tokens, &first, &count);
  for (;;) {
    const RowSum row = join_parts(a, (uint64_t)first + end, heat32(c64));
    const double* powers = kPowers;  // (read here: constants that stand ready for all loops hold 18 registers)
    asm volatile("" : "+s"(powers));
    double mine = 0.0, all = 0.0;
    if (row.sound()) {
#pragma unroll 1
      for (uint32_t v0 = threadIdx.x; v0 < a.vocab; v0 += 4 * kThreads) {
        double z[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const uint32_t v = v0 + i * kThreads;
          const float x = v < a.vocab ? L::one(a.logits, (first + end) * a.logits_row + v) : -INFINITY;
          z[i] = x > -INFINITY ? ((double)x - (double)row.top) * c64 : -INFINITY;  // (2^-1000 is nothing beside 1)
        }
        exp2_64<4>(z, powers);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) mine += z[i];
      }
      run_before(mine, s_sum, &all);
    }
    Children<L> child;
    bool never = false, lost = false;
    const uint64_t todo = child.load(a, first, count, end, end + 1);
    const uint32_t go = choose_child<L>(a, first, count, end, c64, row, child, todo, all, 0.f, &never, &lost, powers);
    if (!go) {
      End done = end_path(a, b, first, end, length, c64, row, lost, writes);
      uint32_t* words = reinterpret_cast<uint32_t*>(&done);  // (the same in all lanes: no vector registers for them)
#pragma unroll
      for (uint32_t i = 0; i < sizeof(End) / 4; ++i) words[i] = __builtin_amdgcn_readfirstlane(words[i]);
      return done;
    }
    end = __builtin_amdgcn_readfirstlane(go);
    if (writes) a.path[first + length] = (int32_t)end;
    ++length;
  }
}

// Up to this many segments every workgroup adds up a whole row itself sooner than a launch
// more would give its sum.  The call, so and with the launch, for chains of up to 5 with draft
// probabilities, us: 24 requests at 2 segments 40 and 50, at 4 42 and 50, at 6 48 and 53, at 8 49 and
// 51, at 12 55 and 52, at 16 56 and 53; 96 requests at 4 51 and 58, at 6 58 and 58, at 8 66 and 63, at
// 12 81 and 65; one request at 8 36 and 33.
constexpr uint32_t kFew = 8;

// Weights of a path's last row, a workgroup a segment; where they are p without the refused
// tokens, the last workgroup chooses.
template <class L>
__global__ __launch_bounds__(kThreads, 4) void k_verify_next(VerifyArgs a) {
  __shared__ double s_sum[kThreads / 64];
  __shared__ uint32_t s_gone[kSeg / 32];  // a bit for each refused token of a segment
  __shared__ uint32_t s_pick[2], s_last;
  const uint32_t b = blockIdx.x / a.segs, own = blockIdx.x - b * a.segs, t = threadIdx.x;
  End end = a.ends[b];
  if (end.mode == kDone) return;
  const double c = heat(a, b);
  if (end.mode == kOpen) {
    end = finish_path<L>(a, b, end, c, own == 0 && t == 0, s_sum);
    if (own == 0 && t == 0) a.ends[a.requests + b] = end;
    if (end.mode == kDone) return;
  }
  double w[kEach];
  if (end.mode == kFromRest && a.segs <= kFew) {
    double mine = 0.0, all;
#pragma unroll 2
    for (uint32_t seg = 0; seg < a.segs; ++seg) {
      exponentials<L>(a, end, c, seg, place<L>, w);
#pragma unroll
      for (uint32_t e = 0; e < kEach; ++e) mine += w[e];
    }
    run_before(mine, s_sum, &all);
    choose_rest<L>(a, b, own, end, c, 1.0 / all, s_sum, s_pick, &s_last);
    return;
  }
  const bool fewer = end.mode == kFromTarget && end.lost;
  auto weights = [&](uint32_t seg, auto at, double (&w)[kEach]) {
    exponentials<L>(a, end, c, seg, at, w);
    if (!fewer) return;
    uint32_t first, count;
    request_rows(a.cu, b, a.tokens, &first, &count);
    __syncthreads();
    for (uint32_t i = t; i < kSeg / 32; i += kThreads) s_gone[i] = 0;
    __syncthreads();
    for (uint32_t j = end.end + 1 + t; j < count; j += kThreads)
      if (a.parents ? a.parents[first + j] == (int32_t)end.end : j == end.end + 1) {
        const uint32_t token = (uint32_t)a.draft[first + j];
        if (token < a.vocab && token / kSeg == seg) atomicOr(&s_gone[token % kSeg / 32], 1u << token % 32);
      }
    __syncthreads();
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e)
      if (s_gone[at(e) / 32] >> at(e) % 32 & 1) w[e] = 0.0;
  };
  weights(own, place<L>, w);
  double* sums = a.sums + (uint64_t)b * a.segs;
  if (put_sum(sums, own, a.segs, sum_of(w, s_sum), &a.ends[b].counter, &s_last) && end.mode == kFromTarget)
    choose_next(a, b, end, sums, weights, s_sum, s_pick);
}

template <class L>
__global__ __launch_bounds__(kThreads) void k_verify_rest(VerifyArgs a) {
  __shared__ double s_sum[kThreads / 64];
  __shared__ uint32_t s_pick[2], s_last;
  const uint32_t b = blockIdx.x / a.segs, own = blockIdx.x - b * a.segs;
  End end = a.ends[b];
  if (end.mode == kOpen) end = a.ends[a.requests + b];
  if (end.mode != kFromRest) return;
  double first;
  const double all = all_sums(a.sums + (uint64_t)b * a.segs, a.segs, &first);
  choose_rest<L>(a, b, own, end, heat(a, b), 1.0 / all, s_sum, s_pick, &s_last);
}

struct VerifyPlan {
  uint32_t segs;
  size_t order_off, counters_off, states_off, sums_off, rest_off, ends_off, bytes;
};

VerifyPlan plan_verify(uint32_t tokens, uint32_t vocab, uint32_t requests) {
  VerifyPlan p;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.segs = (vocab + kSeg - 1) / kSeg;
  take((size_t)tokens * p.segs * 16);  // parts
  p.order_off = take((size_t)tokens * 8);
  p.counters_off = take((size_t)tokens * 4);
  p.states_off = take((size_t)requests * sizeof(State));
  p.sums_off = take((size_t)requests * p.segs * 8);
  p.rest_off = take((size_t)requests * p.segs * 8);
  p.ends_off = take((size_t)requests * 2 * sizeof(End));
  p.bytes = std::max<size_t>(at, 256);
  return p;
}

constexpr uint32_t kMaxVocab = 1u << 22;
bool verify_shape_ok(uint32_t tokens, uint32_t vocab, uint32_t requests) {
  return vocab >= 1 && vocab <= kMaxVocab && requests <= kMaxRequests && tokens <= (1u << 20) &&
         (uint64_t)tokens * ((vocab + kSeg - 1) / kSeg) <= kMaxGroups;
}

template <class L>
int launch_verify(const VerifyArgs& a, hipStream_t st) {
  const uint32_t lds = (a.requests + 1) * 4;  // 32 KB at most
  hipLaunchKernelGGL(k_verify_begin, dim3((std::max(a.tokens, a.requests) + kThreads - 1) / kThreads), dim3(kThreads), lds, st, a);
  if (int rc = launched()) return rc;
  if (a.tokens == 0) return DGT_OK;
  hipLaunchKernelGGL(k_verify_rows<L>, dim3(a.tokens * a.segs), dim3(kThreads), 0, st, a);
  if (int rc = launched()) return rc;
  hipLaunchKernelGGL(k_verify_next<L>, dim3(a.requests * a.segs), dim3(kThreads), 0, st, a);
  if (int rc = launched()) return rc;
  if (!a.probs || a.segs <= kFew) return DGT_OK;
  hipLaunchKernelGGL(k_verify_rest<L>, dim3(a.requests * a.segs), dim3(kThreads), 0, st, a);
  return launched();
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" {

size_t dgt_verify_workspace(uint32_t tokens, uint32_t vocab, uint32_t requests) {
  return verify_shape_ok(tokens, vocab, requests) ? plan_verify(tokens, vocab, requests).bytes : 0;
}

int dgt_verify(uint32_t type, const void* d_logits, uint64_t logits_row, const int32_t* d_draft,
               const float* d_probs, uint64_t probs_row, const int32_t* d_parents, const int32_t* d_cu,
               const float* d_temperature, const float* d_accept, const float* d_sample,
               uint32_t requests, uint32_t tokens, uint32_t vocab, int32_t* d_path,
               int32_t* d_accepted, int32_t* d_next, void* d_ws, size_t ws_bytes, void* stream) {
  if (type != DGT_ELT_F32 && type != DGT_ELT_BF16 && type != DGT_ELT_F16) return DGT_E_UNSUPPORTED;
  if (d_probs && d_parents) return DGT_E_UNSUPPORTED;
  if (!verify_shape_ok(tokens, vocab, requests)) return DGT_E_SHAPE;
  if (tokens > 1 && (logits_row < vocab || (d_probs && probs_row < vocab))) return DGT_E_SHAPE;
  if (requests == 0) return DGT_OK;
  if (!d_cu || !d_accepted || !d_next || !d_sample) return DGT_E_ARG;
  if (tokens && (!d_logits || !d_draft || !d_accept || !d_path)) return DGT_E_ARG;
  if (!d_ws || !aligned(d_ws, 16)) return DGT_E_ARG;
  const VerifyPlan p = plan_verify(tokens, vocab, requests);
  if (ws_bytes < p.bytes) return DGT_E_BUFSIZE;
  if (tokens <= 1) logits_row = probs_row = 0;  // a single row has no stride
  VerifyArgs a;
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  a.logits = d_logits;
  a.probs = d_probs;
  a.temperature = d_temperature;
  a.accept = d_accept;
  a.sample = d_sample;
  a.draft = d_draft;
  a.parents = d_parents;
  a.cu = d_cu;
  a.path = d_path;
  a.accepted = d_accepted;
  a.next = d_next;
  a.parts = reinterpret_cast<uint64_t*>(ws);
  a.order = reinterpret_cast<uint32_t*>(ws + p.order_off);
  a.counters = reinterpret_cast<uint32_t*>(ws + p.counters_off);
  a.states = reinterpret_cast<State*>(ws + p.states_off);
  a.sums = reinterpret_cast<double*>(ws + p.sums_off);
  a.rest = reinterpret_cast<double*>(ws + p.rest_off);
  a.ends = reinterpret_cast<End*>(ws + p.ends_off);
  a.logits_row = logits_row;
  a.probs_row = probs_row;
  a.requests = requests;
  a.tokens = tokens;
  a.vocab = vocab;
  a.segs = p.segs;
  a.wide = aligned(d_logits, 16) && logits_row % (type == DGT_ELT_F32 ? 4 : 8) == 0;
  a.probs_wide = aligned(d_probs, 16) && probs_row % 4 == 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  switch (type) {
    case DGT_ELT_F32: return launch_verify<Logit<F32>>(a, st);
    case DGT_ELT_BF16: return launch_verify<Logit<Bf16>>(a, st);
  }
  return launch_verify<Logit<F16>>(a, st);
}

}  // extern "C"
