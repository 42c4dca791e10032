// Verification of drafted tokens against the target's logits.
#include "dgt_serve.h"

#include <algorithm>

namespace dgt {
namespace serve {
namespace {

struct VerifyArgs {
  const void* logits;
  const float *probs, *temperature, *accept, *sample;
  const int32_t *draft, *parents, *cu;
  int32_t *path, *accepted, *next;
  struct Part* parts;       // [tokens][segs]
  double* rest;             // [requests][segs], sums of max(p - q, 0)
  struct End* ends;         // [requests]
  uint64_t logits_row, probs_row;
  uint32_t requests, tokens, vocab, segs;
  bool wide, probs_wide;    // rows are 16-byte aligned
};

// A row's vocabulary in segments; a segment of a row is what one workgroup looks at.
constexpr uint32_t kSeg = 4096, kThreads = 256, kEach = kSeg / kThreads;

struct Part {  // of a segment
  double sum;  // of exp((l - top) / T)
  float top;   // the largest logit; NaN if there is a NaN
  uint32_t at; // its place, the first of equals (within the vocabulary)
};

struct End {  // of a path whose next token comes from max(p - q, 0)
  double sum;      // of exp((l - top) / T) over the row
  float top;
  uint32_t row, counter;  // row: ~0 where there is nothing to do
};

// 2^z for z <= 0 in fp64: the Taylor series of 2^f on |f| <= 1/2 ends below 2^-37.  A
// uniform number falls between two of a vocabulary's running sums, which lie 1 / vocab
// apart: sums of fp32 exponentials, off by 2^-24, would give another token in one of a
// hundred calls.  Far values are cut at 2^-1100, which is zero.
__device__ __forceinline__ double exp2_64(double z) {
  z = fmax(z, -1100.0);
  const double n = __builtin_rint(z), f = z - n;
  double p = 1.01780860092396997e-7;  // ln(2)^k / k!
  p = fma(p, f, 1.32154867901443095e-6);
  p = fma(p, f, 1.52527338040598403e-5);
  p = fma(p, f, 1.54035303933816099e-4);
  p = fma(p, f, 1.33335581464284434e-3);
  p = fma(p, f, 9.61812910762847716e-3);
  p = fma(p, f, 5.55041086648215800e-2);
  p = fma(p, f, 2.40226506959100712e-1);
  p = fma(p, f, 6.93147180559945309e-1);
  p = fma(p, f, 1.0);
  return __builtin_ldexp(p, (int)n);
}

constexpr double kLog2e = 1.44269504088896340736;
// What logits are multiplied by: 1 / T in powers of two, or 0 for the largest logit's token.
__device__ __forceinline__ double heat(const VerifyArgs& a, uint32_t b) {
  const float t = a.temperature ? a.temperature[b] : 1.f;
  return t > 0.f ? kLog2e / (double)t : 0.0;
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

// A segment's elements of a row; past the vocabulary's end -inf.
template <class L>
__device__ __forceinline__ void load_segment(const void* base, uint64_t row, uint32_t seg, uint32_t vocab, bool wide,
                                             float (&x)[kEach]) {
  const typename L::T* p = static_cast<const typename L::T*>(base) + row + (uint64_t)seg * kSeg;
  const uint32_t left = vocab - seg * kSeg;
  if (wide && left >= kSeg) {
#pragma unroll
    for (uint32_t e = 0; e < kEach; e += L::kPiece) L::piece(p + place<L>(e), x + e);
  } else {
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e) x[e] = place<L>(e) < left ? L::one(p, place<L>(e)) : -INFINITY;
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

// Largest logit, its place and the sum of exponentials of a segment, to every thread.
template <class L>
__device__ __forceinline__ Part segment_part(const float (&x)[kEach], uint32_t seg, double c, float* s_top, uint32_t* s_at,
                                             double* s_sum) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float top = -INFINITY;
  uint32_t at = 0xFFFFFFFFu;
  bool odd = false;
#pragma unroll
  for (uint32_t e = 0; e < kEach; ++e) {
    odd |= x[e] != x[e];
    const bool take = x[e] > top || at == 0xFFFFFFFFu;  // places rise with e
    top = take ? x[e] : top;
    at = take ? seg * kSeg + place<L>(e) : at;
  }
  top = odd ? -INFINITY : top;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) better(top, at, __shfl_xor(top, m, 64), __shfl_xor(at, m, 64));
  odd = __any(odd);
  if (lane == 0) {
    s_top[wave] = odd ? NAN : top;
    s_at[wave] = at;
  }
  __syncthreads();
  top = s_top[0];
  at = s_at[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    odd |= s_top[w] != s_top[w];
    better(top, at, s_top[w], s_at[w]);
  }
  odd |= s_top[0] != s_top[0];
  double sum = 0.0;
  if (c > 0.0 && top > -INFINITY && !odd) {
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e) sum += exp2_64(((double)x[e] - (double)top) * c);
  }
  sum = wave_sum(sum);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  return Part{(s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]), odd ? NAN : top, at};
}

// The request of a row: the last that begins at or before it.
__device__ __forceinline__ uint32_t row_request(const VerifyArgs& a, uint32_t row) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t lo = 0, len = a.requests;
  while (len > 1) {
    const uint32_t step = (len + 63) / 64, at = lane * step;
    const bool before = lane == 0 || (at < len && (uint32_t)max(a.cu[lo + at], 0) <= row);
    const uint32_t hits = (uint32_t)__popcll(__ballot(before));
    const uint32_t skip = (hits - 1) * step;
    lo += skip;
    len = min(step, len - skip);
  }
  return lo;
}

// Every segment of every row.
template <class L>
__global__ __launch_bounds__(kThreads) void k_verify_parts(VerifyArgs a) {
  __shared__ float s_top[4];
  __shared__ uint32_t s_at[4];
  __shared__ double s_sum[4];
  const uint32_t row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
  float x[kEach];
  load_segment<L>(a.logits, row * a.logits_row, seg, a.vocab, a.wide, x);
  const uint32_t b = row_request(a, row);
  uint32_t first, count;
  request_rows(a.cu, b, a.tokens, &first, &count);
  if (row - first >= count) return;  // of no request
  const Part p = segment_part<L>(x, seg, heat(a, b), s_top, s_at, s_sum);
  if (threadIdx.x == 0) a.parts[(uint64_t)row * a.segs + seg] = p;
}

struct RowSum {
  double sum;
  float top;
  uint32_t at;
  bool sound;
};

// A row's parts together, by each wave for itself.
__device__ __forceinline__ RowSum join_row(const Part* parts, uint32_t segs, double c) {
  const uint32_t lane = threadIdx.x & 63;
  float top = -INFINITY;
  uint32_t at = 0xFFFFFFFFu;
  bool odd = false;
  for (uint32_t s = lane; s < segs; s += 64) {
    odd |= parts[s].top != parts[s].top;
    better(top, at, parts[s].top, parts[s].at);
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) better(top, at, __shfl_xor(top, m, 64), __shfl_xor(at, m, 64));
  odd = __any(odd) || !(top > -INFINITY && top < INFINITY);
  double sum = 0.0;
  if (!odd && c > 0.0)
    for (uint32_t s = lane; s < segs; s += 64)
      if (parts[s].sum > 0.0) sum += parts[s].sum * exp2_64(((double)parts[s].top - (double)top) * c);
  return RowSum{wave_sum(sum), top, at, !odd};
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
  // (scan - v is exact enough for choosing a thread, which then adds for itself)
#pragma unroll
  for (uint32_t w = 0; w < kThreads / 64; ++w) {
    if (w < wave) before += s_sum[w];
    all += s_sum[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

// The first place whose running sum passes `border`, where `before` is the sum of all
// places before the segment; w holds the segment's weights, kSeg of them.  If rounding
// leaves none, the last place that has a weight; ~0 if no place has one.
__device__ __forceinline__ uint32_t choose(const double* w, double before, double border, double* s_sum, uint32_t* s_pick) {
  const uint32_t t = threadIdx.x;
  if (t == 0) s_pick[0] = 0xFFFFFFFFu, s_pick[1] = 0;
  double mine = 0.0, all;
  uint32_t last = 0;  // one past the last place with a weight
  for (uint32_t e = 0; e < kEach; ++e) {
    const double v = w[kEach * t + e];
    mine += v;
    if (v > 0.0) last = kEach * t + e + 1;
  }
  double run = before + run_before(mine, s_sum, &all);
  if (last) atomicMax(&s_pick[1], last);
  for (uint32_t e = 0; e < kEach && last; ++e) {
    const double v = w[kEach * t + e];
    run += v;
    if (v > 0.0 && run > border) {
      atomicMin(&s_pick[0], kEach * t + e);
      break;
    }
  }
  __syncthreads();
  const uint32_t pick = s_pick[0], end = s_pick[1];
  __syncthreads();
  return pick != 0xFFFFFFFFu ? pick : end - 1;
}

// The first segment in which the running sum passes border, by every wave for itself;
// sum(s) is its sum.  *before: the sum of those in front.  If rounding leaves none, the
// last segment that has a sum; ~0 if none has.
template <class F>
__device__ __forceinline__ uint32_t choose_segment(uint32_t segs, double border, F sum, double* before) {
  const uint32_t lane = threadIdx.x & 63;
  double run = 0.0;
  uint32_t last = 0xFFFFFFFFu;
  double last_before = 0.0;
  for (uint32_t s0 = 0; s0 < segs; s0 += 64) {
    const double v = s0 + lane < segs ? sum(s0 + lane) : 0.0;
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

// One workgroup a request: the way down the tree (each wave for itself, all alike: a step
// is a few loads), and the next token where it comes from p.
template <class L>
__global__ __launch_bounds__(kThreads) void k_verify_walk(VerifyArgs a) {
  extern __shared__ double s_w[];      // [kSeg] weights of a segment, then [segs] sums
  double* s_seg = s_w + kSeg;
  __shared__ double s_sum[4];
  __shared__ uint32_t s_pick[2];
  const uint32_t b = blockIdx.x, t = threadIdx.x, lane = t & 63;
  uint32_t first, count;
  request_rows(a.cu, b, a.tokens, &first, &count);
  if (a.probs && t == 0) {
    a.ends[b].row = 0xFFFFFFFFu;
    a.ends[b].counter = 0;
  }
  if (count == 0) {
    if (t == 0) {
      a.accepted[b] = 0;
      a.next[b] = -1;
    }
    return;
  }
  const double c = heat(a, b);
  uint32_t end = 0, length = 1;
  int32_t next = -1;
  bool lost = false;  // a child of the end was refused
  RowSum row;
  if (t == 0) a.path[first] = 0;
  for (;;) {
    const uint64_t at = (uint64_t)first + end;
    row = join_row(a.parts + at * a.segs, a.segs, c);
    lost = false;
    if (!row.sound) break;
    auto logit = [&](uint32_t v) { return L::one(a.logits, at * a.logits_row + v); };
    uint32_t go = 0;
    double left = row.sum;  // of the row's sum, without the refused tokens
    // children in the order of their rows, 64 candidates at a time
    for (uint32_t j0 = end + 1; j0 < count && !go; j0 += 64) {
      const uint32_t j = j0 + lane;
      bool child = j < count && (a.parents ? a.parents[first + j] == (int32_t)end : j == end + 1);
      uint64_t todo = __ballot(child);
      if (!a.parents) j0 = count;  // a chain has one
      if (!todo) continue;
      // each lane prepares its own candidate
      uint32_t x = 0xFFFFFFFFu;
      double e = 0.0, u = 0.0;
      if (child) {
        x = (uint32_t)a.draft[first + j];
        u = a.accept[first + j];
        if (x < a.vocab) {
          if (c > 0.0) e = exp2_64(((double)logit(x) - (double)row.top) * c);
          if (a.probs) u *= fmax(a.probs[at * a.probs_row + x], 0.f);  // (a NaN counts as 0)
        }
      }
      while (todo) {
        const int n = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        const uint32_t token = __shfl(x, n, 64), node = (uint32_t)__shfl((int)j, n, 64);
        const double weight = __shfl(e, n, 64), draw = __shfl(u, n, 64);
        bool taken;
        if (c > 0.0) {
          // a token that an earlier sibling had is refused already
          bool before = false;
          if (a.parents && token < a.vocab)
            for (uint32_t i = end + 1 + lane; i < node; i += 64)
              before |= a.parents[first + i] == (int32_t)end && (uint32_t)a.draft[first + i] == token;
          const bool again = __any(before);
          taken = token < a.vocab && !again && draw * (a.probs ? row.sum : left) < weight;
          if (!taken && token < a.vocab && !again) left -= weight;
        } else {
          taken = token == row.at;
        }
        if (taken) {
          go = node;
          break;
        }
        lost = true;
      }
    }
    if (!go) break;
    end = go;
    if (t == 0) a.path[first + length] = (int32_t)end;
    ++length;
  }
  for (uint32_t i = length + t; i < count; i += kThreads) a.path[first + i] = -1;

  const uint64_t at = (uint64_t)first + end;
  if (row.sound && c == 0.0) {
    next = (int32_t)row.at;
  } else if (row.sound && a.probs && lost) {
    if (t == 0) {
      a.ends[b].sum = row.sum;
      a.ends[b].top = row.top;
      a.ends[b].row = (uint32_t)at;
    }
  } else if (row.sound) {
    // p without the refused tokens: their segments are added up again without them
    const Part* parts = a.parts + at * a.segs;
    for (uint32_t s = t; s < a.segs; s += kThreads)
      s_seg[s] = parts[s].sum > 0.0 ? parts[s].sum * exp2_64(((double)parts[s].top - (double)row.top) * c) : 0.0;
    __syncthreads();
    auto weights = [&](uint32_t seg) {  // of a segment, into s_w; returns this thread's sum
      float x[kEach];
      load_segment<L>(a.logits, at * a.logits_row, seg, a.vocab, a.wide, x);
      for (uint32_t e = 0; e < kEach; ++e)
        s_w[place<L>(e)] = x[e] > -INFINITY ? exp2_64(((double)x[e] - (double)row.top) * c) : 0.0;
      __syncthreads();
      if (lost)
        for (uint32_t j = end + 1 + t; j < count; j += kThreads)
          if (a.parents ? a.parents[first + j] == (int32_t)end : j == end + 1) {
            const uint32_t x = (uint32_t)a.draft[first + j];
            if (x < a.vocab && x / kSeg == seg) s_w[x % kSeg] = 0.0;
          }
      __syncthreads();
    };
    if (lost) {
      for (uint32_t j = end + 1; j < count; ++j) {
        if (a.parents ? a.parents[first + j] != (int32_t)end : j != end + 1) continue;
        const uint32_t x = (uint32_t)a.draft[first + j];
        if (x >= a.vocab) continue;
        weights(x / kSeg);
        double mine = 0.0, all;
        for (uint32_t e = 0; e < kEach; ++e) mine += s_w[t + e * kThreads];
        run_before(mine, s_sum, &all);
        if (t == 0) s_seg[x / kSeg] = all;
        __syncthreads();
      }
    }
    double total = 0.0, before;
    for (uint32_t s = lane; s < a.segs; s += 64) total += s_seg[s];
    total = wave_sum(total);
    const double border = (double)a.sample[b] * total;
    const uint32_t seg = choose_segment(a.segs, border, [&](uint32_t s) { return s_seg[s]; }, &before);
    next = (int32_t)row.at;  // where nothing is left
    if (seg != 0xFFFFFFFFu) {
      weights(seg);
      const uint32_t pick = choose(s_w, before, border, s_sum, s_pick);
      if (pick != 0xFFFFFFFFu) next = (int32_t)(seg * kSeg + pick);
    }
  }
  if (t == 0) {
    a.accepted[b] = (int32_t)length;
    a.next[b] = next;
  }
}

// Where a chain was refused: sums of max(p - q, 0) by segment, and the last segment's
// workgroup of a request chooses.
template <class L>
__global__ __launch_bounds__(kThreads) void k_verify_rest(VerifyArgs a) {
  __shared__ double s_w[kSeg];
  __shared__ double s_sum[4];
  __shared__ uint32_t s_pick[2], s_last;
  const uint32_t b = blockIdx.x / a.segs, own = blockIdx.x - b * a.segs, t = threadIdx.x, lane = t & 63;
  const End end = a.ends[b];
  if (end.row == 0xFFFFFFFFu) return;
  const double c = heat(a, b), inv = 1.0 / end.sum;
  auto weights = [&](uint32_t seg) {
    float x[kEach], q[kEach];
    load_segment<L>(a.logits, end.row * a.logits_row, seg, a.vocab, a.wide, x);
    // (places differ with the size of the logits, so the draft's are met in the logits' order)
    const float* p = a.probs + end.row * a.probs_row + (uint64_t)seg * kSeg;
    const uint32_t left = a.vocab - seg * kSeg;
    if (a.probs_wide && left >= kSeg) {
#pragma unroll
      for (uint32_t e = 0; e < kEach; e += 4) {
        const floatx4 v = *reinterpret_cast<const floatx4*>(p + place<L>(e));
#pragma unroll
        for (int j = 0; j < 4; ++j) q[e + j] = v[j];
      }
    } else {
#pragma unroll
      for (uint32_t e = 0; e < kEach; ++e) q[e] = place<L>(e) < left ? p[place<L>(e)] : 0.f;
    }
    double mine = 0.0;
#pragma unroll
    for (uint32_t e = 0; e < kEach; ++e) {
      const double w = fmax((x[e] > -INFINITY ? exp2_64(((double)x[e] - (double)end.top) * c) * inv : 0.0) - (double)fmaxf(q[e], 0.f), 0.0);
      s_w[place<L>(e)] = w;
      mine += w;
    }
    return mine;
  };
  double all;
  run_before(weights(own), s_sum, &all);
  // Sums pass between workgroups that may sit on different dies: agent-scope accesses, and a
  // wait for the store before the count.
  double* rest = a.rest + (uint64_t)b * a.segs;
  if (t == 0) {
    __hip_atomic_store(rest + own, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_s_waitcnt(0);
    s_last = __hip_atomic_fetch_add(&a.ends[b].counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.segs - 1;
  }
  __syncthreads();
  if (!s_last) return;
  auto sum = [&](uint32_t s) { return __hip_atomic_load(rest + s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  double total = 0.0, before;
  for (uint32_t s = lane; s < a.segs; s += 64) total += sum(s);
  total = wave_sum(total);
  const double border = (double)a.sample[b] * total;
  const uint32_t seg = choose_segment(a.segs, border, sum, &before);
  int32_t next;
  if (seg == 0xFFFFFFFFu) {  // rounding has left nothing: the target's most likely token
    next = (int32_t)join_row(a.parts + (uint64_t)end.row * a.segs, a.segs, c).at;
  } else {
    __syncthreads();
    weights(seg);
    __syncthreads();
    next = (int32_t)(seg * kSeg + choose(s_w, before, border, s_sum, s_pick));
  }
  if (t == 0) a.next[b] = next;
}

struct VerifyPlan {
  uint32_t segs;
  size_t rest_off, ends_off, bytes;
};

VerifyPlan plan_verify(uint32_t tokens, uint32_t vocab, uint32_t requests) {
  VerifyPlan p;
  p.segs = (vocab + kSeg - 1) / kSeg;
  p.rest_off = (size_t)tokens * p.segs * sizeof(Part);
  p.ends_off = p.rest_off + (size_t)requests * p.segs * sizeof(double);
  p.bytes = p.ends_off + (size_t)requests * sizeof(End) + 256;
  return p;
}

constexpr uint32_t kMaxVocab = 1u << 22;
bool verify_shape_ok(uint32_t tokens, uint32_t vocab, uint32_t requests) {
  return vocab >= 1 && vocab <= kMaxVocab && requests <= kMaxRequests && tokens <= (1u << 20) &&
         (uint64_t)tokens * ((vocab + kSeg - 1) / kSeg) <= 0x7FFFFFFFull;
}

template <class L>
int launch_verify(const VerifyArgs& a, hipStream_t st) {
  const uint32_t lds = (kSeg + a.segs) * 8;  // 40 KB at most
  if (a.tokens) {
    hipLaunchKernelGGL(k_verify_parts<L>, dim3(a.tokens * a.segs), dim3(kThreads), 0, st, a);
    if (int rc = launched()) return rc;
  }
  hipLaunchKernelGGL(k_verify_walk<L>, dim3(a.requests), dim3(kThreads), lds, st, a);
  if (int rc = launched()) return rc;
  if (!a.probs || a.tokens == 0) return DGT_OK;
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
  a.parts = reinterpret_cast<Part*>(ws);
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
