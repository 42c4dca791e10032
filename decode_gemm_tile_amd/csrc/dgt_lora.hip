// Low-rank adapters of many requests beside a shared projection:
// out[t] = y[t] + s_a * (x[t] A_a^T) B_a^T for the adapter a of t's request.
#include "dgt_serve.h"

#include <algorithm>

namespace dgt {
namespace serve {
namespace {

struct LoraArgs {
  const float* y;
  const uint16_t *x, *a, *b;
  const float* scaling;
  const int32_t *adapters, *cu;
  float *out, *part;
  uint64_t x_row, y_row, out_row;  // element strides
  uint32_t tokens, requests, count, n, k, rank;
  uint32_t splits, split_k;        // pieces of K and their length (a multiple of a stage)
  uint32_t block_n;                // columns of out a workgroup of the second kernel takes
  bool wide_y;                     // rows of y and out are 16-byte aligned
};

// Four consecutive columns of a row, as one access where rows are 16-byte aligned
// (`wide`); columns from n1 on are left alone.
__device__ __forceinline__ floatx4 load4(const float* row, uint32_t n, uint32_t n1, bool wide) {
  if (wide && n + 4 <= n1) return *reinterpret_cast<const floatx4*>(row + n);
  floatx4 v = {};
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    if (n + j < n1) v[j] = row[n + j];
  return v;
}
__device__ __forceinline__ void store4(float* row, uint32_t n, uint32_t n1, bool wide, floatx4 v) {
  if (wide && n + 4 <= n1) {
    *reinterpret_cast<floatx4*>(row + n) = v;
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    if (n + j < n1) row[n + j] = v[j];
}

// ------------------------------------------------------------------- shrink
// part[piece][t][r] = sum over the piece of K of x[t][k] A[r][k]: rank rows are
// the first operand, token rows the second.  Read from memory in the matrix
// instruction's layout, 16 lanes would ask for 16 rows, 16 bytes each, and the
// cache lookups would bound the kernel (a load of 1 KB took 120 cycles); so the
// rows come in whole lines, a stage of K at a time, and turn in LDS.  Eight waves
// share a stage's steps of 32 and are added in LDS at the end.  The next stage is
// on its way in registers while this one is multiplied.  Bound by memory and its
// latency: 64 rows of 56 adapters at K = 16384, rank 16, take 9.1 us for 33 MB from the
// caches and 11.2 from memory.
// (32 tokens a workgroup were slower: 18.6 against 14.4 us for 2050 tokens, K = 4096,
// rank 64.)
constexpr uint32_t kShrinkWaves = 8;

template <int RT>
struct Shrink {
  static constexpr uint32_t kRankRows = 16 * RT, kTokRows = 16, kRows = kRankRows + kTokRows;
  static constexpr uint32_t kStage = kRows <= 48 ? 512 : 256;  // of K
  static constexpr uint32_t kPieces = kStage / 8;              // of a row, 16 bytes each
  static constexpr uint32_t kEach = kRows * kPieces / (64 * kShrinkWaves);
  static constexpr uint32_t kSteps = kStage / 32 / kShrinkWaves;
  static constexpr uint32_t kSums = kShrinkWaves * kRankRows * kTokRows * 4;
  static constexpr uint32_t kBytes = kRows * kStage * 2 > kSums ? kRows * kStage * 2 : kSums;
  // pieces are permuted by the row's number, so that 16 rows' reads spread over the banks
  static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t piece) {
    return row * kPieces + (piece ^ (row & 15));
  }
};

template <int RT>
__global__ __launch_bounds__(64 * kShrinkWaves) void k_lora_shrink(LoraArgs p) {
  using S = Shrink<RT>;
  extern __shared__ u32x4 lds[];
  const uint32_t th = threadIdx.x, lane = th & 63, wave = th >> 6, g = lane >> 4, l16 = lane & 15;
  const uint32_t b = chunk_request(p.cu, p.requests, S::kTokRows, blockIdx.x);
  uint32_t first, rows;
  request_rows(p.cu, b, p.tokens, &first, &rows);
  const uint32_t at = (blockIdx.x - (first / S::kTokRows + b)) * S::kTokRows;
  const uint32_t id = (uint32_t)p.adapters[b];
  if (at >= rows || id >= p.count) return;
  const uint32_t live = min(rows - at, S::kTokRows), t0 = first + at, r0 = blockIdx.z * S::kRankRows;
  const uint32_t ranks = min(p.rank - r0, S::kRankRows);
  const uint32_t k0 = blockIdx.y * p.split_k, k1 = min(k0 + p.split_k, p.k);

  // a thread's pieces: rank rows first, then token rows; those past the end are zero
  const uint16_t* from[S::kEach];
#pragma unroll
  for (uint32_t j = 0; j < S::kEach; ++j) {
    const uint32_t x = th + 64 * kShrinkWaves * j, row = x / S::kPieces, k = 8 * (x % S::kPieces);
    from[j] = row < S::kRankRows
                  ? (row < ranks ? p.a + ((uint64_t)id * p.rank + r0 + row) * p.k + k : nullptr)
                  : (row - S::kRankRows < live ? p.x + (uint64_t)(t0 + row - S::kRankRows) * p.x_row + k : nullptr);
  }
  u32x4 next[S::kEach];
  auto load = [&](uint32_t k) {
#pragma unroll
    for (uint32_t j = 0; j < S::kEach; ++j) {
      const uint32_t x = th + 64 * kShrinkWaves * j;
      // K is a multiple of 8: a piece is all in or all out
      next[j] = from[j] && k + 8 * (x % S::kPieces) < k1 ? *reinterpret_cast<const u32x4*>(from[j] + k) : u32x4{};
    }
  };
  floatx4 acc[RT] = {};
  load(k0);
  for (uint32_t k = k0; k < k1; k += S::kStage) {
#pragma unroll
    for (uint32_t j = 0; j < S::kEach; ++j) {
      const uint32_t x = th + 64 * kShrinkWaves * j;
      lds[S::at(x / S::kPieces, x % S::kPieces)] = next[j];
    }
    __syncthreads();
    if (k + S::kStage < k1) load(k + S::kStage);
#pragma unroll
    for (uint32_t s = 0; s < S::kSteps; ++s) {
      const uint32_t piece = 4 * (wave * S::kSteps + s) + g;
      const u32x4 xv = lds[S::at(S::kRankRows + l16, piece)];
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = Bf16::mfma(lds[S::at(16 * r + l16, piece)], xv, acc[r]);
    }
    __syncthreads();
  }
  float* red = reinterpret_cast<float*>(lds);  // [waves][rank rows][token rows]
  constexpr uint32_t kSum = S::kRankRows * S::kTokRows;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[wave * kSum + (16 * r + 4 * g + j) * S::kTokRows + l16] = acc[r][j];
  __syncthreads();
  for (uint32_t i = th; i < live * S::kRankRows; i += 64 * kShrinkWaves) {
    const uint32_t t = i / S::kRankRows, r = i % S::kRankRows;
    if (r >= ranks) continue;
    float v = 0.f;
#pragma unroll
    for (uint32_t w = 0; w < kShrinkWaves; ++w) v += red[w * kSum + r * S::kTokRows + t];
    p.part[((uint64_t)blockIdx.y * p.tokens + t0 + t) * p.rank + r0 + r] = v;
  }
}

// ------------------------------------------------------------------- expand
// out = y + low B^T on the matrix cores without losing fp32: a product of two
// bf16 values is exact in fp32, and low (the shrunk row times the adapter's
// scaling) is cut into three bf16 parts that add up to all of its 24 bits, so three
// products take the place of one.  They are hidden: the kernel is bound by y and
// out, 8 bytes an element against 6 rank operations.  B's rows (columns of out) are
// the first operand, read from memory in its layout, tokens the second, from LDS.
// Parts are cut off, not rounded: they have low's sign, and none passes the largest
// bf16 value.  A part may be zero where low is not, and zero times an infinity of B is
// NaN; so sums that are NaN are formed again from whole products (looking for them
// takes 26.3 to 27.0 us for 64 single rows, 48.6 to 49.1 for 2050).
//
// Results turn in LDS, so that y and out are met in whole lines a row (in the
// instruction's layout 16 lanes would ask for 16 rows).  MT = 2 takes 32 tokens,
// MT = 1 up to 16.  2050 rows by 14336 columns at rank 64 take 51 us for 235 MB, 64
// single rows by 53248 at rank 16 27 us for 122 MB: 4.6 TB/s, where a large copy moves
// 5.1.  That is with what the caches hold of the call before; on inputs that change from
// call to call they take 61 and 36 us (3.9 and 3.4 TB/s): a pass is one chain of loads,
// products and two barriers, and memory's latency is longer.
template <int MT>
struct Expand {
  static constexpr uint32_t kRows = 16 * MT;
  static constexpr uint32_t kTiles = MT == 1 ? 4 : 2;    // of 16 columns, a wave and pass
  static constexpr uint32_t kCols = 4 * 16 * kTiles;     // a workgroup and pass
  static constexpr uint32_t kTurn = kCols + 4;           // floats of a row in LDS
  static constexpr uint32_t kLanes = kCols / 4, kStep = 256 / kLanes, kIter = kRows / kStep;  // of y and out
  // low: [3][kRows][rank rounded up to 32, and 8 to spread the rows over the banks]
  static __host__ __device__ uint32_t low_row(uint32_t rank) { return (rank + 31) / 32 * 32 + 8; }
  static uint32_t bytes(uint32_t rank) { return 3 * kRows * low_row(rank) * 2 + kRows * kTurn * 4; }
};

// One element of low B^T, product by product: `low` at the token's row of the parts,
// `part` elements apart, `b` the column's row of B.
__device__ __forceinline__ float whole_products(const uint16_t* low, uint32_t part, const uint16_t* b, uint32_t rank) {
  float sum = 0.f;
#pragma unroll 1
  for (uint32_t r = 0; r < rank && !isnan(sum); ++r) {
    const float v = Bf16::up(low[r]) + (Bf16::up(low[part + r]) + Bf16::up(low[2 * part + r]));
    sum = fmaf(v, Bf16::up(b[r]), sum);
  }
  return sum;
}

template <int MT>
__global__ __launch_bounds__(256, 4) void k_lora_expand(LoraArgs p) {
  using X = Expand<MT>;
  constexpr uint32_t kRows = X::kRows;
  constexpr int NT = X::kTiles;
  extern __shared__ u32x4 lds[];
  uint16_t* low = reinterpret_cast<uint16_t*>(lds);
  const uint32_t t = threadIdx.x, lane = t & 63, wave = t >> 6, g = lane >> 4, l16 = lane & 15;
  // one more request than there are: the rows past cu[requests], without adapter
  const uint32_t b = chunk_request(p.cu, p.requests + 1, kRows, blockIdx.x);
  uint32_t first, rows, id = ~0u;
  if (b < p.requests) {
    request_rows(p.cu, b, p.tokens, &first, &rows);
    id = (uint32_t)p.adapters[b];
  } else {
    first = min((uint32_t)max(p.cu[b], 0), p.tokens);
    rows = p.tokens - first;
  }
  const uint32_t at = (blockIdx.x - (first / kRows + b)) * kRows;
  if (at >= rows) return;
  const uint32_t live = min(rows - at, kRows), t0 = first + at;
  const uint32_t n0 = blockIdx.y * p.block_n, n1 = min(n0 + p.block_n, p.n);
  if (id >= p.count) {
    if (p.y != p.out)
      for (uint32_t r = 0; r < live; ++r)
        for (uint32_t n = n0 + t; n < n1; n += 256)
          p.out[(uint64_t)(t0 + r) * p.out_row + n] = p.y[(uint64_t)(t0 + r) * p.y_row + n];
    return;
  }

  const uint32_t row = X::low_row(p.rank), padded = row - 8, part = kRows * row;
  const float scale = p.scaling[id];
  for (uint32_t i = t; i < kRows * padded / 8; i += 256) {
    const uint32_t r = 8 * i % padded, tok = 8 * i / padded;
    float v[8] = {};
    if (tok < live && r < p.rank) {
      const float* from = p.part + (uint64_t)(t0 + tok) * p.rank + r;
      for (uint32_t piece = 0; piece < p.splits; ++piece, from += (uint64_t)p.tokens * p.rank) {
        const floatx4 v0 = *reinterpret_cast<const floatx4*>(from), v1 = *reinterpret_cast<const floatx4*>(from + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] += v0[j];
          v[4 + j] += v1[j];
        }
      }
    }
    u32x4 out[3];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      // v = hi + mid + lo, 8 bits each; an infinity stays in hi alone, and a NaN whose
      // upper bits are an infinity's is one in the next part
      float rest[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) rest[e] = v[j + e] * scale;
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        uint32_t top[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[e] = __float_as_uint(rest[e]) & 0xFFFF0000u;
          const float part = __uint_as_float(top[e]);
          rest[e] = rest[e] == part ? 0.f : rest[e] - part;
        }
        out[x][j / 2] = top[0] >> 16 | top[1];
      }
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) *reinterpret_cast<u32x4*>(low + x * part + tok * row + r) = out[x];
  }
  __syncthreads();

  const uint16_t* mat = p.b + (uint64_t)id * p.n * p.rank;
  float* turn = reinterpret_cast<float*>(low + 3 * part);
  const uint32_t row_t = t / X::kLanes, col_t = 4 * (t % X::kLanes);  // where this thread meets y and out
  for (uint32_t nb = n0; nb < n1; nb += X::kCols) {
    const uint32_t nw = nb + wave * 16 * NT;  // the wave's first column
    floatx4 yv[X::kIter];
#pragma unroll
    for (uint32_t j = 0; j < X::kIter; ++j) {
      const uint32_t r = row_t + j * X::kStep;
      if (r < live) yv[j] = load4(p.y + (uint64_t)(t0 + r) * p.y_row, nb + col_t, n1, p.wide_y);
    }
    floatx4 acc[NT][MT] = {};
    for (uint32_t r0 = 0; r0 < p.rank; r0 += 32) {
      const uint32_t r = r0 + 8 * g;
      u32x4 bv[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const uint32_t n = nw + 16 * c + l16;
        bv[c] = n < n1 && r < p.rank ? *reinterpret_cast<const u32x4*>(mat + (uint64_t)n * p.rank + r) : u32x4{};
      }
#pragma unroll
      for (int x = 2; x >= 0; --x)  // the smallest parts first
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const u32x4 lv = *reinterpret_cast<const u32x4*>(low + x * part + (16 * i + l16) * row + r);
#pragma unroll
          for (int c = 0; c < NT; ++c) acc[c][i] = Bf16::mfma(bv[c], lv, acc[c][i]);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
      if (16 * i + l16 < live) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
          *reinterpret_cast<floatx4*>(turn + (16 * i + l16) * X::kTurn + wave * 16 * NT + 16 * c + 4 * g) = acc[c][i];
      }
    bool odd = false;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < NT; ++c)
        odd |= __builtin_isunordered(acc[c][i][0], acc[c][i][1]) || __builtin_isunordered(acc[c][i][2], acc[c][i][3]);
    if (odd) {
#pragma unroll 1
      for (uint32_t e = 0; e < 4 * NT * MT; ++e) {  // this lane's own sums
        uint32_t tok = 16 * (e / (4 * NT)) + l16;
        const uint32_t col = wave * 16 * NT + 16 * (e / 4 % NT) + 4 * g + e % 4;
        keep_here(tok);
        float* sum = turn + tok * X::kTurn + col;
        if (tok < live && nb + col < n1 && isnan(*sum))
          *sum = whole_products(low + tok * row, part, mat + (uint64_t)(nb + col) * p.rank, p.rank);
      }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < X::kIter; ++j) {
      const uint32_t r = row_t + j * X::kStep;
      if (r < live)
        store4(p.out + (uint64_t)(t0 + r) * p.out_row, nb + col_t, n1, p.wide_y,
               yv[j] + *reinterpret_cast<const floatx4*>(turn + r * X::kTurn + col_t));
    }
    __syncthreads();
  }
}

struct LoraPlan {
  uint32_t splits, split_k, expand_mt, block_n;
};

LoraPlan plan_lora(uint32_t tokens, uint32_t requests, uint32_t n, uint32_t k, uint32_t rank) {
  LoraPlan p;
  const uint32_t each = tokens / std::max(requests, 1u);  // of a request, on the average
  // Pieces of K: one workgroup a CU, none shorter than 1024.  Every workgroup of the
  // second kernel adds the pieces up again, so their number is kept low: for 2050
  // tokens and rank 64 two pieces took 14.4 us and eight 17.7 (and 3 us more in the
  // second kernel), for one token four took 3.3 us and one 5.5.
  const uint32_t chunks = std::max(std::min(tokens / 16 + requests, tokens), 1u) * ((rank + 63) / 64);
  const uint32_t s = std::min(std::min((kCUs + chunks - 1) / chunks, std::max(k / 1024, 1u)), 16u);
  p.split_k = ((k + s - 1) / s + 511) / 512 * 512;
  p.splits = (k + p.split_k - 1) / p.split_k;
  // Tokens and columns of a workgroup of the second kernel: 32 rows where requests
  // have as many (2050 tokens in 6 requests: 49 us, 16 rows 61; single tokens: 37 us
  // against 26), four workgroups a CU (two: 59 and 34 us, sixteen: 58 and 31), all from
  // the caches.
  p.expand_mt = each >= 32 ? 2 : 1;
  const uint32_t cols = p.expand_mt == 2 ? Expand<2>::kCols : Expand<1>::kCols;
  const uint32_t rows2 = 16 * p.expand_mt, chunks2 = std::max(std::min(tokens / rows2 + requests, tokens), 1u);
  const uint32_t blocks = std::max((4 * kCUs + chunks2 - 1) / chunks2, 1u), passes = (n + cols - 1) / cols;
  p.block_n = std::max(passes / blocks, 1u) * cols;
  return p;
}

static_assert(Shrink<4>::kBytes <= 64 * 1024 && Shrink<2>::kBytes <= 64 * 1024, "LDS without an attribute");

bool lora_shape_ok(uint32_t tokens, uint32_t requests, uint32_t n, uint32_t k, uint32_t rank) {
  return requests <= kMaxRequests && tokens <= (1u << 24) && n >= 1 && n <= (1u << 23) && k >= 8 &&
         k <= (1u << 24) && k % 8 == 0 && rank >= 8 && rank <= 256 && rank % 8 == 0;
}

}  // namespace
}  // namespace serve
}  // namespace dgt

using namespace dgt::serve;

extern "C" {

size_t dgt_lora_workspace(uint32_t tokens, uint32_t requests, uint32_t n, uint32_t k, uint32_t rank) {
  if (!lora_shape_ok(tokens, requests, n, k, rank)) return 0;
  const LoraPlan p = plan_lora(tokens, requests, n, k, rank);
  return std::max<size_t>((size_t)p.splits * tokens * rank * 4, 256);
}

int dgt_lora_add(const float* d_y, uint64_t y_row, const uint16_t* d_x, uint64_t x_row,
                 const uint16_t* d_a, const uint16_t* d_b, const float* d_scaling, uint32_t adapters,
                 const int32_t* d_ids, const int32_t* d_cu, uint32_t requests, uint32_t tokens,
                 uint32_t n, uint32_t k, uint32_t rank, float* d_out, uint64_t out_row, void* d_ws,
                 size_t ws_bytes, void* stream) {
  if (!lora_shape_ok(tokens, requests, n, k, rank)) return DGT_E_SHAPE;
  if (tokens == 0) return DGT_OK;
  if (!d_y || !d_out || !d_cu || !d_x || !d_ws) return DGT_E_ARG;
  if ((requests && !d_ids) || (adapters && (!d_a || !d_b || !d_scaling))) return DGT_E_ARG;
  if (tokens == 1) {  // one row has no stride
    x_row = k;
    y_row = out_row = ((uint64_t)n + 3) / 4 * 4;
  }
  if (y_row < n || out_row < n || x_row < k || x_row % 8) return DGT_E_SHAPE;
  if (!aligned(d_x, 16) || !aligned(d_a, 16) || !aligned(d_b, 16) || !aligned(d_ws, 256)) return DGT_E_ARG;
  if (d_out == d_y && out_row != y_row) return DGT_E_ARG;
  if (ws_bytes < dgt_lora_workspace(tokens, requests, n, k, rank)) return DGT_E_BUFSIZE;
  LoraArgs p;
  p.y = d_y;
  p.x = d_x;
  p.a = d_a;
  p.b = d_b;
  p.scaling = d_scaling;
  p.adapters = d_ids;
  p.cu = d_cu;
  p.out = d_out;
  p.part = static_cast<float*>(d_ws);
  p.x_row = x_row;
  p.y_row = y_row;
  p.out_row = out_row;
  p.tokens = tokens;
  p.requests = requests;
  p.count = adapters;
  p.n = n;
  p.k = k;
  p.rank = rank;
  const LoraPlan plan = plan_lora(tokens, requests, n, k, rank);
  p.splits = plan.splits;
  p.split_k = plan.split_k;
  p.block_n = plan.block_n;
  p.wide_y = aligned(d_y, 16) && aligned(d_out, 16) && y_row % 4 == 0 && out_row % 4 == 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (requests && adapters) {
    const uint32_t rt = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
    const dim3 grid(tokens / 16 + requests, p.splits, (rank + rt * 16 - 1) / (rt * 16));
    auto run = [&](auto kernel, uint32_t lds) {
      hipLaunchKernelGGL(kernel, grid, dim3(64 * kShrinkWaves), lds, st, p);
      return launched();
    };
    const int rc = rt == 1   ? run(k_lora_shrink<1>, Shrink<1>::kBytes)
                   : rt == 2 ? run(k_lora_shrink<2>, Shrink<2>::kBytes)
                             : run(k_lora_shrink<4>, Shrink<4>::kBytes);
    if (rc) return rc;
  }
  auto run = [&](auto kernel, uint32_t rows, uint32_t lds) {
    if (lds > 64 * 1024 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)lds) != hipSuccess)
      return (int)DGT_E_HIP;
    const dim3 grid(tokens / rows + requests + 1, (n + p.block_n - 1) / p.block_n);
    hipLaunchKernelGGL(kernel, grid, dim3(256), lds, st, p);
    return launched();
  };
  return plan.expand_mt == 2 ? run(k_lora_expand<2>, 32, Expand<2>::bytes(rank))
                             : run(k_lora_expand<1>, 16, Expand<1>::bytes(rank));
}

}  // extern "C"
