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
  uint32_t splits, split_k;        // pieces of K and their length (a multiple of 32)
};

// ------------------------------------------------------------------- shrink
// part[piece][t][r] = sum over the piece of K of x[t][k] A[r][k]: rank rows are
// the first operand, token rows the second, both read from memory in the
// matrix instruction's own layout (16 bytes a lane).  A workgroup's four waves
// take every fourth step of K and meet in LDS.
template <int RT, int MT>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraArgs p) {
  constexpr uint32_t kRows = 16 * MT;
  __shared__ float red[4][RT * 16][kRows];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const uint32_t b = chunk_request(p.cu, p.requests, kRows, blockIdx.x);
  uint32_t first, rows;
  request_rows(p.cu, b, p.tokens, &first, &rows);
  const uint32_t at = (blockIdx.x - (first / kRows + b)) * kRows;
  const uint32_t id = (uint32_t)p.adapters[b];
  if (at >= rows || id >= p.count) return;
  const uint32_t live = min(rows - at, kRows), t0 = first + at, r0 = blockIdx.z * (RT * 16);
  const uint32_t k0 = blockIdx.y * p.split_k, k1 = min(k0 + p.split_k, p.k);

  // rows past the end read the last one; what they add is not stored
  const uint16_t* xp[MT];
  const uint16_t* ap[RT];
#pragma unroll
  for (int i = 0; i < MT; ++i) xp[i] = p.x + (uint64_t)(t0 + min(16u * i + l16, live - 1)) * p.x_row;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    ap[i] = p.a + ((uint64_t)id * p.rank + min(r0 + 16u * i + l16, p.rank - 1)) * p.k;
  floatx4 acc[RT][MT] = {};
  for (uint32_t k = k0 + wave * 32; k < k1; k += 128) {
    const uint32_t kk = k + 8 * g;
    const bool in = kk < k1;  // K is a multiple of 8: a lane's eight values are all in or all out
    u32x4 xv[MT], av[RT];
#pragma unroll
    for (int i = 0; i < MT; ++i) xv[i] = in ? *reinterpret_cast<const u32x4*>(xp[i] + kk) : u32x4{};
#pragma unroll
    for (int i = 0; i < RT; ++i) av[i] = in ? *reinterpret_cast<const u32x4*>(ap[i] + kk) : u32x4{};
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[r][i] = Bf16::mfma(av[r], xv[i], acc[r][i]);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[wave][16 * r + 4 * g + j][16 * i + l16] = acc[r][i][j];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < live * RT * 16; i += 256) {
    const uint32_t t = i / (RT * 16), r = i % (RT * 16);
    if (r0 + r < p.rank)
      p.part[((uint64_t)blockIdx.y * p.tokens + t0 + t) * p.rank + r0 + r] =
          (red[0][r][t] + red[1][r][t]) + (red[2][r][t] + red[3][r][t]);
  }
}

// ------------------------------------------------------------------- expand
// Eight tokens by 256 columns a workgroup, one column a thread, fp32 throughout.
constexpr uint32_t kExpandRows = 8;

__global__ __launch_bounds__(256) void k_lora_expand(LoraArgs p) {
  extern __shared__ float low[];  // [rows][rank], times the adapter's scaling
  // one more request than there are: the rows past cu[requests], without adapter
  const uint32_t b = chunk_request(p.cu, p.requests + 1, kExpandRows, blockIdx.x);
  uint32_t first, rows, id = ~0u;
  if (b < p.requests) {
    request_rows(p.cu, b, p.tokens, &first, &rows);
    id = (uint32_t)p.adapters[b];
  } else {
    first = min((uint32_t)max(p.cu[b], 0), p.tokens);
    rows = p.tokens - first;
  }
  const uint32_t at = (blockIdx.x - (first / kExpandRows + b)) * kExpandRows;
  const bool adapts = id < p.count;
  if (at >= rows || (!adapts && p.y == p.out)) return;
  const uint32_t live = min(rows - at, kExpandRows), t0 = first + at;
  if (adapts) {
    const float s = p.scaling[id];
    for (uint32_t i = threadIdx.x; i < live * p.rank; i += 256) {
      float v = 0.f;
      for (uint32_t piece = 0; piece < p.splits; ++piece)
        v += p.part[((uint64_t)piece * p.tokens + t0) * p.rank + i];
      low[i] = v * s;
    }
    __syncthreads();
  }
  const uint32_t n = blockIdx.y * 256 + threadIdx.x;
  if (n >= p.n) return;
  float acc[kExpandRows] = {};
  if (adapts) {
    const uint16_t* bp = p.b + ((uint64_t)id * p.n + n) * p.rank;
    for (uint32_t r = 0; r < p.rank; r += 8) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(bp + r);
#pragma unroll
      for (uint32_t t = 0; t < kExpandRows; ++t) {
        if (t < live) {
          const float* l = low + t * p.rank + r;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[t] = fmaf(l[2 * j], Bf16::up(w[j] & 0xFFFFu), acc[t]);
            acc[t] = fmaf(l[2 * j + 1], Bf16::up(w[j] >> 16), acc[t]);
          }
        }
      }
    }
  }
#pragma unroll
  for (uint32_t t = 0; t < kExpandRows; ++t)
    if (t < live)
      p.out[(uint64_t)(t0 + t) * p.out_row + n] = p.y[(uint64_t)(t0 + t) * p.y_row + n] + acc[t];
}

// Pieces of K: enough workgroups to fill the chip, none shorter than 512.
void lora_splits(uint32_t tokens, uint32_t requests, uint32_t k, uint32_t rank, uint32_t* rows,
                 uint32_t* splits, uint32_t* split_k) {
  *rows = tokens / std::max(requests, 1u) >= 32 ? 64 : 16;
  const uint32_t groups = (rank + 63) / 64;
  const uint32_t chunks = std::max(std::min(tokens / *rows + requests, tokens), 1u) * groups;
  uint32_t s = std::min((4 * kCUs + chunks - 1) / chunks, std::max(k / 512, 1u));
  s = std::min(s, 32u);
  *split_k = ((k + s - 1) / s + 31) / 32 * 32;
  *splits = (k + *split_k - 1) / *split_k;
}

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
  uint32_t rows, splits, split_k;
  lora_splits(tokens, requests, k, rank, &rows, &splits, &split_k);
  return std::max<size_t>((size_t)splits * tokens * rank * 4, 256);
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
  uint32_t rows;
  lora_splits(tokens, requests, k, rank, &rows, &p.splits, &p.split_k);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (requests && adapters) {
    const uint32_t rt = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
    const dim3 grid(tokens / rows + requests, p.splits, (rank + rt * 16 - 1) / (rt * 16));
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, p);
      return launched();
    };
    int rc;
    if (rows == 64)
      rc = rt == 1 ? run(k_lora_shrink<1, 4>) : rt == 2 ? run(k_lora_shrink<2, 4>) : run(k_lora_shrink<4, 4>);
    else
      rc = rt == 1 ? run(k_lora_shrink<1, 1>) : rt == 2 ? run(k_lora_shrink<2, 1>) : run(k_lora_shrink<4, 1>);
    if (rc) return rc;
  }
  const dim3 grid(tokens / kExpandRows + requests + 1, (n + 255) / 256);
  hipLaunchKernelGGL(k_lora_expand, grid, dim3(256), kExpandRows * rank * 4, st, p);
  return launched();
}

}  // extern "C"
