/*
 * dgt.h -- C ABI of libdgt: tile-granular lossless rANS coding of LLM weight
 * matrices, decoded on the fly inside the GEMM that consumes them (AMD
 * MI355X / gfx950).
 *
 * Source of the method: the page "arXiv'26 | 无损压缩逼近 Shannon 极限：你的
 * LLM 权重里一半以上的 bit 是白存的" (write-up of "Approaching Shannon Bound
 * with Lossless LLM Weight Compression"), cited below as [P §n]:
 *   §2.2  decode must keep up with memory bandwidth, any tile must decode on
 *         its own, decoded weights go to on-chip memory and never to global
 *         memory;
 *   §3.1  offline, each layer is cut into tiles in the GEMM's tiling geometry,
 *         all tiles share one compact ANS codebook, a light index records each
 *         tile's start offset, every tile stream is split into R lane
 *         sub-streams with one rANS state per lane; at run time tile k+1 is
 *         decoded while tile k is multiplied, in a static tile-swizzle order,
 *         packaged as a kernel a framework can call directly;
 *   §4.1  finite-precision frequency normalisation.
 *
 * Conventions for every entry point:
 *   - Plain C types only.  Pointers prefixed d_ are device (HIP) pointers,
 *     others are host pointers.  `stream` is a hipStream_t passed as void*
 *     (NULL = the default stream).  Device entry points are asynchronous on
 *     that stream and return as soon as the work is enqueued.
 *   - The caller owns every buffer; the library allocates no device memory.
 *   - Return value: DGT_OK (0) or a negative dgt_status.  No exceptions cross
 *     the ABI.  On error nothing has been enqueued.
 *   - Device blobs must be 16-byte aligned.  All multi-byte fields are
 *     little-endian.  Calls are thread-safe.
 *   - Environment: DGT_STAGING=whole|ring overrides the per-layer choice of
 *     how device kernels bring tile streams on chip (whole streams, or a
 *     two-chunk ring for one tile per wave); DGT_ROUNDS=n forces n rounds of
 *     chains per workgroup where the multi-round fused kernel applies (ring
 *     staging, M <= 16 per launch, 64 or 128 lanes) instead of the per-layer
 *     choice (1 = one round); DGT_XM_SINGLE_BUFFER=1 makes the large-M fused
 *     kernel (17 <= M <= 256 per pass, 64 lanes) keep one fragment buffer
 *     instead of two (a comparison point; an error where no such kernel
 *     exists).  Results are identical.  DGT_XM_SUBSETS=0 keeps the 8-wave
 *     large-M kernel where the 16-wave subset form would run (256-row tiles,
 *     64 lanes, 17 <= M <= 128, int4 pairs to 64); results agree within
 *     rounding (another order of additions).  Read at every call;
 *     dgt_gemm_workspace covers every choice.
 *
 * Compressed layer ("blob") format, version 1 (all offsets in bytes):
 *   header (128 B): magic "DGT1", u16 version, u16 header size, u32 fmt,
 *     u32 flags, u32 N, K, tile_n, tile_k, lanes R, prob_bits, alphabet,
 *     tiles; u64 table, index, ktab, streams, raw offsets, u64 total size;
 *     u32 max tile length (4-byte units), u32 kmax (16); zero padding.
 *   table  u16 f[alphabet], sum f = 2^prob_bits (shared by all tiles);
 *          BF16_PAIR and BF16_WORD (alphabet 65536): u32 symbol | f << 16
 *          (BF16_WORD: symbol | (f - 1) << 16) for each symbol with f > 0, in
 *          increasing symbol order, and the header's alphabet field holds the
 *          number of entries.
 *   index  u32 off[tiles+1]: tile t's stream starts at streams + 4*off[t].
 *   ktab   u8 k[tiles]: initial-state payload steps of each tile.
 *   streams per tile: R u32 lane states, u16 words in decode order, zero pad.
 *   raw    (BF16_SPLIT, BF16_EXP, BF16_PAIR) T raw bytes per tile, lane-major.
 * Tile t = bn*(K/tile_k) + bk covers W rows bn*tile_n.. and columns
 * bk*tile_k..  Inside a tile, symbol j = s*R + p (step s, lane p) with
 * s = 8g + e, fragment g = fk*(tile_n/16) + fn: lane p decodes row
 * 16fn + p%16, column fk*R/2 + 8*(p/16) + e.  rANS: state in [2^16, 2^32),
 * INT4_PAIR (and BF16_PAIR, whose symbol is the two weights' high bytes)
 * codes symbol c of a row for the weight pair (2c, 2c+1) and lays
 * out a tile's tile_n*tile_k/2 symbols the same way with 4 symbols per lane
 * per fragment (s = 4g + e, pair column fk*R/4 + 4*(p/16) + e), so a lane's
 * 4 symbols are again its 8 consecutive weights of one row.
 * R = 128 (two states per wave lane; tile_n a multiple of 32): states p < 64
 * order the top tile_n/2 rows and states 64 + p the bottom tile_n/2 rows,
 * each half exactly as an R = 64 tile of tile_n/2 rows; both share the one
 * word stream (interleaving j = s*128 + p); raw byte q = g*1024 + p*8 + e.
 * 16-bit renormalisation words; decode x' = f*(x>>n) + (x mod 2^n) - c_s,
 * then if x' < 2^16 read one word.  The last k[t] steps of a tile decode from
 * y = x - 2^16 without reading words; a valid tile ends with y == 0 on every
 * lane and its stream consumed exactly.
 */
#ifndef DGT_H_
#define DGT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Weight formats ([P §2.1]: the formats whose codes are entropy coded). */
enum dgt_format {
  DGT_FMT_INT8 = 1,       /* int8 codes; GEMM value = the integer (exact bf16) */
  DGT_FMT_INT4 = 2,       /* codes 0..15, zero point 8, bf16 scale per 128 columns */
  DGT_FMT_FP8_E4M3 = 3,   /* OCP e4m3 bytes, per-tensor fp32 weight scale */
  DGT_FMT_BF16_SPLIT = 4, /* bf16: high byte coded, low byte stored raw */
  DGT_FMT_INT4_PAIR = 5,  /* INT4 weights and scales, coded two per symbol:
                             q[n,2c] | q[n,2c+1] << 4 (alphabet 256) */
  DGT_FMT_BF16_EXP = 6,   /* bf16: exponent (bits 14..7) coded, sign and mantissa
                             stored raw as one byte (sign << 7 | mantissa) */
  DGT_FMT_BF16_PAIR = 7,  /* bf16 byte split with the high bytes of two weights
                             adjacent along K coded as one 16-bit symbol
                             hi[n,2c] | hi[n,2c+1] << 8; low bytes raw */
  DGT_FMT_BF16_WORD = 8   /* bf16 whole words: the 16-bit pattern is the symbol,
                             frequency precision prob_bits = 16 ([P §4.1]:
                             16-bit symbols need a precise table), nothing raw */
};

enum dgt_status {
  DGT_OK = 0,
  DGT_E_ARG = -1,         /* null pointer or out-of-range scalar argument */
  DGT_E_SHAPE = -2,       /* N, K not multiples of the tile; bad tile/lane geometry */
  DGT_E_ALPHABET = -3,    /* code outside the format's alphabet */
  DGT_E_BUFSIZE = -4,     /* output / workspace buffer too small */
  DGT_E_FORMAT = -5,      /* blob header not recognised (magic, version, fmt) */
  DGT_E_CORRUPT = -6,     /* blob inconsistent (sizes, index, table, ktab) */
  DGT_E_HIP = -7,         /* a HIP runtime call or kernel launch failed */
  DGT_E_UNSUPPORTED = -8  /* valid request this library does not implement */
};

/* Layer geometry for compression.  prob_bits: frequency precision n (12;
 * BF16_WORD: 16, which the device kernels require for it). */
typedef struct dgt_params {
  uint32_t fmt, n, k, tile_n, tile_k, lanes, prob_bits, flags;
} dgt_params;

/* Parsed, validated view of a blob (filled by dgt_layer_info). */
typedef struct dgt_info {
  uint32_t fmt, n, k, tile_n, tile_k, lanes, prob_bits, alphabet;
  uint32_t tiles, max_tile_words4, kmax, flags;
  uint64_t table_off, index_off, ktab_off, streams_off, raw_off, total_bytes;
  uint64_t stream_bytes;     /* bytes of the streams section */
  double bits_per_weight;    /* 8 * total_bytes / (N*K) */
} dgt_info;

/* Library ABI version (1). */
int dgt_version(void);

/* Human-readable text for a dgt_status code (static storage). */
const char* dgt_status_string(int status);

/* Upper bound of the blob size dgt_compress_layer can produce for `p`
 * (every symbol costing a full word); 0 if `p` is invalid. */
size_t dgt_compress_bound(const dgt_params* p);

/* Offline encoder ([P §3.1] offline stage), host only.
 *   w: N*K weights row-major: one byte per weight for INT8 (two's
 *      complement), INT4 and INT4_PAIR (values 0..15; INT4_PAIR needs even
 *      K and tile_k) and FP8_E4M3; one uint16 bf16 bit pattern per weight
 *      for BF16_SPLIT, BF16_EXP, BF16_PAIR and BF16_WORD.
 *   out/cap: caller buffer of `cap` bytes; *out_size receives the blob size.
 * Errors: E_ARG, E_SHAPE, E_ALPHABET (INT4 code > 15), E_BUFSIZE.
 * Deterministic: the same input always gives the same bytes. */
int dgt_compress_layer(const dgt_params* p, const void* w, void* out, size_t cap,
                       size_t* out_size);

/* Parse and validate a host copy of a blob (header, table sums to 2^n,
 * index monotone and inside the blob, ktab <= min(kmax, steps)).
 * Errors: E_ARG, E_FORMAT, E_CORRUPT. */
int dgt_layer_info(const void* blob, size_t size, dgt_info* out);

/* Decode tiles to global memory (the layer-granular "decompress first" path,
 * kept for tests and the decompress-then-GEMM comparison; [P §2.2] names it
 * as what the fused path avoids).
 *   d_blob: device copy of the blob described by `info`.
 *   d_tile_ids: n_ids tile ids to decode, or NULL for all tiles (n_ids ignored).
 *          An id >= the layer's tile count is skipped on the device: nothing
 *          is written for it (neither d_out nor d_status), and the reads made
 *          in its place stay inside the blob (tile 0's stream).
 *   d_out: the full W layout, row-major [N, K]: uint8 (INT8 bytes, INT4
 *          and INT4_PAIR codes, FP8 bytes) or uint16 bf16 bits (BF16_SPLIT,
 *          BF16_EXP);
 *          only the elements of the decoded tiles are written.
 *   d_status: NULL or int32[tiles]; entry t is set to 0 when tile t decoded
 *          with a consistent stream, else to a positive error mask
 *          (1 = final state, 2 = stream length, 4 = stream overrun).
 * Errors (synchronous): E_ARG, E_UNSUPPORTED (lanes not 32/64/128; R = 32
 * streams too long for on-chip staging), E_HIP. */
int dgt_decode_tiles(const void* d_blob, const dgt_info* info, const uint32_t* d_tile_ids,
                     uint32_t n_ids, void* d_out, int32_t* d_status, void* stream);

/* Workspace bytes dgt_fused_decode_gemm needs for `m` activation rows.  The
 * workspace must be zero-filled before its first use; every call leaves it
 * ready for the next one (its counters return to zero). */
size_t dgt_gemm_workspace(const dgt_info* info, uint32_t m);

/* Fused decode + GEMM ([P §3.1] run-time stage): Y[m, n] = sum_k X[m, k] W[n, k]
 * with W decoded tile by tile on chip, never written to global memory.
 *   d_x: bf16 bits [m, K] row-major; m in 1..65536.  Up to 256 rows run in
 *        one pass in which every tile is decoded once; more rows run in
 *        passes of 256 (the layer is decoded once per pass).
 *   d_scales: INT4 and INT4_PAIR, bf16 bits [N, K/128]; else NULL.
 *   w_scale: FP8 only, per-tensor weight scale (X is quantised to e4m3 per
 *            tensor on the device first); ignored otherwise.
 *   d_y: fp32 [m, N] row-major, overwritten.
 *   d_ws, ws_bytes: workspace of at least dgt_gemm_workspace(info, m) bytes.
 *   d_status: NULL or int32[tiles], as for dgt_decode_tiles.
 * Values: INT8 -> bf16(code); INT4, INT4_PAIR -> bf16_RNE((q-8)*scale); BF16_SPLIT,
 * BF16_EXP -> the bf16 bits;
 * FP8 -> e4m3 products scaled by sx*w_scale; fp32 accumulation.
 * Errors: E_ARG, E_BUFSIZE (workspace), E_UNSUPPORTED, E_HIP. */
int dgt_fused_decode_gemm(const void* d_blob, const dgt_info* info, const uint16_t* d_x,
                          uint32_t m, const uint16_t* d_scales, float w_scale, float* d_y,
                          void* d_ws, size_t ws_bytes, int32_t* d_status, void* stream);

/* Allocation-free variant of dgt_fused_decode_gemm, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, values and errors, but
 * no workspace argument: the workspace is a static device array of
 * dgt_noalloc_scratch_bytes() bytes (64 MiB) that every device the library
 * runs on holds from the library's load until the process ends.  A call whose
 * workspace (dgt_gemm_workspace) would exceed it returns DGT_E_BUFSIZE and
 * enqueues nothing; M <= 16 fits every layer up to 53248 x 16384 (55 MiB at
 * most), and so does M <= 64 for 256 x 64 tiles at 64 lanes (39 MiB at most)
 * and M <= 256 up to 14336 x 4096 (42 MiB).  Each call
 * first zeroes the array's counters with a small kernel on `stream`.  All
 * calls on one device share the array: calls that overlap in time on one
 * device (other streams, other threads) race and give wrong results.  Calls
 * no hipMalloc, hipFree or allocating library routine. */
size_t dgt_noalloc_scratch_bytes(void);
int dgt_fused_decode_gemm_noalloc(const void* d_blob, const dgt_info* info, const uint16_t* d_x,
                                  uint32_t m, const uint16_t* d_scales, float w_scale,
                                  float* d_y, int32_t* d_status, void* stream);

/* Uncompressed baseline: Y = X W^T with W read from global memory, d_w is
 * [N, K] in the same element layout dgt_decode_tiles writes (INT4_PAIR is
 * read as INT4, BF16_EXP, BF16_PAIR and BF16_WORD as BF16_SPLIT), same weight
 * values and epilogue as the fused call.  M = 1 runs a streaming GEMV (K <=
 * 32768), M >= 32 an LDS-tiled MFMA GEMM reading each W block once per 128
 * rows, the rows between in the fused call's strip decomposition.  Workspace
 * from dgt_dense_workspace (zero-filled before first use); M <= 256. */
size_t dgt_dense_workspace(uint32_t fmt, uint32_t n, uint32_t k, uint32_t tile_n,
                           uint32_t m);
int dgt_dense_gemm(uint32_t fmt, uint32_t n, uint32_t k, uint32_t tile_n, const void* d_w,
                   const uint16_t* d_x, uint32_t m, const uint16_t* d_scales, float w_scale,
                   float* d_y, void* d_ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------ serving operators
 * What stands beside the compressed projections when a batch of requests is
 * served and drafted tokens are verified: the page plan of a step, the store of
 * new keys and values into a paged cache, attention over that cache, and
 * low-rank adapters.
 *
 * Shared conventions.  Request b holds ctx[b] tokens in the cache and brings
 * new[b] tokens to the step; the new tokens of all requests lie one after
 * another in `tokens` rows, request b in rows cu[b] .. cu[b+1] - 1 (cu starts
 * at 0 and never falls).  The cache is a pool of `blocks` pages of `block`
 * tokens (a power of two, 8..1024):
 *   keys   [blocks, kv_heads, block, dim]
 *   values [blocks, kv_heads, dim, block]   (each page transposed)
 * A slot is page * block + place in the page (blocks * block < 2^31).  A block
 * table [requests, width] names each request's pages; token p of a request is
 * in page table[b, p / block].  At most 8192 requests a call.
 * Lengths, offsets, tables, slots and ids are device data that the host does
 * not see: the kernels hold every access inside the buffers whatever they hold
 * (lengths are cut to the table, offsets to the rows, a page or adapter id out
 * of range counts as absent; offsets that fall leave the rows undefined). */

/* Element types of cache and activations. */
enum dgt_element {
  DGT_ELT_BF16 = 1,
  DGT_ELT_F16 = 2,
  DGT_ELT_F32 = 3
};

/* Page plan of one step, in one launch.  All arrays are on the device, and no
 * output overlaps an input but for one case: *d_free_head may lie in d_counts, so
 * that a step with fixed buffers goes on from its own last result (d_counts + 1);
 * above 256 tokens that takes a second launch.
 *   d_ctx, d_new: int32[requests]; negative values count as 0.
 *   d_free: int32[free_len] page ids that may be taken, from *d_free_head on.
 *   d_table: int32[requests, width]; columns of pages taken now are written.
 *   d_parents: NULL (the new tokens of a request are a chain) or int32[tokens]:
 *          parent of a drafted token, as an index within its request's new
 *          tokens, below its own index; -1 hangs it off the cached context.
 * Request b is refused if its pages would not fit `width`, its rows would not
 * fit `tokens`, or the free list has too few pages for it and the requests
 * before it; it then takes no page.
 *   d_cu: int32[requests + 1], the exclusive sums of new, cut to `tokens`.
 *   d_slots: int32[tokens], slot of each new token (token i of b is stored at
 *          position ctx[b] + i); -1 for rows of no request or a refused one.
 *   d_positions: int32[tokens]: ctx[b] + i, or ctx[b] + depth in the tree; -1
 *          for rows of no request.
 *   d_mask (with d_parents, else NULL and mask_words 0): uint64[tokens,
 *          mask_words]: bit j is set if j is the token itself or one of its
 *          ancestors.  mask_words <= 1024.
 *   d_counts: int32[3]: rows needed (tokens + 1 if more than `tokens`), the
 *          free list's new head, requests refused.
 * A request's pages are counted by its length, ceil(ctx / block).  Where drafted
 * tokens are dropped again, pages past the kept ones go back to the free list before
 * the next plan, in front of its head: those ids into d_free[head - count ..
 * head - 1], and head - count as the head.
 * A token whose index does not fit the mask, or whose way to the root meets a
 * parent that is not below its child, gets slot -1, position -1 and no bits.
 * Errors: E_ARG, E_SHAPE, E_HIP. */
int dgt_page_plan(const int32_t* d_ctx, const int32_t* d_new, uint32_t requests,
                  const int32_t* d_free, uint32_t free_len, const int32_t* d_free_head,
                  int32_t* d_table, uint32_t width, uint32_t block, uint32_t blocks,
                  uint32_t tokens, const int32_t* d_parents, uint32_t mask_words, int32_t* d_cu,
                  int32_t* d_slots, int32_t* d_positions, uint64_t* d_mask, int32_t* d_counts,
                  void* stream);

/* Write the new tokens' keys and values into their slots.
 *   d_k, d_v: [tokens, heads, dim] of type `source` (a dgt_element), element
 *          strides per row and head given, elements of a head contiguous.
 *   cache: type of the pages, BF16 or F16; `source` is F32 (rounded to nearest
 *          even) or the same type (copied bit for bit).
 *   d_slots: int32[tokens]; slots outside the pool are skipped.  Two rows with
 *          one slot leave it with either's values.
 * dim is a multiple of 8, at most 1024.  Errors: E_ARG, E_SHAPE,
 * E_UNSUPPORTED, E_HIP. */
int dgt_kv_store(const void* d_k, const void* d_v, uint32_t source, int64_t k_row, int64_t k_head,
                 int64_t v_row, int64_t v_head, const int32_t* d_slots, uint32_t tokens,
                 uint32_t heads, uint32_t dim, uint32_t cache, void* d_k_cache, void* d_v_cache,
                 uint32_t blocks, uint32_t block, void* stream);

/* Attention of the new tokens over cached and new keys:
 *   out[i, h] = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale * q[i, h] . k_j),
 * j over the request's ctx[b] cached tokens and those of its new tokens
 * (stored at positions ctx[b] .. ctx[b] + n - 1) that token i sees: j with bit
 * set in its mask row, or without a mask every j <= i.  Query head h reads key
 * head h / (heads / kv_heads).  A row that sees no key is zero; keys that a row
 * does not see do not touch it, whatever their values.  Sums are fp32, weights
 * are rounded to `type` for the product with the values.
 *   type: BF16 or F16, of q, the pages and out.
 *   d_q, d_out: [tokens, heads, dim] with element strides per row and head,
 *          elements of a head contiguous; strides of q multiples of 8, of out
 *          of 2; q 16-byte aligned.  (A single row's stride is not looked at, nor a
 *          single head's.)  Rows past cu[requests] are not written.
 *   d_mask: uint64[tokens, mask_words] or NULL with mask_words 0.
 *   scale > 0.  dim: a multiple of 8 up to 256.
 *   d_ws: dgt_tree_attention_workspace(...) bytes, of which the first
 *          DGT_TREE_ATTENTION_ZEROED are zero-filled before its first use (the rest
 *          may hold anything); every call leaves it ready for the next (on one
 *          stream).  No other entry point's workspace: those would write over the zeros.
 * One launch; the order of all sums is fixed by the lengths and shapes.
 * Errors: E_ARG, E_SHAPE, E_BUFSIZE, E_UNSUPPORTED, E_HIP. */
#define DGT_TREE_ATTENTION_ZEROED 9216
size_t dgt_tree_attention_workspace(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim,
                                    uint32_t requests);
int dgt_tree_attention(uint32_t type, const void* d_q, uint64_t q_row, uint64_t q_head,
                       const void* d_k_cache, const void* d_v_cache, uint32_t blocks, uint32_t block,
                       const int32_t* d_table, uint32_t width, const int32_t* d_ctx, const int32_t* d_cu,
                       uint32_t requests, uint32_t tokens, uint32_t heads, uint32_t kv_heads,
                       uint32_t dim, const uint64_t* d_mask, uint32_t mask_words, float scale,
                       void* d_out, uint64_t out_row, uint64_t out_head, void* d_ws, size_t ws_bytes,
                       void* stream);

/* Low-rank adapters: out[t] = y[t] + scaling[a] * (x[t] A_a^T) B_a^T for the
 * adapter a = ids[b] of row t's request (cu as above); rows of a request whose
 * id is outside 0..adapters-1, or of no request, get out[t] = y[t].
 *   d_x: bf16 [tokens, k]; d_a: bf16 [adapters, rank, k]; d_b: bf16 [adapters,
 *          n, rank]; d_scaling: float[adapters]; d_y, d_out: fp32 [tokens, n];
 *          x_row, y_row, out_row are element strides of the rows, no shorter than a
 *          row (not looked at where tokens is 1).
 *   d_out may be d_y (then rows without an adapter are not touched); otherwise
 *          they do not overlap.
 * k is a multiple of 8, rank a multiple of 8 up to 256; x_row a multiple of 8; x, a, b 16-byte
 * aligned.  All sums are fp32 and of a fixed order.  d_ws: dgt_lora_workspace
 * bytes, any contents.  Errors: E_ARG, E_SHAPE, E_BUFSIZE, E_HIP. */
size_t dgt_lora_workspace(uint32_t tokens, uint32_t requests, uint32_t n, uint32_t k, uint32_t rank);
int dgt_lora_add(const float* d_y, uint64_t y_row, const uint16_t* d_x, uint64_t x_row,
                 const uint16_t* d_a, const uint16_t* d_b, const float* d_scaling, uint32_t adapters,
                 const int32_t* d_ids, const int32_t* d_cu, uint32_t requests, uint32_t tokens,
                 uint32_t n, uint32_t k, uint32_t rank, float* d_out, uint64_t out_row, void* d_ws,
                 size_t ws_bytes, void* stream);

/* Queries, keys and values of the new tokens out of the projection's rows: norms of
 * queries and keys for each head and the rotation by position in one pass, the
 * queries into 16-bit rows for the attention, keys and values into the paged cache.
 *   x^ = w x / sqrt(mean(x^2) + eps) over the dim elements of a head (without a
 *        weight array x^ = x);
 *   the first 2 * pairs elements of x^ are turned in pairs by the angle
 *        a_i = position * freqs[i]:  (x, y) -> (x cos a - y sin a, y cos a + x sin a);
 *        pairs are (i, i + pairs), or (2 i, 2 i + 1) with interleaved != 0.
 * All in fp32 (angles in fp64), rounded once to nearest even; values are only rounded.
 *   d_q [tokens, heads, dim], d_k, d_v [tokens, kv_heads, dim] of type `source`: F32,
 *          or the type of the cache; element strides per row and head, elements of a
 *          head contiguous.
 *   d_positions: int32[tokens]; rows with a negative one are skipped altogether.
 *   d_slots: int32[tokens]; keys and values of slots outside the pool are skipped (the
 *          queries are not).  Two rows with one slot leave it with either's values.
 *   d_freqs: double[pairs], radians a position; pairs <= dim / 2, 0 for no rotation.
 *   d_q_weight, d_k_weight: float[dim] or NULL.  eps >= 0.
 *   type: BF16 or F16, of d_q_out and the pages.  d_q_out [tokens, heads, dim], strides
 *          multiples of 8; it does not overlap an input.
 * dim: a multiple of 8 up to 256.  d_q_out and the pages are 16-byte aligned.  tokens <= 2^20,
 * and what the launch can count: about 2^29 token heads.
 * Errors: E_ARG, E_SHAPE, E_UNSUPPORTED, E_HIP. */
int dgt_rope_store(const void* d_q, const void* d_k, const void* d_v, uint32_t source, int64_t q_row,
                   int64_t q_head, int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                   const int32_t* d_positions, const int32_t* d_slots, uint32_t tokens, uint32_t heads,
                   uint32_t kv_heads, uint32_t dim, const double* d_freqs, uint32_t pairs,
                   uint32_t interleaved, const float* d_q_weight, const float* d_k_weight, float eps,
                   uint32_t type, void* d_q_out, int64_t out_row, int64_t out_head, void* d_k_cache,
                   void* d_v_cache, uint32_t blocks, uint32_t block, void* stream);

/* Attention of a chunk of new tokens (a prompt or a part of one) over cached and new
 * keys: what dgt_tree_attention computes without a mask, with its layouts and the
 * same values up to rounding, made for many new tokens a request: tiles of rows end at
 * their own last key, and long ones are split over the keys.
 * Which of the two (bf16, 32 query heads on 8 of 128): up to 16 new tokens a request
 * dgt_tree_attention takes less (32 requests behind 4000 tokens: one token 105 us, here 166;
 * 16 tokens 107, here 152), from 128 on this one (4000 of one prompt: 177 us, there 491); between
 * them it depends on the batch.  A step that mixes pieces of prompts with single tokens is best cut
 * where they differ most: 500 tokens behind 2000 and 32 single ones behind 4000 take 130 us there
 * and 192 here, 2000 tokens of a prompt beside them 260 and 189.
 *   d_ws: dgt_chunk_attention_workspace(...) bytes, any contents.  It has room for the parts of
 *          split tiles whatever the lengths are, and little of its size hangs on the arguments:
 *          68 MB for heads of up to 64 elements, 136 up to 128, 270 up to 256.  One serves all
 *          layers and steps of a stream.
 * Offsets whose rows are more than `tokens` (they fall somewhere) are not computed: nothing is written.
 * Three launches; the order of all sums is fixed by the lengths and shapes.
 * Errors: E_ARG, E_SHAPE, E_BUFSIZE, E_UNSUPPORTED, E_HIP. */
size_t dgt_chunk_attention_workspace(uint32_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim,
                                     uint32_t requests);
int dgt_chunk_attention(uint32_t type, const void* d_q, uint64_t q_row, uint64_t q_head,
                        const void* d_k_cache, const void* d_v_cache, uint32_t blocks, uint32_t block,
                        const int32_t* d_table, uint32_t width, const int32_t* d_ctx, const int32_t* d_cu,
                        uint32_t requests, uint32_t tokens, uint32_t heads, uint32_t kv_heads,
                        uint32_t dim, float scale, void* d_out, uint64_t out_row, uint64_t out_head,
                        void* d_ws, size_t ws_bytes, void* stream);

/* Verification of drafted tokens: which of them the target's probabilities accept,
 * and the token that follows, so that what comes out is distributed as the target's
 * own samples are.  Row 0 of a request is a token that is decided already; the others
 * are drafted, row i with token d_draft[i] to follow row parent(i) (d_parents as for
 * dgt_page_plan; NULL: a chain).  Rows whose way up does not end in row 0 are never
 * accepted.  At the path's end e (at first row 0), with p = softmax(logits[e] / T):
 *   the children of e are looked at in the order of their rows.  Without draft
 *   probabilities the drafts are taken as given: child i is accepted if
 *   u_i * Z < p(x_i), Z = 1 - the sum of p over the tokens of e refused so far; a token
 *   refused once is refused again.  With them (chains only): accepted if
 *   u_i * q(x_i) < p(x_i), q = d_probs[e].  The first accepted child becomes the end.
 *   With no child left the next token is the first v whose running sum of r passes
 *   s * sum(r): r = p without the refused tokens, or max(p - q, 0) after a refusal.
 * T = d_temperature[b] (NULL: 1); T <= 0 (or not a number): a child is accepted if its
 * token is the row's largest logit's (the first of equals), and so is the next token.  With
 * T = +inf all tokens that are not excluded weigh the same.
 * Decisions are those of fp64 sums over the vocabulary (of exponentials off by 2^-39): fp32
 * sums are only trusted where a draft's number lies further from its border than they can be off.
 *   d_logits: [tokens, vocab] of type `type` (F32, BF16, F16), row stride in elements;
 *          -inf excludes a token.  A row with a NaN or +inf, or of -inf alone, ends the
 *          path, and the next token is -1.
 *   d_draft: int32[tokens]; ids outside the vocabulary are refused.
 *   d_probs: NULL or float[tokens, vocab], row stride given: row e is what the token
 *          after row e was drawn from.  Values that are negative or NaN count as 0.
 *   d_accept: float[tokens], u of each row, in [0, 1); row 0's is not used.
 *   d_sample: float[requests], s, in [0, 1).
 *   d_path: int32[tokens]: the accepted rows as indexes within the request, row 0 first,
 *          then -1 to the request's end; rows past cu[requests] are not written.
 *   d_accepted: int32[requests], how many (0 for a request of no rows).
 *   d_next: int32[requests] (-1 for a request of no rows).
 *   d_ws: dgt_verify_workspace(...) bytes, any contents.
 * vocab <= 2^22; tokens * ceil(vocab / 4096) < 2^24 (tokens * vocab may pass 2^32).
 * Errors: E_ARG, E_SHAPE, E_BUFSIZE, E_UNSUPPORTED (draft probabilities of a tree), E_HIP. */
size_t dgt_verify_workspace(uint32_t tokens, uint32_t vocab, uint32_t requests);
int dgt_verify(uint32_t type, const void* d_logits, uint64_t logits_row, const int32_t* d_draft,
               const float* d_probs, uint64_t probs_row, const int32_t* d_parents, const int32_t* d_cu,
               const float* d_temperature, const float* d_accept, const float* d_sample,
               uint32_t requests, uint32_t tokens, uint32_t vocab, int32_t* d_path,
               int32_t* d_accepted, int32_t* d_next, void* d_ws, size_t ws_bytes, void* stream);

/* Pages of a cache: what a step keeps, requests that share pages, requests that end.
 * Caches here may hold several layers, [layers, blocks, ...] with the pages of each as
 * above; a page id means the same page in all of them.  A free list is int32[free_len],
 * its free ids from `head` on; pages go back in front of it.  d_free_head is read;
 * d_counts[0] is the new head (d_free_head may lie in d_counts).  Nothing else overlaps
 * but where it is said.  Elements are 16 bits and are copied bit for bit. */

/* After a step: of request b the first d_kept[b] rows of its path are kept (cut to its new
 * tokens).  Their keys and values move to the places of its first new tokens, in all
 * layers; its length becomes ctx[b] + kept; pages past that length go back to the list,
 * request by request, and their columns of the table become -1 (those too whose tokens the
 * plan gave no slot: they are looked up in the table, as the plan left it).
 *   d_path: int32[tokens] as dgt_verify writes it: row cu[b] + j holds the index, within
 *          the request, of the j-th kept row; or NULL: the first rows are kept.  The
 *          indexes rise; where one is out of range, or below j, the j-th place is left as it is.
 *          A row without a slot (dgt_page_plan gives none to a node past the mask or behind a
 *          bad link) was never stored: it is not kept, nor is what follows it or a place
 *          without a slot on the path, and the length does not count them.
 *   d_slots: int32[tokens], the step's slots (dgt_page_plan).  A request whose first new
 *          token has no slot (the plan refused it) keeps nothing and returns nothing.
 *   d_lens: int32[requests], the new lengths; may be d_ctx.
 *   d_counts: int32[2]: the list's new head, the pages that went back.
 * Errors: E_ARG, E_SHAPE, E_HIP. */
int dgt_page_keep(const int32_t* d_path, const int32_t* d_kept, const int32_t* d_ctx, const int32_t* d_cu,
                  const int32_t* d_slots, uint32_t requests, uint32_t tokens, int32_t* d_free,
                  uint32_t free_len, const int32_t* d_free_head, int32_t* d_table, uint32_t width,
                  uint32_t layers, uint32_t heads, uint32_t dim, uint32_t blocks, uint32_t block,
                  void* d_k_cache, void* d_v_cache, int32_t* d_lens, int32_t* d_counts, void* stream);

/* Fork: row dst[i] of the table becomes a request that holds what row src[i] holds.  Full
 * pages are shared; of a last page that is not full a copy is made, into a page of the
 * free list.  Both requests can then grow independently.
 *   d_shares: int32[blocks], how many requests hold a page besides the first; zero for
 *          pages that the plan hands out.
 *   d_lens: int32[requests]; dst[i] must be empty (length 0) and gets src[i]'s length.
 * Fork i is refused, and changes nothing, if src or dst is out of range, src is empty or
 * its pages do not fit the table, dst is not empty, an earlier i names the same dst, or the
 * list has no page left for it.
 *   d_counts: int32[2]: the list's new head, the forks that were refused.
 * forks and requests are at most 8192.  Errors: E_ARG, E_SHAPE, E_HIP. */
int dgt_page_fork(const int32_t* d_src, const int32_t* d_dst, uint32_t forks, int32_t* d_lens,
                  int32_t* d_table, uint32_t requests, uint32_t width, const int32_t* d_free,
                  uint32_t free_len, const int32_t* d_free_head, int32_t* d_shares, uint32_t layers,
                  uint32_t heads, uint32_t dim, uint32_t blocks, uint32_t block, void* d_k_cache,
                  void* d_v_cache, int32_t* d_counts, void* stream);

/* End of requests: the pages of rows d_rows, as far as their lengths go (pages that a plan took
 * for a step go back with dgt_page_keep, d_kept 0, first), lose a holder, and those that nobody else
 * holds go back to the list, in the order of their ids.  Their lengths become 0, their columns
 * of the table -1.  Rows out of range or named before are passed over.
 *   d_counts: int32[2]: the list's new head, the pages that went back.
 *   d_ws: dgt_page_free_workspace(blocks) bytes, zero-filled before its first use; every
 *          call leaves it ready for the next (on one stream).
 * count and requests are at most 8192.  Errors: E_ARG, E_SHAPE, E_BUFSIZE, E_HIP. */
size_t dgt_page_free_workspace(uint32_t blocks);
int dgt_page_free(const int32_t* d_rows, uint32_t count, int32_t* d_lens, int32_t* d_table,
                  uint32_t requests, uint32_t width, int32_t* d_free, uint32_t free_len,
                  const int32_t* d_free_head, int32_t* d_shares, uint32_t blocks, uint32_t block,
                  int32_t* d_counts, void* d_ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DGT_H_ */
