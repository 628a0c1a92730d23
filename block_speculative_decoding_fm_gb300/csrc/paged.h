// paged.h -- the paged KV cache's kernel argument blocks and launchers, shared by its host calls
// (paged.cu) and its kernels.
//
// A layer's pool is [pages][kv heads][page rows][head dim], K and V apart, of f16 or bf16: a head's rows
// of a page are one contiguous run, which a 2-D tensor map over all rows of the pool cuts into boxes of
// 64 dims x up to 64 rows (128 bytes wide, the tensor cores' swizzle).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

struct fm_paged;

namespace fm {

int paged_device(const fm_paged *c);   // the device that a cache is on

constexpr int kPagedBox = 64;          // rows of a tensor-map box at most (a page's, if it has fewer)
constexpr int kPagedMaxRows = 1 << 30; // rows of a sequence (sums of two of them stay within 32 bits)

// What every launch knows of the batch and of the cache.
struct PagedBatch {
  const int32_t *starts;    // [n_seqs + 1]
  const int32_t *lengths;   // [n_seqs]
  const int32_t *table;     // [n_seqs][table_pages], table_ld apart
  int64_t table_ld;
  int32_t n_seqs, n_tokens, table_pages;
  int32_t page_log;         // log2 of a page's rows
  int32_t n_pages;          // of a layer
  int32_t page0;            // the layer's first page, counted over the pool
  int32_t n_kv, group;
  int32_t tile_tokens;      // whole tokens of a 128-row tile
  uint32_t group_inv;       // r / group = r group_inv / 2^16 for r < 128
  int32_t *err;             // [0] a bounded wait gave up, [1] the batch points outside the cache
};

// Rows [tokens][heads][head dim]: elements between tokens and between heads.
struct PagedRows {
  void *p;
  int64_t ld, hs;
};

struct PagedWriteArgs {
  PagedBatch b;
  PagedRows q, k, v, qo;    // q.p or k.p may be null: nothing of these
  void *k_pool, *v_pool;
  const float *q_norm, *k_norm;   // [head dim], or null: no norm
  const uint64_t *freq;     // [rot / 2] turns a position, in units of 2^-64
  int32_t hd, rot, half;    // half: pairs (i, i + rot/2), otherwise (2i, 2i + 1)
  float eps, gain;
  int32_t in_f32, bf16;     // rows are f32 (otherwise of the pool's type); the pool is bf16 (otherwise f16)
  int32_t slots;            // heads of a token that are to be done: q, then k, then v
  int32_t tokens, split;    // tokens a CTA, CTAs that share a token's heads
};

struct PagedAttnArgs {
  CUtensorMap tk, tv;       // the pool's rows: [all rows][head dim], box 64 dims x min(page rows, 64)
  CUtensorMap tq;           // the queries: [tokens][heads][head dim], box 64 dims x group x 128 / group (chunks only)
  PagedBatch b;
  PagedRows q, out;
  const void *v_pool;       // (read again where a hidden row of V holds an infinity or a NaN)
  int32_t oob_row;          // a row past the pool's last: boxes there read as zeros
  int32_t causal, window, sinks;   // window 0: none
  float scale_log2;
  float *part_o;            // [2 CTAs][unit rows][head dim] unnormalised sums of a unit's parts
  float2 *part_ml;          // [2 CTAs][unit rows] (reference in the log2 domain, sum of weights)
  int4 *desc;               // [CTAs] the unit that CTA i begins and does not end: sequence, KV head, tile, parts
};

// units of `rows` query rows, at most `ctas` CTAs: what the workspace has to hold
struct PagedShape {
  int32_t rows, ctas;
};

cudaError_t launch_paged_write(const PagedWriteArgs &a, int n_sm, cudaStream_t s);
// kind: 0 few rows (16 a unit), 1 one tile of 128 rows, 2 two tiles
template <int HD> PagedShape paged_attn_shape(int kind, int n_sm);
template <int HD> cudaError_t paged_attn_call(const PagedAttnArgs &a, int kind, bool bf16, int n_sm, cudaStream_t s);

}  // namespace fm
