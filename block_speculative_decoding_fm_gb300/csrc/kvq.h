// kvq.h -- the 4-bit KV cache's memory layout, kernel argument blocks and
// launchers, shared by its host calls (kvq.cu) and its kernels.
//
// A plane holds one KV head of one sequence and layer in tiles of 64 rows.  A
// tile is one contiguous run [K codes | K scales | V codes | V scales]:
//   codes   64 rows of hd / 2 bytes.  A 16-byte unit holds the 32 values of a
//           group, value e in bits 4 e of the unit; the row's units are permuted
//           by unit ^ kvq_swz(row), so that the eight rows of an 8 x 16-byte
//           matrix fetch (ldmatrix) hit eight distinct bank groups.
//   scales  f16.  K: [row][group], a row's scales together.  V: [group][row % 8 / 2]
//           [row / 8][row % 2]: the pairs of neighbouring rows that one lane column of a
//           tensor-core fragment multiplies, together.
// So one bulk copy lands whole tiles in shared memory as the matrix
// instructions read them, K alone is contiguous too, and a row is written and
// moved without touching its neighbours' bytes.
#pragma once

#include <cstddef>
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

struct fm_kvq;

namespace fm {

int kvq_device(const fm_kvq *c);   // the device that a cache is on

constexpr int kKvqTile = 64;       // rows a tile
constexpr int kKvqSeqs = 64;       // sequences a launch
// tiles a stage, what the attention kernel fetches and deals out (four warps' strips of 32 or 16 rows)
__host__ __device__ constexpr int kvq_stage_tiles(int hd) { return hd == 256 ? 1 : 2; }
// what beginning and ending a unit costs a CTA, in stages: a unit takes that many places before its stages' where shares
// are dealt out, so that shares of many short units are as long as shares of one long one
constexpr int kKvqUnitCost = 4;
constexpr int kKvqMaxNQ = 4;       // a unit carries 8 nq query rows (block row x head of the group), nq <= 4

enum KvqType : int32_t { KVQ_F32 = 0, KVQ_F16 = 1, KVQ_BF16 = 2 };

__host__ __device__ constexpr int kvq_tile_bytes(int hd) { return 72 * hd; }
__host__ __device__ constexpr int kvq_k_bytes(int hd) { return 36 * hd; }       // K codes and scales
__host__ __device__ constexpr int kvq_scale_off(int hd) { return 32 * hd; }     // inside a K or V half
// which way row r's 16-byte units are permuted: r / (rows per 128 bytes), modulo the units a row
__host__ __device__ constexpr int kvq_swz(int r, int hd) {
  return hd == 64 ? (r >> 2) & 1 : hd == 128 ? (r >> 1) & 3 : r & 7;
}
// byte offset of unit u (group u's codes) of row r, and of its scale, inside a K or V half tile
__host__ __device__ constexpr int kvq_unit(int r, int u, int hd) { return r * (hd / 2) + ((u ^ kvq_swz(r, hd)) << 4); }
__host__ __device__ constexpr int kvq_kscale(int r, int u, int hd) { return kvq_scale_off(hd) + (r * (hd / 32) + u) * 2; }
__host__ __device__ constexpr int kvq_vscale(int r, int u, int hd) {
  return kvq_scale_off(hd) + ((u * 4 + (r & 7) / 2) * 16 + (r >> 3) * 2 + (r & 1)) * 2;
}
__host__ __device__ constexpr int kvq_scale(int r, int u, int hd, bool v) {
  return v ? kvq_vscale(r, u, hd) : kvq_kscale(r, u, hd);
}

// What every launch knows of the cache (pointers of the call's layer).
struct KvqCache {
  uint8_t *planes;        // [seqs][kv heads] planes of plane_bytes
  size_t plane_bytes;
  float *weights;         // [seqs][kv heads][rows_pad] accumulated attention weights
  int32_t rows_pad;       // rows of a plane (a multiple of 64)
  int32_t n_kv;
  int32_t *err;           // raised when a bounded wait gives up
};

// append and read: rows packed by sequence <-> cache rows at[i] .. at[i] + rows[i] - 1
struct KvqRowsArgs {
  KvqCache c;
  const void *k, *v;      // append: source rows [n][n_kv][hd], row stride ld elements
  void *ko, *vo;          // read: destination rows (each may be null)
  int64_t ld;
  float *wo;              // read: weights out [call sequences][n_kv][ldw], or null
  const float *wi;        // set_weights: weights in, or null
  int64_t ldw;
  int32_t n, type;
  int32_t tiles;          // tiles touched, all sequences (grid x)
  int32_t call0;          // the first sequence's place in the call (rows of wo)
  int64_t row0[kKvqSeqs];
  int32_t seq[kKvqSeqs], at[kKvqSeqs], rows[kKvqSeqs];
  int32_t tile0[kKvqSeqs + 1];   // prefix sums of the tiles each sequence touches
};
cudaError_t launch_kvq_append(const KvqRowsArgs &a, int hd, cudaStream_t s);
cudaError_t launch_kvq_read(const KvqRowsArgs &a, int hd, cudaStream_t s);
cudaError_t launch_kvq_set_weights(const KvqRowsArgs &a, cudaStream_t s);

struct KvqAttnArgs {
  KvqCache c;
  const void *q;          // [rows][n_heads][hd], row stride ldq elements
  void *out;              // the same shape, row stride ldo
  int64_t ldq, ldo;
  int32_t type;           // KvqType of q and out
  int32_t group;          // query heads a KV head
  int32_t nq;             // query rows of a unit / 8
  float scale_log2;       // scale * log2(e)
  int32_t causal, first;  // row t of T sees rows first <= j < (causal ? len - T + t + 1 : len)
  int32_t n;              // sequences of this launch
  // CTAs of the launch, and their shares of the W = st0[n] places.  share > 0: CTA b takes share = W / ctas, and one more
  // where b < extra = W % ctas, whatever units they belong to.  share 0: a unit of sequence i has parts[i] CTAs of its own.
  int32_t ctas, share, extra;
  int32_t parts[kKvqSeqs];
  int32_t cta0[kKvqSeqs + 1];    // share 0: prefix sums of units x parts
  float *part_o;          // [2 ctas][8 nq][hd] unnormalised partial outputs
  float2 *part_ml;        // [2 ctas][8 nq] (reference, row sum)
  float *lse;             // [units][8 nq] log2 of the row sums, for the weights; or null
  int32_t wtiles;         // weights: tiles a CTA
  float decay;            // weights: w = decay w + this call's
  float *w_out;           // [call sequences][n_kv][ldw] or null
  int64_t ldw;
  int32_t call0;
  int64_t row0[kKvqSeqs];
  int32_t seq[kKvqSeqs], len[kKvqSeqs], rows[kKvqSeqs];
  // A unit is a (KV head, tile of 8 nq query rows) of a sequence; its keys are stages, one at least.
  int32_t stages[kKvqSeqs];      // of a unit
  int32_t st0[kKvqSeqs + 1];     // prefix sums of units x (kKvqUnitCost + stages)
  int32_t unit0[kKvqSeqs + 1];   // prefix sums of row tiles (lse is by (row tile, KV head))
  int32_t wt0[kKvqSeqs + 1];     // weights: prefix sums of the CTAs of each sequence
};
// attention (weights false) or its pass over the weights, which follows it
template <int HD>
cudaError_t kvq_attn_call(const KvqAttnArgs &a, bool weights, cudaStream_t s);
// the attention kernel's CTAs an SM, and the groups of four warps a CTA that take its stages in turn
struct KvqShape {
  int ctas, groups;
};
template <int HD>
KvqShape kvq_attn_shape(int type, int nq);
constexpr int kKvqMaxCtas = 2;
constexpr int kKvqWeightTiles = 16;   // tiles a CTA of the weights pass covers at most

struct KvqEvictArgs {
  KvqCache c;
  int32_t n, keep, recent;
  int32_t n_sm;           // of the device, by which the launches are shaped
  int32_t *kept;          // [call sequences][n_kv][keep] or null
  int32_t *list;          // [n][n_kv][rows_pad] scratch: the rows kept, in order
  int32_t call0;
  int32_t src[kKvqSeqs], dst[kKvqSeqs], len[kKvqSeqs];
};
cudaError_t launch_kvq_evict(const KvqEvictArgs &a, int hd, cudaStream_t s);

int &kvq_launches();   // this thread's launches since a call began

// lets a kernel have its dynamic shared memory, once a device (done: a bit a device)
template <typename K>
inline cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename K, typename... Args>
inline cudaError_t kvq_launch(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ++kvq_launches();
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace fm
