// paged.cu -- the paged KV cache's host calls: argument checks, the rotation's frequencies, tensor maps, the choice of the
// attention kernel, the launches (k_paged_write.cu; paged_rows.cuh and paged_chunk.cuh by way of k_paged_attn64.cu,
// k_paged_attn128.cu and k_paged_attn256.cu).
//
// The pool, the batch's metadata and the attention's workspace are the caller's; a handle holds the configuration, the
// frequencies, the pool's tensor maps and an error word, and calls change nothing in it: they allocate nothing, copy
// nothing and may be captured into a graph, which is then replayed with other starts, lengths and pages.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include <cudaTypedefs.h>

#include "../../include/fm.h"
#include "fm_internal.h"
#include "paged.h"

using namespace fm;

struct fm_paged {
  fm_paged_config cfg{};
  int device = 0, n_sm = 0;
  void *k_pool = nullptr, *v_pool = nullptr;
  int page_log = 0;
  int64_t rows = 0;              // of the pool
  CUtensorMap tk, tv;
  void *block = nullptr;         // all device memory: frequencies, error words
  uint64_t *freq = nullptr;
  int32_t *dev_err = nullptr;    // what went wrong: a wait gave up, a batch pointed outside
  int32_t *taken = nullptr;      // the error that a check takes, under its lock
  std::mutex taking;
};

namespace {

thread_local char g_paged_error[512] = "";
thread_local int g_paged_launches = 0;

fm_status pfail(fm_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_paged_error, sizeof g_paged_error, fmt, ap);
  va_end(ap);
  return s;
}

#define PCK(expr)                                                                              \
  do {                                                                                         \
    cudaError_t e_ = (expr);                                                                   \
    if (e_ != cudaSuccess) {                                                                   \
      cudaGetLastError();                                                                      \
      return pfail(FM_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_));                      \
    }                                                                                          \
  } while (0)
#define PTRY(expr)              \
  do {                          \
    fm_status s_ = (expr);      \
    if (s_ != FM_OK) return s_; \
  } while (0)

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  return fn;
}

bool encode(CUtensorMap *map, const void *p, int dims, const cuuint64_t *size, const cuuint64_t *stride, const cuuint32_t *box) {
  const auto fn = encoder();
  const cuuint32_t one[3] = {1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, const_cast<void *>(p), size, stride, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;   // (16-bit words; zeros outside)
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Angle a position of pair i, in turns (rotary positions; by parts: Peng et al., "YaRN", section 3.2).
double turns(const fm_paged_config &g, int i) {
  const double pi = 3.14159265358979323846;
  const double f = std::pow((double)g.theta, -2.0 * i / g.rot_dims) / (2.0 * pi);
  if (g.rope_scaling == FM_ROPE_LINEAR) return f / g.rope_factor;
  if (g.rope_scaling == FM_ROPE_BY_PARTS) {
    const double r = std::min(1.0, std::max(0.0, (g.rope_rows * f - g.rope_low) / ((double)g.rope_high - g.rope_low)));
    return f * (r + (1.0 - r) / g.rope_factor);
  }
  return f;
}

fm_status check_config(const fm_paged_config &g) {
  if (g.n_layers < 1 || g.n_layers > 1024 || g.n_pages < 1 || g.n_kv_heads < 1 || g.n_kv_heads > 256 || g.n_heads < g.n_kv_heads ||
      g.n_heads % g.n_kv_heads)
    return pfail(FM_ERR_INVALID_ARG, "%d layers, %d pages, %d heads over %d KV heads", g.n_layers, g.n_pages, g.n_heads, g.n_kv_heads);
  if (g.n_heads / g.n_kv_heads > 128) return pfail(FM_ERR_UNSUPPORTED, "%d heads a KV head: at most 128", g.n_heads / g.n_kv_heads);
  if (g.head_dim != 64 && g.head_dim != 128 && g.head_dim != 256)
    return pfail(FM_ERR_UNSUPPORTED, "head_dim %d: 64, 128 or 256", g.head_dim);
  if (g.page_rows != 16 && g.page_rows != 32 && g.page_rows != 64 && g.page_rows != 128 && g.page_rows != 256)
    return pfail(FM_ERR_UNSUPPORTED, "page_rows %d: 16, 32, 64, 128 or 256", g.page_rows);
  if (g.dtype != FM_DTYPE_F16 && g.dtype != FM_DTYPE_BF16) return pfail(FM_ERR_INVALID_ARG, "dtype %d: f16 or bf16", g.dtype);
  if (!(g.eps >= 0.f) || !std::isfinite(g.eps)) return pfail(FM_ERR_INVALID_ARG, "eps %g", g.eps);
  if ((double)g.n_layers * g.n_pages * g.n_kv_heads * g.page_rows > 2147483391.0)
    return pfail(FM_ERR_UNSUPPORTED, "the pool has over 2^31 - 257 rows of heads");
  if (g.rot_dims < 0 || g.rot_dims > g.head_dim || g.rot_dims % 16)
    return pfail(FM_ERR_INVALID_ARG, "rot_dims %d: a multiple of 16 up to head_dim", g.rot_dims);
  if (g.rot_dims == 0) return FM_OK;
  if (g.rot_layout != FM_ROPE_INTERLEAVED && g.rot_layout != FM_ROPE_HALF) return pfail(FM_ERR_INVALID_ARG, "rot_layout %d", g.rot_layout);
  if (g.rope_scaling != FM_ROPE_PLAIN && g.rope_scaling != FM_ROPE_LINEAR && g.rope_scaling != FM_ROPE_BY_PARTS)
    return pfail(FM_ERR_INVALID_ARG, "rope_scaling %d", g.rope_scaling);
  if (!(g.theta >= 1.f) || !std::isfinite(g.theta)) return pfail(FM_ERR_INVALID_ARG, "theta %g: at least 1", g.theta);
  if (!std::isfinite(g.rope_gain) || !(g.rope_gain > 0.f)) return pfail(FM_ERR_INVALID_ARG, "rope_gain %g", g.rope_gain);
  if (g.rope_scaling != FM_ROPE_PLAIN && (!(g.rope_factor >= 1.f) || !std::isfinite(g.rope_factor)))
    return pfail(FM_ERR_INVALID_ARG, "rope_factor %g: at least 1", g.rope_factor);
  if (g.rope_scaling == FM_ROPE_BY_PARTS && (g.rope_rows < 1 || !(g.rope_high > g.rope_low) || !(g.rope_low >= 0.f) || !std::isfinite(g.rope_high)))
    return pfail(FM_ERR_INVALID_ARG, "by parts: %d rows, turns %g to %g", g.rope_rows, g.rope_low, g.rope_high);
  return FM_OK;
}

// One error taken out of the handle's words: read and cleared in one step, so that one that another stream raises meanwhile stays
// for the next check, as the second kind does where there are both.
__global__ void paged_take_kernel(int32_t *err, int32_t *taken) {
  const int wait = atomicExch(err, 0);
  taken[0] = wait;
  taken[1] = wait ? 0 : atomicExch(err + 1, 0);
}

void release(fm_paged *c) {
  if (c->block) cudaFree(c->block);
  delete c;
}

fm_status setup(fm_paged *c, cudaStream_t s) {
  const fm_paged_config &g = c->cfg;
  PCK(cudaGetDevice(&c->device));
  PCK(cudaDeviceGetAttribute(&c->n_sm, cudaDevAttrMultiProcessorCount, c->device));
  while ((1 << c->page_log) < g.page_rows) ++c->page_log;
  c->rows = (int64_t)g.n_layers * g.n_pages * g.n_kv_heads * g.page_rows;
  const cuuint64_t size[2] = {(cuuint64_t)g.head_dim, (cuuint64_t)c->rows}, stride[1] = {(cuuint64_t)g.head_dim * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)std::min(g.page_rows, kPagedBox)};
  if (!encode(&c->tk, c->k_pool, 2, size, stride, box) || !encode(&c->tv, c->v_pool, 2, size, stride, box))
    return pfail(FM_ERR_CUDA, "the pool's tensor maps could not be made");
  if (cudaMalloc(&c->block, 1024 + 256) != cudaSuccess) {   // up to 128 frequencies
    cudaGetLastError();
    c->block = nullptr;
    return pfail(FM_ERR_OOM, "the device allocation failed");
  }
  c->freq = static_cast<uint64_t *>(c->block);
  c->dev_err = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(c->block) + 1024);
  c->taken = c->dev_err + 32;   // (a line of its own)
  uint64_t host[(1024 + 256) / 8] = {};
  for (int i = 0; i < g.rot_dims / 2; ++i) {
    // f / 2 pi in units of 2^-64: two 32-bit digits, the second from the first's exact remainder
    const double t = std::ldexp(turns(g, i), 32), hi = std::floor(t);
    host[i] = ((uint64_t)hi << 32) + (uint64_t)std::llround(std::ldexp(t - hi, 32));
  }
  PCK(cudaMemcpyAsync(c->block, host, sizeof host, cudaMemcpyHostToDevice, s));
  PCK(cudaStreamSynchronize(s));
  return FM_OK;
}

fm_status check_call(const fm_paged *c, int layer, const fm_paged_batch *b, PagedBatch *out) {
  g_paged_launches = 0;
  int dev = -1;
  PCK(cudaGetDevice(&dev));
  if (dev != c->device) return pfail(FM_ERR_INVALID_ARG, "the current device is %d, the cache's is %d", dev, c->device);
  const fm_paged_config &g = c->cfg;
  if (layer < 0 || layer >= g.n_layers) return pfail(FM_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, g.n_layers);
  if (!b) return pfail(FM_ERR_INVALID_ARG, "null batch");
  if (b->n_seqs < 0 || b->n_tokens < 0 || b->max_new < 0 || b->table_pages < 0)
    return pfail(FM_ERR_INVALID_ARG, "a batch of %d sequences, %d tokens (%d a sequence), %d pages", b->n_seqs, b->n_tokens, b->max_new,
                 b->table_pages);
  if (b->n_seqs > 65536) return pfail(FM_ERR_UNSUPPORTED, "%d sequences: at most 65536", b->n_seqs);
  if ((int64_t)b->n_tokens * (g.n_heads + 2 * g.n_kv_heads) > INT32_MAX)
    return pfail(FM_ERR_UNSUPPORTED, "%d tokens of %d heads: at most 2^31 - 1 rows of heads", b->n_tokens, g.n_heads + 2 * g.n_kv_heads);
  if ((int64_t)b->table_pages * g.page_rows > kPagedMaxRows)
    return pfail(FM_ERR_UNSUPPORTED, "%d pages of %d rows a sequence: at most 2^30 rows", b->table_pages, g.page_rows);
  if (b->n_seqs > 0 && b->n_tokens > 0) {
    if (!b->starts || !b->lengths || !aligned4(b->starts) || !aligned4(b->lengths))
      return pfail(FM_ERR_INVALID_ARG, "starts or lengths: a null or misaligned pointer (4 bytes)");
    if (b->table_pages > 0 && (!b->table || !aligned4(b->table) || b->table_ld < b->table_pages))
      return pfail(FM_ERR_INVALID_ARG, "table: a null or misaligned pointer (4 bytes), or a row stride of %lld below %d pages",
                   (long long)b->table_ld, b->table_pages);
  }
  *out = {b->starts, b->lengths, b->table, b->table_ld, b->n_seqs, b->n_tokens, b->table_pages, c->page_log, g.n_pages,
          layer * g.n_pages, g.n_kv_heads, g.n_heads / g.n_kv_heads, 128 / (g.n_heads / g.n_kv_heads),
          65536u / (uint32_t)(g.n_heads / g.n_kv_heads) + 1, c->dev_err};
  return FM_OK;
}

// Rows [n_tokens][heads][head_dim]: strides that do not matter are made whole ones.
fm_status check_rows(const char *what, const fm_paged_rows *r, int n_tokens, int heads, int hd, int size, PagedRows *out) {
  if (!r->data || !aligned16(r->data)) return pfail(FM_ERR_INVALID_ARG, "%s: a null or misaligned pointer (16 bytes)", what);
  *out = {r->data, r->token_stride, r->head_stride};
  if (heads == 1) out->hs = hd;
  if (out->hs < hd || out->hs * size % 16 || out->hs > (int64_t)1 << 31)
    return pfail(FM_ERR_INVALID_ARG, "%s: head stride %lld (at least %d, whole 16 bytes, at most 2^31)", what, (long long)out->hs, hd);
  if (n_tokens == 1) out->ld = out->hs * heads;
  if (out->ld < hd || out->ld * size % 16 || out->ld > (int64_t)1 << 36)
    return pfail(FM_ERR_INVALID_ARG, "%s: token stride %lld (at least %d, whole 16 bytes, at most 2^36)", what, (long long)out->ld, hd);
  return FM_OK;
}

// The attention kernel for at most max_new new tokens a sequence.  Up to 16 (token, head) rows a KV head: tiles of 16 rows.
// More: tiles of 128, two at a time where a sequence may have more than one and two fit tensor memory (head dims 64, 128).
// One choice serves a whole call; a sequence with fewer rows costs a tile of its own, which memory, not the tile, bounds.
int kind_of(const fm_paged_config &g, int max_new) {
  const int group = g.n_heads / g.n_kv_heads;
  if ((int64_t)max_new * group <= 16) return 0;
  return g.head_dim < 256 && max_new > 128 / group ? 2 : 1;
}
PagedShape shape_of(const fm_paged *c, int kind) {
  const int hd = c->cfg.head_dim;
  return hd == 64 ? paged_attn_shape<64>(kind, c->n_sm) : hd == 128 ? paged_attn_shape<128>(kind, c->n_sm) : paged_attn_shape<256>(kind, c->n_sm);
}
// parts, their sums, the units that are cut: every part of the workspace on a 16-byte boundary
int64_t shape_bytes(const PagedShape &s, int hd) { return (int64_t)2 * s.ctas * s.rows * (4 * hd + 8) + 16ll * s.ctas; }

int64_t workspace_of(const fm_paged *c, int max_new) {
  int64_t bytes = 0;
  for (int kind = 0; kind <= kind_of(c->cfg, max_new); ++kind) bytes = std::max(bytes, shape_bytes(shape_of(c, kind), c->cfg.head_dim));
  return bytes;
}

}  // namespace

int fm::paged_device(const fm_paged *c) { return c->device; }

extern "C" {

fm_status fm_paged_create(const fm_paged_config *cfg, void *k_pool_dev, void *v_pool_dev, void *stream, fm_paged **out) {
  if (!out) return pfail(FM_ERR_INVALID_ARG, "null out");
  *out = nullptr;
  if (!cfg) return pfail(FM_ERR_INVALID_ARG, "null config");
  PTRY(check_config(*cfg));
  if (!k_pool_dev || !v_pool_dev || !aligned16(k_pool_dev) || !aligned16(v_pool_dev) || k_pool_dev == v_pool_dev)
    return pfail(FM_ERR_INVALID_ARG, "k_pool, v_pool: null, misaligned (16 bytes) or the same");
  fm_paged *c = new (std::nothrow) fm_paged();
  if (!c) return pfail(FM_ERR_OOM, "out of host memory");
  c->cfg = *cfg;
  c->k_pool = k_pool_dev;
  c->v_pool = v_pool_dev;
  const fm_status s = setup(c, static_cast<cudaStream_t>(stream));
  if (s != FM_OK) {
    release(c);
    return s;
  }
  *out = c;
  return FM_OK;
}

fm_status fm_paged_write(fm_paged *c, int32_t layer, const fm_paged_batch *batch, const fm_paged_rows *q, const fm_paged_rows *k,
                         const fm_paged_rows *v, int32_t dtype, const float *q_norm_dev, const float *k_norm_dev,
                         const fm_paged_rows *q_out, void *stream) {
  if (!c) return pfail(FM_ERR_INVALID_ARG, "null cache");
  PagedWriteArgs a = {};
  PTRY(check_call(c, layer, batch, &a.b));
  const fm_paged_config &g = c->cfg;
  if (dtype != g.dtype && dtype != FM_DTYPE_F32) return pfail(FM_ERR_INVALID_ARG, "dtype %d: f32, or the pool's %d", dtype, g.dtype);
  if ((k != nullptr) != (v != nullptr)) return pfail(FM_ERR_INVALID_ARG, "k without v, or v without k");
  if ((q != nullptr) != (q_out != nullptr)) return pfail(FM_ERR_INVALID_ARG, "q without q_out, or q_out without q");
  if (!q && !k) return pfail(FM_ERR_INVALID_ARG, "neither q nor k");
  if ((q_norm_dev && !aligned16(q_norm_dev)) || (k_norm_dev && !aligned16(k_norm_dev)))
    return pfail(FM_ERR_INVALID_ARG, "norm weights: a misaligned pointer (16 bytes)");
  const int size = dtype == FM_DTYPE_F32 ? 4 : 2;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return FM_OK;
  if (q) {
    PTRY(check_rows("q", q, batch->n_tokens, g.n_heads, g.head_dim, size, &a.q));
    PTRY(check_rows("q_out", q_out, batch->n_tokens, g.n_heads, g.head_dim, 2, &a.qo));
    // (a row is read as a whole before it is written, by the lanes that write it)
    if (q->data == q_out->data && (size != 2 || a.q.ld != a.qo.ld || a.q.hs != a.qo.hs))
      return pfail(FM_ERR_INVALID_ARG, "q_out in the place of q has another type or other strides");
  }
  if (k) {
    PTRY(check_rows("k", k, batch->n_tokens, g.n_kv_heads, g.head_dim, size, &a.k));
    PTRY(check_rows("v", v, batch->n_tokens, g.n_kv_heads, g.head_dim, size, &a.v));
  }
  a.k_pool = c->k_pool;
  a.v_pool = c->v_pool;
  a.q_norm = q_norm_dev;
  a.k_norm = k_norm_dev;
  a.freq = c->freq;
  a.hd = g.head_dim;
  a.rot = g.rot_dims;
  a.half = g.rot_layout == FM_ROPE_HALF;
  a.eps = g.eps;
  a.gain = g.rope_gain;
  a.in_f32 = dtype == FM_DTYPE_F32;
  a.bf16 = g.dtype == FM_DTYPE_BF16;
  a.slots = (q ? g.n_heads : 0) + (k ? 2 * g.n_kv_heads : 0);
  PCK(launch_paged_write(a, c->n_sm, static_cast<cudaStream_t>(stream)));
  g_paged_launches = 1;
  return FM_OK;
}

fm_status fm_paged_workspace_bytes(const fm_paged *c, int32_t max_new, int64_t *bytes) {
  if (!c || !bytes || max_new < 0) return pfail(FM_ERR_INVALID_ARG, "null cache or bytes, or max_new %d", max_new);
  *bytes = workspace_of(c, max_new);
  return FM_OK;
}

fm_status fm_paged_attend(fm_paged *c, int32_t layer, const fm_paged_batch *batch, const fm_paged_rows *q, const fm_paged_rows *out,
                          float scale, int32_t causal, int32_t window, int32_t sinks, void *workspace_dev, int64_t workspace_bytes,
                          void *stream) {
  if (!c) return pfail(FM_ERR_INVALID_ARG, "null cache");
  PagedAttnArgs a = {};
  PTRY(check_call(c, layer, batch, &a.b));
  const fm_paged_config &g = c->cfg;
  if (!q || !out) return pfail(FM_ERR_INVALID_ARG, "null q or out");
  if (!(scale >= 1e-30f && scale <= 1e30f)) return pfail(FM_ERR_INVALID_ARG, "scale %g: 1e-30 to 1e30", scale);
  if (window < 0 || sinks < 0) return pfail(FM_ERR_INVALID_ARG, "window %d, sinks %d", window, sinks);
  if (window > 0 && !causal) return pfail(FM_ERR_INVALID_ARG, "a window without causal order");
  if (sinks > 0 && window == 0) return pfail(FM_ERR_INVALID_ARG, "sinks without a window");
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return FM_OK;
  PTRY(check_rows("q", q, batch->n_tokens, g.n_heads, g.head_dim, 2, &a.q));
  PTRY(check_rows("out", out, batch->n_tokens, g.n_heads, g.head_dim, 2, &a.out));
  if (q->data == out->data) return pfail(FM_ERR_INVALID_ARG, "out in the place of q");
  const int64_t need = workspace_of(c, batch->max_new);
  if (!workspace_dev || !aligned16(workspace_dev) || workspace_bytes < need)
    return pfail(FM_ERR_INVALID_ARG, "workspace: null, misaligned (16 bytes) or %lld bytes of %lld", (long long)workspace_bytes, (long long)need);
  const int kind = kind_of(g, batch->max_new);
  const PagedShape shape = shape_of(c, kind);
  a.tk = c->tk;
  a.tv = c->tv;
  if (kind > 0) {
    const cuuint64_t size[3] = {(cuuint64_t)g.head_dim, (cuuint64_t)g.n_heads, (cuuint64_t)batch->n_tokens};
    const cuuint64_t stride[2] = {(cuuint64_t)a.q.hs * 2, (cuuint64_t)a.q.ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.b.group, (cuuint32_t)(128 / a.b.group)};
    if (!encode(&a.tq, a.q.p, 3, size, stride, box)) return pfail(FM_ERR_CUDA, "the queries' tensor map could not be made");
  }
  a.v_pool = c->v_pool;
  a.oob_row = (int32_t)c->rows;
  a.causal = causal != 0;
  a.window = window < kPagedMaxRows ? window : 0;   // (no sequence is longer)
  a.sinks = std::min(sinks, kPagedMaxRows);
  a.scale_log2 = scale * 1.4426950408889634f;
  uint8_t *w = static_cast<uint8_t *>(workspace_dev);
  a.desc = reinterpret_cast<int4 *>(w);
  w += 16ll * shape.ctas;
  a.part_o = reinterpret_cast<float *>(w);
  w += (int64_t)2 * shape.ctas * shape.rows * g.head_dim * 4;
  a.part_ml = reinterpret_cast<float2 *>(w);
  const bool bf = g.dtype == FM_DTYPE_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PCK(g.head_dim == 64 ? paged_attn_call<64>(a, kind, bf, c->n_sm, s)
      : g.head_dim == 128 ? paged_attn_call<128>(a, kind, bf, c->n_sm, s)
                          : paged_attn_call<256>(a, kind, bf, c->n_sm, s));
  g_paged_launches = 2;
  return FM_OK;
}

fm_status fm_paged_get_config(const fm_paged *c, fm_paged_config *cfg) {
  if (!c || !cfg) return pfail(FM_ERR_INVALID_ARG, "null cache or config");
  *cfg = c->cfg;
  return FM_OK;
}

fm_status fm_paged_last_launch_count(const fm_paged *c, int32_t *count) {
  if (!c || !count) return pfail(FM_ERR_INVALID_ARG, "null cache or count");
  *count = g_paged_launches;
  return FM_OK;
}

fm_status fm_paged_synchronize(fm_paged *c, void *stream) {
  if (!c) return pfail(FM_ERR_INVALID_ARG, "null cache");
  int dev = -1;
  PCK(cudaGetDevice(&dev));
  if (dev != c->device) return pfail(FM_ERR_INVALID_ARG, "the current device is %d, the cache's is %d", dev, c->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t e[2] = {0, 0};
  PCK(cudaMemcpyAsync(e, c->dev_err, sizeof e, cudaMemcpyDeviceToHost, s));
  PCK(cudaStreamSynchronize(s));
  if (!e[0] && !e[1]) return FM_OK;
  std::lock_guard<std::mutex> lock(c->taking);
  paged_take_kernel<<<1, 1, 0, s>>>(c->dev_err, c->taken);
  PCK(cudaGetLastError());
  PCK(cudaMemcpyAsync(e, c->taken, sizeof e, cudaMemcpyDeviceToHost, s));
  PCK(cudaStreamSynchronize(s));
  if (!e[0] && !e[1]) return FM_OK;   // (another thread's check has reported it)
  return e[0] ? pfail(FM_ERR_TIMEOUT, "a bounded device wait gave up")
              : pfail(FM_ERR_INVALID_ARG, "a batch's starts, lengths or pages lay outside the batch, its table or the pool");
}

fm_status fm_paged_selftest_wait_timeout(fm_paged *c, int32_t budget_us, void *stream) {
  if (!c) return pfail(FM_ERR_INVALID_ARG, "null cache");
  if (budget_us < 1 || budget_us > 1000000) return pfail(FM_ERR_INVALID_ARG, "budget_us %d outside [1, 1e6]", budget_us);
  int dev = -1;
  PCK(cudaGetDevice(&dev));
  if (dev != c->device) return pfail(FM_ERR_INVALID_ARG, "the current device is %d, the cache's is %d", dev, c->device);
  int khz = 0;
  PCK(cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, c->device));
  PCK(launch_wait_selftest(c->dev_err, (long long)budget_us * (khz / 1000), static_cast<cudaStream_t>(stream)));
  return FM_OK;
}

const char *fm_paged_last_error(const fm_paged *) { return g_paged_error; }

void fm_paged_destroy(fm_paged *c) {
  if (!c) return;
  // On the cache's device; and a capture that this thread may be in goes on (a Python object may be collected any time).
  // (Freeing waits for what runs.)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  int dev = -1;
  cudaThreadExchangeStreamCaptureMode(&mode);
  cudaGetDevice(&dev);
  const int own = c->device;
  if (dev != own) cudaSetDevice(own);
  release(c);
  if (dev != own) cudaSetDevice(dev);
  cudaThreadExchangeStreamCaptureMode(&mode);
}

}  // extern "C"
