// kvq.cu -- the 4-bit KV cache's host calls: argument checks, the lengths, the
// split of a call's work over the SMs, the launches (k_kvq_rows.cu,
// kvq_attn.cuh by way of k_kvq_attn64.cu, k_kvq_attn128.cu and k_kvq_attn256.cu,
// k_kvq_evict.cu).
//
// Every value that a call needs on the device rides in the kernels' argument
// blocks (64 sequences a launch), so nothing is copied or allocated after
// fm_kvq_create and a call can be captured into a graph.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/fm.h"
#include "fm_internal.h"
#include "kvq.h"

using namespace fm;

int &fm::kvq_launches() {
  thread_local int n = 0;
  return n;
}

struct fm_kvq {
  fm_kvq_config cfg{};
  int device = 0, n_sm = 0;
  int rows_pad = 0;
  size_t plane_bytes = 0;
  void *block = nullptr;          // all device memory
  uint8_t *planes = nullptr;
  float *weights = nullptr, *part_o = nullptr, *lse = nullptr;
  float2 *part_ml = nullptr;
  int32_t *list = nullptr, *dev_err = nullptr;
  int slots = 0;                  // partial results the workspace holds
  int64_t bytes = 0;
  std::vector<int32_t> len;       // [layers][seqs]
  std::vector<uint32_t> mark;     // [seqs] the last call that named a sequence (as a destination)
  uint32_t call = 0;
  cudaEvent_t done = nullptr;     // the last eager call's work
  unsigned long long last = 0;    // its stream's id (a handle may come back as another stream's)
  bool has_last = false;
  unsigned long long stream = 0;  // this call's
  bool eager = true;              // it is not captured
  int launches = 0;               // kernels that the last call launched
  char err[512] = "";
};

int fm::kvq_device(const fm_kvq *c) { return c->device; }

namespace {

constexpr int kMaxUnits = 1 << 15;   // (row tile, KV head) units of a launch
constexpr int kMaxRows = 1 << 24;

thread_local char g_kvq_error[512] = "";

// (the attention kernels are instantiated in a translation unit a head dim)
KvqShape attn_shape(int hd, int type, int nq) {
  return hd == 64 ? kvq_attn_shape<64>(type, nq) : hd == 128 ? kvq_attn_shape<128>(type, nq) : kvq_attn_shape<256>(type, nq);
}
cudaError_t launch_kvq_attn(const KvqAttnArgs &a, int hd, bool weights, cudaStream_t s) {
  return hd == 64 ? kvq_attn_call<64>(a, weights, s) : hd == 128 ? kvq_attn_call<128>(a, weights, s) : kvq_attn_call<256>(a, weights, s);
}

fm_status kfail(fm_kvq *c, fm_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(c ? c->err : g_kvq_error, sizeof g_kvq_error, fmt, ap);
  va_end(ap);
  return s;
}

#define KCK(expr)                                                                                 \
  do {                                                                                            \
    cudaError_t e_ = (expr);                                                                      \
    if (e_ != cudaSuccess) return kfail(c, FM_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_)); \
  } while (0)
#define KTRY(expr)          \
  do {                      \
    fm_status s_ = (expr);  \
    if (s_ != FM_OK) return s_; \
  } while (0)

int32_t *lengths(fm_kvq *c, int layer) { return c->len.data() + (size_t)layer * c->cfg.n_seqs; }

KvqCache view(const fm_kvq *c, int layer) {
  const size_t p0 = (size_t)layer * c->cfg.n_seqs * c->cfg.n_kv_heads;
  KvqCache v;
  v.planes = c->planes + p0 * c->plane_bytes;
  v.plane_bytes = c->plane_bytes;
  v.weights = c->weights + p0 * c->rows_pad;
  v.rows_pad = c->rows_pad;
  v.n_kv = c->cfg.n_kv_heads;
  v.err = c->dev_err;
  return v;
}

// the checks that every call begins with
fm_status check_call(fm_kvq *c, int layer, int n, const int32_t *ids) {
  int dev = -1;
  KCK(cudaGetDevice(&dev));
  if (dev != c->device) return kfail(c, FM_ERR_INVALID_ARG, "the current device is %d, the cache's is %d", dev, c->device);
  if (layer < 0 || layer >= c->cfg.n_layers)
    return kfail(c, FM_ERR_INVALID_ARG, "layer %d outside [0, %d)", layer, c->cfg.n_layers);
  if (n < 1 || n > c->cfg.n_seqs) return kfail(c, FM_ERR_INVALID_ARG, "n_seqs %d outside [1, %d]", n, c->cfg.n_seqs);
  if (!ids) return kfail(c, FM_ERR_INVALID_ARG, "null sequence ids");
  for (int i = 0; i < n; ++i)
    if (ids[i] < 0 || ids[i] >= c->cfg.n_seqs)
      return kfail(c, FM_ERR_INVALID_ARG, "sequence %d outside [0, %d)", ids[i], c->cfg.n_seqs);
  return FM_OK;
}

uint32_t next_call(fm_kvq *c) {
  if (++c->call == 0) {   // wrapped: no old mark may look new
    std::fill(c->mark.begin(), c->mark.end(), 0u);
    c->call = 1;
  }
  return c->call;
}

fm_status check_distinct(fm_kvq *c, int n, const int32_t *ids) {
  const uint32_t call = next_call(c);
  for (int i = 0; i < n; ++i) {
    if (c->mark[ids[i]] == call) return kfail(c, FM_ERR_INVALID_ARG, "sequence %d named twice", ids[i]);
    c->mark[ids[i]] = call;
  }
  return FM_OK;
}

fm_status type_of(fm_kvq *c, int dtype, int32_t *type, int *size) {
  switch (dtype) {
    case FM_DTYPE_F32: *type = KVQ_F32, *size = 4; return FM_OK;
    case FM_DTYPE_F16: *type = KVQ_F16, *size = 2; return FM_OK;
    case FM_DTYPE_BF16: *type = KVQ_BF16, *size = 2; return FM_OK;
  }
  return kfail(c, FM_ERR_INVALID_ARG, "dtype %d: f32, f16 or bf16", dtype);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

fm_status check_words(fm_kvq *c, const char *what, const void *p) {
  if (reinterpret_cast<uintptr_t>(p) & 3) return kfail(c, FM_ERR_INVALID_ARG, "%s: a misaligned pointer (4 bytes)", what);
  return FM_OK;
}

fm_status check_rows(fm_kvq *c, const char *what, const void *p, int64_t ld, int64_t width, int size) {
  if (!p || !aligned16(p)) return kfail(c, FM_ERR_INVALID_ARG, "%s: a null or misaligned pointer (16 bytes)", what);
  if (ld < width || (ld * size) % 16)
    return kfail(c, FM_ERR_INVALID_ARG, "%s: row stride %lld (at least %lld, whole 16 bytes)", what, (long long)ld,
                 (long long)width);
  return FM_OK;
}

// Calls share the lengths' rows, the weights and the workspace, so work that
// another stream was given earlier comes first.  (A captured call cannot wait
// for eager work, nor eager work for a graph: the caller orders those.)
bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &st) != cudaSuccess) {
    cudaGetLastError();
    return true;
  }
  return st != cudaStreamCaptureStatusNone;
}

fm_status begin(fm_kvq *c, cudaStream_t s) {
  kvq_launches() = 0;
  c->eager = !capturing(s);
  if (!c->eager) return FM_OK;
  KCK(cudaStreamGetId(s, &c->stream));
  if (c->has_last && c->stream != c->last) KCK(cudaStreamWaitEvent(s, c->done, 0));
  return FM_OK;
}

fm_status end(fm_kvq *c, cudaStream_t s) {
  c->launches = kvq_launches();
  if (!c->eager) return FM_OK;
  KCK(cudaEventRecord(c->done, s));
  c->last = c->stream;
  c->has_last = true;
  return FM_OK;
}

// Stages of a unit over `len` rows of which those from `first` on are seen: one at least.
int stages_of(int len, int first, int stage_rows) {
  const int s0 = first / stage_rows, s1 = (len + stage_rows - 1) / stage_rows;
  return s1 > s0 ? s1 - s0 : 1;
}

// The octets of query rows that a unit carries, 0 where the call has too many units.  A stage costs about 1 + nq (its codes
// are unpacked once, then used for each octet), beginning and ending a unit 5 nq (9 nq for 256 dims) of the same: short
// caches want many narrow units, long ones few wide ones.  (8 rows of 24 heads over 4 KV heads of 256, f32: 64 rows 5.3 us
// with nq 1, 10.5 with 3; 16384 rows 38.0 and 31.2, and 34.3 with 2, which the rule takes.  16 rows of 16 heads of 128, bf16:
// 4161 rows 9.6 us with nq 1, 10.3 with 2; 16384 rows 19.3 and 17.0.)  In the pass over the weights a CTA takes a sequence's
// row tiles one after another, about 7 each.  (With weights, 8 rows of 32 heads over 8 KV heads of 128, 1042 rows: 13.3 us,
// 16.8 with nq 1, which the rule without that term takes.)
int choose_nq(int n_seqs, const int32_t *seq, const int32_t *rows, const int32_t *len, int first, int group, int nkv, int hd,
              int n_sm, int64_t widest, bool weights) {
  const int stage_rows = kKvqTile * kvq_stage_tiles(hd), most = (int)(widest < 8 * kKvqMaxNQ ? (widest + 7) / 8 : kKvqMaxNQ);
  int best = 0;
  int64_t least = 0;
  for (int nq = 1; nq <= most; ++nq) {
    int64_t work = 0;
    bool fits = true;
    for (int i = 0; i < n_seqs; ++i) {
      const int64_t units = ((int64_t)rows[i] * group + 8 * nq - 1) / (8 * nq) * nkv;
      const int stages = stages_of(len[seq[i]], first, stage_rows);
      fits = fits && units <= kMaxUnits && units * (stages + kKvqUnitCost) <= INT_MAX;
      work += units * stages;
    }
    int64_t cost = (int64_t)nq * (hd == 256 ? 9 : 5) * n_sm + work * (1 + nq);
    if (weights) cost += (widest + 8 * nq - 1) / (8 * nq) * 7 * n_sm;
    if (fits && (!best || cost < least)) best = nq, least = cost;
  }
  return best;
}

// Deals the launch's stages to at most `most` CTAs (what the SMs hold at once).  Equal shares balance best, but a share
// that ends one unit and begins another pays for two (queries loaded, outputs written: about kKvqUnitCost stages).
// Where the units are no more than the CTAs, each gets CTAs of its own unless that makes the longest share that much
// longer.  (16 rows of 16 heads over 4161 rows of 128: 10.9 us by equal shares, 9.7 us this way; 8 rows of 24 heads over 64
// rows of 4 x 256, f32: 9.7 and 5.3; 32 ragged sequences whose longest would set the pace stay with equal shares.)
void deal(KvqAttnArgs &a, int64_t most, int groups, int nkv, int unit_rows) {
  const int64_t W = a.st0[a.n];
  auto units = [&](int i) { return ((int64_t)a.rows[i] * a.group + unit_rows - 1) / unit_rows * nkv; };
  // (a CTA's groups take its stages in turn: fewer stages than groups leave some idle, and make more parts to join)
  const int64_t wanted = (W + groups + kKvqUnitCost - 1) / (groups + kKvqUnitCost);
  a.ctas = (int32_t)(wanted < most ? wanted : most);
  a.share = (int32_t)(W / a.ctas);
  a.extra = (int32_t)(W % a.ctas);
  int64_t all = 0, stages = 0;
  int longest = 1;
  for (int i = 0; i < a.n; ++i) {
    all += units(i);
    stages += units(i) * a.stages[i];
    if (a.rows[i] > 0 && a.stages[i] > longest) longest = a.stages[i];
  }
  if (all > most) return;
  // the least number of stages a CTA with which the CTAs suffice
  const int even = (int)((stages + most - 1) / most);   // stages a CTA if they could be dealt out evenly
  int lo = even < groups ? groups : even, hi = longest < lo ? lo : longest;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    int64_t n = 0;
    for (int i = 0; i < a.n; ++i) n += units(i) * ((a.stages[i] + mid - 1) / mid);
    if (n <= most)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (lo > even + kKvqUnitCost + even / 8) return;
  a.share = 0;
  int ctas = 0;
  for (int i = 0; i < a.n; ++i) {
    a.cta0[i] = ctas;
    a.parts[i] = (a.stages[i] + lo - 1) / lo;
    ctas += (int)units(i) * a.parts[i];
  }
  a.cta0[a.n] = ctas;
  a.ctas = ctas;
}

void release(fm_kvq *c) {
  if (c->block) cudaFree(c->block);
  if (c->done) cudaEventDestroy(c->done);
  delete c;
}

fm_status setup(fm_kvq *c, cudaStream_t s) {
  const fm_kvq_config &g = c->cfg;
  KCK(cudaGetDevice(&c->device));
  KCK(cudaDeviceGetAttribute(&c->n_sm, cudaDevAttrMultiProcessorCount, c->device));
  const int stage_rows = kKvqTile * kvq_stage_tiles(g.head_dim);   // (the attention kernel fetches whole stages)
  c->rows_pad = (g.max_rows + stage_rows - 1) / stage_rows * stage_rows;
  c->plane_bytes = (size_t)(c->rows_pad / kKvqTile) * kvq_tile_bytes(g.head_dim);
  const size_t planes = (size_t)g.n_layers * g.n_seqs * g.n_kv_heads;
  c->slots = 2 * kKvqMaxCtas * c->n_sm;
  // one allocation, every part on a 256-byte boundary
  const size_t sizes[7] = {planes * c->plane_bytes,
                           planes * c->rows_pad * sizeof(float),
                           (size_t)c->slots * 8 * kKvqMaxNQ * g.head_dim * sizeof(float),
                           (size_t)c->slots * 8 * kKvqMaxNQ * sizeof(float2),
                           (size_t)kMaxUnits * 8 * kKvqMaxNQ * sizeof(float),
                           (size_t)(g.n_seqs < kKvqSeqs ? g.n_seqs : kKvqSeqs) * g.n_kv_heads * c->rows_pad * sizeof(int32_t),
                           4 * sizeof(int32_t)};
  size_t at[7], total = 0;
  for (int i = 0; i < 7; ++i) {
    at[i] = total;
    total += (sizes[i] + 255) / 256 * 256;
  }
  // (more planes than any address space holds would wrap the product)
  if (planes > ((size_t)1 << 48) / c->plane_bytes || cudaMalloc(&c->block, total) != cudaSuccess) {
    cudaGetLastError();
    return kfail(c, FM_ERR_OOM, "%zu planes of %zu bytes: the device allocation failed", planes, c->plane_bytes);
  }
  c->bytes = (int64_t)total;
  uint8_t *b = static_cast<uint8_t *>(c->block);
  c->planes = b + at[0];
  c->weights = reinterpret_cast<float *>(b + at[1]);
  c->part_o = reinterpret_cast<float *>(b + at[2]);
  c->part_ml = reinterpret_cast<float2 *>(b + at[3]);
  c->lse = reinterpret_cast<float *>(b + at[4]);
  c->list = reinterpret_cast<int32_t *>(b + at[5]);
  c->dev_err = reinterpret_cast<int32_t *>(b + at[6]);
  // rows behind a sequence's end are read with the last tile: they hold finite values from the start
  KCK(cudaMemsetAsync(b, 0, at[2], s));   // (weights too)
  KCK(cudaMemsetAsync(c->dev_err, 0, 16, s));
  KCK(cudaEventCreateWithFlags(&c->done, cudaEventDisableTiming));
  KCK(cudaStreamSynchronize(s));
  return FM_OK;
}

}  // namespace

extern "C" {

fm_status fm_kvq_create(const fm_kvq_config *cfg, void *stream, fm_kvq **out) {
  if (!out) return kfail(nullptr, FM_ERR_INVALID_ARG, "null out");
  *out = nullptr;
  if (!cfg) return kfail(nullptr, FM_ERR_INVALID_ARG, "null config");
  const fm_kvq_config g = *cfg;
  if (g.head_dim != 64 && g.head_dim != 128 && g.head_dim != 256)
    return kfail(nullptr, FM_ERR_UNSUPPORTED, "head_dim %d: 64, 128 or 256", g.head_dim);
  if (g.n_layers < 1 || g.n_layers > 1024 || g.n_seqs < 1 || g.n_seqs > 65536 || g.n_kv_heads < 1 || g.n_kv_heads > 256 ||
      g.max_rows < 1 || g.max_rows > kMaxRows)
    return kfail(nullptr, FM_ERR_INVALID_ARG, "n_layers %d, n_seqs %d, n_kv_heads %d or max_rows %d out of range", g.n_layers,
                 g.n_seqs, g.n_kv_heads, g.max_rows);
  fm_kvq *c = new (std::nothrow) fm_kvq();
  if (!c) return kfail(nullptr, FM_ERR_OOM, "host allocation failed");
  c->cfg = g;
  fm_status st;
  try {
    c->len.assign((size_t)g.n_layers * g.n_seqs, 0);
    c->mark.assign(g.n_seqs, 0u);
    st = setup(c, static_cast<cudaStream_t>(stream));
  } catch (const std::bad_alloc &) {
    st = kfail(c, FM_ERR_OOM, "host allocation failed");
  }
  if (st != FM_OK) {
    memcpy(g_kvq_error, c->err, sizeof c->err);
    release(c);
    return st;
  }
  *out = c;
  return FM_OK;
}

fm_status fm_kvq_append(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host, const int32_t *n_rows_host,
                        const int32_t *start_host, const void *k_dev, const void *v_dev, int32_t dtype, int64_t ld,
                        void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  KTRY(check_call(c, layer, n_seqs, seq_ids_host));
  if (!n_rows_host || !start_host) return kfail(c, FM_ERR_INVALID_ARG, "null row counts or starts");
  KTRY(check_distinct(c, n_seqs, seq_ids_host));
  int32_t type;
  int size;
  KTRY(type_of(c, dtype, &type, &size));
  int32_t *len = lengths(c, layer);
  int64_t total = 0;
  for (int i = 0; i < n_seqs; ++i) {
    const int s = seq_ids_host[i];
    if (n_rows_host[i] < 0) return kfail(c, FM_ERR_INVALID_ARG, "sequence %d: %d rows", s, n_rows_host[i]);
    if (start_host[i] < 0 || start_host[i] > len[s])
      return kfail(c, FM_ERR_STATE, "sequence %d: start %d, length %d", s, start_host[i], len[s]);
    if ((int64_t)start_host[i] + n_rows_host[i] > c->cfg.max_rows)
      return kfail(c, FM_ERR_CONTEXT_FULL, "sequence %d: %d + %d rows, the cache holds %d", s, start_host[i], n_rows_host[i],
                   c->cfg.max_rows);
    total += n_rows_host[i];
  }
  const int64_t width = (int64_t)c->cfg.n_kv_heads * c->cfg.head_dim;
  if (total > 0) {
    KTRY(check_rows(c, "k", k_dev, ld, width, size));
    KTRY(check_rows(c, "v", v_dev, ld, width, size));
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KTRY(begin(c, s));
  KvqRowsArgs a;
  memset(&a, 0, sizeof a);
  a.c = view(c, layer);
  a.k = k_dev;
  a.v = v_dev;
  a.ld = ld;
  a.type = type;
  int64_t row0 = 0;
  for (int i0 = 0; i0 < n_seqs; i0 += kKvqSeqs) {
    a.n = 0;
    a.tiles = 0;
    for (int i = i0; i < n_seqs && i < i0 + kKvqSeqs; ++i) {
      const int n = n_rows_host[i], at = start_host[i];
      if (n > 0) {
        a.seq[a.n] = seq_ids_host[i];
        a.at[a.n] = at;
        a.rows[a.n] = n;
        a.row0[a.n] = row0;
        a.tile0[a.n++] = a.tiles;
        a.tiles += (at + n - 1) / kKvqTile - at / kKvqTile + 1;
        row0 += n;
      }
    }
    a.tile0[a.n] = a.tiles;
    if (a.n) KCK(launch_kvq_append(a, c->cfg.head_dim, s));
    for (int i = i0; i < n_seqs && i < i0 + kKvqSeqs; ++i) len[seq_ids_host[i]] = start_host[i] + n_rows_host[i];
  }
  return end(c, s);
}

fm_status fm_kvq_read(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host, const int32_t *row_host,
                      const int32_t *n_rows_host, void *k_dev, void *v_dev, int32_t dtype, int64_t ld, float *weights_dev,
                      int64_t ldw, void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  KTRY(check_call(c, layer, n_seqs, seq_ids_host));
  if (!n_rows_host || !row_host) return kfail(c, FM_ERR_INVALID_ARG, "null row counts or first rows");
  int32_t type;
  int size;
  KTRY(type_of(c, dtype, &type, &size));
  const int32_t *len = lengths(c, layer);
  int64_t total = 0;
  int most = 0;
  for (int i = 0; i < n_seqs; ++i) {
    const int s = seq_ids_host[i];
    if (n_rows_host[i] < 0 || row_host[i] < 0 || (int64_t)row_host[i] + n_rows_host[i] > len[s])
      return kfail(c, FM_ERR_INVALID_ARG, "sequence %d: rows %d + %d, length %d", s, row_host[i], n_rows_host[i], len[s]);
    total += n_rows_host[i];
    most = n_rows_host[i] > most ? n_rows_host[i] : most;
  }
  KTRY(check_words(c, "weights", weights_dev));
  const int64_t width = (int64_t)c->cfg.n_kv_heads * c->cfg.head_dim;
  if (total > 0) {
    if (k_dev) KTRY(check_rows(c, "k", k_dev, ld, width, size));
    if (v_dev) KTRY(check_rows(c, "v", v_dev, ld, width, size));
    if (weights_dev && ldw < most)
      return kfail(c, FM_ERR_INVALID_ARG, "weights: row stride %lld, %d rows", (long long)ldw, most);
    if (!k_dev && !v_dev && !weights_dev) return kfail(c, FM_ERR_INVALID_ARG, "nothing to read into");
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KTRY(begin(c, s));
  KvqRowsArgs a;
  memset(&a, 0, sizeof a);
  a.c = view(c, layer);
  a.ko = k_dev;
  a.vo = v_dev;
  a.ld = ld;
  a.type = type;
  a.wo = weights_dev;
  a.ldw = ldw;
  int64_t row0 = 0;
  for (int i0 = 0; i0 < n_seqs; i0 += kKvqSeqs) {
    a.n = 0;
    a.tiles = 0;
    a.call0 = i0;
    // (every sequence keeps its place: the weights' rows go by it)
    for (int i = i0; i < n_seqs && i < i0 + kKvqSeqs; ++i) {
      const int n = n_rows_host[i], at = row_host[i];
      a.seq[a.n] = seq_ids_host[i];
      a.at[a.n] = at;
      a.rows[a.n] = n;
      a.row0[a.n] = row0;
      a.tile0[a.n++] = a.tiles;
      if (n > 0) a.tiles += (at + n - 1) / kKvqTile - at / kKvqTile + 1;
      row0 += n;
    }
    a.tile0[a.n] = a.tiles;
    if (a.tiles) KCK(launch_kvq_read(a, c->cfg.head_dim, s));
  }
  return end(c, s);
}

fm_status fm_kvq_set_weights(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host, const float *weights_dev,
                             int64_t ldw, void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  KTRY(check_call(c, layer, n_seqs, seq_ids_host));
  KTRY(check_distinct(c, n_seqs, seq_ids_host));
  const int32_t *len = lengths(c, layer);
  int most = 0;
  for (int i = 0; i < n_seqs; ++i) most = len[seq_ids_host[i]] > most ? len[seq_ids_host[i]] : most;
  if (most > 0 && (!weights_dev || ldw < most))
    return kfail(c, FM_ERR_INVALID_ARG, "weights: null, or row stride %lld with %d rows", (long long)ldw, most);
  KTRY(check_words(c, "weights", weights_dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KTRY(begin(c, s));
  KvqRowsArgs a;
  memset(&a, 0, sizeof a);
  a.c = view(c, layer);
  a.wi = weights_dev;
  a.ldw = ldw;
  for (int i0 = 0; i0 < n_seqs; i0 += kKvqSeqs) {
    a.n = 0;
    a.call0 = i0;
    for (int i = i0; i < n_seqs && i < i0 + kKvqSeqs; ++i) {
      a.seq[a.n] = seq_ids_host[i];
      a.rows[a.n++] = len[seq_ids_host[i]];
    }
    KCK(launch_kvq_set_weights(a, s));
  }
  return end(c, s);
}

fm_status fm_kvq_attend(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *seq_ids_host, const int32_t *n_rows_host,
                        const void *q_dev, int32_t dtype, int32_t n_heads, int64_t ldq, float scale, int32_t causal,
                        int32_t first_row, void *out_dev, int64_t ldo, float decay, float *weights_dev, int64_t ldw,
                        void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  KTRY(check_call(c, layer, n_seqs, seq_ids_host));
  if (!n_rows_host) return kfail(c, FM_ERR_INVALID_ARG, "null row counts");
  int32_t type;
  int size;
  KTRY(type_of(c, dtype, &type, &size));
  const int nkv = c->cfg.n_kv_heads, hd = c->cfg.head_dim;
  if (n_heads < 1 || n_heads % nkv || n_heads / nkv > 1024)
    return kfail(c, FM_ERR_INVALID_ARG, "%d query heads over %d KV heads", n_heads, nkv);
  if (!std::isfinite(scale)) return kfail(c, FM_ERR_INVALID_ARG, "scale is not finite");
  if (first_row < 0) return kfail(c, FM_ERR_INVALID_ARG, "first_row %d", first_row);
  if (first_row > c->cfg.max_rows) first_row = c->cfg.max_rows;   // (past every row either way)
  if (!(decay == decay) || std::isinf(decay)) return kfail(c, FM_ERR_INVALID_ARG, "decay is not finite");
  const bool keep_w = decay >= 0.f;
  KTRY(check_words(c, "weights", weights_dev));
  if (!keep_w && weights_dev) return kfail(c, FM_ERR_INVALID_ARG, "weights wanted, but decay < 0 keeps none");
  if (keep_w) KTRY(check_distinct(c, n_seqs, seq_ids_host));
  const int32_t *len = lengths(c, layer);
  const int group = n_heads / nkv;
  int64_t total = 0, widest = 1;
  int most = 0;
  for (int i = 0; i < n_seqs; ++i) {
    const int64_t r = (int64_t)n_rows_host[i] * group;
    widest = r > widest ? r : widest;
  }
  const int stage_rows = kKvqTile * kvq_stage_tiles(hd);
  for (int i = 0; i < n_seqs; ++i) {
    const int n = n_rows_host[i];
    if (n < 0 || n > (1 << 16)) return kfail(c, FM_ERR_INVALID_ARG, "sequence %d: %d query rows", seq_ids_host[i], n);
    total += n;
    if (n > 0 && len[seq_ids_host[i]] > most) most = len[seq_ids_host[i]];
  }
  const int nq = choose_nq(n_seqs, seq_ids_host, n_rows_host, len, first_row, group, nkv, hd, c->n_sm, widest, keep_w),
            unit_rows = 8 * nq;
  if (!nq) return kfail(c, FM_ERR_UNSUPPORTED, "%lld query rows of a KV head in one call", (long long)widest);
  const int64_t width = (int64_t)n_heads * hd;
  if (total > 0) {
    KTRY(check_rows(c, "q", q_dev, ldq, width, size));
    KTRY(check_rows(c, "out", out_dev, ldo, width, size));
    if (q_dev == out_dev) return kfail(c, FM_ERR_INVALID_ARG, "out is q: rows are still read when others are written");
    if (weights_dev && ldw < most)
      return kfail(c, FM_ERR_INVALID_ARG, "weights: row stride %lld, %d rows", (long long)ldw, most);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KTRY(begin(c, s));
  KvqAttnArgs a;
  memset(&a, 0, sizeof a);
  a.c = view(c, layer);
  a.q = q_dev;
  a.out = out_dev;
  a.ldq = ldq;
  a.ldo = ldo;
  a.type = type;
  a.group = group;
  a.nq = nq;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal != 0;
  a.first = first_row;
  a.part_o = c->part_o;
  a.part_ml = c->part_ml;
  a.lse = keep_w ? c->lse : nullptr;
  a.decay = decay;
  a.w_out = weights_dev;
  a.ldw = ldw;
  int64_t row0 = 0;
  for (int i0 = 0; i0 < n_seqs;) {
    // the sequences of this launch: 64, and as many units as the workspace has row sums for
    int64_t units = 0, work = 0;
    int un = 0, wt = 0;
    a.n = 0;
    a.call0 = i0;
    int i = i0;
    for (; i < n_seqs && a.n < kKvqSeqs; ++i) {
      const int n = n_rows_host[i], L = len[seq_ids_host[i]], j = a.n;
      const int rts = (int)(((int64_t)n * group + unit_rows - 1) / unit_rows);
      const int t1 = (L + kKvqTile - 1) / kKvqTile;
      const int stages = stages_of(L, first_row, stage_rows);
      const int64_t more = (int64_t)rts * nkv * (stages + kKvqUnitCost);
      if (j && (units + (int64_t)rts * nkv > kMaxUnits || work + more > INT_MAX)) break;
      a.seq[j] = seq_ids_host[i];
      a.len[j] = L;
      a.rows[j] = n;
      a.row0[j] = row0;
      a.stages[j] = stages;
      a.st0[j] = (int32_t)work;
      a.unit0[j] = un;
      row0 += n;
      units += (int64_t)rts * nkv;
      work += more;
      un += rts;
      if (rts > 0) wt += t1;
      ++a.n;
    }
    a.st0[a.n] = (int32_t)work;
    a.unit0[a.n] = un;
    // the weights pass: tiles a CTA so that the CTAs are whole rounds of what the SMs hold (about four each)
    if (keep_w && wt > 0) {
      const int64_t room = 4ll * c->n_sm, tiles = (int64_t)wt * nkv, rounds = (tiles + room * kKvqWeightTiles - 1) / (room * kKvqWeightTiles);
      const int64_t even = (tiles + room * rounds - 1) / (room * rounds);
      a.wtiles = (int32_t)(even < 2 ? even : (even + 1) / 2 * 2);   // (whole pairs)
      wt = 0;
      for (int j = 0; j < a.n; ++j) {
        a.wt0[j] = wt;
        if (a.rows[j] > 0) wt += ((a.len[j] + kKvqTile - 1) / kKvqTile + a.wtiles - 1) / a.wtiles;
      }
      a.wt0[a.n] = wt;
    }
    if (work > 0) {
      const KvqShape sh = attn_shape(hd, type, nq);
      deal(a, (int64_t)c->n_sm * sh.ctas, sh.groups, nkv, unit_rows);
      KCK(launch_kvq_attn(a, hd, false, s));
      if (keep_w && wt > 0) KCK(launch_kvq_attn(a, hd, true, s));
    }
    i0 = i;
  }
  return end(c, s);
}

fm_status fm_kvq_evict(fm_kvq *c, int32_t layer, int32_t n_seqs, const int32_t *src_ids_host, const int32_t *dst_ids_host,
                       int32_t keep, int32_t recent, int32_t *kept_dev, void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  KTRY(check_call(c, layer, n_seqs, src_ids_host));
  KTRY(check_call(c, layer, n_seqs, dst_ids_host));
  if (keep < 0 || keep > c->cfg.max_rows || recent < 0 || recent > keep)
    return kfail(c, FM_ERR_INVALID_ARG, "keep %d (of at most %d), recent %d", keep, c->cfg.max_rows, recent);
  KTRY(check_words(c, "kept rows", kept_dev));
  KTRY(check_distinct(c, n_seqs, dst_ids_host));
  // a sequence that is written is read by its own move alone
  for (int i = 0; i < n_seqs; ++i)
    if (src_ids_host[i] != dst_ids_host[i] && c->mark[src_ids_host[i]] == c->call)
      return kfail(c, FM_ERR_INVALID_ARG, "sequence %d is read and written", src_ids_host[i]);
  int32_t *len = lengths(c, layer);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KTRY(begin(c, s));
  KvqEvictArgs a;
  memset(&a, 0, sizeof a);
  a.c = view(c, layer);
  a.keep = keep;
  a.n_sm = c->n_sm;
  a.recent = recent;
  a.kept = kept_dev;
  a.list = c->list;
  for (int i0 = 0; i0 < n_seqs; i0 += kKvqSeqs) {
    a.n = 0;
    a.call0 = i0;
    for (int i = i0; i < n_seqs && i < i0 + kKvqSeqs; ++i) {
      a.src[a.n] = src_ids_host[i];
      a.dst[a.n] = dst_ids_host[i];
      a.len[a.n++] = len[src_ids_host[i]];
    }
    KCK(launch_kvq_evict(a, c->cfg.head_dim, s));
    for (int j = 0; j < a.n; ++j) len[a.dst[j]] = a.len[j] < keep ? a.len[j] : keep;
  }
  return end(c, s);
}

fm_status fm_kvq_length(const fm_kvq *c, int32_t layer, int32_t seq, int32_t *length) {
  if (!c || !length || layer < 0 || layer >= c->cfg.n_layers || seq < 0 || seq >= c->cfg.n_seqs) return FM_ERR_INVALID_ARG;
  *length = c->len[(size_t)layer * c->cfg.n_seqs + seq];
  return FM_OK;
}

fm_status fm_kvq_get_config(const fm_kvq *c, fm_kvq_config *cfg) {
  if (!c || !cfg) return FM_ERR_INVALID_ARG;
  *cfg = c->cfg;
  return FM_OK;
}

fm_status fm_kvq_last_launch_count(const fm_kvq *c, int32_t *count) {
  if (!c || !count) return FM_ERR_INVALID_ARG;
  *count = c->launches;
  return FM_OK;
}

fm_status fm_kvq_memory_bytes(const fm_kvq *c, int64_t *bytes) {
  if (!c || !bytes) return FM_ERR_INVALID_ARG;
  *bytes = c->bytes;
  return FM_OK;
}

fm_status fm_kvq_synchronize(fm_kvq *c, void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t e = 0;
  KCK(cudaMemcpyAsync(&e, c->dev_err, 4, cudaMemcpyDeviceToHost, s));
  KCK(cudaStreamSynchronize(s));
  if (e) {
    KCK(cudaMemsetAsync(c->dev_err, 0, 4, s));
    return kfail(c, FM_ERR_TIMEOUT, "a bounded device wait gave up");
  }
  return FM_OK;
}

fm_status fm_kvq_selftest_wait_timeout(fm_kvq *c, int32_t budget_us, void *stream) {
  if (!c) return FM_ERR_INVALID_ARG;
  if (budget_us < 1 || budget_us > 1000000) return kfail(c, FM_ERR_INVALID_ARG, "budget_us outside [1, 1000000]");
  int dev = -1, khz = 0;
  KCK(cudaGetDevice(&dev));
  if (dev != c->device) return kfail(c, FM_ERR_INVALID_ARG, "the current device is %d, the cache's is %d", dev, c->device);
  KCK(cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, dev));
  if (khz <= 0) khz = 2000000;
  KCK(launch_wait_selftest(c->dev_err, (long long)budget_us * (khz / 1000), static_cast<cudaStream_t>(stream)));
  c->launches = 1;
  return FM_OK;
}

const char *fm_kvq_last_error(const fm_kvq *c) { return c ? c->err : g_kvq_error; }

void fm_kvq_destroy(fm_kvq *c) {
  if (!c) return;
  // On the cache's device; and a capture that this thread may be in goes on (a Python object may be collected any time),
  // which a synchronisation of the device would end.  (Freeing waits for what runs, graphs too.)
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  int dev = -1;
  cudaThreadExchangeStreamCaptureMode(&mode);
  cudaGetDevice(&dev);
  const int own = c->device;
  if (dev != own) cudaSetDevice(own);
  if (c->has_last) cudaEventSynchronize(c->done);
  release(c);
  if (dev != own) cudaSetDevice(dev);
  cudaThreadExchangeStreamCaptureMode(&mode);
}

}  // extern "C"
