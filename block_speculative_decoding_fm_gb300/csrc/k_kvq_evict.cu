// k_kvq_evict.cu -- eviction from the 4-bit KV cache by accumulated attention
// weight: per (sequence, KV head) the last `recent` rows stay, and of the rows
// before them the keep - recent with the largest weight (ties: the lowest row; NaN
// below everything), in their order.
//
// Two launches:
//   select   one CTA a plane, or a cluster of eight: the weight of rank keep - recent by
//            radix selection on the ordered bits, eight at a time, then the rows that stay
//            are listed in their order, a run of rows a warp (scans, no atomics whose order
//            could show);
//   move     16 bytes of codes and their scale an item.  Into another sequence, CTAs
//            of 64 rows and a plane each, all over the GPU (512 planes, 2048 rows of 128
//            kept in each: 52 us, 5.9 TB/s).  In place, a cluster of eight CTAs a plane
//            goes through the rows in rounds: a kept row never moves up, so the rows that a round
//            writes lie below every row that a later round reads, and a cluster barrier
//            between a round's loads and its stores is all that is needed.
// Bound by memory: 4 bytes a row of weights, and the kept rows read and written once.
#include <cooperative_groups.h>

#include <utility>

#include "dev_common.cuh"
#include "kvq.h"
#include "kvq_load.cuh"

namespace cg = cooperative_groups;

namespace fm {
namespace {

constexpr int kThreads = 512;    // in place
constexpr int kCopies = 8;       // of a histogram
constexpr int kMoveThreads = 256;
constexpr int kSelectRoom[2] = {200 * 1024, 90 * 1024};   // bytes of keys in shared memory: a CTA an SM, two
constexpr int kCluster = 8;      // in place; select, where planes are few
constexpr int kMoveItems = 4;    // 16-byte units a thread moves a round

// weights as unsigned integers of the same order; -0 counts as 0, NaN as less than everything
__device__ __forceinline__ uint32_t ordered(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  return w != w ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// exclusive sum over the block's NT threads of v; red holds NT / 32 words
template <int NT>
__device__ __forceinline__ int block_scan(int v, int *red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the last call's words have been read
  if (lane == 31) red[w] = x;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int j = 0; j < NT / 32; ++j) base += j < w ? red[j] : 0;
  return base + x - v;
}

// rows a warp's run has, whole turns of 128: nc rows over `warps`
__host__ __device__ inline int select_run(int nc, int warps) { return (nc + warps * 128 - 1) / (warps * 128) * 128; }

// A plane's rows over CS CTAs (a cluster of eight where planes are few), an equal run of rows a warp.  Histograms of 8-bit
// digits are kept in eight copies, a lane's by its number and a bin's copies side by side: weights crowd into few bins, and
// lanes that meet in a bank go one after the other.  A pass over few planes costs its waits: the first one reads the
// weights, and where they fit (cached) every later one has them from shared memory, in the thread that put them there.
// With many planes other CTAs fill the waits, and shared memory taken from L1 made the launches around this one slower.
// The passes end early where all of the selected bin stay, for distinct weights after three mostly.
// (512 planes of 512 to 8192 rows: 18 us; 4 of 65535 rows: 15 us, 18 without the cache; 8 of 262144: 32 us, 41 without.)
template <int CS>
__global__ void __launch_bounds__(CS == 1 ? 256 : 512, CS == 1 ? 4 : 2) kvq_select_kernel(const __grid_constant__ KvqEvictArgs a, bool cached) {
  constexpr int NT = CS == 1 ? 256 : 512, NWarp = NT / 32;
  extern __shared__ __align__(16) uint32_t s_keys[];   // [warp][per], where cached
  __shared__ __align__(16) int hist[256 * kCopies];
  __shared__ int bins[2][256];                         // (two: a CTA may still read the last pass's)
  __shared__ int red[NWarp];
  __shared__ int s_found[3];
  __shared__ int2 s_cnt[NWarp];
  __shared__ int2 s_all;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = CS == 1 ? 0 : blockIdx.x % CS, pl = blockIdx.x / CS, i = pl / a.c.n_kv, head = pl - i * a.c.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, len = a.len[i];
  const float *ws = a.c.weights + ((size_t)a.src[i] * a.c.n_kv + head) * a.c.rows_pad;
  int32_t *list = a.list + (size_t)pl * a.c.rows_pad;
  int32_t *kept = a.kept ? a.kept + ((size_t)(a.call0 + i) * a.c.n_kv + head) * a.keep : nullptr;
  pdl_trigger();
  pdl_wait();
  auto put = [&](int pos, int row) {
    list[pos] = row;
    if (kept) kept[pos] = row;
  };
  if (len <= a.keep) {
    for (int r = rank * NT + tid; r < len; r += CS * NT) put(r, r);
    return;
  }
  const int nc = len - a.recent, m = a.keep - a.recent;   // m of the first nc rows stay
  for (int r = rank * NT + tid; r < a.recent; r += CS * NT) put(m + r, nc + r);
  if (m == 0) return;
  // a warp's run of rows; four rows' keys (a plane's rows are padded to 64)
  const int per = select_run(nc, CS * NWarp);
  const int r_beg = (rank * NWarp + w) * per, r_end = min(nc, r_beg + per);
  uint32_t *mine = s_keys + w * per - r_beg;
  auto read = [&](int r, uint32_t (&k)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(ws + r);
    k[0] = ordered(v.x), k[1] = ordered(v.y), k[2] = ordered(v.z), k[3] = ordered(v.w);
  };
  auto keys = [&](int r, uint32_t (&k)[4]) {
    if (CS > 1 && cached) {
      const uint4 v = *reinterpret_cast<const uint4 *>(mine + r);
      k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
    } else {
      read(r, k);
    }
  };
  uint32_t prefix = 0;   // the selected weight's leading bits
  int want = m;          // its rank among the rows that share them
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int x = tid; x < 256 * kCopies / 4; x += NT) reinterpret_cast<int4 *>(hist)[x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    int *h = hist + lane % kCopies;
    if (shift == 24) {
#pragma unroll 4
      for (int r = r_beg + 4 * lane; r < r_end; r += 128) {
        uint32_t k[4];
        read(r, k);
        if (CS > 1 && cached) *reinterpret_cast<uint4 *>(mine + r) = make_uint4(k[0], k[1], k[2], k[3]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r + q < r_end) atomicAdd(h + (k[q] >> 24) * kCopies, 1);
      }
    } else {
#pragma unroll 4
      for (int r = r_beg + 4 * lane; r < r_end; r += 128) {
        uint32_t k[4];
        keys(r, k);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r + q < r_end && (k[q] >> (shift + 8)) == prefix) atomicAdd(h + ((k[q] >> shift) & 255) * kCopies, 1);
      }
    }
    __syncthreads();
    // bins from the top: thread t has bin 255 - t, of all CTAs
    int n = 0, *b = bins[shift >> 3 & 1];
    if (tid < 256) {
#pragma unroll
      for (int c = 0; c < kCopies; c += 4) {   // (lanes begin at different copies: their banks differ)
        const int4 v = *reinterpret_cast<const int4 *>(hist + (255 - tid) * kCopies + (c + 4 * (tid / (32 / kCopies))) % kCopies);
        n += (v.x + v.y) + (v.z + v.w);
      }
      if (CS > 1) b[tid] = n;
    }
    if (CS > 1) {
      cl.sync();
      if (tid < 256) {
        n = 0;
#pragma unroll
        for (int c = 0; c < CS; ++c) n += *cl.map_shared_rank(b + tid, c);
      }
    }
    const int before = block_scan<NT>(n, red);
    if (before < want && before + n >= want) s_found[0] = 255 - tid, s_found[1] = want - before, s_found[2] = n;
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)s_found[0];
    want = s_found[1];
    if (want == s_found[2]) {   // all of the bin stay: whatever is above what lies below it (they are not all rows)
      prefix = (prefix << shift) - 1u;
      want = 0;
      break;
    }
  }
  // Rows above the selected weight stay, and the first `want` that equal it: a warp counts both kinds in its run,
  // and with the counts before it writes its own, in order.
  int2 cnt = make_int2(0, 0);   // above, equal
#pragma unroll 4
  for (int r = r_beg + 4 * lane; r < r_end; r += 128) {
    uint32_t k[4];
    keys(r, k);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (r + q < r_end) cnt.x += k[q] > prefix, cnt.y += k[q] == prefix;
  }
  cnt.x = __reduce_add_sync(0xffffffffu, cnt.x);
  cnt.y = __reduce_add_sync(0xffffffffu, cnt.y);
  if (lane == 0) s_cnt[w] = cnt;
  __syncthreads();
  int pos = 0, eq = 0;
  if (CS > 1) {
    if (tid == 0) {
      int2 t = make_int2(0, 0);
      for (int v = 0; v < NWarp; ++v) t.x += s_cnt[v].x, t.y += s_cnt[v].y;
      s_all = t;
    }
    cl.sync();
    for (int c = 0; c < rank; ++c) {
      const int2 t = *cl.map_shared_rank(&s_all, c);
      pos += t.x, eq += t.y;
    }
  }
  for (int v = 0; v < w; ++v) pos += s_cnt[v].x, eq += s_cnt[v].y;
  pos += min(eq, want);
#pragma unroll 2
  for (int r0 = r_beg; r0 < r_end; r0 += 128) {
    const int r = r0 + 4 * lane;
    uint32_t k[4] = {};
    if (r < r_end) keys(r, k);
    int ne = 0, ng = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) ne += r + q < r_end && k[q] == prefix, ng += r + q < r_end && k[q] > prefix;
    // both counts in one scan (at most 128 each)
    const int both = ne << 16 | ng;
    int x = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int all = __shfl_sync(0xffffffffu, x, 31), before = x - both;
    int er = eq + (before >> 16);                                       // equal rows before this thread's
    int at = pos + (before & 0xffff) + min(er, want) - min(eq, want);   // kept rows before them
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (r + q >= r_end) break;
      const bool same = k[q] == prefix;
      if (k[q] > prefix || (same && er < want)) put(at++, r + q);
      er += same;
    }
    pos += (all & 0xffff) + min(eq + (all >> 16), want) - min(eq, want);
    eq += all >> 16;
  }
  if (CS > 1) cl.sync();   // no CTA leaves while another may read its shared memory
}

// Rows [r0, r0 + RB) of the list: found, loaded, stored.  kItems 16-byte units a thread.
template <int HD, int NT, int kItems>
struct Mover {
  static constexpr int U = HD / 32;                    // units of K (and of V) a row
  static constexpr int RB = NT * kItems / (2 * U);     // rows a round
  static constexpr int WR = (RB + NT - 1) / NT;        // weights a thread
  uint4 code[kItems];
  int row[kItems], mine[WR];
  uint16_t sc[kItems];
  float wt[WR];
  __device__ __forceinline__ void find(const int32_t *list, int r0, int left, int tid) {
#pragma unroll
    for (int q = 0; q < kItems; ++q) {
      const int r = r0 + (q * NT + tid) / (2 * U);
      row[q] = r < left ? (int)ldg32(list + r) : -1;
    }
#pragma unroll
    for (int x = 0; x < WR; ++x) {
      const int r = x * NT + tid;
      mine[x] = r < RB && r0 + r < left ? (int)ldg32(list + r0 + r) : -1;
    }
  }
  __device__ __forceinline__ void load(const uint8_t *src, const float *ws, int tid) {
#pragma unroll
    for (int q = 0; q < kItems; ++q) {
      const int u = (q * NT + tid) % (2 * U);
      if (row[q] >= 0) {
        const int tr = row[q] % kKvqTile;
        const uint8_t *h = src + (size_t)(row[q] / kKvqTile) * kvq_tile_bytes(HD) + (u >= U ? kvq_k_bytes(HD) : 0);
        code[q] = *reinterpret_cast<const uint4 *>(h + kvq_unit(tr, u % U, HD));
        sc[q] = *reinterpret_cast<const uint16_t *>(h + kvq_scale(tr, u % U, HD, u >= U));
      }
    }
#pragma unroll
    for (int x = 0; x < WR; ++x)
      if (mine[x] >= 0) wt[x] = ws[mine[x]];
  }
  __device__ __forceinline__ void store(uint8_t *dst, float *wd, int r0, int left, int tid) const {
#pragma unroll
    for (int q = 0; q < kItems; ++q) {
      const int it = q * NT + tid, r = r0 + it / (2 * U), u = it % (2 * U);
      if (r < left) {
        const int tr = r % kKvqTile;
        uint8_t *h = dst + (size_t)(r / kKvqTile) * kvq_tile_bytes(HD) + (u >= U ? kvq_k_bytes(HD) : 0);
        *reinterpret_cast<uint4 *>(h + kvq_unit(tr, u % U, HD)) = code[q];
        *reinterpret_cast<uint16_t *>(h + kvq_scale(tr, u % U, HD, u >= U)) = sc[q];
      }
    }
#pragma unroll
    for (int x = 0; x < WR; ++x) {
      const int r = x * NT + tid;
      if (r < RB && r0 + r < left) wd[r0 + r] = wt[x];
    }
  }
};

// into other sequences: grid (rounds, planes)
template <int HD>
__global__ void __launch_bounds__(kMoveThreads) kvq_move_kernel(const __grid_constant__ KvqEvictArgs a) {
  using M = Mover<HD, kMoveThreads, kMoveItems>;
  const int pl = blockIdx.y, i = pl / a.c.n_kv, head = pl - i * a.c.n_kv;
  const int left = min(a.keep, a.len[i]), r0 = blockIdx.x * M::RB;
  const size_t ps = (size_t)a.src[i] * a.c.n_kv + head, pd = (size_t)a.dst[i] * a.c.n_kv + head;
  pdl_trigger();
  pdl_wait();
  if (a.src[i] == a.dst[i]) return;
  if (r0 >= left) return;
  M m;
  m.find(a.list + (size_t)pl * a.c.rows_pad, r0, left, threadIdx.x);
  m.load(a.c.planes + ps * a.c.plane_bytes, a.c.weights + ps * a.c.rows_pad, threadIdx.x);
  m.store(a.c.planes + pd * a.c.plane_bytes, a.c.weights + pd * a.c.rows_pad, r0, left, threadIdx.x);
}

// In place: grid (cluster of a plane).  A round's rows are loaded by all before any of them is stored.  With many planes
// other clusters fill the waits (two CTAs an SM).  With few, a round is twice as long, and the next one's loads and the
// list's for the one after are on their way while the barrier is waited for: they read behind every row written so far.
// (One sequence of 8 planes, 65536 of 262144 rows kept: 96 us with the selection, 52 us more without the loads ahead; 256 planes,
// 2048 of 4096 kept: 63 us, 86 with them.)
template <int HD, bool Few>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, Few ? 1 : 2)
    kvq_move_in_place_kernel(const __grid_constant__ KvqEvictArgs a) {
  using M = Mover<HD, kThreads, Few ? 2 * kMoveItems : kMoveItems>;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = blockIdx.x % kCluster, pl = blockIdx.x / kCluster, i = pl / a.c.n_kv, head = pl - i * a.c.n_kv;
  pdl_trigger();
  pdl_wait();
  if (a.src[i] != a.dst[i] || a.len[i] <= a.keep) return;   // (all eight CTAs)
  const size_t p = (size_t)a.src[i] * a.c.n_kv + head;
  uint8_t *plane = a.c.planes + p * a.c.plane_bytes;
  float *ws = a.c.weights + p * a.c.rows_pad;
  const int32_t *list = a.list + (size_t)pl * a.c.rows_pad;
  constexpr int step = kCluster * M::RB;
  const int first = rank * M::RB, tid = threadIdx.x;
  if constexpr (!Few) {
    for (int base = 0; base < a.keep; base += step) {
      M m;
      m.find(list, base + first, a.keep, tid);
      m.load(plane, ws, tid);
      cl.sync();
      m.store(plane, ws, base + first, a.keep, tid);
    }
  } else {
    M m[2];
    m[0].find(list, first, a.keep, tid);
    m[0].load(plane, ws, tid);
    m[1].find(list, first + step, a.keep, tid);
    for (int base = 0; base < a.keep; base += 2 * step) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r0 = base + h * step + first;
        if (base + h * step >= a.keep) break;   // (the same for the cluster)
        auto token = cl.barrier_arrive();
        m[1 - h].load(plane, ws, tid);
        m[h].find(list, r0 + 2 * step, a.keep, tid);
        cl.barrier_wait(std::move(token));
        m[h].store(plane, ws, r0, a.keep, tid);
      }
    }
  }
}

template <int HD>
cudaError_t evict_hd(const KvqEvictArgs &a, cudaStream_t s) {
  const int planes = a.n * a.c.n_kv;
  cudaError_t e;
  // a cluster a plane while two CTAs an SM hold them all (38 planes of 32,768 rows: select and move 45 us, 72 with a CTA a
  // plane; 8 planes: 18 and 49; of 4,096 rows 38 planes: 22 and 14 to 16, 8 planes: 12 and 14)
  if (planes * kCluster <= 2 * a.n_sm) {
    // (longer planes are read again in each pass)
    int longest = 0;
    for (int i = 0; i < a.n; ++i) longest = a.len[i] > longest ? a.len[i] : longest;
    const int bytes = select_run(longest, kCluster * 16) * 16 * 4;
    const bool cached = bytes <= kSelectRoom[planes * kCluster > a.n_sm];
    static std::atomic<uint64_t> done{0};
    e = allow_smem(kvq_select_kernel<kCluster>, kSelectRoom[0], done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(planes * kCluster);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = cached ? bytes : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    ++kvq_launches();
    e = cudaLaunchKernelEx(&cfg, kvq_select_kernel<kCluster>, a, cached);
  } else {
    e = kvq_launch(kvq_select_kernel<1>, dim3(planes), dim3(256), 0, s, a, false);
  }
  int most = 0;   // rows that go to another sequence
  bool same = false;
  for (int i = 0; i < a.n; ++i) {
    const int left = a.len[i] < a.keep ? a.len[i] : a.keep;
    if (a.src[i] == a.dst[i])
      same = same || a.len[i] > a.keep;
    else
      most = left > most ? left : most;
  }
  if (e == cudaSuccess && most > 0) {
    const int rb = Mover<HD, kMoveThreads, kMoveItems>::RB;
    e = kvq_launch(kvq_move_kernel<HD>, dim3((most + rb - 1) / rb, planes), dim3(kMoveThreads), 0, s, a);
  }
  if (e == cudaSuccess && same)
    e = kvq_launch(planes * kCluster <= a.n_sm ? kvq_move_in_place_kernel<HD, true> : kvq_move_in_place_kernel<HD, false>,
                   dim3(planes * kCluster), dim3(kThreads), 0, s, a);
  return e;
}

}  // namespace

cudaError_t launch_kvq_evict(const KvqEvictArgs &a, int hd, cudaStream_t s) {
  return hd == 64 ? evict_hd<64>(a, s) : hd == 128 ? evict_hd<128>(a, s) : evict_hd<256>(a, s);
}

}  // namespace fm
