// k_kvq_evict.cu -- eviction from the 4-bit KV cache by accumulated attention
// weight: per (sequence, KV head) the last `recent` rows stay, and of the rows
// before them the keep - recent with the largest weight (ties: the lowest row; NaN
// below everything), in their order.
//
// One cluster of eight CTAs per plane, one launch for everything:
//   select   the weight of rank keep - recent by radix selection on the ordered
//            bits (11 + 11 + 10), each CTA counting its eighth of the rows in a shared
//            histogram, the counts joined through distributed shared memory;
//   list     every CTA writes the rows that its eighth keeps, from the counts of
//            the eighths before it: the order is the rows' own, no atomics;
//   move     16 bytes of codes and their scale an item, all items of a round loaded before
//            the first is stored.  In place, a kept row never moves up, so the rows that a
//            round writes lie below every row that a later round reads, and a
//            cluster barrier between a round's loads and its stores is all that is needed.
// Bound by memory: 4 bytes a row of weights, and the kept rows read and written once.
#include <cooperative_groups.h>

#include "dev_common.cuh"
#include "kvq.h"

namespace cg = cooperative_groups;

namespace fm {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kBins = 2048;
constexpr int kItems = 4;        // 16-byte units a thread moves a round

// weights as unsigned integers of the same order; -0 counts as 0, NaN as less than everything
__device__ __forceinline__ uint32_t ordered(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  return w != w ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// exclusive sum over the block's threads of v, and the total; red holds kWarps + 1 words
__device__ __forceinline__ int block_scan(int v, int *red, int &total) {
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
  int base = 0, all = 0;
#pragma unroll
  for (int j = 0; j < kWarps; ++j) {
    base += j < w ? red[j] : 0;
    all += red[j];
  }
  total = all;
  return base + x - v;
}

template <int HD>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    kvq_evict_kernel(const __grid_constant__ KvqEvictArgs a) {
  constexpr int U = HD / 32;                          // units of K (and of V) a row
  constexpr int RB = kThreads * kItems / (2 * U);     // rows a CTA moves a round
  __shared__ int hist[kBins];
  __shared__ int red[kWarps + 1];
  __shared__ int s_found[2], s_cnt[2];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = blockIdx.x % kCluster, pl = blockIdx.x / kCluster;
  const int i = pl / a.c.n_kv, head = pl - i * a.c.n_kv;
  const int tid = threadIdx.x;
  const int len = a.len[i], left = min(a.keep, len);
  const bool in_place = a.src[i] == a.dst[i];
  const size_t ps = (size_t)a.src[i] * a.c.n_kv + head, pd = (size_t)a.dst[i] * a.c.n_kv + head;
  const float *ws = a.c.weights + ps * a.c.rows_pad;
  int32_t *list = a.list + (size_t)pl * a.c.rows_pad;
  int32_t *kept = a.kept ? a.kept + ((size_t)(a.call0 + i) * a.c.n_kv + head) * a.keep : nullptr;
  pdl_trigger();
  pdl_wait();

  auto put = [&](int pos, int row) {
    list[pos] = row;
    if (kept) kept[pos] = row;
  };
  if (len <= a.keep) {
    for (int r = rank * kThreads + tid; r < len; r += kCluster * kThreads) put(r, r);
  } else {
    const int nc = len - a.recent, m = a.keep - a.recent;   // m of the first nc rows stay
    for (int r = rank * kThreads + tid; r < a.recent; r += kCluster * kThreads) put(m + r, nc + r);
    const int per = (nc + kCluster - 1) / kCluster;
    const int b = min(nc, rank * per), e = min(nc, b + per);
    uint32_t prefix = 0;       // the selected weight's leading bits
    int want = m;              // its rank among the rows that share them
    if (m > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        for (int x = tid; x < kBins; x += kThreads) hist[x] = 0;
        __syncthreads();
        for (int r = b + tid; r < e; r += kThreads) {
          const uint32_t k = ordered(ws[r]);
          if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
        }
        cl.sync();
        // bins from the top: thread t has bins kBins - 1 - 4 t .. - 3
        int cnt[4], sum = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          cnt[q] = 0;
          for (int c = 0; c < kCluster; ++c) cnt[q] += *cl.map_shared_rank(&hist[kBins - 1 - 4 * tid - q], c);
          sum += cnt[q];
        }
        int total;
        int before = block_scan(sum, red, total);
        if (before < want && before + sum >= want) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (before < want && before + cnt[q] >= want) {
              s_found[0] = kBins - 1 - 4 * tid - q;
              s_found[1] = want - before;
              break;
            }
            before += cnt[q];
          }
        }
        cl.sync();   // the histograms have been read, s_found is written
        prefix = (prefix << bits) | (uint32_t)s_found[0];
        want = s_found[1];
        __syncthreads();
      }
    }
    // rows above the selected weight stay, and the first `want` that equal it
    int ng = 0, ne = 0;
    if (m > 0)
      for (int r = b + tid; r < e; r += kThreads) {
        const uint32_t k = ordered(ws[r]);
        ng += k > prefix;
        ne += k == prefix;
      }
    int tg, te;
    block_scan(ng, red, tg);
    block_scan(ne, red, te);
    if (tid == 0) s_cnt[0] = tg, s_cnt[1] = te;
    cl.sync();
    int pos = 0, eq = 0;   // rows kept, and rows equal to the weight, before this eighth
    for (int c = 0; c < rank; ++c) {
      const int *sc = cl.map_shared_rank(s_cnt, c);
      const int g = sc[0], q = sc[1];
      pos += g + min(q, max(0, want - eq));
      eq += q;
    }
    if (m > 0)
      for (int r0 = b; r0 < e; r0 += kThreads) {
        const int r = r0 + tid;
        const uint32_t k = r < e ? ordered(ws[r]) : 0u;
        const bool same = r < e && k == prefix, more = r < e && k > prefix;
        int t1, t2;
        const int er = block_scan(same, red, t1);
        const bool keep = more || (same && eq + er < want);
        const int kr = block_scan(keep, red, t2);
        if (keep) put(pos + kr, r);
        eq += t1;
        pos += t2;
      }
  }
  cl.sync();   // the list is whole, and every weight has been read
  if (!(in_place && len <= a.keep)) {
    const uint8_t *src = a.c.planes + ps * a.c.plane_bytes;
    uint8_t *dst = a.c.planes + pd * a.c.plane_bytes;
    for (int base = 0; base < left; base += kCluster * RB) {
      const int r0 = base + rank * RB;
      uint4 code[kItems];
      uint16_t sc[kItems];
      float wt = 0.f;
#pragma unroll
      for (int q = 0; q < kItems; ++q) {
        const int it = q * kThreads + tid, r = r0 + it / (2 * U), u = it % (2 * U);
        if (r < left) {
          const int row = __ldcg(list + r), t = row / kKvqTile, tr = row % kKvqTile;
          const uint8_t *h = src + (size_t)t * kvq_tile_bytes(HD) + (u >= U ? kvq_k_bytes(HD) : 0);
          code[q] = *reinterpret_cast<const uint4 *>(h + kvq_unit(tr, u % U, HD));
          sc[q] = *reinterpret_cast<const uint16_t *>(h + kvq_scale(tr, u % U, HD, u >= U));
        }
      }
      const bool has_w = tid < RB && r0 + tid < left;
      if (has_w) wt = ws[__ldcg(list + r0 + tid)];
      if (in_place) cl.sync();
#pragma unroll
      for (int q = 0; q < kItems; ++q) {
        const int it = q * kThreads + tid, r = r0 + it / (2 * U), u = it % (2 * U);
        if (r < left) {
          const int t = r / kKvqTile, tr = r % kKvqTile;
          uint8_t *h = dst + (size_t)t * kvq_tile_bytes(HD) + (u >= U ? kvq_k_bytes(HD) : 0);
          *reinterpret_cast<uint4 *>(h + kvq_unit(tr, u % U, HD)) = code[q];
          *reinterpret_cast<uint16_t *>(h + kvq_scale(tr, u % U, HD, u >= U)) = sc[q];
        }
      }
      if (has_w) a.c.weights[pd * a.c.rows_pad + r0 + tid] = wt;
    }
    if (!in_place && rank == 0 && tid == 0) a.c.vmax[pd] = a.c.vmax[ps];
  }
  cl.sync();   // no CTA leaves while another may read its shared memory
}

template <int HD>
cudaError_t evict_hd(const KvqEvictArgs &a, cudaStream_t s) {
  return kvq_launch(kvq_evict_kernel<HD>, dim3(a.n * a.c.n_kv * kCluster), dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kvq_evict(const KvqEvictArgs &a, int hd, cudaStream_t s) {
  return hd == 64 ? evict_hd<64>(a, s) : hd == 128 ? evict_hd<128>(a, s) : evict_hd<256>(a, s);
}

}  // namespace fm
