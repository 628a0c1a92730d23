// paged_dev.cuh -- what the paged cache's kernels share: reading a batch's metadata, the key tiles that a
// unit of query rows sees, and how the tiles of a launch are dealt to its CTAs.
//
// A unit is (sequence, KV head, tile of query rows: token x query head of the group); it sees a list of key
// tiles, those of the first `sinks` rows and those from the window's first row to the causal end.  The
// lengths are on the device (a captured call is replayed with other lengths), so every CTA adds up the
// launch's tiles by itself and takes an equal, contiguous share: about 1 us for 32 sequences, once a launch,
// against a second launch for a plan.  A unit that is cut between CTAs leaves unnormalised parts, which the
// join kernel adds in the order of their CTAs (so the same call gives the same bits).
#pragma once

#include "dev_common.cuh"
#include "paged.h"

namespace fm {

__device__ __forceinline__ void tma_2d_row(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// A bounded wait as mbar_wait_bounded, without a time hint: a thread wakes 30 cycles sooner (82 after the arrival, where the
// hinted form takes 112), which counts where products and weights hand over to each other every 1,000 cycles.
__device__ __forceinline__ bool paged_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool paged_wait_long(uint32_t bar, uint32_t parity, int32_t *err) {
  const long long t0 = clock64();
  long long next = t0 + 8192;
  while (!paged_try(bar, parity)) {
    const long long t = clock64();
    if (t > next) {
      if (*reinterpret_cast<volatile int32_t *>(err)) return false;
      if (t - t0 > kWaitBudgetCycles) {
        atomicExch(err, 1);
        return false;
      }
      next = t + 8192;
    }
  }
  return true;
}
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, int32_t *err) {
  if (paged_try(bar, parity)) return true;
  return paged_wait_long(bar, parity, err);
}
__device__ __forceinline__ bool paged_wait_warp(uint32_t bar, uint32_t parity, int32_t *err) {
  const bool ok = paged_wait(bar, parity, err);
  return __all_sync(0xffffffffu, ok);
}

// Two f32 values in one 64-bit register: packed arithmetic at two results an instruction.
__device__ __forceinline__ uint64_t f2_make(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_get(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}

// The halves of a word that are infinite or NaN, as a mask of their bits.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  constexpr uint32_t e = BF16 ? 0x7f80u : 0x7c00u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w >> 16 & e) == e ? 0xffff0000u : 0u);
}

struct PagedSeq {
  int s0, n_new, len;   // first packed row, new rows, rows held (the new ones are the last)
};

// Sequence i, or one without rows where its numbers point outside the batch or the table (ok: they do not).
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch &b, int i, bool &ok) {
  PagedSeq q;
  const int s0 = __ldcg(b.starts + i), s1 = __ldcg(b.starts + i + 1), len = __ldcg(b.lengths + i);
  ok = s0 >= 0 && s1 >= s0 && s1 <= b.n_tokens && len >= 0 && (int64_t)len <= ((int64_t)b.table_pages << b.page_log);
  if (!ok) b.err[1] = 1;
  q.s0 = ok ? s0 : 0;
  q.n_new = ok ? s1 - s0 : 0;
  q.len = ok ? len : 0;
  return q;
}
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch &b, int i) {
  bool ok;
  return paged_seq(b, i, ok);
}

// The key tiles (of kTile rows) that query tokens ta .. tb of a sequence see between them.
struct PagedSpan {
  int lo, hi;        // rows lo <= j < hi, and those below `sinks`
  int lt, ns, n;     // the list: tiles 0 .. ns - 1, then lt, lt + 1, ...; n in all, one at least
  int all_hi, all_lo;   // rows below all_hi are ahead of every token's end, those from all_lo on inside every window
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : lt + i - ns; }
};

template <int kTile>
__device__ __forceinline__ PagedSpan paged_span(const PagedAttnArgs &a, const PagedSeq &q, int ta, int tb) {
  PagedSpan s;
  const int pos0 = q.len - q.n_new;
  s.hi = a.causal ? max(0, min(q.len, pos0 + tb + 1)) : q.len;
  s.all_hi = a.causal ? pos0 + ta + 1 : q.len;
  s.lo = a.window ? max(0, pos0 + ta - a.window + 1) : 0;
  s.all_lo = a.window ? pos0 + tb - a.window + 1 : 0;
  if (s.lo > s.hi) s.lo = s.hi;
  s.lt = s.lo / kTile;
  const int ht = (s.hi + kTile - 1) / kTile;
  s.ns = a.window ? min((min(a.sinks, s.hi) + kTile - 1) / kTile, s.lt) : 0;
  s.n = max(1, s.ns + max(0, ht - s.lt));
  return s;
}

// Whether some token of the unit does not see some row of the tile.
template <int kTile>
__device__ __forceinline__ bool paged_masked(const PagedAttnArgs &a, const PagedSpan &s, int key0) {
  return key0 + kTile > s.all_hi || (key0 < s.all_lo && key0 + kTile > a.sinks);
}
// Whether the token at position pos sees row j (j >= 0).
__device__ __forceinline__ bool paged_sees(const PagedAttnArgs &a, const PagedSeq &q, int pos, int j) {
  return j < q.len && (!a.causal || j <= pos) && (!a.window || j > pos - a.window || j < a.sinks);
}

// Whether some token of the unit sees row j.
__device__ __forceinline__ bool paged_seen(const PagedAttnArgs &a, const PagedSpan &s, int j) {
  return j < s.hi && (j >= s.lo || (a.window && j < a.sinks));
}

// A weight is exp2(score scale - reference scale), one multiply-add whose second product is rounded: all weights of a reference are
// off by the same factor, which falls out, as long as an exponent holds it.  Past this size of the product the kernels see to it
// that it is exact.
constexpr float kFarReference = 16777216.f;

// What a row's summed outputs are multiplied by: 1 / the sum of its weights.  Without weight are a row that sees nothing (zeros) and
// one that sees only scores of minus infinity (0 / 0).
__device__ __forceinline__ float paged_inv(const PagedAttnArgs &a, const PagedSeq &q, int pos, float l) {
  if (l != 0.f) return 1.f / l;
  return q.len > 0 && (!a.causal || pos >= 0) ? __int_as_float(0x7fc00000) : 0.f;
}

// Where row `row` of the sequence lies in the pool (a page the unit does not see, or one that the table has no
// valid number for, reads as zeros): the tensor map's row.
__device__ __forceinline__ int paged_row(const PagedAttnArgs &a, const PagedSpan &s, int seq, int head, int row) {
  const PagedBatch &b = a.b;
  const int pg = row >> b.page_log, r0 = pg << b.page_log, r1 = r0 + (1 << b.page_log);
  if (!((r0 < s.hi && r1 > s.lo) || (a.window && r0 < min(a.sinks, s.hi)))) return a.oob_row;
  const int id = __ldcg(b.table + seq * b.table_ld + pg);
  if (id < 0 || id >= b.n_pages) {
    b.err[1] = 1;
    return a.oob_row;
  }
  return (((b.page0 + id) * b.n_kv + head) << b.page_log) + (row - r0);
}

// A unit's shape: kFlat: kRows consecutive (token, head) rows; otherwise kSub tiles of whole tokens, 128 / group each.
template <int kRows, bool kFlat>
struct PagedTiles {
  static constexpr int kSub = kFlat ? 1 : kRows / 128;
  static __device__ __forceinline__ int count(const PagedSeq &q, const PagedBatch &b) {
    if (kFlat) return (q.n_new * b.group + kRows - 1) / kRows;
    const int t = kSub * b.tile_tokens;
    return (q.n_new + t - 1) / t;
  }
  static __device__ __forceinline__ int first(int tile, const PagedBatch &b) {
    return kFlat ? tile * kRows / b.group : tile * kSub * b.tile_tokens;
  }
  static __device__ __forceinline__ int last(const PagedSeq &q, int tile, const PagedBatch &b) {
    if (kFlat) return (min(q.n_new * b.group, (tile + 1) * kRows) - 1) / b.group;
    return min(q.n_new, (tile + 1) * kSub * b.tile_tokens) - 1;
  }
};

// One CTA's part of a unit: key tiles begin .. end - 1 of its list.
struct PagedSeg {
  PagedSeq q;
  PagedSpan s;
  int seq, head, tile, begin, end;
  __device__ __forceinline__ bool whole() const { return begin == 0 && end == s.n; }
};

struct PagedStart {       // where a CTA's share begins
  long long left;         // places of its share
  long long share;
  PagedSeq q;
  int seq, head, tile, off;
};

// Walks a CTA's share.  A unit takes kCost places before its tiles', what beginning and ending one costs in tiles.
template <int kRows, bool kFlat, int kTile, int kCost>
struct PagedWalk {
  using Tiles = PagedTiles<kRows, kFlat>;
  long long left, share;
  int seq, head, tile, off, tiles;
  PagedSeq q;
  bool loaded;

  __device__ __forceinline__ void init(const PagedStart &p, const PagedBatch &b) {
    left = p.left, share = p.share, seq = p.seq, head = p.head, tile = p.tile, off = p.off;
    q = p.q;
    tiles = left > 0 ? Tiles::count(q, b) : 0;
    loaded = true;
  }
  // The CTAs that the unit of a segment with begin == 0 is cut into: this share ended with the segment, the rest of the
  // unit fills the shares behind it.
  __device__ __forceinline__ int parts(const PagedSeg &g) const {
    return 1 + (int)((g.s.n - g.end + share - 1) / share);
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs &a, PagedSeg &g) {
    const PagedBatch &b = a.b;
    while (left > 0 && seq < b.n_seqs) {
      if (!loaded) {
        q = paged_seq(b, seq);
        tiles = Tiles::count(q, b);
        loaded = true;
      }
      if (tiles == 0) {
        ++seq;
        loaded = false;
        continue;
      }
      g.q = q;
      g.seq = seq, g.head = head, g.tile = tile;
      g.s = paged_span<kTile>(a, q, Tiles::first(tile, b), Tiles::last(q, tile, b));
      const int total = g.s.n + kCost;
      const int take = (int)min((long long)(total - off), left);
      g.begin = max(0, off - kCost);
      g.end = max(0, off + take - kCost);
      left -= take;
      off += take;
      if (off == total) {
        off = 0;
        if (++tile == tiles) {
          tile = 0;
          if (++head == b.n_kv) {
            head = 0;
            ++seq;
            loaded = false;
          }
        }
      }
      if (g.end > g.begin) return true;
    }
    return false;
  }
};

// A warp's walk and its present segment, in shared memory: the tile loops need the registers.  The next segment may be worked
// out ahead (look), while something else is waited for: finding it takes one thread 1,300 cycles.
template <class Walk>
struct PagedWarp {
  Walk walk;
  PagedSeg g[2];
  int more, at;
  bool ahead;
  __device__ __forceinline__ void init(const PagedStart &p, const PagedBatch &b, int lane) {
    if (lane == 0) {
      walk.init(p, b);
      at = 1;
      ahead = false;
    }
  }
  // by one thread
  __device__ __forceinline__ void look(const PagedAttnArgs &a) {
    more = walk.next(a, g[at ^ 1]);
    ahead = true;
  }
  __device__ __forceinline__ bool step(const PagedAttnArgs &a) {
    if (!ahead) look(a);
    ahead = false;
    at ^= 1;
    return more != 0;
  }
  __device__ __forceinline__ bool next(const PagedAttnArgs &a, int lane) {
    __syncwarp();
    if (lane == 0) step(a);
    __syncwarp();
    return more != 0;
  }
  __device__ __forceinline__ const PagedSeg &seg() const { return g[at]; }
};

// Adds up the launch's places and finds where this CTA's share begins.  Every thread of the CTA calls it; sh: a
// long long a warp, and the start, in shared memory.  Shares are at least kLeast places.
template <int kRows, bool kFlat, int kTile, int kCost, int kLeast, int kThreads>
__device__ __forceinline__ void paged_plan(const PagedAttnArgs &a, long long *sh, PagedStart *out) {
  using Tiles = PagedTiles<kRows, kFlat>;
  const PagedBatch &b = a.b;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr int kWarps = kThreads / 32;
  // places of one KV head of a sequence; sequences of many tiles are summed by the whole warp
  auto one = [&](const PagedSeq &q, int i) -> int {
    return paged_span<kTile>(a, q, Tiles::first(i, b), Tiles::last(q, i, b)).n + kCost;
  };
  auto cost = [&](int i, PagedSeq &q) -> long long {
    q = {0, 0, 0};
    if (i < b.n_seqs) q = paged_seq(b, i);
    const int nt = Tiles::count(q, b);
    long long c = 0;
    if (nt <= 4)
      for (int j = 0; j < nt; ++j) c += one(q, j);
    for (uint32_t m = __ballot_sync(0xffffffffu, nt > 4); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      PagedSeq r;
      r.s0 = 0;
      r.n_new = __shfl_sync(0xffffffffu, q.n_new, src);
      r.len = __shfl_sync(0xffffffffu, q.len, src);
      const int n = __shfl_sync(0xffffffffu, nt, src);
      long long x = 0;
      for (int j = lane; j < n; j += 32) x += one(r, j);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == src) c = x;
    }
    return c;
  };
  // Sums of the threads' places, in the order of the sequences.  One round of kThreads sequences: its scan gives the sum as
  // well; more: a first walk for the sum, a second that stops at the share's sequence.
  const int rounds = (b.n_seqs + kThreads - 1) / kThreads;
  PagedSeq q;
  long long mine = 0, all = 0;
  if (rounds > 1) {
    for (int r = 0; r < rounds; ++r) all += cost(r * kThreads + t, q);
    all *= b.n_kv;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) sh[warp] = all;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += sh[w];
    __syncthreads();
  }
  if (t == 0) {
    out->left = 0;
    out->seq = b.n_seqs;
  }
  long long before = 0, share = 0, from = 0;
  for (int r = 0; r < rounds; ++r) {
    mine = cost(r * kThreads + t, q) * b.n_kv;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    long long lower = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) lower += sh[w];
      before += sh[w];
    }
    if (rounds == 1) all = before;
    if (r == 0) {
      share = (all >> 31) ? (all + gridDim.x - 1) / gridDim.x : (long long)(((uint32_t)all + gridDim.x - 1) / gridDim.x);
      if (share < kLeast) share = kLeast;
      from = share * blockIdx.x;
    }
    const long long end = lower + x, begin = end - mine;
    const uint32_t holds = __ballot_sync(0xffffffffu, from >= begin && from < end);
    if (holds) {   // this warp has the sequence that holds place `from`: the KV head and the tile in it
      const int src = __ffs(holds) - 1;
      PagedSeq h;
      h.s0 = __shfl_sync(0xffffffffu, q.s0, src);
      h.n_new = __shfl_sync(0xffffffffu, q.n_new, src);
      h.len = __shfl_sync(0xffffffffu, q.len, src);
      const long long rest = __shfl_sync(0xffffffffu, from - begin, src), of = __shfl_sync(0xffffffffu, mine, src) / b.n_kv;
      const int head = (rest >> 31) || (of >> 31) ? (int)(rest / of) : (int)((uint32_t)rest / (uint32_t)of);
      const int nt = Tiles::count(h, b);
      long long in = rest - head * of;
      for (int j0 = 0; j0 < nt; j0 += 32) {
        const int j = j0 + lane;
        const int c = j < nt ? one(h, j) : 0;
        long long e = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, e, o);
          if (lane >= o) e += y;
        }
        if (c > 0 && in >= e - c && in < e) {
          out->share = share;
          out->left = min(share, all - from);
          out->q = h;
          out->seq = r * kThreads + (warp << 5) + src;
          out->head = head;
          out->tile = j;
          out->off = (int)(in - (e - c));
        }
        const long long sum = __shfl_sync(0xffffffffu, e, 31);
        if (in < sum) break;
        in -= sum;
      }
    }
    __syncthreads();
    if (before > from) break;   // (the same for every thread)
  }
}

// The infinite and NaN values of V, columns d .. d + kCols - 1, in masked tiles of the segment, that the token at `pos` sees, added to
// sum (each counted with weight 1, which gives the infinity or NaN that any positive weight would).  Only asked where the
// segment met one in a row that some token of it sees: such values are taken out of the tile ahead of the product, where a
// weight of 0 would make NaN of them for rows that do not see them.  Keys outside, columns inside: a row's place is looked up
// once a page, and the threads of a warp read the same words.
template <int kTile, bool BF16, int kCols>
__device__ __noinline__ void paged_poison(const PagedAttnArgs &a, const PagedSeg &g, int hd, int pos, int d, float *sum) {
  const uint16_t *v = static_cast<const uint16_t *>(a.v_pool) + d;
  const int in_page = (1 << a.b.page_log) - 1;
  for (int i = g.begin; i < g.end; ++i) {
    const int key0 = g.s.tile(i) * kTile;
    if (!paged_masked<kTile>(a, g.s, key0)) continue;
    const int end = min(key0 + kTile, g.s.hi);
    int row = a.oob_row;
    for (int j = key0; j < end; ++j) {
      if (j == key0 || (j & in_page) == 0)
        row = paged_row(a, g.s, g.seq, g.head, j);
      else if (row != a.oob_row)
        ++row;
      if (row == a.oob_row || !paged_sees(a, g.q, pos, j)) continue;
      const uint4 *x = reinterpret_cast<const uint4 *>(v + (int64_t)row * hd);
#pragma unroll 1
      for (int c = 0; c < kCols / 8; ++c) {
        const uint4 y = x[c];
        if (!(not_finite<BF16>(y.x) | not_finite<BF16>(y.y) | not_finite<BF16>(y.z) | not_finite<BF16>(y.w))) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t h = word(y, e >> 1) >> (16 * (e & 1)) & 0xffffu;
          if (not_finite<BF16>(h)) sum[8 * c + e] += BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
        }
      }
    }
  }
}

// Where column d of a row of a part lies: 4 columns of every row together, so that threads a row each write and read next to
// one another.
template <int HD, int kRows>
__device__ __forceinline__ float *paged_part(const PagedAttnArgs &a, size_t slot, int row, int d) {
  return a.part_o + ((slot * (HD / 4) + (d >> 2)) * kRows + row) * 4 + (d & 3);
}

// Joins the parts of the units that were cut.  Blocks take the CTAs' cut units in turn (x), 64 columns each (y), and rows in
// steps; a thread takes 8 columns of a row, kSplit threads share a row's parts.  Parts lie so that neighbouring threads,
// neighbouring rows, read on from each other.  (One block a unit and warp a row read as well, but the blocks of calls that cut
// little took 4 us to come and go.)
constexpr int kJoinThreads = 512;
template <int HD, int kRows, bool kFlat, bool BF16, int kSplit>
__global__ void __launch_bounds__(kJoinThreads) fm_paged_join_kernel(const __grid_constant__ PagedAttnArgs a, int ctas) {
  using Tiles = PagedTiles<kRows, kFlat>;
  constexpr int kStep = kJoinThreads / (8 * kSplit);      // rows at a time
  static_assert(kStep <= kRows, "rows of a step");
  __shared__ float acc[kSplit > 1 ? kSplit - 1 : 1][kSplit > 1 ? kStep * 8 : 1][9];
  pdl_trigger();
  pdl_wait();
  const int group = a.b.group, zs = gridDim.z;
  const int r = threadIdx.x % kStep, c = threadIdx.x / kStep % 8, sub = threadIdx.x / (kStep * 8);
  for (int cta = blockIdx.x; cta < ctas; cta += gridDim.x) {
    const int4 d = __ldcg(a.desc + cta);
    if (d.w == 0) continue;
    const PagedSeq q = paged_seq(a.b, d.x);
    auto slot = [&](int p) -> size_t { return p == 0 ? 2 * (size_t)cta + 1 : 2 * (size_t)(cta + p); };
    for (int r0 = blockIdx.z * kStep; r0 < kRows; r0 += zs * kStep) {
      const int row = r0 + r;
      int token, head;
      bool valid;
      if (kFlat) {
        const int f = d.z * kRows + row;
        token = f / group;
        head = f - token * group;
        valid = f < q.n_new * group;
      } else {
        const int tt = a.b.tile_tokens, in = row & 127, tk = in * a.b.group_inv >> 16;
        token = (d.z * Tiles::kSub + (row >> 7)) * tt + tk;
        head = in - tk * group;
        valid = in < tt * group && token < q.n_new;
      }
      // one pass with the running maximum, kAhead parts in flight
      constexpr int kAhead = 4;
      float top = -INFINITY, l = 0.f, o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
      if (valid)
        for (int p0 = sub; p0 < d.w; p0 += kSplit * kAhead) {
          float2 ml[kAhead];
          float4 x[kAhead][2];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const int p = p0 + u * kSplit;
            ml[u] = make_float2(-INFINITY, 0.f);
            if (p < d.w) {
              const int d0 = blockIdx.y * 64 + 8 * c;
              ml[u] = __ldcg(a.part_ml + slot(p) * kRows + row);
              x[u][0] = __ldcg(reinterpret_cast<const float4 *>(paged_part<HD, kRows>(a, slot(p), row, d0)));
              x[u][1] = __ldcg(reinterpret_cast<const float4 *>(paged_part<HD, kRows>(a, slot(p), row, d0 + 4)));
            }
          }
          float t = top;
#pragma unroll
          for (int u = 0; u < kAhead; ++u) t = fmaxf(t, ml[u].x);
          const float f = top == -INFINITY ? 0.f : ex2(top - t);
          top = t;
          l *= f;
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            if (ml[u].y == 0.f) continue;   // (no part, or no weight in it; one whose scores are all NaN has a sum of NaN)
            const float w = ex2(ml[u].x - t);
            l += w * ml[u].y;
            o[0] += w * x[u][0].x, o[1] += w * x[u][0].y, o[2] += w * x[u][0].z, o[3] += w * x[u][0].w;
            o[4] += w * x[u][1].x, o[5] += w * x[u][1].y, o[6] += w * x[u][1].z, o[7] += w * x[u][1].w;
          }
        }
      if constexpr (kSplit > 1) {
        __shared__ float2 tl[kSplit][kStep * 8];
        const int at = c * kStep + r;
        __syncthreads();
        tl[sub][at] = make_float2(top, l);
        __syncthreads();
        float t = -INFINITY;
#pragma unroll
        for (int u = 0; u < kSplit; ++u) t = fmaxf(t, tl[u][at].x);
        const float f = top == -INFINITY ? 0.f : ex2(top - t);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f;
        if (sub > 0)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[sub - 1][at][e] = o[e];
        __syncthreads();
        if (sub == 0) {
          l = 0.f;
#pragma unroll
          for (int u = 0; u < kSplit; ++u) {
            const float2 x = tl[u][at];
            l += x.y == 0.f ? 0.f : ex2(x.x - t) * x.y;
          }
#pragma unroll
          for (int u = 1; u < kSplit; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] += acc[u - 1][at][e];
        }
      }
      if (valid && sub == 0) {
        const float inv = paged_inv(a, q, q.len - q.n_new + token, l);
        uint16_t *out = static_cast<uint16_t *>(a.out.p) + (int64_t)(q.s0 + token) * a.out.ld +
                        (int64_t)(d.y * group + head) * a.out.hs + blockIdx.y * 64 + 8 * c;
        *reinterpret_cast<uint4 *>(out) = make_uint4(pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv),
                                                     pack2<BF16>(o[4] * inv, o[5] * inv), pack2<BF16>(o[6] * inv, o[7] * inv));
      }
    }
  }
}

}  // namespace fm
