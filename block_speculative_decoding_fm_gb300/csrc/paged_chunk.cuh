// paged_chunk.cuh -- attention of a chunk of new tokens over a paged cache: more than 16 (token, head) rows a KV head.
//
// The same one pass as paged_rows.cuh, on the tensor cores' 128-row tiles: S = Q K^T (M = 128 query rows, N = 128 keys) into
// tensor memory, a thread a row turns its 128 scores into weights and puts them back over the scores as 16-bit operand, and
// O += P V (P from tensor memory, V from shared memory) stays in tensor memory over the unit's keys.  A row is (token, query
// head of the group): the heads of a group share every key tile, so a tile holds 128 / group whole tokens.
//   warp 0         the queries of a unit (one box a tile and 64 dims) and the key tiles (a box a page and 64 dims) into a ring
//   warp 1         the products; an elected lane issues them
//   warps 2, 3     see that masked tiles of V hold finite values only, and note where a row that is seen did not
//   warps 4 ..     four a query tile, a thread a row: scores -> weights, the outputs
// Two query tiles (kNT = 2, head dims 64 and 128) share every K and V tile and take turns: while one's scores become
// weights, the other's products run.  With one tile (kNT = 1: head dim 256, whose outputs fill half of tensor memory, or
// at most 128 rows a unit) the next key tile's scores are computed ahead into a second buffer instead.
// Products of one CTA run in the order they were issued, so a score buffer may be written behind the product that
// reads the weights in it.
//
// P enters the second product rounded once to the pool's type, as paged_rows.cuh says; sums, outputs and references are f32.
//
// Bound: 4 * 128 * 128 * head_dim flop a query and a key tile against 4 * 128 * head_dim bytes: the tensor pipe for chunks, memory
// for a few tokens over a long cache.  Measured, calls one after another for seconds: 2,048 rows over 34,816 of 16 x 128 bf16 454 us
// (1.25 PFLOP/s, 0.64 of the measured bf16 rate; the card is at its power limit then, at 1,485 of 2,070 MHz -- the first tens of
// calls take 390-405 us, 1.40-1.45 PFLOP/s, tensor pipe 67 %); prompts of 33-4,001 rows of 24/4 x 256 817 us (1.00 PFLOP/s; 790 in
// a short graph).  In short graphs: 1-17 rows of 32 sequences of 16 x 128 over 512-8,192 in pages of 64 179 us (0.88 of the copy
// rate), of 16 206; 512 rows over 8,704 of 8 x 128 34 (floor 9); eight prompts of 1,024 of 16 x 128 68-72 (floor 20).  What is
// left: a tile's chain (scores, 890 cycles of weights with a warp a scheduler, products) against 2,048 cycles of products a
// pair of tiles; in short chunks the units' ends and starts.
#pragma once

#include "paged_dev.cuh"

namespace fm {

constexpr int kChunkKeys = 128;    // keys a tile
// A unit's own cost in tiles, and the places a share has at least.  (1 and 2: prompts of 24/4 x 256 846 us; 2 and 3: 811; 3 and 4:
// 803, but eight rows over 4,161 21.0 us for 19.5 and prompts of 1,024 of 16 x 128 73.9 for 70.6.)
constexpr int kChunkCost = 2;
constexpr int kChunkLeast = 3;

template <int HD, int NT>
struct ChunkCfg {
  using Walk = PagedWalk<128 * NT, false, kChunkKeys, kChunkCost>;
  static constexpr int kP = HD / 64;                        // panels of 64 dims
  static constexpr int kDims = HD < 128 ? HD : 128;         // dims a ring stage: 128 keys, 16 or 32 KB
  static constexpr int kSub = HD / kDims;                   // stages a tile
  static constexpr int kStage = kChunkKeys * kDims * 2;
  static constexpr int kPanel = kChunkKeys * 128;
  static constexpr int kQ = NT * 128 * HD * 2;
  static constexpr int kStages = (HD == 64 ? 10 : 5) + (HD == 128 && NT == 1 ? 1 : 0);
  static constexpr int kThreads = 128 + 128 * NT;
  static constexpr int kSums = 16;                          // long longs that the plan takes
  static constexpr int kSmem = kQ + kStages * kStage + 16 * kStages + 128 + 8 * kSums + sizeof(PagedStart) + (4 + 4 * NT) * sizeof(PagedWarp<Walk>);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static constexpr int kO = 256;                            // first column of the outputs (scores: 0 .. 255)
  // place in the ring's order of tile j's K and V, of a segment of n tiles
  __device__ static int kpos(int j, int n) { return NT == 2 ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
  __device__ static int vpos(int j, int n) { return NT == 2 ? 2 * j + 1 : j < n - 1 ? 2 * j + 2 : 2 * n - 1; }
};

// kind::f16 with A in tensor memory
__device__ __forceinline__ void umma_ts_elect16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Shared-memory descriptors of 128-byte-swizzled operands as their low word (the address, and for operands stored [keys]
// [dims] the distance of panels of 64 dims); the high word (8 rows are 1024 bytes) is a constant, so that a product needs
// one register of its own an operand: the instruction takes uniform registers, and each value moved there costs it time.
__device__ __forceinline__ uint32_t lo_k(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t lo_n(uint32_t saddr, uint32_t lbo) { return (saddr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(d) : "r"(lo), "n"((1024 >> 4) | 1 << 14 | 2 << 29));
  return d;
}
// 32 columns of this thread's lane, without waiting for them
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float *f) {
  uint32_t *v = reinterpret_cast<uint32_t *>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// The bits below bit n.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
// 0 x w + sum in both halves: a sum stays 0 until a half of w is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t none(uint32_t w, uint32_t sum) {
  if constexpr (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %0;\n" : "+r"(sum) : "r"(w), "r"(0));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %0;\n" : "+r"(sum) : "r"(w), "r"(0));
  return sum;
}
// Four lanes' 16-byte pieces, transposed: lane q had pieces 0 .. 3 of its row, and has piece q of the four lanes' rows.
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int lane) {
  auto swap = [&](uint4 &x, uint4 &y, int step, bool upper) {   // y of the lower lane for x of the upper one
    uint4 s = upper ? x : y, r;
    r.x = __shfl_xor_sync(0xffffffffu, s.x, step);
    r.y = __shfl_xor_sync(0xffffffffu, s.y, step);
    r.z = __shfl_xor_sync(0xffffffffu, s.z, step);
    r.w = __shfl_xor_sync(0xffffffffu, s.w, step);
    if (upper)
      x = r;
    else
      y = r;
  };
  swap(v[0], v[1], 1, lane & 1);
  swap(v[2], v[3], 1, lane & 1);
  swap(v[0], v[2], 2, lane & 2);
  swap(v[1], v[3], 2, lane & 2);
}

template <int HD, int NT, bool BF16>
__global__ void __launch_bounds__(ChunkCfg<HD, NT>::kThreads, 1)
    fm_paged_chunk_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = ChunkCfg<HD, NT>;
  constexpr int kRows = 128 * NT;
  using Tiles = PagedTiles<kRows, false>;
  extern __shared__ __align__(1024) uint8_t gbase[];
  const uint32_t base = smem_u32(gbase);
  const uint32_t qbuf = base, ring = base + C::kQ;
  const uint32_t bars = ring + C::kStages * C::kStage;
  auto full = [&](uint32_t c) { return bars + 8 * (c % C::kStages); };
  auto empty = [&](uint32_t c) { return bars + 8 * (C::kStages + c % C::kStages); };
  auto phase = [&](uint32_t c) { return (c / C::kStages) & 1; };
  const uint32_t b2 = bars + 16 * C::kStages;
  const uint32_t qfull = b2, qfree = b2 + 8;
  auto sfull = [&](int s) { return b2 + 16 + 8 * s; };     // a score buffer's products are done
  auto pfull = [&](int s) { return b2 + 32 + 8 * s; };     // its weights are stored
  auto pvdone = [&](int s) { return b2 + 48 + 8 * s; };    // O += P V is done: kNT = 2 a query tile's last, kNT = 1 a buffer's
  const uint32_t drained = b2 + 64, tslot = b2 + 72;
  const uint32_t vready = b2 + 96, vclean = b2 + 104;      // a masked tile's V is there, and holds finite values only
  int *poison = reinterpret_cast<int *>(gbase + (b2 - base) + 80);             // [4]: a segment that met a non-finite V
  long long *sh = reinterpret_cast<long long *>(gbase + (b2 - base) + 128);    // [kSums]
  PagedStart *start = reinterpret_cast<PagedStart *>(sh + C::kSums);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PagedWarp<typename C::Walk> &w = reinterpret_cast<PagedWarp<typename C::Walk> *>(start + 1)[warp];
  const PagedBatch &b = a.b;

  // Tensor memory ahead of the trigger: a later launch that started first could take it, and would wait for this one.
  if (warp == 1) {
    tmem_alloc<512>(tslot);
    pdl_trigger();
  }
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.tk)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.tv)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.tq)) : "memory");
    for (uint32_t s = 0; s < (uint32_t)C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qfree, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(sfull(s), 1);
      mbar_init(pfull(s), 128);
      mbar_init(pvdone(s), 1);
      poison[s] = poison[2 + s] = 0;
    }
    mbar_init(drained, 1);
    mbar_init(vready, 1);
    mbar_init(vclean, 64);
    mbar_fence_init();
  }
  pdl_wait();
  tc_fence_before();
  paged_plan<kRows, false, kChunkKeys, kChunkCost, kChunkLeast, C::kThreads>(a, sh, start);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(tslot);
  w.init(*start, b, lane);
  const int tt = b.tile_tokens;
  // query rows of tile t of the segment's unit
  auto rows_of = [&](const PagedSeg &s, int t) {
    return max(0, min(tt, s.q.n_new - (s.tile * NT + t) * tt)) * b.group;
  };

  // registers of a thread: 384 at 168 become 256 at 208 for scores and weights, and 128 at 88
  if (NT == 2 && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
  if (warp == 0) {
    const int box_log = min(b.page_log, 6), boxes = kChunkKeys >> box_log;
    const int box = lane & (boxes - 1), panel = lane / boxes;
    const bool mine = panel < C::kDims / 64;
    uint32_t c = 0, segs = 0;
    bool ok = true;
    while (ok && w.next(a, lane)) {
      const PagedSeg &g = w.seg();
      const int n = g.end - g.begin, nt = NT == 2 && rows_of(g, 1) > 0 ? 2 : 1;
      // where this lane's rows of a key tile lie
      auto row_of = [&](int j) {
        return mine && j < n ? paged_row(a, g.s, g.seq, g.head, g.s.tile(g.begin + j) * kChunkKeys + (box << box_log)) : 0;
      };
      auto fetch = [&](const CUtensorMap *map, int row) {
#pragma unroll
        for (int sub = 0; ok && sub < C::kSub; ++sub) {
          ok = paged_wait_warp(empty(c), phase(c) ^ 1, b.err);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(full(c), C::kStage);
          __syncwarp();
          if (mine)
            tma_2d_row(ring + (c % C::kStages) * C::kStage + panel * C::kPanel + (box << box_log) * 128, map,
                       sub * C::kDims + panel * 64, row, full(c));
          ++c;
        }
      };
      ok = paged_wait_warp(qfree, (segs & 1) ^ 1, b.err);
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_tx(qfull, nt * C::kP * tt * b.group * 128);
        for (int t = 0; t < nt; ++t)
          for (int p = 0; p < C::kP; ++p)
            tma_3d_box(qbuf + (t * C::kP + p) * 16384, &a.tq, p * 64, g.head * b.group, g.q.s0 + (g.tile * NT + t) * tt, qfull);
      }
      ++segs;
      // (the table is asked two tiles ahead)
      int before = 0, row = row_of(0), next = row_of(1);
      for (int j = 0; ok && j <= n; ++j) {
        const int ahead = row_of(j + 2);
        if (j < n) fetch(&a.tk, row);
        if (NT == 2 && j < n) fetch(&a.tv, row);
        if (NT == 1 && j > 0) fetch(&a.tv, before);   // V behind the next tile's K: the scores run a tile ahead
        before = row, row = next, next = ahead;
      }
    }
    // the CTA leaves only after its copies have landed
    for (uint32_t u = c > (uint32_t)C::kStages ? c - C::kStages : 0; u < c; ++u) mbar_wait_drain(full(u), phase(u));
    if (segs) mbar_wait_drain(qfull, (segs - 1) & 1);
  } else if (warp == 1) {
    // A product takes the tensor pipe 64 cycles and this warp 36 to issue; the pipe holds eight.  A wait costs 90 cycles and a
    // commit 100 even where nothing is waited for, so there are few: key tiles are waited for while products are queued, and
    // with two query tiles the ring's stages are given back by the warps that see the scores behind them (with one, whose
    // ring holds little more than a tile of head dim 256, at once).  (Two threads that issue, one a query
    // tile, cost less each, but the tiles then run in step and weights and products take turns: 585 us for 454.)
    constexpr uint32_t IS = umma_idesc(128, kChunkKeys, BF16);
    constexpr uint32_t IO = umma_idesc(128, C::kDims, BF16) | (1u << 16);   // V with its dims contiguous
    uint32_t c0 = 0, segs = 0, tiles = 0;      // ring places, segments and (kNT = 1) tiles behind
    uint32_t np[2] = {0, 0}, nv = 0;           // weights taken from each score buffer, masked tiles behind
    bool ok = true;
    while (ok && w.next(a, lane)) {
      const PagedSeg &g = w.seg();
      const PagedSpan span = g.s;
      const int n = g.end - g.begin, begin = g.begin, nt = NT == 2 && rows_of(g, 1) > 0 ? 2 : 1;
      auto stage = [&](int pos) { return ring + ((c0 + pos) % C::kStages) * C::kStage; };
      auto wait_stage = [&](int pos) {
#pragma unroll
        for (int s = 0; s < C::kSub; ++s) {
          const uint32_t c = c0 + pos * C::kSub + s;
          ok = ok && paged_wait_warp(full(c), phase(c), b.err);
        }
      };
      auto free_stage = [&](int pos) {
#pragma unroll
        for (int s = 0; s < C::kSub; ++s) umma_commit_elect(empty(c0 + pos * C::kSub + s));
      };
      // scores of query tile t against key tile j into buffer s
      auto scores = [&](int t, int j, int s) {
        const uint32_t d = tmem + 128 * s, q0 = lo_k(qbuf + t * C::kP * 16384);
#pragma unroll
        for (int sub = 0; sub < C::kSub; ++sub) {
          const uint32_t k0 = lo_k(stage(C::kpos(j, n) * C::kSub + sub));
#pragma unroll
          for (int kk = 0; kk < C::kDims / 16; ++kk)
            umma_ss_elect(d, desc_of(q0 + ((sub * (C::kDims / 64) + (kk >> 2)) * 16384 + (kk & 3) * 32) / 16),
                          desc_of(k0 + ((kk >> 2) * C::kPanel + (kk & 3) * 32) / 16), IS, sub || kk ? 1u : 0u);
        }
        umma_commit_elect(sfull(s));
      };
      // outputs of query tile t += its weights of tile j, V
      auto product = [&](int t, int j, int s) {
        const uint32_t d = tmem + C::kO + t * HD, pt = tmem + 128 * s;
#pragma unroll
        for (int sub = 0; sub < C::kSub; ++sub) {
          const uint32_t v0 = lo_n(stage(C::vpos(j, n) * C::kSub + sub), C::kPanel);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts_elect16(d + sub * C::kDims, pt + 8 * kk, desc_of(v0 + kk * 2048 / 16), IO, kk ? 1u : j ? 1u : 0u);
        }
      };
      // a masked tile's V, once it is there, is handed to the warps that look it over
      auto clean = [&](int j) {
        if (!paged_masked<kChunkKeys>(a, span, span.tile(begin + j) * kChunkKeys)) return;
        if (ok && lane == 0) mbar_arrive(vready);
        ok = ok && paged_wait_warp(vclean, nv++ & 1, b.err);
      };
      ok = paged_wait_warp(qfull, segs & 1, b.err);
      wait_stage(C::kpos(0, n));
      if (!ok) break;
      tc_fence_after();
      if (NT == 2) {
        for (int t = 0; t < nt; ++t) scores(t, 0, t);
      } else {
        scores(0, 0, tiles & 1);
        free_stage(C::kpos(0, n));
        if (n > 1) {
          wait_stage(C::kpos(1, n));
          if (!ok) break;
          scores(0, 1, (tiles + 1) & 1);
          free_stage(C::kpos(1, n));
        }
      }
      for (int j = 0; ok && j < n; ++j) {
        wait_stage(C::vpos(j, n));
        clean(j);
        if (NT == 2) {
          if (j + 1 < n) wait_stage(C::kpos(j + 1, n));
          for (int t = 0; ok && t < nt; ++t) {
            ok = paged_wait_warp(pfull(t), np[t]++ & 1, b.err);
            if (!ok) break;
            tc_fence_after();
            product(t, j, t);
            if (j + 1 < n)
              scores(t, j + 1, t);
            else
              umma_commit_elect(pvdone(t));
          }
        } else {
          const int s = (tiles + j) & 1;
          ok = ok && paged_wait_warp(pfull(s), np[s]++ & 1, b.err);
          if (!ok) break;
          tc_fence_after();
          product(0, j, s);
          umma_commit_elect(pvdone(s));
          free_stage(C::vpos(j, n));
          if (j + 2 < n) {                     // (the ring may not hold it before V is free)
            wait_stage(C::kpos(j + 2, n));
            if (!ok) break;
            scores(0, j + 2, s);
            free_stage(C::kpos(j + 2, n));
          }
        }
      }
      c0 += 2 * n * C::kSub;
      tiles += n;
      ++segs;
    }
    umma_commit_elect(drained);   // every product issued above has completed when this arrives
    mbar_wait_drain(drained, 0);
  } else if (warp < 4) {
    // Masked tiles of V: infinities and NaN out of them (a weight of 0 times one would be NaN), while the scores become
    // weights.  (The ring's own barriers cannot be waited on here: they may be a whole turn behind.)
    // A word is one fused multiply-add, four sums at a time; the loop is short because it runs once or twice a unit, from
    // instructions that have left the caches since (exponents compared by three integer operations a word and both
    // halves of head dim 256 unrolled: 153 us for the windowed chunk of 8,191 rows, 146 so; 148 with the place of what is found
    // looked at, so that garbage in hidden rows stays cheap).
    uint32_t c0 = 0, segs = 0, nv = 0;
    bool ok = true;
    while (ok && w.next(a, lane)) {
      const PagedSeg &g = w.seg();
      const int n = g.end - g.begin;
      for (int j = 0; ok && j < n; ++j) {
        if (!paged_masked<kChunkKeys>(a, g.s, g.s.tile(g.begin + j) * kChunkKeys)) continue;
        ok = paged_wait_warp(vready, nv++ & 1, b.err);
        if (!ok) break;
#pragma unroll 1
        for (int sub = 0; sub < C::kSub; ++sub) {
          const uint32_t vt = ring + ((c0 + C::vpos(j, n) * C::kSub + sub) % C::kStages) * C::kStage + ((warp & 1) * 32 + lane) * 16;
          uint4 sum = make_uint4(0, 0, 0, 0);
#pragma unroll 4
          for (int u = 0; u < C::kStage; u += 64 * 16) {
            const uint4 x = lds128(vt + u);
            sum = make_uint4(none<BF16>(x.x, sum.x), none<BF16>(x.y, sum.y), none<BF16>(x.z, sum.z), none<BF16>(x.w, sum.w));
          }
          if ((sum.x | sum.y | sum.z | sum.w) & 0x7fff7fffu) {
            const int key0 = g.s.tile(g.begin + j) * kChunkKeys;
#pragma unroll 1
            for (int u = 0; u < C::kStage; u += 64 * 16) {
              const uint4 x = lds128(vt + u);
              const uint4 f = make_uint4(not_finite<BF16>(x.x), not_finite<BF16>(x.y), not_finite<BF16>(x.z), not_finite<BF16>(x.w));
              if (!(f.x | f.y | f.z | f.w)) continue;
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(vt + u), "r"(x.x & ~f.x), "r"(x.y & ~f.y), "r"(x.z & ~f.z),
                           "r"(x.w & ~f.w)
                           : "memory");
              const int row = (((warp & 1) * 32 + lane) * 16 + u) / 128 % kChunkKeys;
              if (paged_seen(a, g.s, key0 + row)) poison[segs & 3] = (int)segs + 1;
            }
            fence_proxy_async();
          }
        }
        mbar_arrive(vclean);
      }
      c0 += 2 * n * C::kSub;
      ++segs;
    }
  } else {
    // ---- four warps a query tile, a thread a row ----
    if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    const int t = (warp - 4) >> 2, quad = warp & 3, in = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const float thr = 8.f / a.scale_log2;       // a row's reference moves where a score beats it by 2^8
    // For far references the power of two below the scale, whose products are exact; a weight w becomes up to sqrt(w), but there a
    // score's last bit is a factor of two or more.  (The reference taken off every score: 10 % slower.)
    const float far = __int_as_float(__float_as_int(a.scale_log2) & 0x7f800000);
    uint32_t c0 = 0, segs = 0, tiles = 0;
    uint32_t ns[2] = {0, 0}, npv = 0;           // scores taken from each buffer, products behind
    bool ok = true;
    if (threadIdx.x == 128) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    while (w.next(a, lane)) {
      const PagedSeg &g = w.seg();
      const int n = g.end - g.begin;
      const int rows = rows_of(g, t), token = (g.tile * NT + t) * tt + (int)(in * b.group_inv >> 16);
      if (threadIdx.x == 128 && g.begin == 0 && !g.whole()) a.desc[blockIdx.x] = make_int4(g.seq, g.head, g.tile, w.walk.parts(g));
      if (rows == 0) {                          // (the unit has no second tile)
        c0 += 2 * n * C::kSub;
        ++segs;
        continue;
      }
      const bool active = quad * 32 < rows;     // some row of this warp is one
      // the thread that gives the ring's stages back: scores of the last query tile are there when all before them is done
      const bool frees = quad == 0 && lane == 0 && (NT == 1 || t == 1 || rows_of(g, 1) == 0);
      const int pos = g.q.len - g.q.n_new + token;
      float m = -INFINITY, by = a.scale_log2;   // the row's reference, and what its scores are multiplied by
      uint64_t sum[2] = {0, 0};                 // of weights: two packed pairs
      for (int j = 0; j < n; ++j) {
        const int s = NT == 2 ? t : (tiles + j) & 1;
        const int key0 = g.s.tile(g.begin + j) * kChunkKeys;
        const bool masked = paged_masked<kChunkKeys>(a, g.s, key0);
        if (ok) ok = paged_wait_warp(sfull(s), ns[s] & 1, b.err);
        ++ns[s];
        if (frees && ok) {
          if (NT == 2 && j > 0) mbar_arrive(empty(c0 + C::vpos(j - 1, n)));
          if (NT == 2) mbar_arrive(empty(c0 + C::kpos(j, n)));
          if (j == n - 1) mbar_arrive(qfree);
        }
        if (ok && active) {
          tc_fence_after();
          float x[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32_async(lanes + 128 * s + 32 * q, x + 32 * q);
          tmem_wait_ld();
          if (masked) {
            // a bit a key: ahead of the end, and inside the window or among the first
            const int hi = a.causal ? min(g.q.len, pos + 1) : g.q.len, lo = a.window ? pos - a.window + 1 : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int k = key0 + 32 * q;
              const uint32_t see = below(hi - k) & (~below(lo - k) | below((a.window ? a.sinks : 0) - k));
              if (__any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[32 * q + e] = see & (1u << e) ? x[32 * q + e] : -INFINITY;
              }
            }
          }
          float tops[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tops[q] = x[q];
#pragma unroll
            for (int e = 4 + q; e < 128; e += 8) tops[q] = fmaxf(fmaxf(tops[q], x[e]), e + 4 < 128 ? x[e + 4] : x[e]);
          }
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
          const bool move = top > m + thr;
          if (__any_sync(0xffffffffu, move)) {
            const float f = move ? ex2((m - top) * a.scale_log2) : 1.f;
            if (move) m = top, by = fabsf(top * a.scale_log2) > kFarReference ? far : a.scale_log2;
            const uint64_t f2 = f2_make(f, f);
            sum[0] = f2_fma(sum[0], f2, 0);
            sum[1] = f2_fma(sum[1], f2, 0);
            if (j > 0) {
              if (NT == 1) ok = paged_wait_warp(pvdone(s ^ 1), (ns[s ^ 1] - 1) & 1, b.err);   // (the last tile's product)
              if (ok) {
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < HD / 32; ++q) {
                  float o[32];
                  tmem_ld32(lanes + C::kO + t * HD + 32 * q, o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] *= f;
                  tmem_st32(lanes + C::kO + t * HD + 32 * q, o);
                }
              }
            }
          }
          const float off = m == -INFINITY ? 0.f : -m * by;
          const uint64_t scale2 = f2_make(by, by), off2 = f2_make(off, off);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              f2_get(f2_fma(f2_make(x[32 * q + 2 * e], x[32 * q + 2 * e + 1]), scale2, off2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[e & 1] = f2_add(sum[e & 1], f2_make(p0, p1));
              p[e] = pack2<BF16>(p0, p1);
            }
            tmem_st16_async(lanes + 128 * s + 16 * q, p);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(pfull(s));
      }
      // ---- the outputs ----
      float l, l2;
      f2_get(f2_add(sum[0], sum[1]), l, l2);
      l += l2;
      const int last = NT == 2 ? t : (tiles + n - 1) & 1;
      const bool starts = g.begin == 0, whole = g.whole();
      if (lane == 0) w.look(a);                 // (while the last product runs)
      if (ok) ok = paged_wait_warp(pvdone(last), (NT == 2 ? npv++ : ns[last] - 1) & 1, b.err);
      if (NT == 2 && frees && ok) mbar_arrive(empty(c0 + C::vpos(n - 1, n)));
      tc_fence_after();
      if (ok && active) {
        const bool valid = in < rows;
        const bool bad = reinterpret_cast<volatile int *>(poison)[segs & 3] == (int)segs + 1;
        const size_t slot = 2 * (size_t)blockIdx.x + (starts ? 1 : 0);
        const float inv = paged_inv(a, g.q, pos, l);
        // a quad of lanes writes 64 bytes of its four rows, one after another
        int64_t at[4];
        bool there[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (in & ~3) + i, tk = r * b.group_inv >> 16;
          there[i] = r < rows;
          at[i] = (int64_t)(g.q.s0 + (g.tile * NT + t) * tt + tk) * a.out.ld + (int64_t)(g.head * b.group + r - tk * b.group) * a.out.hs +
                  8 * (lane & 3);
        }
        uint16_t *out = static_cast<uint16_t *>(a.out.p);
        if (valid && !whole)
          a.part_ml[slot * kRows + 128 * t + in] = make_float2(m == -INFINITY ? m : m * a.scale_log2, l);
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float o[32];
          tmem_ld32(lanes + C::kO + t * HD + c, o);
          if (bad) {
            if (valid) {
              const PagedSeg held = g;
              float more[32] = {};
              paged_poison<kChunkKeys, BF16, 32>(a, held, HD, pos, c, more);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] += more[e];
            }
            __syncwarp();
          }
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = make_uint4(pack2<BF16>(o[8 * i] * inv, o[8 * i + 1] * inv), pack2<BF16>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                pack2<BF16>(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack2<BF16>(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
            transpose4(v, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (there[i]) *reinterpret_cast<uint4 *>(out + at[i] + c) = v[i];
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(paged_part<HD, kRows>(a, slot, 128 * t + in, c + e)) =
                  make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      c0 += 2 * n * C::kSub;
      tiles += n;
      ++segs;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<512>(tmem);
  }
}

}  // namespace fm
