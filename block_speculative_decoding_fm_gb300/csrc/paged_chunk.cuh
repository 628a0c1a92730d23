// paged_chunk.cuh -- attention of a chunk of new tokens over a paged cache: more than 16 (token, head) rows a KV head.
//
// The same one pass as paged_rows.cuh, on the tensor cores' 128-row tiles: S = Q K^T (M = 128 query rows, N = 128 keys) into
// tensor memory, a thread a row turns its 128 scores into weights and puts them back over the scores as 16-bit operand, and
// O += P V (P from tensor memory, V from shared memory) stays in tensor memory over the unit's keys.  A row is (token, query
// head of the group): the heads of a group share every key tile, so a tile holds 128 / group whole tokens.
//   warp 0         the queries of a unit (one box a tile and 64 dims) and the key tiles (a box a page and 64 dims) into a ring
//   warp 1         the products; an elected lane issues them
//   warps 2 ..     four a query tile: scores -> weights, the outputs
// Two query tiles (kNT = 2, head dims 64 and 128) share every K and V tile and take turns: while one's scores become
// weights, the other's products run.  With one tile (kNT = 1: head dim 256, whose outputs fill half of tensor memory, or
// at most 128 rows a unit) the next key tile's scores are computed ahead into a second buffer instead.
// Products of one CTA run in the order they were issued, so a score buffer may be written behind the product that
// reads the weights in it.
//
// Bound: 4 * 128 * 128 * head_dim flop a pair of tiles against 4 * 128 * head_dim bytes: the tensor pipe for chunks, memory
// for a few tokens over a long cache.
#pragma once

#include "paged_dev.cuh"

namespace fm {

constexpr int kChunkKeys = 128;    // keys a tile
constexpr int kChunkCost = 2;      // a unit's own cost in tiles
constexpr int kChunkLeast = 4;     // places a share has at least

template <int HD, int NT>
struct ChunkCfg {
  static constexpr int kP = HD / 64;                        // panels of 64 dims
  static constexpr int kKeys = HD == 256 ? 64 : 128;        // keys a ring stage: 16 or 32 KB
  static constexpr int kSub = kChunkKeys / kKeys;           // stages a tile
  static constexpr int kStage = kKeys * HD * 2;
  static constexpr int kPanel = kKeys * 128;
  static constexpr int kQ = NT * 128 * HD * 2;
  static constexpr int kStages = (HD == 64 ? 10 : 5) + (HD == 128 && NT == 1 ? 1 : 0);
  static constexpr int kSmem = kQ + kStages * kStage + 16 * kStages + 16 * 8 + 16 * 8 + 8 * 32 + 64;
  static constexpr int kThreads = 64 + 128 * NT;
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
// operand stored [keys][dims] with dims (N) contiguous: panels of 64 dims `lbo` bytes apart, 8 keys 1024 bytes apart
__device__ __forceinline__ uint64_t desc_n_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
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
__device__ __forceinline__ void tmem_st32_async(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

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
  auto pvdone = [&](int t) { return b2 + 48 + 8 * t; };    // a tile's O += P V is done
  const uint32_t drained = b2 + 64, tslot = b2 + 72;
  const uint32_t vready = b2 + 96;                         // a masked tile's V is there
  int *poison = reinterpret_cast<int *>(gbase + (b2 - base) + 80);             // [4]: a segment that met a non-finite V
  long long *sh = reinterpret_cast<long long *>(gbase + (b2 - base) + 128);    // [kThreads / 32 + 1]
  PagedStart *start = reinterpret_cast<PagedStart *>(sh + 12);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedBatch &b = a.b;

  pdl_trigger();
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
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc<512>(tslot);
  pdl_wait();
  tc_fence_before();
  paged_plan<kRows, false, kChunkKeys, kChunkCost, kChunkLeast, C::kThreads>(a, sh, start);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(tslot);
  PagedWalk<kRows, false, kChunkKeys, kChunkCost> walk;
  walk.init(*start);
  PagedSeg g;
  const int tt = Tiles::tokens(b.group);
  // query rows of tile t of the segment's unit
  auto rows_of = [&](const PagedSeg &s, int t) {
    return max(0, min(tt, s.q.n_new - (s.tile * NT + t) * tt)) * b.group;
  };

  if (warp == 0) {
    const int box_log = min(b.page_log, 6), boxes = C::kKeys >> box_log;
    const int box = lane & (boxes - 1), panel = lane / boxes;
    const bool mine = panel < C::kP;
    uint32_t c = 0, segs = 0;
    bool ok = true;
    while (ok && walk.next(a, g)) {
      const int n = g.end - g.begin, nt = NT == 2 && rows_of(g, 1) > 0 ? 2 : 1;
      auto row_of = [&](int u) {   // of the u-th stage of the segment
        const int e = u / C::kSub, sub = u % C::kSub;
        const int j = NT == 2 ? e >> 1 : e == 0 ? 0 : (e & 1) ? min((e + 1) >> 1, n - 1) : (e - 2) >> 1;
        return mine ? paged_row(a, g.s, g.seq, g.head, g.s.tile(g.begin + j) * kChunkKeys + sub * C::kKeys + (box << box_log)) : 0;
      };
      int row = row_of(0);
      ok = mbar_wait_warp(qfree, (segs & 1) ^ 1, b.err);
      if (!ok) break;
      if (lane == 0) {
        mbar_expect_tx(qfull, nt * C::kP * tt * b.group * 128);
        for (int t = 0; t < nt; ++t)
          for (int p = 0; p < C::kP; ++p)
            tma_3d_box(qbuf + (t * C::kP + p) * 16384, &a.tq, p * 64, g.head * b.group, g.q.s0 + (g.tile * NT + t) * tt, qfull);
      }
      ++segs;
      for (int u = 0; u < 2 * n * C::kSub; ++u) {
        const int e = u / C::kSub;
        const bool is_k = NT == 2 ? !(e & 1) : e == 0 || ((e & 1) && e < 2 * n - 1);
        const int next = u + 1 < 2 * n * C::kSub ? row_of(u + 1) : 0;
        ok = mbar_wait_warp(empty(c), phase(c) ^ 1, b.err);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full(c), C::kStage);
        __syncwarp();
        if (mine)
          tma_2d_row(ring + (c % C::kStages) * C::kStage + panel * C::kPanel + (box << box_log) * 128, is_k ? &a.tk : &a.tv,
                     panel * 64, row, full(c));
        ++c;
        row = next;
      }
    }
    // the CTA leaves only after its copies have landed
    for (uint32_t u = c > (uint32_t)C::kStages ? c - C::kStages : 0; u < c; ++u) mbar_wait_drain(full(u), phase(u));
    if (segs) mbar_wait_drain(qfull, (segs - 1) & 1);
  } else if (warp == 1) {
    constexpr uint32_t IS = umma_idesc(128, C::kKeys, BF16);
    constexpr uint32_t IO = umma_idesc(128, HD, BF16) | (1u << 16);   // V with its dims contiguous
    uint32_t c0 = 0, segs = 0, tiles = 0;      // ring places, segments and (kNT = 1) tiles behind
    uint32_t np[2] = {0, 0};                   // weights taken from each score buffer
    bool ok = true;
    while (ok && walk.next(a, g)) {
      const int n = g.end - g.begin, nt = NT == 2 && rows_of(g, 1) > 0 ? 2 : 1;
      auto wait_stage = [&](int pos) {
        for (int s = 0; ok && s < C::kSub; ++s) {
          const uint32_t c = c0 + pos * C::kSub + s;
          ok = mbar_wait_warp(full(c), phase(c), b.err);
        }
      };
      auto free_stage = [&](int pos) {
        for (int s = 0; s < C::kSub; ++s) umma_commit_elect(empty(c0 + pos * C::kSub + s));
      };
      // scores of query tile t against key tile j into buffer s
      auto scores = [&](int t, int j, int s) {
#pragma unroll
        for (int sub = 0; sub < C::kSub; ++sub) {
          const uint32_t kt = ring + ((c0 + C::kpos(j, n) * C::kSub + sub) % C::kStages) * C::kStage;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_ss_elect(tmem + 128 * s + C::kKeys * sub, umma_desc_sw128(qbuf + (t * C::kP + (kk >> 2)) * 16384) + 2 * (kk & 3),
                          umma_desc_sw128(kt + (kk >> 2) * C::kPanel) + 2 * (kk & 3), IS, kk > 0 ? 1u : 0u);
        }
        umma_commit_elect(sfull(s));
      };
      auto product = [&](int t, int j, int s) {
#pragma unroll
        for (int kk = 0; kk < kChunkKeys / 16; ++kk) {
          const int sub = kk / (C::kKeys / 16), in = kk % (C::kKeys / 16);
          const uint32_t vt = ring + ((c0 + C::vpos(j, n) * C::kSub + sub) % C::kStages) * C::kStage;
          umma_ts_elect16(tmem + C::kO + t * HD, tmem + 128 * s + 8 * kk, desc_n_sw128(vt + in * 2048, C::kPanel), IO,
                          (j | kk) ? 1u : 0u);
        }
        umma_commit_elect(pvdone(t));
      };
      ok = mbar_wait_warp(qfull, segs & 1, b.err);
      wait_stage(C::kpos(0, n));
      if (!ok) break;
      tc_fence_after();
      if (NT == 2) {
        for (int t = 0; t < nt; ++t) scores(t, 0, t);
        free_stage(C::kpos(0, n));
      } else {
        for (int j = 0; j < 2 && j < n; ++j) {
          if (j) wait_stage(C::kpos(j, n));
          if (!ok) break;
          scores(0, j, (tiles + j) & 1);
          free_stage(C::kpos(j, n));
        }
      }
      if (ok && n <= (NT == 2 ? 1 : 2)) umma_commit_elect(qfree);
      for (int j = 0; ok && j < n; ++j) {
        wait_stage(C::vpos(j, n));
        if (ok && lane == 0 && paged_masked<kChunkKeys>(a, g.s, g.s.tile(g.begin + j) * kChunkKeys)) mbar_arrive(vready);
        __syncwarp();
        for (int t = 0; ok && t < nt; ++t) {
          const int s = NT == 2 ? t : (tiles + j) & 1;
          ok = ok && mbar_wait_warp(pfull(s), np[s] & 1, b.err);
          if (!ok) break;
          ++np[s];
          tc_fence_after();
          product(t, j, s);
          if (t == nt - 1) free_stage(C::vpos(j, n));
          const int jn = j + (NT == 2 ? 1 : 2);
          if (jn < n) {
            if (t == 0) wait_stage(C::kpos(jn, n));
            if (!ok) break;
            scores(t, jn, s);
            if (t == nt - 1) {
              free_stage(C::kpos(jn, n));
              if (jn == n - 1) umma_commit_elect(qfree);
            }
          }
        }
      }
      c0 += 2 * n * C::kSub;
      tiles += n;
      ++segs;
    }
    umma_commit_elect(drained);   // every product issued above has completed when this arrives
    mbar_wait_drain(drained, 0);
  } else {
    const int t = NT == 2 ? (warp - 2) >> 2 : 0, quad = warp & 3, in = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const float thr = 8.f / a.scale_log2;
    uint32_t c0 = 0, segs = 0, tiles = 0;
    uint32_t ns[2] = {0, 0}, npv = 0, nv = 0;   // scores taken from each buffer, products behind, masked tiles behind
    bool ok = true;
    int4 desc = make_int4(0, 0, 0, 0);
    while (walk.next(a, g)) {
      const int n = g.end - g.begin;
      const int rows = rows_of(g, t), token = (g.tile * NT + t) * tt + in / b.group;
      if (g.begin == 0 && !g.whole()) desc = make_int4(g.seq, g.head, g.tile, walk.parts(g));
      if (rows == 0) {       // (the unit has no second tile)
        c0 += 2 * n * C::kSub;
        ++segs;
        continue;
      }
      const bool active = quad * 32 < rows;      // some row of this warp is one
      const int pos = g.q.len - g.q.n_new + token;
      const int hi = a.causal ? min(g.q.len, pos + 1) : g.q.len;
      const int lo = a.window ? pos - a.window + 1 : 0, sink = a.window ? a.sinks : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int s = NT == 2 ? t : (tiles + j) & 1;
        const int key0 = g.s.tile(g.begin + j) * kChunkKeys;
        const bool masked = paged_masked<kChunkKeys>(a, g.s, key0);
        if (masked && t == 0) {
          // infinities and NaN of V: out of the tile (a weight of 0 times one would be NaN)
          // (the ring's own barriers cannot be waited on here: they may be a whole turn behind)
          bool bad = false;
          if (ok) ok = mbar_wait_warp(vready, nv & 1, b.err);
          ++nv;
          for (int sub = 0; sub < C::kSub; ++sub) {
            const uint32_t c = c0 + C::vpos(j, n) * C::kSub + sub;
            const uint32_t vt = ring + (c % C::kStages) * C::kStage;
            for (int u = in; ok && u < C::kStage / 16; u += 128) {
              const uint4 x = lds128(vt + u * 16);
              const uint4 w = make_uint4(not_finite<BF16>(x.x), not_finite<BF16>(x.y), not_finite<BF16>(x.z), not_finite<BF16>(x.w));
              if (w.x | w.y | w.z | w.w) {
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(vt + u * 16), "r"(x.x & ~w.x), "r"(x.y & ~w.y),
                             "r"(x.z & ~w.z), "r"(x.w & ~w.w)
                             : "memory");
                bad = true;
              }
            }
          }
          if (bad) {
            fence_proxy_async();
            poison[segs & 3] = (int)segs + 1;
          }
        }
        if (ok) ok = mbar_wait_warp(sfull(s), ns[s] & 1, b.err);
        ++ns[s];
        if (ok && active) {
          tc_fence_after();
          float x[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32_async(lanes + 128 * s + 32 * q, x + 32 * q);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int e = 0; e < 128; ++e) {
              const int key = key0 + e;
              if (!(key < hi && (key >= lo || key < sink))) x[e] = -INFINITY;
            }
          }
          float top = x[0];
#pragma unroll
          for (int e = 1; e < 128; ++e) top = fmaxf(top, x[e]);
          const bool move = top > m + thr;
          if (__any_sync(0xffffffffu, move)) {
            const float f = move ? ex2((m - top) * a.scale_log2) : 1.f;
            if (move) m = top;
            l *= f;
            if (j > 0) {
              if (NT == 1) ok = mbar_wait_warp(pvdone(0), (npv + j - 1) & 1, b.err);
              if (ok) {
#pragma unroll
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
          const float off = m == -INFINITY ? 0.f : m * a.scale_log2;
          uint32_t w[64];
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            const float p0 = ex2(fmaf(x[2 * e], a.scale_log2, -off)), p1 = ex2(fmaf(x[2 * e + 1], a.scale_log2, -off));
            l += p0 + p1;
            w[e] = pack2<BF16>(p0, p1);
          }
          tmem_st32_async(lanes + 128 * s, w);
          tmem_st32_async(lanes + 128 * s + 32, w + 32);
          tmem_wait_st();
          tc_fence_before();
        }
        // With one tile the scores run a tile ahead of the products: the last product but one is waited for here, ahead of
        // this warp's arrival, since its phase cannot be told from the next but one once the last product is done.
        if (NT == 1 && j > 0 && j == n - 1 && ok) ok = mbar_wait_warp(pvdone(0), (npv + j - 1) & 1, b.err);
        mbar_arrive(pfull(s));
      }
      // ---- the outputs ----
      if (ok) ok = mbar_wait_warp(pvdone(t), (npv + n - 1) & 1, b.err);
      npv += n;
      tc_fence_after();
      if (ok && active) {
        const bool valid = in < rows, whole = g.whole();
        const bool bad = reinterpret_cast<volatile int *>(poison)[segs & 3] == (int)segs + 1;
        const size_t slot = 2 * (size_t)blockIdx.x + (g.begin == 0 ? 1 : 0);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t *out = static_cast<uint16_t *>(a.out.p) + (int64_t)(g.q.s0 + token) * a.out.ld +
                        (int64_t)(g.head * b.group + in % b.group) * a.out.hs;
        float *po = a.part_o + (slot * kRows + 128 * t + in) * HD;
        if (valid && !whole) a.part_ml[slot * kRows + 128 * t + in] = make_float2(m == -INFINITY ? m : m * a.scale_log2, l);
#pragma unroll
        for (int q = 0; q < HD / 32; ++q) {
          float o[32];
          tmem_ld32(lanes + C::kO + t * HD + 32 * q, o);
          if (valid && bad) {
            const PagedSeg held = g;
            for (int e = 0; e < 32; ++e) {
              const float x = paged_poison<kChunkKeys, BF16>(a, held, HD, pos, 32 * q + e);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k == e) o[k] += x;
            }
          }
          if (valid && whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4 *>(out + 32 * q + e) =
                  make_uint4(pack2<BF16>(o[e] * inv, o[e + 1] * inv), pack2<BF16>(o[e + 2] * inv, o[e + 3] * inv),
                             pack2<BF16>(o[e + 4] * inv, o[e + 5] * inv), pack2<BF16>(o[e + 6] * inv, o[e + 7] * inv));
          } else if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(po + 32 * q + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      c0 += 2 * n * C::kSub;
      tiles += n;
      ++segs;
    }
    if (threadIdx.x == 64) a.desc[blockIdx.x] = desc;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free<512>(tmem);
  }
}

}  // namespace fm
