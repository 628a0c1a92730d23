// paged_rows.cuh -- attention of few query rows over a paged cache: single tokens, draft blocks, anything up to
// 16 (token, head) rows a KV head at its best.
//
// out = sum_j p_j v_j / sum_j p_j, p_j = exp2(scale_log2 q.k_j - m): one pass over the keys, with a reference m a row that
// moves only where a score beats it by 2^8 (then sums and outputs are scaled once), so a step costs no rescaling.
//
// Bound: memory, 4 head_dim bytes a key against 4 * 16 * head_dim flop.  A CTA is one warp that fetches and four that
// compute.  The fetching warp walks the share's key stages (64 rows of K and of V) and asks for a box a page and 64 dims
// into a ring of mbarriers; a computing warp takes 16 of a stage's rows: S = Q K^T and O += P V by m16n8k16 products with
// f32 sums (16 query rows are the products' M: at most a quarter of the legacy pipe's rate is needed to keep up with HBM,
// and the tcgen05 form would need P through tensor memory for 16 rows of 128).  The four warps' sums meet at a
// unit's end.  P enters the product rounded once to the pool's type, as the matrix instructions need it: half a step of
// each weight, averaged over the keys (below the output's own rounding); the sum of weights stays f32.
#pragma once

#include "paged_dev.cuh"

namespace fm {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
  else
    mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
}

constexpr int kRowsUnit = 16;      // query rows a unit
constexpr int kRowsKeys = 64;      // keys a stage
// A unit's own cost in stages (queries, first fetch, outputs), and the places a share has at least.  (3 and 6: 22.0 us for a
// windowed token of 32 sequences, 97 us for 16 rows over 65,537; 4 and 5: 21.9 and 96.)
constexpr int kRowsCost = 4;
constexpr int kRowsLeast = 5;
constexpr int kRowsThreads = 160;

template <int HD>
struct RowsCfg {
  using Walk = PagedWalk<kRowsUnit, true, kRowsKeys, kRowsCost>;
  static constexpr int kStage = 2 * kRowsKeys * HD * 2;                   // K then V, panels of 64 dims
  static constexpr int kStages = HD == 64 ? 4 : 3;
  static constexpr int kCtas = HD == 64 ? 3 : HD == 128 ? 2 : 1;          // an SM holds
  static constexpr int kMerge = 2 * kRowsUnit * HD * 4;
  static constexpr int kSmem = kStages * kStage + kMerge + 4 * kRowsUnit * 8 + 16 * kStages + 16 + 2 * sizeof(PagedWarp<Walk>);
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

template <int HD, bool BF16>
__global__ void __launch_bounds__(kRowsThreads, RowsCfg<HD>::kCtas)
    fm_paged_rows_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = RowsCfg<HD>;
  constexpr int kP = HD / 64;                     // panels of 64 dims
  constexpr int kPanel = kRowsKeys * 128;         // bytes
  extern __shared__ __align__(1024) uint8_t gbase[];
  const uint32_t base = smem_u32(gbase);
  float *merge = reinterpret_cast<float *>(gbase + C::kStages * C::kStage);           // [2][16][HD]
  float2 *ml = reinterpret_cast<float2 *>(merge + 2 * kRowsUnit * HD);                // [4][16]
  const uint32_t bars = smem_u32(ml + 4 * kRowsUnit);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (C::kStages + s); };
  // (the plan's, read before the first stage is there; the sums' memory afterwards)
  long long *sh = reinterpret_cast<long long *>(ml);                                         // [8]
  PagedStart *start = reinterpret_cast<PagedStart *>(sh + 8);
  int *poison = reinterpret_cast<int *>(gbase + (bars - base) + 16 * C::kStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PagedWarp<typename C::Walk> &w = reinterpret_cast<PagedWarp<typename C::Walk> *>(poison + 4)[warp < 4 ? 0 : 1];   // (one for the four)
  const PagedBatch &b = a.b;

  pdl_trigger();
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.tk)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&a.tv)) : "memory");
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4);
    }
    mbar_fence_init();
    *poison = 0;
  }
  pdl_wait();
  paged_plan<kRowsUnit, true, kRowsKeys, kRowsCost, kRowsLeast, kRowsThreads>(a, sh, start);
  if (warp == 0 || warp == 4) w.init(*start, b, lane);

  if (warp == 4) {
    // ---- fetch: a lane a (page box, panel) ----
    const int box_log = min(b.page_log, 6), boxes = kRowsKeys >> box_log;
    const int box = lane & (boxes - 1), panel = lane / boxes;
    const bool mine = panel < kP;
    uint32_t c = 0;                               // stages asked for
    bool ok = true;
    while (ok && w.next(a, lane)) {
      const PagedSeg &g = w.seg();
      auto row_of = [&](int i) { return mine ? paged_row(a, g.s, g.seq, g.head, g.s.tile(i) * kRowsKeys + (box << box_log)) : 0; };
      int row = row_of(g.begin), next = g.begin + 1 < g.end ? row_of(g.begin + 1) : 0;
      for (int i = g.begin; i < g.end; ++i) {
        const int ahead = i + 2 < g.end ? row_of(i + 2) : 0;   // (the table is asked two stages ahead)
        const int s = c % C::kStages;
        ok = paged_wait_warp(empty(s), ((c / C::kStages) & 1) ^ 1, a.b.err);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(full(s), C::kStage);
        __syncwarp();
        if (mine) {
          const uint32_t dst = base + s * C::kStage + panel * kPanel + (box << box_log) * 128;
          tma_2d_row(dst, &a.tk, panel * 64, row, full(s));
          tma_2d_row(dst + kP * kPanel, &a.tv, panel * 64, row, full(s));
        }
        ++c;
        row = next, next = ahead;
      }
    }
    // the CTA leaves only after its copies have landed
    for (uint32_t u = c > (uint32_t)C::kStages ? c - C::kStages : 0; u < c; ++u)
      mbar_wait_drain(full(u % C::kStages), (u / C::kStages) & 1);
    return;
  }

  // ---- compute: warp w takes keys 16 w .. 16 w + 15 of each stage; lane: rows g8 and g8 + 8 of the products ----
  const int g8 = lane >> 2, c4 = lane & 3;
  const float thr = 8.f / a.scale_log2;           // a reference moves where a score beats it by 2^8
  // ldmatrix addresses inside a panel: row and 16-byte unit, permuted by the row
  const int krow = 16 * warp + (lane & 7) + (lane >> 4) * 8, kun = (lane >> 3) & 1;     // K: keys by halves, dims by units
  const int vrow = 16 * warp + (lane & 15), vun = lane >> 4;                            // V transposed
  uint32_t c = 0;
  bool ok = true;
  if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  for (;;) {
    if (threadIdx.x == 0) w.step(a);
    named_sync(1, 128);
    if (!w.more) break;
    const PagedSeg &g = w.seg();
    const int r0 = g.tile * kRowsUnit, rows = min(kRowsUnit, g.q.n_new * b.group - r0);
    const int pos0 = g.q.len - g.q.n_new;
    int tok[2];
    uint32_t qf[HD / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + min(g8 + 8 * h, rows - 1);     // (rows past the unit's repeat its last, and are not stored)
      tok[h] = r / b.group;
      const uint16_t *src = static_cast<const uint16_t *>(a.q.p) + (int64_t)(g.q.s0 + tok[h]) * a.q.ld +
                            (int64_t)(g.head * b.group + r - tok[h] * b.group) * a.q.hs + 2 * c4;
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        qf[k][h] = __ldcg(reinterpret_cast<const unsigned int *>(src + 16 * k));
        qf[k][2 + h] = __ldcg(reinterpret_cast<const unsigned int *>(src + 16 * k + 8));
      }
    }
    float o[HD / 8][4];
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int i = g.begin; i < g.end; ++i, ++c) {
      const int st = c % C::kStages, key0 = g.s.tile(i) * kRowsKeys;
      const bool masked = paged_masked<kRowsKeys>(a, g.s, key0);
      if (ok) ok = paged_wait_warp(full(st), (c / C::kStages) & 1, a.b.err);
      const uint32_t kt = base + st * C::kStage, vt = kt + kP * kPanel;
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < HD / 16; ++k) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kt + (k >> 2) * kPanel + krow * 128 + ((((k & 3) * 2 + kun) ^ (krow & 7)) << 4), b0, b1, b2, b3);
        mma16<BF16>(s[0], qf[k], b0, b1);
        mma16<BF16>(s[1], qf[k], b2, b3);
      }
      if (masked) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!paged_sees(a, g.q, pos0 + tok[e >> 1], key0 + 16 * warp + 8 * n + 2 * c4 + (e & 1))) s[n][e] = -INFINITY;
        // infinities and NaN of this warp's rows of V: out of the tile (a weight of 0 times one would be NaN)
        for (int u = lane; u < 16 * HD / 8; u += 32) {
          const uint32_t at = vt + (u / 128) * kPanel + 16 * warp * 128 + (u % 128) * 16;
          const uint4 x = lds128(at);
          const uint4 n = make_uint4(not_finite<BF16>(x.x), not_finite<BF16>(x.y), not_finite<BF16>(x.z), not_finite<BF16>(x.w));
          if (n.x | n.y | n.z | n.w) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(x.x & ~n.x), "r"(x.y & ~n.y),
                         "r"(x.z & ~n.z), "r"(x.w & ~n.w)
                         : "memory");
            fence_proxy_async();   // (the stage's next copy comes after this store)
            if (paged_seen(a, g.s, key0 + 16 * warp + (u % 128) / 8)) *poison = 1;   // (read at the unit's end)
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool move = top > m[h] + thr;       // (m = -inf: with the first score)
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? ex2((m[h] - top) * a.scale_log2) : 1.f;
          if (move) m[h] = top;
          l[h] *= f;
#pragma unroll
          for (int d = 0; d < HD / 8; ++d) {
            o[d][2 * h] *= f;
            o[d][2 * h + 1] *= f;
          }
        }
        float off = m[h] == -INFINITY ? 0.f : m[h] * a.scale_log2, first = 0.f;
        if (fabsf(off) > kFarReference) first = m[h], off = 0.f;   // (taken off the score itself)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float &p = s[n][2 * h + e];
            p = ex2(fmaf(p - first, a.scale_log2, -off));
            l[h] += p;
          }
      }
      const uint32_t pf[4] = {pack2<BF16>(s[0][0], s[0][1]), pack2<BF16>(s[0][2], s[0][3]), pack2<BF16>(s[1][0], s[1][1]),
                              pack2<BF16>(s[1][2], s[1][3])};
#pragma unroll
      for (int d = 0; d < HD / 16; ++d) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_trans(vt + (d >> 2) * kPanel + vrow * 128 + ((((d & 3) * 2 + vun) ^ (vrow & 7)) << 4), b0, b1, b2, b3);
        mma16<BF16>(o[2 * d], pf, b0, b1);
        mma16<BF16>(o[2 * d + 1], pf, b2, b3);
      }
      // The stage is given back once every lane's reads of it are done: without the fence the last V fragments can still be
      // on their way when the next copy lands in their place (costs nothing that shows: 106 us for a token of 32 sequences).
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
    }
    // ---- the four warps' sums ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (c4 == 0) ml[warp * kRowsUnit + g8 + 8 * h] = make_float2(m[h], l[h]);
    }
    named_sync(1, 128);
    const bool any_bad = *reinterpret_cast<volatile int *>(poison) != 0;
    float top[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) t = fmaxf(t, ml[w * kRowsUnit + g8 + 8 * h].x);
      top[h] = t;
      const float f = m[h] == -INFINITY ? 0.f : ex2((m[h] - t) * a.scale_log2);
#pragma unroll
      for (int d = 0; d < HD / 8; ++d) {
        o[d][2 * h] *= f;
        o[d][2 * h + 1] *= f;
      }
    }
    auto cell = [&](int w, int row, int d) { return merge + (w * kRowsUnit + row) * HD + (d ^ ((row & 7) << 3)); };
    if (warp >= 2)
#pragma unroll
      for (int d = 0; d < HD / 8; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2 *>(cell(warp - 2, g8 + 8 * h, 8 * d + 2 * c4)) = make_float2(o[d][2 * h], o[d][2 * h + 1]);
    named_sync(1, 128);
    if (warp < 2)
#pragma unroll
      for (int d = 0; d < HD / 8; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float2 *x = reinterpret_cast<float2 *>(cell(warp, g8 + 8 * h, 8 * d + 2 * c4));
          *x = make_float2(x->x + o[d][2 * h], x->y + o[d][2 * h + 1]);
        }
    named_sync(1, 128);
    const bool whole = g.whole();
    const size_t slot = 2 * (size_t)blockIdx.x + (g.begin == 0 ? 1 : 0);
    if (threadIdx.x == 0 && !whole && g.begin == 0) a.desc[blockIdx.x] = make_int4(g.seq, g.head, g.tile, w.walk.parts(g));
    for (int u = threadIdx.x; u < kRowsUnit * HD / 8; u += 128) {
      const int row = u / (HD / 8), d = (u % (HD / 8)) * 8;
      if (row >= rows) break;
      const int r = r0 + row, t = r / b.group;
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mt = fmaxf(mt, ml[w * kRowsUnit + row].x);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 x = ml[w * kRowsUnit + row];
        lt += x.y == 0.f ? 0.f : ex2((x.x - mt) * a.scale_log2) * x.y;   // (scores that are all NaN: a sum of NaN)
      }
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 x = *reinterpret_cast<const float4 *>(cell(0, row, d) + e);
        const float4 y = *reinterpret_cast<const float4 *>(cell(1, row, d) + e);
        v[e] = x.x + y.x;
        v[e + 1] = x.y + y.y;
        v[e + 2] = x.z + y.z;
        v[e + 3] = x.w + y.w;
      }
      if (any_bad) {
        const PagedSeg held = g;
        float more[8] = {};
        paged_poison<kRowsKeys, BF16, 8>(a, held, HD, pos0 + t, d, more);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += more[e];
      }
      if (whole) {
        const float inv = paged_inv(a, g.q, pos0 + t, lt);
        uint16_t *out = static_cast<uint16_t *>(a.out.p) + (int64_t)(g.q.s0 + t) * a.out.ld +
                        (int64_t)(g.head * b.group + r - t * b.group) * a.out.hs + d;
        *reinterpret_cast<uint4 *>(out) =
            make_uint4(pack2<BF16>(v[0] * inv, v[1] * inv), pack2<BF16>(v[2] * inv, v[3] * inv),
                       pack2<BF16>(v[4] * inv, v[5] * inv), pack2<BF16>(v[6] * inv, v[7] * inv));
      } else {
        *reinterpret_cast<float4 *>(paged_part<HD, kRowsUnit>(a, slot, row, d)) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(paged_part<HD, kRowsUnit>(a, slot, row, d + 4)) = make_float4(v[4], v[5], v[6], v[7]);
        if (d == 0) a.part_ml[slot * kRowsUnit + row] = make_float2(mt == -INFINITY ? mt : mt * a.scale_log2, lt);
      }
    }
    named_sync(1, 128);   // (the sums' memory is free)
    if (any_bad) {
      if (threadIdx.x == 0) *poison = 0;
      named_sync(1, 128);
    }
  }
}

}  // namespace fm
