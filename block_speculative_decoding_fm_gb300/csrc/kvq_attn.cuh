// kvq_attn.cuh -- attention over the 4-bit KV cache, and the attention weight
// that each cache row collects.
//
//   O[r] = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp2(t_rj - m_r),
//   t_rj = scale log2(e) q_r . k_j  over the rows j that r sees,
// one pass over the cache with a running reference m and sum.  A unit is a
// (sequence, KV head, 8 nq query rows), its keys stages of 128 rows (64 for head
// dim 256).  Either a unit has CTAs of its own, or the units lie end to end and every CTA
// takes an equal share of them (kvq.cu chooses); a second, short launch joins the parts of
// units that several CTAs share, in their order.
//
// A CTA's warps work in groups of four with a ring of stages of their own (K and V codes and scales in one bulk
// copy).  A warp forms the scores of a quarter of the stage's keys, S^T = K Q^T, and puts its P into
// shared memory; then each warp takes a quarter of the dims over all the stage's keys, O^T += V^T P^T, so
// that it holds 8 accumulators a query octet for head dim 128 (64, were the output split by keys), many warps fit an
// SM, and a unit's end needs no exchange inside a group.  The group shares one reference a row; it moves
// only when a score beats it by 2^8, and the barrier that hands P over tells everyone whether one did.
//
// One query row is bound by memory: 524288 rows of 8 KV heads of 128 in 105 us, 5.8 TB/s (0.85 of a plain copy), 24 heads
// over 4 of 256 in 112 us, 5.4 TB/s.  Sixteen are bound by the chain of a warp's steps (codes unpacked, product, exponential,
// barrier, product), each waiting for the one before, with 16 warps an SM to fill the waits: the tensor pipe is 38 to 39 % busy
// and the issue slots 47 to 49 %.  bf16 147 us (4.1 TB/s), f16 160 us, f32 246 us, whose queries and probabilities are two
// operands each.  Short caches are a chain of waits between CTAs: of 26 us over 32769 rows of 16 heads, 18 are the stream, 2 the
// queries, 1 the output, 3 the join.
//
// With at most 32 query rows the product is a skinny one, and the codes pass from shared memory (ldmatrix)
// through a few integer operations straight into mma.sync fragments: they never go back to shared
// memory as f16, which a tcgen05 operand would need (64 KB written and read again per 128 rows of
// head dim 128: 1024 cycles of shared memory against the 784 cycles in which an SM's share of HBM
// delivers their 18 KB).  (A first operand in TMEM, which the scores could have, has not been tried.)
#include <atomic>
#include <type_traits>

#include "kvq_dev.cuh"

namespace fm {
namespace {

using namespace kvq;

constexpr float kLazy = 8.f;               // log2 of the growth a reference tolerates
constexpr int kWThreads = 128;             // the weights pass
// its pairs of tiles in shared memory: about 37 KB, with which an SM holds the four CTAs that the pass is dealt out for (more
// at once share unevenly: 16 rows over 32768 of 128 dims 48 us with two or three pairs, 41 with four; 256 dims 36 us with
// two, 38 with four)
__host__ __device__ constexpr int w_slots(int hd) { return 512 / hd; }

constexpr int imin(int a, int b) { return a < b ? a : b; }
constexpr int imax(int a, int b) { return a > b ? a : b; }

// The attention kernel's shape: CTAs an SM, groups of four warps a CTA, P once or twice.  Two CTAs an SM where two groups
// each fit them (one's ends of units pass under the other's work), else one CTA with as many groups as fit, four at
// most; fewer where many query rows want more registers than 128 a thread.
template <int HD, typename T, int NQ>
struct Shape : Kind<HD, T, NQ> {
  using K = Kind<HD, T, NQ>;
  using QT = QTile<HD, K::QS, NQ>;
  using PT = PTile<NQ, K::PS, K::KS>;
  static constexpr int KT = kvq_stage_tiles(HD), SB = KT * kvq_tile_bytes(HD);
  static constexpr int GP = K::G < 4 ? 1 : K::G / 4;      // groups of dims a warp takes
  static constexpr int KP = K::G < 4 ? 4 / K::G : 1;      // ways the keys are split in the second product
  static constexpr int NS = HD == 64 ? 3 : 2;
  static constexpr int kJoin = HD * K::RT * 4;            // one output, when a CTA's are joined
  static constexpr int p_bytes(int ng, int db) { return imax((1 + db) * PT::kBytes, ((ng * KP - 1) * kJoin / ng + 127) / 128 * 128); }
  static constexpr int kMore = 4 * K::RT * 4 * 2 + K::RT * 4 + 32 + 2 * NS * 8;   // maxima, sums, references, cursor, barriers
  static constexpr int bytes(int ng, int db) { return ng * (NS * SB + p_bytes(ng, db) + kMore) + QT::kBytes; }
  static constexpr int kRoom1 = 226 * 1024, kRoom2 = 112 * 1024 + 512;
  static constexpr int kMost = NQ <= 2 ? 4 : HD == 256 && NQ == 4 ? 2 : 3;        // groups an SM, by registers
  static constexpr bool kTwo = kMost == 4 && bytes(2, 0) <= kRoom2;
  static constexpr int fits(int ng) { return ng == 1 || bytes(ng, 0) <= kRoom1 ? ng : fits(ng - 1); }
  static constexpr int MB = kTwo ? 2 : 1, NG = kTwo ? 2 : fits(kMost);
  static constexpr int DB = bytes(NG, 1) <= (kTwo ? kRoom2 : kRoom1) ? 1 : 0;
  static constexpr int kP = p_bytes(NG, DB), kBytes = bytes(NG, DB), kThreads = 128 * NG;
  static_assert(kBytes <= kRoom1, "a group fits an SM");
};

template <typename T>
__device__ __forceinline__ void store4(T *p, float4 v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(p) = v;
  } else {
    uint2 w;
    if constexpr (std::is_same<T, __half>::value) {
      const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
      w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
      w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    *reinterpret_cast<uint2 *>(p) = w;
  }
}

// A CTA's share of the places: [w_beg, w_end)
__device__ __forceinline__ void share_of(const KvqAttnArgs &a, int b, int &w_beg, int &w_end) {
  if (a.share) {
    w_beg = b * a.share + min(b, a.extra);
    w_end = w_beg + a.share + (b < a.extra);
  } else {
    const int i = find_seq<int32_t>(a.cta0, a.n, b), n = a.parts[i], S = a.stages[i];
    const int unit = (b - a.cta0[i]) / n, p = b - a.cta0[i] - unit * n;
    const int u0 = a.st0[i] + unit * (S + kKvqUnitCost) + kKvqUnitCost;   // the unit's first stage
    const int q = S / n, r = S - q * n;
    w_beg = u0 + p * q + min(p, r);
    w_end = w_beg + q + (p < r);
  }
}
// the CTA with a place, shares equal
__device__ __forceinline__ int cta_of(const KvqAttnArgs &a, int stage) {
  const int wide = a.extra * (a.share + 1);
  return stage < wide ? stage / (a.share + 1) : a.extra + (stage - wide) / a.share;
}

// A stretch of a share: stages [s0, s0 + n) of one unit, `places` places long (n is 0 where they end before its stages).
struct Stretch {
  int i, head, rt, s0, n, places, u0;   // u0: the place of the unit's first stage
  __device__ __forceinline__ Stretch(const KvqAttnArgs &a, int at, int end) {
    i = find_seq<int32_t>(a.st0, a.n, at);
    const int rel = at - a.st0[i], V = a.stages[i] + kKvqUnitCost, unit = rel / V, r0 = rel - unit * V;
    places = min(V - r0, end - at);
    s0 = max(0, r0 - kKvqUnitCost);
    n = max(0, r0 + places - kKvqUnitCost) - s0;
    u0 = at - r0 + kKvqUnitCost;
    const int rts = (a.rows[i] * a.group + 8 * a.nq - 1) / (8 * a.nq);
    head = unit / rts;
    rt = unit - head * rts;
  }
};

// Where a group's copies have got to (in shared memory: one lane's business, once a stage).
struct Cursor {
  const uint8_t *src;     // the next stage
  int32_t at;             // the share's place after the stretch that the cursor is in
  int32_t left;           // stages of the stretch that are the group's
  int32_t issued;
};
static_assert(sizeof(Cursor) <= 32, "a cursor's place in shared memory");

// the group's next stage, from where its stretch is used up; false where there is none
template <int HD, typename Sh>
__device__ __forceinline__ bool find_stage(const KvqAttnArgs &a, Cursor *cu, int w_end, int grp) {
  while (cu->left == 0) {
    const int at = cu->at;
    if (at >= w_end) return false;
    const Stretch x(a, at, w_end);
    // (a unit that sees no rows has one stage, whatever is there: every score of it is masked)
    const int t = min((a.first / (kKvqTile * Sh::KT) + x.s0 + grp) * Sh::KT, a.c.rows_pad / kKvqTile - Sh::KT);
    cu->left = (x.n - grp + Sh::NG - 1) / Sh::NG;
    cu->src = a.c.planes + ((size_t)a.seq[x.i] * a.c.n_kv + x.head) * a.c.plane_bytes + (size_t)t * kvq_tile_bytes(HD);
    cu->at = at + x.places;
  }
  return true;
}
// The next of the group's stages into its ring; false where a wait gave up.
template <int HD, typename Sh>
__device__ __forceinline__ bool issue_stage(const KvqAttnArgs &a, Cursor *cu, int w_end, int grp, uint32_t ring,
                                            uint32_t full, uint32_t empty) {
  if (!find_stage<HD, Sh>(a, cu, w_end, grp)) return true;
  const uint8_t *src = cu->src;
  const int left = cu->left;
  const int g = cu->issued, slot = g % Sh::NS;
  if (g >= Sh::NS && !mbar_wait_bounded(empty + slot * 8, (g / Sh::NS - 1) & 1, a.c.err)) return false;
  mbar_expect_tx(full + slot * 8, Sh::SB);
  bulk_g2s(ring + slot * Sh::SB, src, Sh::SB, full + slot * 8);   // (whole stages: planes are padded to them)
  cu->left = left - 1;
  cu->src = src + Sh::NG * Sh::SB;
  cu->issued = g + 1;
  return true;
}

template <int HD, typename T, int NQ, bool W>
__global__ void __launch_bounds__(Shape<HD, T, NQ>::kThreads, Shape<HD, T, NQ>::MB)
    kvq_attend_kernel(const __grid_constant__ KvqAttnArgs a) {
  using Sh = Shape<HD, T, NQ>;
  using QT = typename Sh::QT;
  using PT = typename Sh::PT;
  constexpr bool QS = Sh::QS, SV = Sh::SV, SK = QS || W;
  constexpr int PS = Sh::PS, DB = Sh::DB;
  constexpr int NG = Sh::NG, NS = Sh::NS, SB = Sh::SB, TB = kvq_tile_bytes(HD), RT = Sh::RT, KS = Sh::KS, MT = Sh::MT;
  constexpr int GP = Sh::GP, KP = Sh::KP, NT = Sh::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 s_row[RT];              // references and sums of the query rows, all groups
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, grp = NG == 1 ? 0 : w >> 2, wq = w & 3;
  const int g8 = lane >> 2, c = lane & 3;
  // rings first (128-byte aligned), then P tiles, the queries, and the rest
  const uint32_t ring = smem_u32(smem) + grp * NS * SB;
  uint8_t *ptile = smem + NG * NS * SB + grp * Sh::kP;
  uint8_t *qs = smem + NG * (NS * SB + Sh::kP);
  uint8_t *more = qs + QT::kBytes;
  uint64_t *bar = reinterpret_cast<uint64_t *>(more);                              // [group][full, empty][stage]
  Cursor *cu = reinterpret_cast<Cursor *>(more + NG * 2 * NS * 8) + grp;
  float *gm = reinterpret_cast<float *>(more + NG * (2 * NS * 8 + 32));            // [group][row] references
  float *wl = gm + NG * RT;                                                        // [group][warp][row] sums
  float *wx = wl + NG * 4 * RT + grp * 4 * RT;                                     // [group][warp][row] maxima
  const uint32_t full = smem_u32(bar + grp * 2 * NS), empty = full + NS * 8, qt = smem_u32(qs);
  int w_beg, w_end;
  share_of(a, blockIdx.x, w_beg, w_end);

  // what comes of the arguments alone is done before the wait
  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < NG * 2 * NS; ++s) mbar_init(smem_u32(bar + s), s / NS & 1 ? 4 : 1);
    mbar_fence_init();
  }
  const bool copies = lane == 0 && wq == 0;   // the lane that sends for its group's stages
  bool ok = true;
  if (copies) {
    cu->at = w_beg;
    cu->left = 0;
    cu->issued = 0;
    find_stage<HD, Sh>(a, cu, w_end, grp);
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();   // (after the wait: whoever starts behind this launch finds what came before it done)
  if (copies)
    for (int k = 0; k < NS - 1; ++k) ok = issue_stage<HD, Sh>(a, cu, w_end, grp, ring, full, empty);

  // first product: this warp's strip; second: its groups of dims gw, gw + 4 over the 32-row blocks kp, kp + KP, ...
  const int strip = wq * KS;
  const LaneAt<HD, KS> la(strip % kKvqTile, lane);
  const uint32_t kcode = ring + strip / kKvqTile * TB + la.code, kscale = ring + strip / kKvqTile * TB + la.scale;
  const int gw = KP == 1 ? wq : wq % Sh::G, kp = KP == 1 ? 0 : wq / Sh::G;
  const uint32_t vcode = ring + kvq_k_bytes(HD) + kvq_unit(lane, 0, HD);
  const uint32_t vscale = ring + kvq_k_bytes(HD) + kvq_vscale(2 * c, gw, HD);
  int slot = 0, buf = 0;
  uint32_t par = 0;
  for (int at = w_beg; at < w_end;) {
    const Stretch x(a, at, w_end);
    at += x.places;
    if (x.n == 0) continue;
    const int len = a.len[x.i], T_rows = a.rows[x.i], R = T_rows * a.group, rq = x.rt * RT;
    load_q<HD, QS, SK, NQ, NT>(static_cast<const T *>(a.q) + a.row0[x.i] * a.ldq + (int64_t)x.head * a.group * HD, a.ldq, a.group,
                           rq, R, a.scale_log2, qs, tid);
    __syncthreads();
    const int lim_all = a.causal ? len - T_rows + rq / a.group + 1 : len;   // the rows that every query row sees end here

    float o[GP][2][NQ][4], cor[GP][NQ][4], m[NQ][2];
    int shift = 15;                          // of this warp's V scales
#pragma unroll
    for (int u = 0; u < GP; ++u)
#pragma unroll
      for (int n = 0; n < NQ; ++n) cor[u][n][0] = cor[u][n][1] = cor[u][n][2] = cor[u][n][3] = 0.f;
    uint64_t l[NQ];                          // row sums of this warp's strips
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n] = 0ull;
#pragma unroll
      for (int u = 0; u < GP; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) o[u][t][n][0] = o[u][t][n][1] = o[u][t][n][2] = o[u][t][n][3] = 0.f;
    }
    int tile0 = (a.first / (kKvqTile * Sh::KT) + x.s0 + grp) * Sh::KT;
    for (int k = grp; k < x.n; k += NG, tile0 += NG * Sh::KT) {
      // a stage ahead of the ring's end; then this one (a wait that gave up ends the group's work, not its barriers)
      if (copies && ok) ok = issue_stage<HD, Sh>(a, cu, w_end, grp, ring, full, empty);
      ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(full + slot * 8, par, a.c.err));
      const int key0 = tile0 * kKvqTile + strip;
      const uint32_t pt = smem_u32(ptile) + buf * PT::kBytes;
      float s[MT][NQ][4];
      uint64_t sp[MT][NQ][2];
      strip_scores<HD, QS, SK, NQ, KS>(kcode + slot * SB, kscale + slot * SB, qt, lane, sp);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          unpack2(sp[i][n][0], s[i][n][0], s[i][n][1]);
          unpack2(sp[i][n][1], s[i][n][2], s[i][n][3]);
        }
      if (key0 < a.first || key0 + KS > lim_all) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // (rows past R follow the last: they are not stored)
            const int row = min(rq + 8 * n + 2 * c + h, R - 1);
            const int lim = a.causal ? len - T_rows + row / a.group + 1 : len;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = key0 + 16 * i + 8 * e + g8;
                if (key < a.first || key >= lim) s[i][n][2 * e + h] = -INFINITY;
              }
          }
      }
      // P with the references as they are; who beats one by 2^8 says so at the barrier
      float p[MT][NQ][4];
      uint64_t add[NQ];
      bool beat = false;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float2 mu = *reinterpret_cast<const float2 *>(qs + QT::kMult + (8 * n + 2 * c) * 4);
        const float b0 = kBias - (m[n][0] == -INFINITY ? 0.f : m[n][0]), b1 = kBias - (m[n][1] == -INFINITY ? 0.f : m[n][1]);
        const uint64_t mm = pack2(mu.x, mu.y), bb = pack2(b0, b1);
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t0, t1;
            x0 = fmaxf(x0, s[i][n][2 * e]);
            x1 = fmaxf(x1, s[i][n][2 * e + 1]);
            unpack2(fma2(pack2(s[i][n][2 * e], s[i][n][2 * e + 1]), mm, bb), t0, t1);
            p[i][n][2 * e] = ex2(t0);
            p[i][n][2 * e + 1] = ex2(t1);
            const uint64_t pp = pack2(p[i][n][2 * e], p[i][n][2 * e + 1]);
            add[n] = i + e ? add2(add[n], pp) : pp;
          }
        beat |= x0 * mu.x > m[n][0] + kLazy || x1 * mu.y > m[n][1] + kLazy;
      }
      if (!DB) named_sync(1 + grp, 128);   // the last stage's P has been used
      put_p<NQ, PS, KS>(pt, strip, lane, p);
      if (bar_any(1 + grp, 128, beat)) {
        // the group's new references, what it holds brought to them, and P again
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const float2 mu = *reinterpret_cast<const float2 *>(qs + QT::kMult + (8 * n + 2 * c) * 4);
          float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) x0 = fmaxf(x0, s[i][n][2 * e]), x1 = fmaxf(x1, s[i][n][2 * e + 1]);
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, sh));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, sh));
          }
          if (g8 == 0) *reinterpret_cast<float2 *>(wx + wq * RT + 8 * n + 2 * c) = make_float2(x0 * mu.x, x1 * mu.y);
        }
        named_sync(1 + grp, 128);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float n0 = m[n][0], n1 = m[n][1];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float2 y = *reinterpret_cast<const float2 *>(wx + v * RT + 8 * n + 2 * c);
            n0 = fmaxf(n0, y.x), n1 = fmaxf(n1, y.y);
          }
          const float f0 = n0 == m[n][0] ? 1.f : ex2(m[n][0] - n0), f1 = n1 == m[n][1] ? 1.f : ex2(m[n][1] - n1);
          m[n][0] = n0, m[n][1] = n1;
          l[n] = mul2(l[n], pack2(f0, f1));
#pragma unroll
          for (int u = 0; u < GP; ++u)
#pragma unroll
            for (int t = 0; t < 2; ++t) o[u][t][n][0] *= f0, o[u][t][n][1] *= f1, o[u][t][n][2] *= f0, o[u][t][n][3] *= f1;
          if constexpr (!SV) {   // (by query row lane / 4: the factor of column lane / 4)
            const float e0 = __shfl_sync(0xffffffffu, f0, (lane & ~3) | (g8 >> 1)), e1 = __shfl_sync(0xffffffffu, f1, (lane & ~3) | (g8 >> 1));
            const float f = g8 & 1 ? e1 : e0;
#pragma unroll
            for (int u = 0; u < GP; ++u) cor[u][n][0] *= f, cor[u][n][1] *= f, cor[u][n][2] *= f, cor[u][n][3] *= f;
          }
          const float2 mu = *reinterpret_cast<const float2 *>(qs + QT::kMult + (8 * n + 2 * c) * 4);
          const float b0 = kBias - (n0 == -INFINITY ? 0.f : n0), b1 = kBias - (n1 == -INFINITY ? 0.f : n1);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              p[i][n][2 * e] = ex2(fmaf(s[i][n][2 * e], mu.x, b0));
              p[i][n][2 * e + 1] = ex2(fmaf(s[i][n][2 * e + 1], mu.y, b1));
              const uint64_t pp = pack2(p[i][n][2 * e], p[i][n][2 * e + 1]);
              add[n] = i + e ? add2(add[n], pp) : pp;
            }
        }
        put_p<NQ, PS, KS>(pt, strip, lane, p);
        named_sync(1 + grp, 128);
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) l[n] = add2(l[n], add[n]);
      {
        // the warp's blocks of 32 rows (KP > 1: every KP-th) and their scales
        constexpr int NB = 2 * Sh::KT / KP;
        uint32_t sc[NB][GP][4];
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
          for (int u = 0; u < GP; ++u) {
            const int key = 32 * (kb * KP + kp);
            const uint4 v = lds128(vscale + slot * SB + key / kKvqTile * TB + 4 * u * 128 + key % kKvqTile / 2);
            sc[kb][u][0] = v.x, sc[kb][u][1] = v.y, sc[kb][u][2] = v.z, sc[kb][u][3] = v.w;
          }
        // Rows outside the view -- behind the end they are whatever the slot held before -- count with a scale of 0.
        if (tile0 * kKvqTile < a.first || (tile0 + Sh::KT) * kKvqTile > len) {
#pragma unroll
          for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = tile0 * kKvqTile + 32 * (kb * KP + kp) + 8 * j + 2 * c;   // (the word's low half; its high half: row + 1)
              const uint32_t keep = (row >= a.first && row < len ? 0xffffu : 0u) | (row + 1 >= a.first && row + 1 < len ? 0xffff0000u : 0u);
#pragma unroll
              for (int u = 0; u < GP; ++u) sc[kb][u][j] &= keep;
            }
        }
        // does one ask for a lower shift?  (1 to 3 % of the time; looked for ahead of P's barrier, in scales fetched
        // twice, 9 %)
        __half2 top2 = __habs2(h2(sc[0][0][0]));
#pragma unroll
        for (int kb = 0; kb < NB; ++kb)
#pragma unroll
          for (int u = 0; u < GP; ++u)
#pragma unroll
            for (int j = kb + u == 0; j < 4; ++j) top2 = __hmax2(top2, __habs2(h2(sc[kb][u][j])));
        uint32_t top = max(u32(top2) & 0xffffu, u32(top2) >> 16);
        if (__any_sync(0xffffffffu, top >= shift_limit(shift))) {
          top = __reduce_max_sync(0xffffffffu, top);
          const int to = shift_for(top);
          const float f = pow2f(to - shift);
          shift = to;
#pragma unroll
          for (int u = 0; u < GP; ++u)
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[u][0][n][e] *= f, o[u][1][n][e] *= f;
                if constexpr (!SV) cor[u][n][e] *= f;
              }
            }
        }
        if (shift != 0) {
          const __half2 up = shift_factor(shift > 0 ? shift : shift - shift / 2);
#pragma unroll
          for (int kb = 0; kb < NB; ++kb)
#pragma unroll
            for (int u = 0; u < GP; ++u)
#pragma unroll
              for (int j = 0; j < 4; ++j) sc[kb][u][j] = u32(__hmul2(h2(sc[kb][u][j]), up));
        }
        auto pv = [&](auto low, __half2 by) {
#pragma unroll
          for (int kb = 0; kb < NB; ++kb) {
            const int key = 32 * (kb * KP + kp);
#pragma unroll
            for (int u = 0; u < GP; ++u)
              tile_pv<HD, PS, SV, decltype(low)::value, NQ, KS>(vcode + slot * SB + key / kKvqTile * TB + key % kKvqTile * (HD / 2),
                                                                gw + 4 * u, sc[kb][u], by, pt, key, lane, o[u], cor[u]);
          }
        };
        if (shift >= 0)
          pv(std::false_type(), h2(0));
        else
          pv(std::true_type(), shift_factor(shift / 2));
      }
      // The stage is given back once every lane's reads of it are done: an arrival does not wait for a lane's last loads, and
      // the next copy lands in their place (nothing that shows: 102 us for 16 rows of 32 sequences over 512-8,192 of 16 x 128,
      // 21.0 for a token of 32 sequences of 24/4 x 256; without it 102.7 and 21.9 had been measured).
      __threadfence_block();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + slot * 8);
      if (++slot == NS) slot = 0, par ^= 1;
      buf ^= DB;
    }

    // the groups' references and the warps' sums, then the outputs
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float l0, l1;
      unpack2(l[n], l0, l1);
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
        l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
      }
      if (g8 == 0) {
        *reinterpret_cast<float2 *>(wl + (grp * 4 + wq) * RT + 8 * n + 2 * c) = make_float2(l0, l1);
        if (wq == 0) *reinterpret_cast<float2 *>(gm + grp * RT + 8 * n + 2 * c) = make_float2(m[n][0], m[n][1]);
      }
    }
    __syncthreads();
    if (tid < RT) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int u = 0; u < NG; ++u) M = fmaxf(M, gm[u * RT + tid]);
#pragma unroll
      for (int u = 0; u < NG; ++u) {
        const float *y = wl + u * 4 * RT + tid;
        const float mu = gm[u * RT + tid];
        L += (mu == M ? 1.f : ex2(mu - M)) * ((y[0] + y[RT]) + (y[2 * RT] + y[3 * RT]));
      }
      s_row[tid] = make_float2(M, L);
    }
    __syncthreads();
    const float undo = pow2f(-shift);
    // in the values' own unit and with the rows' common references; every part but the first group's into shared memory
    float *ob = reinterpret_cast<float *>(smem + NG * NS * SB) + (size_t)((grp * KP + kp - 1) * Sh::G + (GP == 1 ? gw : wq * GP)) * (2 * NQ * 128) + lane * 4;
#pragma unroll
    for (int u = 0; u < GP; ++u)
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float M0 = s_row[8 * n + 2 * c].x, M1 = s_row[8 * n + 2 * c + 1].x;
        const float f0 = undo * (m[n][0] == M0 ? 1.f : ex2(m[n][0] - M0)), f1 = undo * (m[n][1] == M1 ? 1.f : ex2(m[n][1] - M1));
        float c0 = 0.f, c1 = 0.f;
        if constexpr (!SV) {
          const float all = 8.f * (cor[u][n][0] + cor[u][n][2]);   // of query row lane / 4
          c0 = __shfl_sync(0xffffffffu, all, 8 * c);
          c1 = __shfl_sync(0xffffffffu, all, 8 * c + 4);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float unit = SV ? 1.f : t ? 1.f / kUnitHi : 1.f / kUnitLo;
          float(&y)[4] = o[u][t][n];
          y[0] = fmaf(y[0], unit, -c0) * f0, y[1] = fmaf(y[1], unit, -c1) * f1;
          y[2] = fmaf(y[2], unit, -c0) * f0, y[3] = fmaf(y[3], unit, -c1) * f1;
          if (grp > 0 || kp > 0) *reinterpret_cast<float4 *>(ob + ((u * NQ + n) * 2 + t) * 128) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
    const bool whole = x.n == a.stages[x.i];
    float *lse = a.lse ? a.lse + ((size_t)(a.unit0[x.i] + x.rt) * a.c.n_kv + x.head) * RT : nullptr;
    const size_t slot_g = (size_t)blockIdx.x * 2 + (x.s0 == 0);   // a unit begun here, or one continued
    __syncthreads();
    if (grp == 0 && kp == 0) {
#pragma unroll
      for (int u = 0; u < GP; ++u)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int v = 1; v < NG * KP; ++v) {
            const float *y = reinterpret_cast<const float *>(smem + NG * NS * SB) +
                             (size_t)((v - 1) * Sh::G + (GP == 1 ? gw : wq * GP)) * (2 * NQ * 128) + lane * 4;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const float4 z = *reinterpret_cast<const float4 *>(y + ((u * NQ + n) * 2 + t) * 128);
              o[u][t][n][0] += z.x, o[u][t][n][1] += z.y, o[u][t][n][2] += z.z, o[u][t][n][3] += z.w;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // four dims of a query row: tiles' first rows, second rows
            const int r = 8 * n + 2 * c + h, qr = rq + r, d = 32 * (gw + 4 * u) + 4 * g8;
            const float4 y = make_float4(o[u][0][n][h], o[u][1][n][h], o[u][0][n][2 + h], o[u][1][n][2 + h]);
            if (!whole) {
              *reinterpret_cast<float4 *>(a.part_o + (slot_g * RT + r) * HD + d) = y;
            } else if (qr < R) {
              const float L = s_row[r].y, inv = L == 0.f ? 0.f : 1.f / L;
              const int t = qr / a.group;
              store4(static_cast<T *>(a.out) + (a.row0[x.i] + t) * a.ldo + ((int64_t)x.head * a.group + qr - t * a.group) * HD + d,
                     make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
            }
          }
        }
    }
    if (tid < RT) {
      const float M = s_row[tid].x, L = s_row[tid].y;
      if (!whole)
        a.part_ml[slot_g * RT + tid] = make_float2(M, L);
      else if (lse)
        lse[tid] = L == 0.f ? INFINITY : M + log2f(L) - kBias;
    }
    if (at < w_end) __syncthreads();   // the next stretch writes the queries, the references and the outputs' place
  }
  // nothing is left in flight when the CTA ends (a consumer may have given up)
  if (copies)
    for (int k = max(0, cu->issued - NS); k < cu->issued; ++k) mbar_wait_drain(full + k % NS * 8, (k / NS) & 1);
  __syncthreads();
}

// The parts of the units that several CTAs share into their output rows, in part order.  Many: the units are no more
// than the CTAs, and block x takes unit x; its four quarters take a quarter of the parts each, their loads in flight
// together (grid y: 64 float4 of a unit's outputs).  Else block x takes the boundary between CTAs x and x + 1, if it is
// the first one inside a unit: few parts, one after another (grid y: 256 float4).
constexpr int kJoinThreads = 256;
struct Joined {
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  // parts c0 .. c1 of which `first` is in its CTA's second slot; NB parts' loads in flight together
  template <int NB>
  __device__ __forceinline__ void add(const KvqAttnArgs &a, int RT, int HD, int r, int d, int c0, int c1, int first) {
    for (int c = c0; c <= c1; c += NB) {
      float2 ml[NB];
      float4 v[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int p = min(c + k, c1);
        const size_t slot = (size_t)p * 2 + (p == first);
        ml[k] = ldg64f(&a.part_ml[slot * RT + r]);
        v[k] = ldg128f(a.part_o + (slot * RT + r) * HD + d);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (c + k > c1) break;
        add_one(ml[k], v[k]);
      }
    }
  }
  __device__ __forceinline__ void add_one(float2 ml, float4 v) {
    const float m = fmaxf(M, ml.x), f = M == m ? 1.f : ex2(M - m), g = ml.x == m ? 1.f : ex2(ml.x - m);
    M = m;
    L = fmaf(L, f, g * ml.y);
    acc.x = fmaf(acc.x, f, g * v.x);
    acc.y = fmaf(acc.y, f, g * v.y);
    acc.z = fmaf(acc.z, f, g * v.z);
    acc.w = fmaf(acc.w, f, g * v.w);
  }
};
template <int HD, typename T, int NQ, bool Many>
__global__ void __launch_bounds__(kJoinThreads) kvq_join_kernel(const __grid_constant__ KvqAttnArgs a) {
  constexpr int RT = 8 * NQ, TX = Many ? 64 : kJoinThreads;
  pdl_trigger();
  int at, first, last;   // a place of the unit; the CTAs that have parts of it
  if (Many) {
    const int i = find_seq<int32_t>(a.unit0, a.n, (int)blockIdx.x / a.c.n_kv), unit = (int)blockIdx.x - a.unit0[i] * a.c.n_kv;
    at = a.st0[i] + unit * (a.stages[i] + kKvqUnitCost);
    if (!a.share) first = a.cta0[i] + unit * a.parts[i], last = first + a.parts[i] - 1;
  } else {
    at = (blockIdx.x + 1) * a.share + min((int)blockIdx.x + 1, a.extra);
  }
  const Stretch x(a, at, a.st0[a.n]);
  if (!Many || a.share) first = cta_of(a, x.u0), last = cta_of(a, x.u0 + a.stages[x.i] - 1);
  pdl_wait();   // every block, so that a later launch that waits for this one waits for what came before too
  if (first == last || (!Many && first != (int)blockIdx.x)) return;
  const int q = Many ? threadIdx.x >> 6 : 0, e = blockIdx.y * TX + threadIdx.x % TX;
  const int r = e / (HD / 4), d = 4 * (e % (HD / 4)), qr = x.rt * RT + r;
  const bool mine = r < RT && qr < a.rows[x.i] * a.group;
  Joined j;
  if (Many) {
    const int per = (last - first + 4) / 4, c0 = first + q * per;
    if (mine) j.add<8>(a, RT, HD, r, d, c0, min(last, c0 + per - 1), first);
    __shared__ float4 s_acc[4][64];
    __shared__ float2 s_ml[4][64];
    s_acc[q][threadIdx.x & 63] = j.acc;
    s_ml[q][threadIdx.x & 63] = make_float2(j.M, j.L);
    __syncthreads();
    if (q > 0 || !mine) return;
#pragma unroll
    for (int k = 1; k < 4; ++k) j.add_one(s_ml[k][threadIdx.x], s_acc[k][threadIdx.x]);
  } else {
    if (!mine) return;
    j.add<2>(a, RT, HD, r, d, first, last, first);
  }
  const float inv = j.L == 0.f ? 0.f : 1.f / j.L;
  const int t = qr / a.group;
  store4(static_cast<T *>(a.out) + (a.row0[x.i] + t) * a.ldo + ((int64_t)x.head * a.group + qr - t * a.group) * HD + d,
         make_float4(j.acc.x * inv, j.acc.y * inv, j.acc.z * inv, j.acc.w * inv));
  if (a.lse && d == 0)
    a.lse[((size_t)(a.unit0[x.i] + x.rt) * a.c.n_kv + x.head) * RT + r] = j.L == 0.f ? INFINITY : j.M + log2f(j.L) - kBias;
}

// weights[j] = decay weights[j] + sum_r p_rj / sum_j p_rj: with every row's sum
// known, K alone is read again (from L2 where it still is there) and the scores
// formed a second time, which needs no store of rows x keys.  One CTA owns a
// run of tiles, so nothing is added atomically.  Grid (sequence x run, KV head).
// Bound by unpacking the codes and by the exponentials (issue 55 %, tensor pipe 24 %): 524288 rows of 8 KV heads of 128,
// 16 query rows: 108 us, 2.8 TB/s; 32769 rows of 16: 13 us.
template <int HD, typename T, int NQ>
__global__ void __launch_bounds__(kWThreads) kvq_weights_kernel(const __grid_constant__ KvqAttnArgs a) {
  constexpr bool QS = sizeof(T) == 4;
  constexpr int KB = kvq_k_bytes(HD), RT = 8 * NQ, KS = 32;
  using QT = QTile<HD, QS, NQ>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *qs = smem + w_slots(HD) * 2 * KB;
  // a row's sum so far (a warp's own rows: lane 4 g + j has key 8 j + g of its strip of a pair of tiles)
  float *acc = reinterpret_cast<float *>(qs + QT::kBytes);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g8 = lane >> 2, c = lane & 3;
  const int i = find_seq<int32_t>(a.wt0, a.n, blockIdx.x), head = blockIdx.y;
  const int len = a.len[i], T_rows = a.rows[i], R = T_rows * a.group, rts = (R + RT - 1) / RT;
  const int t0 = (blockIdx.x - a.wt0[i]) * a.wtiles;
  const int nt = min(a.wtiles, (len + kKvqTile - 1) / kKvqTile - t0), np = (nt + 1) / 2;
  const size_t plane = (size_t)a.seq[i] * a.c.n_kv + head;
  pdl_trigger();
  const uint8_t *src = a.c.planes + plane * a.c.plane_bytes + (size_t)t0 * kvq_tile_bytes(HD);
  auto fetch = [&](int p) {   // the K halves of pair p
    if (p < np)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (2 * p + h < nt)
          for (int e = tid; e < KB / 16; e += kWThreads)
            cp_async16(smem_u32(smem) + (p % w_slots(HD) * 2 + h) * KB + e * 16, src + (size_t)(2 * p + h) * kvq_tile_bytes(HD) + e * 16, 16);
    cp_async_commit();
  };
  const LaneAt<HD, KS> la((w & 1) * 32, lane);
  auto key_of = [&](int p) { return (t0 + 2 * p + (w >> 1)) * kKvqTile + (w & 1) * 32 + 8 * c + g8; };
  float *ws = a.c.weights + plane * a.c.rows_pad;
  for (int p = 0; p < np; ++p) {   // (what the rows collected before is there too, like the rows: below)
    const int key = key_of(p);
    acc[p * kWThreads + tid] = a.decay != 0.f && 2 * p + (w >> 1) < nt && key < len ? a.decay * __uint_as_float(ldg32(ws + key)) : 0.f;
  }
  for (int rt = 0; rt < rts; ++rt) {
    if (rt) __syncthreads();
#pragma unroll
    for (int p = 0; p < w_slots(HD) - 1; ++p) fetch(p);
    load_q<HD, QS, true, NQ, kWThreads>(static_cast<const T *>(a.q) + a.row0[i] * a.ldq + (int64_t)head * a.group * HD, a.ldq,
                                  a.group, rt * RT, R, a.scale_log2, qs, tid);
    // The attention has begun everywhere before this launch begins, and lets nothing begin before what came ahead of it
    // is done: rows, weights and queries are there already, its sums are what is waited for.
    if (rt == 0) pdl_wait();
    const float *lse = a.lse + ((size_t)(a.unit0[i] + rt) * a.c.n_kv + head) * RT;
    float ls[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * n + 2 * c + h;
        ls[n][h] = rt * RT + r < R ? __uint_as_float(ldg32(lse + r)) : INFINITY;
      }
    __syncthreads();
    const int lim_all = a.causal ? len - T_rows + rt * RT / a.group + 1 : len;
    float mu[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) mu[n][h] = *reinterpret_cast<const float *>(qs + QT::kMult + (8 * n + 2 * c + h) * 4);
#pragma unroll 1
    for (int k = 0; k < np; ++k) {
      cp_async_wait<w_slots(HD) - 2>();
      __syncthreads();   // everyone's copies of this pair; everyone is done with the pair before it, whose place is next
      fetch(k + w_slots(HD) - 1);
      const int t = 2 * k + (w >> 1), key0 = (t0 + t) * kKvqTile + (w & 1) * 32;
      if (t >= nt || key0 >= len || key0 + 32 <= a.first) continue;
      const uint32_t kb = smem_u32(smem) + (k % w_slots(HD) * 2 + (w >> 1)) * KB;
      uint64_t sp[2][NQ][2];
      strip_scores<HD, QS, true, NQ, KS>(kb + la.code, kb + la.scale, smem_u32(qs), lane, sp);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};     // keys 8 j + lane / 4
      if (key0 >= a.first && key0 + 32 <= lim_all) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // (a row without keys, or past the last: the log of its sum is inf, p 0)
            float s0, s1;
            unpack2(sp[j >> 1][n][j & 1], s0, s1);
            sum[j] += ex2(fmaf(s0, mu[n][0], -ls[n][0])) + ex2(fmaf(s1, mu[n][1], -ls[n][1]));
          }
      } else {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = rt * RT + 8 * n + 2 * c + h, lim = a.causal ? len - T_rows + row / a.group + 1 : len;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float s[2];
              unpack2(sp[j >> 1][n][j & 1], s[0], s[1]);
              const int key = key0 + 8 * j + g8;
              if (key >= a.first && key < lim) sum[j] += ex2(fmaf(s[h], mu[n][h], -ls[n][h]));
            }
          }
      }
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y = sum[j];
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        if (c == j) v = y;
      }
      acc[k * kWThreads + tid] += v;
    }
  }
  for (int k = 0; k < np; ++k) {
    const int key = key_of(k);
    if (2 * k + (w >> 1) < nt && key < len) {
      const float v = acc[k * kWThreads + tid];
      ws[key] = v;
      if (a.w_out) a.w_out[((size_t)(a.call0 + i) * a.c.n_kv + head) * a.ldw + key] = v;
    }
  }
}

template <int HD, typename T, int NQ>
cudaError_t attend_t(const KvqAttnArgs &a, cudaStream_t s) {
  using Sh = Shape<HD, T, NQ>;
  static_assert(Sh::kBytes <= 226 * 1024, "shared memory of a CTA");
  // (f32 rows take their codes signed anyway)
  constexpr bool W = sizeof(T) != 4;
  static std::atomic<uint64_t> done[2];
  auto kern = W && a.lse ? kvq_attend_kernel<HD, T, NQ, W> : kvq_attend_kernel<HD, T, NQ, false>;
  cudaError_t e = allow_smem(kern, Sh::kBytes, done[W && a.lse]);
  if (e != cudaSuccess) return e;
  e = kvq_launch(kern, dim3(a.ctas), dim3(Sh::kThreads), Sh::kBytes, s, a);
  // nothing to join where every share is a unit
  bool whole = a.extra == 0 || a.share == 0;
  for (int i = 0; i < a.n; ++i) whole = whole && (a.rows[i] == 0 || (a.share ? a.stages[i] + kKvqUnitCost == a.share : a.parts[i] == 1));
  if (e != cudaSuccess || whole) return e;
  const int units = a.unit0[a.n] * a.c.n_kv, items = 8 * NQ * HD / 4;
  if (units <= a.ctas) return kvq_launch(kvq_join_kernel<HD, T, NQ, true>, dim3(units, items / 64), dim3(kJoinThreads), 0, s, a);
  return kvq_launch(kvq_join_kernel<HD, T, NQ, false>, dim3(a.ctas - 1, (items + kJoinThreads - 1) / kJoinThreads),
                    dim3(kJoinThreads), 0, s, a);
}
template <int HD, typename T, int NQ>
cudaError_t weights_t(const KvqAttnArgs &a, cudaStream_t s) {
  constexpr int smem = w_slots(HD) * 2 * kvq_k_bytes(HD) + QTile<HD, sizeof(T) == 4, NQ>::kBytes + kKvqWeightTiles / 2 * kWThreads * 4;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kvq_weights_kernel<HD, T, NQ>, smem, done);
  if (e != cudaSuccess) return e;
  return kvq_launch(kvq_weights_kernel<HD, T, NQ>, dim3(a.wt0[a.n], a.c.n_kv), dim3(kWThreads), smem, s, a);
}

template <typename Sh>
constexpr KvqShape shape_of() {
  return {Sh::MB, Sh::NG};
}
template <int HD, typename T>
KvqShape shape_t(int nq) {
  return nq == 1   ? shape_of<Shape<HD, T, 1>>()
         : nq == 2 ? shape_of<Shape<HD, T, 2>>()
         : nq == 3 ? shape_of<Shape<HD, T, 3>>()
                   : shape_of<Shape<HD, T, 4>>();
}
template <int HD, typename T>
cudaError_t call_t(const KvqAttnArgs &a, bool weights, cudaStream_t s) {
  switch (a.nq) {
    case 1: return weights ? weights_t<HD, T, 1>(a, s) : attend_t<HD, T, 1>(a, s);
    case 2: return weights ? weights_t<HD, T, 2>(a, s) : attend_t<HD, T, 2>(a, s);
    case 3: return weights ? weights_t<HD, T, 3>(a, s) : attend_t<HD, T, 3>(a, s);
    default: return weights ? weights_t<HD, T, 4>(a, s) : attend_t<HD, T, 4>(a, s);
  }
}

}  // namespace

// one translation unit a head dim (KVQ_HD), so that they compile side by side
template <int HD>
cudaError_t kvq_attn_call(const KvqAttnArgs &a, bool weights, cudaStream_t s) {
  if (a.type == KVQ_F32) return call_t<HD, float>(a, weights, s);
  if (a.type == KVQ_F16) return call_t<HD, __half>(a, weights, s);
  return call_t<HD, __nv_bfloat16>(a, weights, s);
}
template <int HD>
KvqShape kvq_attn_shape(int type, int nq) {
  return type == KVQ_F32 ? shape_t<HD, float>(nq) : type == KVQ_F16 ? shape_t<HD, __half>(nq) : shape_t<HD, __nv_bfloat16>(nq);
}
template cudaError_t kvq_attn_call<KVQ_HD>(const KvqAttnArgs &, bool, cudaStream_t);
template KvqShape kvq_attn_shape<KVQ_HD>(int, int);

}  // namespace fm
