// k_kvq_attn.cu -- attention over the 4-bit KV cache, and the attention weight
// that each cache row collects.
//
//   O[r] = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp2(t_rj - m_r),
//   t_rj = scale log2(e) q_r . k_j  over the rows j that r sees,
// one pass over the cache with a running reference m and sum; a
// call's (sequence, KV head, 16 query rows) units lie end to end and every CTA
// takes an equal share of their stages (two tiles, 128 rows); where a unit is
// shared, the CTA that finishes last joins the parts, in their order.
//
// A CTA carries 16 query rows (block row x head of the KV head's group) at a time.  Its
// warps work in groups of four: a group has its own ring of stages (K and V codes
// and scales of 128 rows in one bulk copy) and its warps take a strip of 32 rows each.  With 16 query rows the
// product is a skinny one, and the codes pass from shared memory (ldmatrix)
// through a few integer and f16 operations straight into mma.sync fragments:
// they never go back to shared memory as f16, which a tcgen05 operand would need
// (64 KB written and read again per 128 rows of head dim 128: 1024 cycles of shared
// memory against the 784 cycles in which the SM's share of HBM delivers their 18 KB).
#include <type_traits>

#include "kvq_dev.cuh"

namespace fm {
namespace {

using namespace kvq;

constexpr float kLazy = 8.f;               // log2 of the growth a reference tolerates
constexpr int kWThreads = 128;             // the weights pass

// The attention kernel's shape: groups of four warps (they take the stages in turn) and ring stages; one
// CTA an SM, as wide as the registers allow, so that a unit is in few parts.
template <int HD, typename T>
struct Shape {
  static constexpr bool QS = sizeof(T) == 4;                          // f32 queries: f16 hi + lo
  static constexpr bool PS = !std::is_same<T, __nv_bfloat16>::value;  // f16 and f32 outputs: P' too
  static constexpr bool SV = sizeof(T) == 4;                          // f32 outputs: signed codes (no sums to take off)
  static constexpr int NG = HD == 64 ? 4 : HD == 128 ? 3 : 2;
  static constexpr int NS = HD == 64 ? 4 : HD == 128 ? 3 : 2;         // of a group's own ring
  static constexpr int NW = 4 * NG, kThreads = 128 * NG;
  static constexpr int SB = kKvqStage * kvq_tile_bytes(HD);
  static constexpr int HC = 64;                                       // dims joined at a time
  static constexpr int kFold = NW > 8 ? 8 : NW > 4 ? 4 : 2;           // warps left after the first step of the joining
  static constexpr int kScratch = (NW - kFold > kFold / 2 ? NW - kFold : kFold / 2) * 16 * HC * 4;
  static constexpr int kBytes = NG * NS * SB + kScratch + QTile<HD, QS>::kBytes + 2 * NW * 16 * 4 + NG * 2 * NS * 8 + NG * 32;
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

// A CTA's share of the stages
__device__ __forceinline__ int share_begin(const KvqAttnArgs &a, int b) { return b * a.share + min(b, a.extra); }
__device__ __forceinline__ int cta_of(const KvqAttnArgs &a, int stage) {
  const int wide = a.extra * (a.share + 1);
  return stage < wide ? stage / (a.share + 1) : a.extra + (stage - wide) / a.share;
}

// A stretch of a share: stages [s0, s0 + n) of one unit.
struct Stretch {
  int i, head, rt, s0, n;
  __device__ __forceinline__ Stretch(const KvqAttnArgs &a, int at, int end) {
    i = find_seq<int32_t>(a.st0, a.n, at);
    const int rel = at - a.st0[i], S = a.stages[i], unit = rel / S;
    s0 = rel - unit * S;
    n = min(S - s0, end - at);
    const int rts = (a.rows[i] * a.group + kKvqQRows - 1) / kKvqQRows;
    head = unit / rts;
    rt = unit - head * rts;
  }
};

// Where a group's copies have got to (in shared memory: one lane's business, once a stage).
struct Cursor {
  const uint8_t *src;     // the next stage
  int32_t at;             // the share's stage after the stretch that the cursor is in
  int32_t left;           // stages of the stretch that are the group's
  int32_t tiles;          // tiles from the next stage to the unit's end
  int32_t issued;
};
static_assert(sizeof(Cursor) <= 32, "a cursor's place in shared memory");

// The next of the group's stages into its ring; false where a wait gave up.
template <int HD, typename Sh>
__device__ __forceinline__ bool issue_stage(const KvqAttnArgs &a, Cursor *cu, int w_end, int grp, uint32_t ring,
                                            uint32_t full, uint32_t empty) {
  constexpr int TB = kvq_tile_bytes(HD);
  int left = cu->left, tiles = cu->tiles;
  const uint8_t *src = cu->src;
  while (left == 0) {
    const int at = cu->at;
    if (at >= w_end) return true;
    const Stretch x(a, at, w_end);
    const int t = a.first / kKvqTile + (x.s0 + grp) * kKvqStage;
    left = (x.n - grp + Sh::NG - 1) / Sh::NG;
    tiles = (a.len[x.i] + kKvqTile - 1) / kKvqTile - t;
    src = a.c.planes + ((size_t)a.seq[x.i] * a.c.n_kv + x.head) * a.c.plane_bytes + (size_t)t * TB;
    cu->at = at + x.n;
  }
  const int g = cu->issued, slot = g % Sh::NS;
  if (g >= Sh::NS && !mbar_wait_bounded(empty + slot * 8, (g / Sh::NS - 1) & 1, a.c.err)) return false;
  if (tiles > 0) {
    const uint32_t bytes = min(kKvqStage, tiles) * TB;
    mbar_expect_tx(full + slot * 8, bytes);
    bulk_g2s(ring + slot * Sh::SB, src, bytes, full + slot * 8);
  } else {
    mbar_arrive(full + slot * 8);   // a unit without keys has one stage of nothing
  }
  cu->left = left - 1;
  cu->tiles = tiles - Sh::NG * kKvqStage;
  cu->src = src + Sh::NG * Sh::SB;
  cu->issued = g + 1;
  return true;
}

// The parts of a split unit into its output rows, in part order: CTA `first` has the unit's first stages (its
// second slot), the CTAs after it up to `last` the rest.
template <int HD, typename T, int NT>
__device__ __forceinline__ void join_parts(const KvqAttnArgs &a, const Stretch &x, int first, int last, float undo, float bias,
                                           float *lse, int tid) {
  constexpr int NB = 8;    // parts whose loads are in flight together
  const int R = a.rows[x.i] * a.group;
  for (int e = tid; e < 16 * HD / 4; e += NT) {
    const int r = e / (HD / 4), d = 4 * (e % (HD / 4)), qr = x.rt * kKvqQRows + r;
    if (qr >= R) break;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = first; c <= last; c += NB) {
      float2 ml[NB];
      float4 v[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const size_t slot = (size_t)min(c + k, last) * 2 + (c + k == first);
        ml[k] = __ldcg(&a.part_ml[slot * 16 + r]);
        v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + (slot * 16 + r) * HD + d));
      }
      float m = M;
#pragma unroll
      for (int k = 0; k < NB; ++k) m = fmaxf(m, ml[k].x);
      const float f = M == m ? 1.f : ex2(M - m);
      M = m;
      L *= f, acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (c + k > last) break;
        const float g = ml[k].x == M ? 1.f : ex2(ml[k].x - M);
        L = fmaf(g, ml[k].y, L);
        acc.x = fmaf(g, v[k].x, acc.x);
        acc.y = fmaf(g, v[k].y, acc.y);
        acc.z = fmaf(g, v[k].z, acc.z);
        acc.w = fmaf(g, v[k].w, acc.w);
      }
    }
    const float inv = L == 0.f ? 0.f : undo / L;
    const int t = qr / a.group;
    store4(static_cast<T *>(a.out) + (a.row0[x.i] + t) * a.ldo + ((int64_t)x.head * a.group + qr - t * a.group) * HD + d,
           make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (lse && d == 0) lse[r] = L == 0.f ? INFINITY : M + log2f(L) - bias;
  }
}

template <int HD, typename T>
__global__ void __launch_bounds__(Shape<HD, T>::kThreads, 1)
    kvq_attend_kernel(const __grid_constant__ KvqAttnArgs a) {
  using Sh = Shape<HD, T>;
  using QT = QTile<HD, Sh::QS>;
  constexpr bool QS = Sh::QS, PS = Sh::PS, SV = Sh::SV;
  constexpr int NG = Sh::NG, NS = Sh::NS, NW = Sh::NW, SB = Sh::SB, TB = kvq_tile_bytes(HD), HC = Sh::HC;
  constexpr int kCons = Sh::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  float *scratch = reinterpret_cast<float *>(smem + NG * NS * SB);
  uint8_t *qs = smem + NG * NS * SB + Sh::kScratch;
  float *wm = reinterpret_cast<float *>(qs + QT::kBytes), *wl = wm + NW * 16;   // [warp][row] reference and sum
  uint64_t *bar = reinterpret_cast<uint64_t *>(wl + NW * 16);                   // [group][full, empty][stage]
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int grp = NG == 1 ? 0 : w >> 2;     // a group takes the stages grp, grp + NG, ... of a stretch
  __shared__ int s_last;
  __shared__ float2 s_row[16];               // references and sums of the query rows, all warps
  Cursor *cu = reinterpret_cast<Cursor *>(bar + NG * 2 * NS) + grp;
  const uint32_t full = smem_u32(bar + grp * 2 * NS), empty = full + NS * 8, ring = smem_u32(smem) + grp * NS * SB;
  const int w_beg = share_begin(a, blockIdx.x), w_end = share_begin(a, blockIdx.x + 1);

  pdl_trigger();
  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < NG * 2 * NS; ++s) mbar_init(smem_u32(bar + s), s / NS & 1 ? 4 : 1);
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  const bool copies = lane == 0 && (w & 3) == 0;   // the lane that sends for its group's stages
  bool ok = true;
  if (copies) {
    cu->at = w_beg;
    cu->left = 0;
    cu->issued = 0;
    for (int k = 0; k < NS - 1; ++k) ok = issue_stage<HD, Sh>(a, cu, w_end, grp, ring, full, empty);
  }

  const int wt = (w >> 1) & 1, r0 = (w & 1) * 32;
  const LaneAt<HD> la(r0, lane);
  const uint32_t qt = smem_u32(qs);
  const uint32_t code0 = ring + wt * TB + la.code, scale0 = ring + wt * TB + la.scale;
  const int row = lane >> 2;
  int slot = 0;
  uint32_t par = 0;
  for (int at = w_beg; at < w_end;) {
    const Stretch x(a, at, w_end);
    const int len = a.len[x.i], T_rows = a.rows[x.i], R = T_rows * a.group, rq = x.rt * kKvqQRows;
    const size_t plane = (size_t)a.seq[x.i] * a.c.n_kv + x.head;
    load_q<HD, QS, kCons>(static_cast<const T *>(a.q) + a.row0[x.i] * a.ldq + (int64_t)x.head * a.group * HD, a.ldq, a.group,
                          rq, R, a.scale_log2, qs, tid);
    const PRange<PS> range(__ldcg(a.c.vmax + plane));
    __syncthreads();
    const float2 mu = *reinterpret_cast<const float2 *>(qs + QT::kMult + row * 8);
    // the rows that this lane's two query rows see end at lim; rows past R follow the last (they are not stored)
    const int ra = min(rq + row, R - 1), rb = min(rq + row + 8, R - 1);
    const int lim0 = a.causal ? len - T_rows + ra / a.group + 1 : len;
    const int lim1 = a.causal ? len - T_rows + rb / a.group + 1 : len;
    const int lim_all = a.causal ? len - T_rows + rq / a.group + 1 : len;

    float o[HD / 8][4], cor[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY;
    uint64_t l0 = 0ull, l1 = 0ull;          // row sums, even and odd keys apart
    int key0 = (a.first / kKvqTile + (x.s0 + grp) * kKvqStage + wt) * kKvqTile + r0;
    for (int k = grp; k < x.n; k += NG) {
      // a stage ahead of the ring's end; then this one (a wait that gave up ends the warp's work, not its barriers)
      if (copies && ok) ok = issue_stage<HD, Sh>(a, cu, w_end, grp, ring, full, empty);
      ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(full + slot * 8, par, a.c.err));
      if (!ok) break;
      if (key0 < len && key0 + 32 > a.first) {
        const uint32_t code = code0 + slot * SB, scale = scale0 + slot * SB;
        uint64_t sp[4][2];
        strip_scores<HD, QS>(code, scale, qt, lane, sp);
        float s[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack2(sp[j][0], s[j][0], s[j][1]), unpack2(sp[j][1], s[j][2], s[j][3]);
        if (key0 < a.first || key0 + 32 > lim_all) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 8 * j + 2 * (lane & 3) + (e & 1);
              if (key < a.first || key >= (e < 2 ? lim0 : lim1)) s[j][e] = -INFINITY;
            }
        }
        float x0 = fmaxf(s[0][0], s[0][1]), x1 = fmaxf(s[0][2], s[0][3]);
#pragma unroll
        for (int j = 1; j < 4; ++j) {
          x0 = fmaxf(x0, fmaxf(s[j][0], s[j][1]));
          x1 = fmaxf(x1, fmaxf(s[j][2], s[j][3]));
        }
#pragma unroll
        for (int sh = 1; sh < 4; sh <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, sh));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, sh));
        }
        x0 *= mu.x, x1 *= mu.y;
        if (__any_sync(0xffffffffu, x0 > m0 + kLazy || x1 > m1 + kLazy)) {
          const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
          const float f0 = n0 == m0 ? 1.f : ex2(m0 - n0), f1 = n1 == m1 ? 1.f : ex2(m1 - n1);
          m0 = n0, m1 = n1;
          l0 = mul2(l0, pack2(f0, f0)), l1 = mul2(l1, pack2(f1, f1));
#pragma unroll
          for (int n = 0; n < HD / 8; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
          if constexpr (!SV) cor[0] *= f0, cor[1] *= f0, cor[2] *= f1, cor[3] *= f1;
        }
        const float b0 = range.bias - (m0 == -INFINITY ? 0.f : m0), b1 = range.bias - (m1 == -INFINITY ? 0.f : m1);
        const uint64_t mu0 = pack2(mu.x, mu.x), mu1 = pack2(mu.y, mu.y), bb0 = pack2(b0, b0), bb1 = pack2(b1, b1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float t[4];
          unpack2(fma2(pack2(s[j][0], s[j][1]), mu0, bb0), t[0], t[1]);
          unpack2(fma2(pack2(s[j][2], s[j][3]), mu1, bb1), t[2], t[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = ex2(t[e]);
          l0 = add2(l0, pack2(t[0], t[1]));
          l1 = add2(l1, pack2(t[2], t[3]));
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = t[e];
        }
        strip_pv<HD, PS, SV>(code + kvq_k_bytes(HD), scale + kvq_k_bytes(HD), lane, range, s, o, cor);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + slot * 8);
      if (++slot == NS) slot = 0, par ^= 1;
      key0 += NG * kKvqStage * kKvqTile;
    }

    // the warps' results: references and sums first, then the outputs pairwise
    float ls0, ls1, lt;
    unpack2(l0, ls0, lt);
    ls0 += lt;
    unpack2(l1, ls1, lt);
    ls1 += lt;
#pragma unroll
    for (int sh = 1; sh < 4; sh <<= 1) {
      ls0 += __shfl_xor_sync(0xffffffffu, ls0, sh);
      ls1 += __shfl_xor_sync(0xffffffffu, ls1, sh);
    }
    if ((lane & 3) == 0) {
      wm[w * 16 + row] = m0;
      wm[w * 16 + row + 8] = m1;
      wl[w * 16 + row] = ls0;
      wl[w * 16 + row + 8] = ls1;
    }
    __syncthreads();
    if (tid < 16) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int u = 0; u < NW; ++u) M = fmaxf(M, wm[u * 16 + tid]);
#pragma unroll
      for (int u = 0; u < NW; ++u) L += (wm[u * 16 + tid] == M ? 1.f : ex2(wm[u * 16 + tid] - M)) * wl[u * 16 + tid];
      s_row[tid] = make_float2(M, L);
    }
    __syncthreads();
    const float M0 = s_row[row].x, M1 = s_row[row + 8].x;
    finish_o<HD, SV>(o, cor, lane, m0 == M0 ? 1.f : ex2(m0 - M0), m1 == M1 ? 1.f : ex2(m1 - M1));
    const bool whole = x.n == a.stages[x.i];
    const size_t slot_g = (size_t)blockIdx.x * 2 + (x.s0 == 0);   // a unit begun here, or one continued
    float *lse = a.lse ? a.lse + ((size_t)(a.unit0[x.i] + x.rt) * a.c.n_kv + x.head) * 16 : nullptr;
#pragma unroll
    for (int c0 = 0; c0 < HD; c0 += HC) {
#pragma unroll
      for (int half = Sh::kFold; half >= 1; half >>= 1) {
        float4 *buf = reinterpret_cast<float4 *>(scratch) + (w & (half - 1)) * (16 * HC / 4) + lane;
        if (w >= half && w < 2 * half) {
#pragma unroll
          for (int n = 0; n < HC / 8; ++n) {
            const float(&v)[4] = o[c0 / 8 + n];
            buf[n * 32] = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        __syncthreads();
        if (w < half && w + half < NW) {
#pragma unroll
          for (int n = 0; n < HC / 8; ++n) {
            const float4 v = buf[n * 32];
            float(&y)[4] = o[c0 / 8 + n];
            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
          }
        }
      }
      if (w == 0) {   // as rows: columns 2 c, 2 c + 1 of tile n are dims d, d + 4
#pragma unroll
        for (int n = 0; n < HC / 8; ++n) {
          const int d = 32 * (n >> 2) + 8 * (lane & 3) + (n & 3);
          const float(&v)[4] = o[c0 / 8 + n];
          scratch[row * HC + d] = v[0];
          scratch[row * HC + d + 4] = v[1];
          scratch[(row + 8) * HC + d] = v[2];
          scratch[(row + 8) * HC + d + 4] = v[3];
        }
      }
      __syncthreads();
#pragma unroll
      for (int e = tid; e < 16 * HC / 4; e += kCons) {
        const int r = e / (HC / 4), d = 4 * (e % (HC / 4)), qr = rq + r;
        const float4 v = *reinterpret_cast<const float4 *>(scratch + r * HC + d);
        const float M = s_row[r].x, L = s_row[r].y;
        if (!whole) {
          *reinterpret_cast<float4 *>(a.part_o + (slot_g * 16 + r) * HD + c0 + d) = v;
          if (c0 + d == 0) a.part_ml[slot_g * 16 + r] = make_float2(M, L);
        } else if (qr < R) {
          const float inv = L == 0.f ? 0.f : range.undo / L;
          const int t = qr / a.group;
          store4(static_cast<T *>(a.out) + (a.row0[x.i] + t) * a.ldo +
                     ((int64_t)x.head * a.group + qr - t * a.group) * HD + c0 + d,
                 make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
          if (lse && c0 + d == 0) lse[r] = L == 0.f ? INFINITY : M + log2f(L) - range.bias;
        }
      }
      if (c0 + HC < HD) __syncthreads();
    }
    if (!whole) {   // the CTA that finishes the last part of a unit joins them all, in their order
      int32_t *ticket = a.tickets + (size_t)(a.unit0[x.i] + x.rt) * a.c.n_kv + x.head;
      const int u0 = at - x.s0, first = cta_of(a, u0), last = cta_of(a, u0 + a.stages[x.i] - 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(ticket, 1) == last - first;
      __syncthreads();
      if (s_last) {
        __threadfence();
        if (tid == 0) *ticket = 0;
        join_parts<HD, T, kCons>(a, x, first, last, range.undo, range.bias, lse, tid);
      }
    }
    at += x.n;
    if (at < w_end) __syncthreads();   // the next stretch writes the queries, the references and the scratch
  }
  // nothing is left in flight when the CTA ends (a consumer may have given up)
  if (copies)
    for (int k = max(0, cu->issued - NS); k < cu->issued; ++k) mbar_wait_drain(full + k % NS * 8, (k / NS) & 1);
  __syncthreads();
}

// weights[j] = decay weights[j] + sum_r p_rj / sum_j p_rj: with every row's sum
// known, K alone is read again (from L2 where it still is there) and the scores
// formed a second time, which needs no store of rows x keys.  One CTA owns a
// run of 8 tiles, so nothing is added atomically.  Grid (sequence x run, KV head).
template <int HD, typename T>
__global__ void __launch_bounds__(kWThreads) kvq_weights_kernel(const __grid_constant__ KvqAttnArgs a) {
  constexpr bool QS = sizeof(T) == 4;
  constexpr int KB = kvq_k_bytes(HD), NW = kKvqWeightTiles / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  using QT = QTile<HD, QS>;
  uint8_t *qs = smem + kKvqWeightTiles * KB;
  const uint32_t bars = smem_u32(qs + QT::kBytes);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int i = find_seq<int32_t>(a.wt0, a.n, blockIdx.x), head = blockIdx.y;
  const int len = a.len[i], T_rows = a.rows[i], R = T_rows * a.group;
  const int rts = (R + kKvqQRows - 1) / kKvqQRows;
  const int t0 = (blockIdx.x - a.wt0[i]) * kKvqWeightTiles;
  const int nt = min(kKvqWeightTiles, (len + kKvqTile - 1) / kKvqTile - t0);
  const size_t plane = (size_t)a.seq[i] * a.c.n_kv + head;
  pdl_trigger();
  if (tid == 0) {
    for (int t = 0; t < nt; ++t) mbar_init(bars + t * 8, 1);
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  if (tid == 0)
    for (int t = 0; t < nt; ++t) {
      mbar_expect_tx(bars + t * 8, KB);
      bulk_g2s(smem_u32(smem + t * KB), a.c.planes + plane * a.c.plane_bytes + (size_t)(t0 + t) * kvq_tile_bytes(HD), KB,
               bars + t * 8);
    }
  const LaneAt<HD> la((w & 1) * 32, lane);
  float acc[NW][4][2];
#pragma unroll
  for (int k = 0; k < NW; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[k][j][0] = acc[k][j][1] = 0.f;
  bool ok = true;
  for (int rt = 0; rt < rts; ++rt) {
    if (rt) __syncthreads();
    load_q<HD, QS, kWThreads>(static_cast<const T *>(a.q) + a.row0[i] * a.ldq + (int64_t)head * a.group * HD, a.ldq,
                              a.group, rt * kKvqQRows, R, a.scale_log2, qs, tid);
    __syncthreads();
    const int row0 = rt * kKvqQRows + (lane >> 2), row1 = row0 + 8;
    const float *lse = a.lse + ((size_t)(a.unit0[i] + rt) * a.c.n_kv + head) * 16;
    const float ls0 = row0 < R ? __ldcg(lse + (lane >> 2)) : INFINITY, ls1 = row1 < R ? __ldcg(lse + (lane >> 2) + 8) : INFINITY;
    const float2 mu = *reinterpret_cast<const float2 *>(qs + QT::kMult + (lane >> 2) * 8);
    const int lim0 = a.causal ? len - T_rows + row0 / a.group + 1 : len;
    const int lim1 = a.causal ? len - T_rows + row1 / a.group + 1 : len;
    const int lim_all = a.causal ? len - T_rows + rt * kKvqQRows / a.group + 1 : len;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int t = 2 * k + (w >> 1), key0 = (t0 + t) * kKvqTile + (w & 1) * 32;
      if (t >= nt || key0 >= len || key0 + 32 <= a.first) continue;
      if (rt == 0 && !mbar_wait_warp(bars + t * 8, 0, a.c.err)) ok = false;
      if (!ok) continue;
      uint64_t sp[4][2];
      strip_scores<HD, QS>(smem_u32(smem + t * KB) + la.code, smem_u32(smem + t * KB) + la.scale, smem_u32(qs), lane, sp);
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) unpack2(sp[j][0], s[j][0], s[j][1]), unpack2(sp[j][1], s[j][2], s[j][3]);
      const bool whole = key0 >= a.first && key0 + 32 <= lim_all;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = ex2(fmaf(s[j][e], e < 2 ? mu.x : mu.y, e < 2 ? -ls0 : -ls1));
          if (!whole) {
            const int key = key0 + 8 * j + 2 * (lane & 3) + (e & 1);
            if (key < a.first || key >= (e < 2 ? lim0 : lim1)) p = 0.f;
          }
          // a row without keys, or past the last, has no weight to give
          if ((e < 2 ? ls0 : ls1) == INFINITY) p = 0.f;
          acc[k][j][e & 1] += p;
        }
    }
  }
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    const int t = 2 * k + (w >> 1), key0 = (t0 + t) * kKvqTile + (w & 1) * 32;
    if (t >= nt) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = acc[k][j][e];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) v += __shfl_xor_sync(0xffffffffu, v, sh);
        const int key = key0 + 8 * j + 2 * (lane & 3) + e;
        if (lane < 4 && key < len && ok) {
          float *p = a.c.weights + plane * a.c.rows_pad + key;
          if (a.decay != 0.f) v = fmaf(a.decay, *p, v);
          *p = v;
          if (a.w_out) a.w_out[((size_t)(a.call0 + i) * a.c.n_kv + head) * a.ldw + key] = v;
        }
      }
  }
  // (a strip that no query row sees was not waited for: nothing is left in flight when the CTA ends)
  if (tid == 0)
    for (int t = 0; t < nt; ++t) mbar_wait_drain(bars + t * 8, 0);
  __syncthreads();
}

template <int HD, bool QS>
constexpr int weights_smem() {
  return kKvqWeightTiles * kvq_k_bytes(HD) + QTile<HD, QS>::kBytes + kKvqWeightTiles * 8;
}

template <int HD, typename T>
cudaError_t attend_t(const KvqAttnArgs &a, cudaStream_t s) {
  constexpr int smem = Shape<HD, T>::kBytes;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(kvq_attend_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return kvq_launch(kvq_attend_kernel<HD, T>, dim3(a.ctas), dim3(Shape<HD, T>::kThreads), smem, s, a);
}
template <int HD, typename T>
cudaError_t weights_t(const KvqAttnArgs &a, cudaStream_t s) {
  constexpr int smem = weights_smem<HD, sizeof(T) == 4>();
  cudaError_t e = cudaFuncSetAttribute(kvq_weights_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return kvq_launch(kvq_weights_kernel<HD, T>, dim3(a.wt0[a.n], a.c.n_kv), dim3(kWThreads), smem, s, a);
}
template <int HD, typename T>
int ctas_t() {
  constexpr int smem = Shape<HD, T>::kBytes;
  int n = 0;
  if (cudaFuncSetAttribute(kvq_attend_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kvq_attend_kernel<HD, T>, Shape<HD, T>::kThreads, smem) != cudaSuccess)
    return 1;
  return n < 1 ? 1 : n;
}

#define KVQ_DISPATCH(fn, ...)                                                                       \
  switch (hd * 4 + type) {                                                                          \
    case 64 * 4 + KVQ_F32: return fn<64, float>(__VA_ARGS__);                                       \
    case 64 * 4 + KVQ_F16: return fn<64, __half>(__VA_ARGS__);                                      \
    case 64 * 4 + KVQ_BF16: return fn<64, __nv_bfloat16>(__VA_ARGS__);                              \
    case 128 * 4 + KVQ_F32: return fn<128, float>(__VA_ARGS__);                                     \
    case 128 * 4 + KVQ_F16: return fn<128, __half>(__VA_ARGS__);                                    \
    case 128 * 4 + KVQ_BF16: return fn<128, __nv_bfloat16>(__VA_ARGS__);                            \
    case 256 * 4 + KVQ_F32: return fn<256, float>(__VA_ARGS__);                                     \
    case 256 * 4 + KVQ_F16: return fn<256, __half>(__VA_ARGS__);                                    \
    default: return fn<256, __nv_bfloat16>(__VA_ARGS__);                                            \
  }

}  // namespace

int kvq_attn_ctas_per_sm(int hd, int type) { KVQ_DISPATCH(ctas_t) }
cudaError_t launch_kvq_attend(const KvqAttnArgs &a, int hd, cudaStream_t s) {
  const int type = a.type;
  KVQ_DISPATCH(attend_t, a, s)
}
cudaError_t launch_kvq_weights(const KvqAttnArgs &a, int hd, cudaStream_t s) {
  const int type = a.type;
  KVQ_DISPATCH(weights_t, a, s)
}

}  // namespace fm
