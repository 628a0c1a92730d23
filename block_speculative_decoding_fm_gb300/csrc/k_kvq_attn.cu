// k_kvq_attn.cu -- attention over the 4-bit KV cache, and the attention weight
// that each cache row collects.
//
//   O[r] = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp2(t_rj - m_r),
//   t_rj = scale log2(e) q_r . k_j  over the rows j that r sees,
// one pass over the cache with a running reference m and sum; the keys of a
// (sequence, KV head) are dealt to CTAs in chunks of whole tiles, and a second,
// short launch joins the chunks of sequences that have more than one.
//
// A CTA carries 16 query rows (block row x head of the KV head's group): warp 4
// streams stages of two tiles (128 rows, K and V codes and scales in one bulk copy)
// into a ring; warps 0..3 take a strip of 32 rows each.  With 16 query rows the
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

constexpr int kCons = 128;                 // consumer threads
constexpr int kThreads = kCons + 32;
constexpr float kLazy = 8.f;               // log2 of the growth a reference tolerates

template <int HD>
constexpr int n_stages() {
  return HD == 256 ? 3 : 4;
}
template <int HD, bool QS>
constexpr int attend_smem() {
  return n_stages<HD>() * 2 * kvq_tile_bytes(HD) + q_bytes<HD, QS>() + 16 * 4 + 2 * 4 * 16 * 4 + 2 * n_stages<HD>() * 8;
}

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

// Grid (sequence x chunk x row tile, KV head).
template <int HD, typename T>
__global__ void __launch_bounds__(kThreads) kvq_attend_kernel(const __grid_constant__ KvqAttnArgs a) {
  // f32 queries are split into f16 hi + lo; f16 and f32 outputs keep P split too (a once-rounded
  // P' alone is as far off as an f16 output's own rounding)
  constexpr bool QS = sizeof(T) == 4, PS = !std::is_same<T, __nv_bfloat16>::value;
  constexpr int NS = n_stages<HD>(), SB = 2 * kvq_tile_bytes(HD);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *qs = smem + NS * SB;
  float *mult = reinterpret_cast<float *>(qs + q_bytes<HD, QS>());
  float *wm = mult + 16, *wl = wm + 4 * 16;             // [warp][row] reference and sum
  const uint32_t bars = smem_u32(wl + 4 * 16);
  auto full = [&](int i) { return bars + i * 8; };
  auto empty = [&](int i) { return bars + (NS + i) * 8; };
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;

  const int i = find_seq(a.cta0, a.n, blockIdx.x);
  const int head = blockIdx.y;
  const int len = a.len[i], T_rows = a.rows[i], R = T_rows * a.group;
  const int rts = (R + kKvqQRows - 1) / kKvqQRows;
  const int in_seq = blockIdx.x - a.cta0[i];
  const int chunk = in_seq / rts, rt = in_seq - chunk * rts;
  const int chunks = (a.cta0[i + 1] - a.cta0[i]) / rts;
  const int t_end_all = (len + kKvqTile - 1) / kKvqTile;
  const int t0 = min(t_end_all, a.first / kKvqTile + chunk * a.chunk), t1 = min(t_end_all, t0 + a.chunk);
  const int nst = (t1 - t0 + 1) / 2;
  const size_t plane = (size_t)a.seq[i] * a.c.n_kv + head;

  pdl_trigger();
  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4);
    }
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();

  if (w == 4) {
    if (lane == 0) {
      const uint8_t *src = a.c.planes + plane * a.c.plane_bytes + (size_t)t0 * kvq_tile_bytes(HD);
      int st = 0;
      for (; st < nst; ++st) {
        const int slot = st % NS;
        if (st >= NS && !mbar_wait_bounded(empty(slot), ((st / NS) - 1) & 1, a.c.err)) break;
        const uint32_t bytes = (uint32_t)min(2, t1 - t0 - 2 * st) * kvq_tile_bytes(HD);
        mbar_expect_tx(full(slot), bytes);
        bulk_g2s(smem_u32(smem + slot * SB), src + (size_t)st * SB, bytes, full(slot));
      }
      // nothing is left in flight when the CTA ends (a consumer may have given up)
      for (int s = max(0, st - NS); s < st; ++s) mbar_wait_drain(full(s % NS), (s / NS) & 1);
    }
    __syncthreads();
    return;
  }

  load_q<HD, QS, kCons>(static_cast<const T *>(a.q) + a.row0[i] * a.ldq + (int64_t)head * a.group * HD, a.ldq, a.group,
                        rt * kKvqQRows, R, a.scale_log2, qs, mult, tid);
  named_sync(1, kCons);
  const PRange<PS> range(__ldcg(a.c.vmax + plane));
  const float bias = range.bias;
  const float mu0 = mult[lane >> 2], mu1 = mult[(lane >> 2) + 8];
  // the rows that this lane's two query rows see end at lim; rows past R follow the last (they are not stored)
  const int ra = min(rt * kKvqQRows + (lane >> 2), R - 1), rb = min(rt * kKvqQRows + (lane >> 2) + 8, R - 1);
  const int lim0 = a.causal ? len - T_rows + ra / a.group + 1 : len;
  const int lim1 = a.causal ? len - T_rows + rb / a.group + 1 : len;
  const int lim_all = a.causal ? len - T_rows + rt * kKvqQRows / a.group + 1 : len;

  float o[HD / 8][4];
#pragma unroll
  for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  const uint32_t qf = smem_u32(qs);
  for (int st = 0; st < nst; ++st) {
    const int slot = st % NS;
    if (!mbar_wait_warp(full(slot), (st / NS) & 1, a.c.err)) break;
    const int tile = t0 + 2 * st + (w >> 1), r0 = (w & 1) * 32, key0 = tile * kKvqTile + r0;
    if (tile < t1 && key0 < len && key0 + 32 > a.first) {
      const uint32_t kb = smem_u32(smem + slot * SB + (w >> 1) * kvq_tile_bytes(HD));
      float s[4][4];
      strip_scores<HD, QS>(kb, r0, qf, lane, s);
      const bool whole = key0 >= a.first && key0 + 32 <= lim_all;
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[j][e] *= e < 2 ? mu0 : mu1;
          if (!whole) {
            const int key = key0 + 8 * j + 2 * (lane & 3) + (e & 1);
            if (key < a.first || key >= (e < 2 ? lim0 : lim1)) s[j][e] = -INFINITY;
          }
        }
        x0 = fmaxf(x0, fmaxf(s[j][0], s[j][1]));
        x1 = fmaxf(x1, fmaxf(s[j][2], s[j][3]));
      }
#pragma unroll
      for (int sh = 1; sh < 4; sh <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, sh));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, sh));
      }
      if (__any_sync(0xffffffffu, x0 > m0 + kLazy || x1 > m1 + kLazy)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float f0 = n0 == m0 ? 1.f : ex2(m0 - n0), f1 = n1 == m1 ? 1.f : ex2(m1 - n1);
        m0 = n0, m1 = n1;
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int n = 0; n < HD / 8; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
      }
      const float b0 = (m0 == -INFINITY ? 0.f : m0) - bias, b1 = (m1 == -INFINITY ? 0.f : m1) - bias;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j][0] = ex2(s[j][0] - b0);
        s[j][1] = ex2(s[j][1] - b0);
        s[j][2] = ex2(s[j][2] - b1);
        s[j][3] = ex2(s[j][3] - b1);
        l0 += s[j][0] + s[j][1];
        l1 += s[j][2] + s[j][3];
      }
      strip_pv<HD, PS>(kb + kvq_k_bytes(HD), r0, lane, range, s, o);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(slot));
  }
#pragma unroll
  for (int sh = 1; sh < 4; sh <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
    l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
  }
  // the four warps' results, in warp order, in the ring (every copy into it has landed and been read)
  if ((lane & 3) == 0) {
    wm[w * 16 + (lane >> 2)] = m0;
    wm[w * 16 + (lane >> 2) + 8] = m1;
    wl[w * 16 + (lane >> 2)] = l0;
    wl[w * 16 + (lane >> 2) + 8] = l1;
  }
  __syncthreads();   // with the copying warp, whose copies have all landed
  float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    M0 = fmaxf(M0, wm[v * 16 + (lane >> 2)]);
    M1 = fmaxf(M1, wm[v * 16 + (lane >> 2) + 8]);
  }
  const float f0 = m0 == M0 ? 1.f : ex2(m0 - M0), f1 = m1 == M1 ? 1.f : ex2(m1 - M1);
  float *ob = reinterpret_cast<float *>(smem) + w * 16 * HD;
#pragma unroll
  for (int n = 0; n < HD / 8; ++n) {
    const int d = 32 * (n >> 2) + 8 * (lane & 3) + (n & 3);   // columns 2 c, 2 c + 1 of tile n: dims d, d + 4
    ob[(lane >> 2) * HD + d] = o[n][0] * f0;
    ob[(lane >> 2) * HD + d + 4] = o[n][1] * f0;
    ob[((lane >> 2) + 8) * HD + d] = o[n][2] * f1;
    ob[((lane >> 2) + 8) * HD + d + 4] = o[n][3] * f1;
  }
  named_sync(1, kCons);
  const size_t slot_g = ((size_t)a.slot0[i] + in_seq) * a.c.n_kv + head;
#pragma unroll
  for (int it = tid; it < 16 * HD / 4; it += kCons) {
    const int r = it / (HD / 4), d = 4 * (it % (HD / 4));
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int v = 0; v < 4; ++v) M = fmaxf(M, wm[v * 16 + r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float mv = wm[v * 16 + r];
      L += (mv == M ? 1.f : ex2(mv - M)) * wl[v * 16 + r];
      const float4 x = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem) + (v * 16 + r) * HD + d);
      acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
    }
    const int row = rt * kKvqQRows + r;
    if (chunks > 1) {
      *reinterpret_cast<float4 *>(a.part_o + (slot_g * 16 + r) * HD + d) = acc;
      if (d == 0) a.part_ml[slot_g * 16 + r] = make_float2(M, L);
    } else if (row < R) {
      const float inv = L == 0.f ? 0.f : range.undo / L;
      const int t = row / a.group;
      store4(static_cast<T *>(a.out) + (a.row0[i] + t) * a.ldo + ((int64_t)head * a.group + row - t * a.group) * HD + d,
             make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
      if (a.lse && d == 0)
        a.lse[((size_t)(a.unit0[i] + rt) * a.c.n_kv + head) * 16 + r] = L == 0.f ? INFINITY : M + log2f(L) - bias;
    }
  }
}

// Joins the chunks of a split unit in chunk order.  Grid (split row tile, KV head, 16 HD / 4 / 128 row groups).
template <int HD, typename T>
__global__ void __launch_bounds__(128) kvq_merge_kernel(const __grid_constant__ KvqAttnArgs a) {
  pdl_trigger();
  const int i = find_seq(a.split0, a.n, blockIdx.x);
  const int head = blockIdx.y, rt = blockIdx.x - a.split0[i];
  const int R = a.rows[i] * a.group, rts = (R + kKvqQRows - 1) / kKvqQRows;
  const int chunks = (a.cta0[i + 1] - a.cta0[i]) / rts;
  const int it = blockIdx.z * 128 + threadIdx.x;
  const int r = it / (HD / 4), d = 4 * (it % (HD / 4)), row = rt * kKvqQRows + r;
  const size_t step = (size_t)rts * a.c.n_kv;
  const size_t s0 = ((size_t)a.slot0[i] + rt) * a.c.n_kv + head;
  pdl_wait();
  if (row >= R) return;
  float M = -INFINITY, L = 0.f;
#pragma unroll 8
  for (int c = 0; c < chunks; ++c) M = fmaxf(M, __ldcg(&a.part_ml[(s0 + c * step) * 16 + r]).x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int c = 0; c < chunks; ++c) {
    const float2 ml = __ldcg(&a.part_ml[(s0 + c * step) * 16 + r]);
    const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.part_o + ((s0 + c * step) * 16 + r) * HD + d));
    const float f = ml.x == M ? 1.f : ex2(ml.x - M);
    L = fmaf(f, ml.y, L);
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  const PRange<!std::is_same<T, __nv_bfloat16>::value> range(__ldcg(a.c.vmax + (size_t)a.seq[i] * a.c.n_kv + head));
  const float inv = L == 0.f ? 0.f : range.undo / L;
  const int t = row / a.group;
  store4(static_cast<T *>(a.out) + (a.row0[i] + t) * a.ldo + ((int64_t)head * a.group + row - t * a.group) * HD + d,
         make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (a.lse && d == 0)
    a.lse[((size_t)(a.unit0[i] + rt) * a.c.n_kv + head) * 16 + r] = L == 0.f ? INFINITY : M + log2f(L) - range.bias;
}

// weights[j] = decay weights[j] + sum_r p_rj / sum_j p_rj: with every row's sum
// known, K alone is read again (from L2 where it still is there) and the scores
// formed a second time, which needs no store of rows x keys.  One CTA owns a
// run of 8 tiles, so nothing is added atomically.  Grid (sequence x run, KV head).
template <int HD, typename T>
__global__ void __launch_bounds__(kCons) kvq_weights_kernel(const __grid_constant__ KvqAttnArgs a) {
  constexpr bool QS = sizeof(T) == 4;
  constexpr int KB = kvq_k_bytes(HD), NW = kKvqWeightTiles / 2;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *qs = smem + kKvqWeightTiles * KB;
  float *mult = reinterpret_cast<float *>(qs + q_bytes<HD, QS>());
  const uint32_t bars = smem_u32(mult + 16);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int i = find_seq(a.wt0, a.n, blockIdx.x), head = blockIdx.y;
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
  float acc[NW][4][2];
#pragma unroll
  for (int k = 0; k < NW; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[k][j][0] = acc[k][j][1] = 0.f;
  bool ok = true;
  for (int rt = 0; rt < rts; ++rt) {
    if (rt) __syncthreads();
    load_q<HD, QS, kCons>(static_cast<const T *>(a.q) + a.row0[i] * a.ldq + (int64_t)head * a.group * HD, a.ldq, a.group,
                          rt * kKvqQRows, R, a.scale_log2, qs, mult, tid);
    __syncthreads();
    const int row0 = rt * kKvqQRows + (lane >> 2), row1 = row0 + 8;
    const float *lse = a.lse + ((size_t)(a.unit0[i] + rt) * a.c.n_kv + head) * 16;
    const float ls0 = row0 < R ? __ldcg(lse + (lane >> 2)) : INFINITY, ls1 = row1 < R ? __ldcg(lse + (lane >> 2) + 8) : INFINITY;
    const float mu0 = mult[lane >> 2], mu1 = mult[(lane >> 2) + 8];
    const int lim0 = a.causal ? len - T_rows + row0 / a.group + 1 : len;
    const int lim1 = a.causal ? len - T_rows + row1 / a.group + 1 : len;
    const int lim_all = a.causal ? len - T_rows + rt * kKvqQRows / a.group + 1 : len;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int t = 2 * k + (w >> 1), r0 = (w & 1) * 32, key0 = (t0 + t) * kKvqTile + r0;
      if (t >= nt || key0 >= len || key0 + 32 <= a.first) continue;
      if (rt == 0 && !mbar_wait_warp(bars + t * 8, 0, a.c.err)) ok = false;
      if (!ok) continue;
      float s[4][4];
      strip_scores<HD, QS>(smem_u32(smem + t * KB), r0, smem_u32(qs), lane, s);
      const bool whole = key0 >= a.first && key0 + 32 <= lim_all;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = ex2(fmaf(s[j][e], e < 2 ? mu0 : mu1, e < 2 ? -ls0 : -ls1));
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
  return kKvqWeightTiles * kvq_k_bytes(HD) + q_bytes<HD, QS>() + 16 * 4 + kKvqWeightTiles * 8;
}

template <int HD, typename T>
cudaError_t attend_t(const KvqAttnArgs &a, cudaStream_t s) {
  constexpr int smem = attend_smem<HD, sizeof(T) == 4>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static_assert(n_stages<HD>() * 2 * kvq_tile_bytes(HD) >= 4 * 16 * HD * 4, "the warps' results fit the ring");
  cudaError_t e = cudaFuncSetAttribute(kvq_attend_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return kvq_launch(kvq_attend_kernel<HD, T>, dim3(a.cta0[a.n], a.c.n_kv), dim3(kThreads), smem, s, a);
}
template <int HD, typename T>
cudaError_t merge_t(const KvqAttnArgs &a, cudaStream_t s) {
  return kvq_launch(kvq_merge_kernel<HD, T>, dim3(a.split0[a.n], a.c.n_kv, 16 * HD / 4 / 128), dim3(128), 0, s, a);
}
template <int HD, typename T>
cudaError_t weights_t(const KvqAttnArgs &a, cudaStream_t s) {
  constexpr int smem = weights_smem<HD, sizeof(T) == 4>();
  cudaError_t e = cudaFuncSetAttribute(kvq_weights_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return kvq_launch(kvq_weights_kernel<HD, T>, dim3(a.wt0[a.n], a.c.n_kv), dim3(kCons), smem, s, a);
}
template <int HD, typename T>
int ctas_t() {
  constexpr int smem = attend_smem<HD, sizeof(T) == 4>();
  int n = 0;
  if (cudaFuncSetAttribute(kvq_attend_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kvq_attend_kernel<HD, T>, kThreads, smem) != cudaSuccess)
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
cudaError_t launch_kvq_merge(const KvqAttnArgs &a, int hd, cudaStream_t s) {
  const int type = a.type;
  KVQ_DISPATCH(merge_t, a, s)
}
cudaError_t launch_kvq_weights(const KvqAttnArgs &a, int hd, cudaStream_t s) {
  const int type = a.type;
  KVQ_DISPATCH(weights_t, a, s)
}

}  // namespace fm
