// k_paged_write.cu -- a batch's new rows into a paged cache: per-head RMSNorm of queries and keys, the position
// rotation, the store to q_out and to the pages, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;   (u, v) -> gain (u cos t - v sin t, u sin t + v cos t) for the pairs of the first
//   rot dims, t = pos f_i;   V is stored as it is
// Sums and rotation are f32; the one rounding is the store's.  Angles: positions go far and f_i need not be small, so the
// turns pos f_i / 2 pi are taken in 64-bit fixed point (f_i / 2 pi in units of 2^-64, whole turns fall out of the
// product; what is left of the error is f_i's own, an f64's), and only the fraction of a turn becomes an f32.
//
// Bound: memory (each value read and written once).  A CTA takes `tokens` tokens (one where the batch is small, so that a
// single token's heads spread over `split` CTAs): its threads first compute the tokens' sines and cosines, one a thread, and
// lay out where each head's rows are read and written; then each group of head_dim / 8 lanes takes heads of a token, 8 values
// a lane: one or two 16-byte loads, the mean by shuffles, the partner of a pair from the same lane or, in the half layout,
// from the lane rot / 16 away.  What counts is instructions a row: choosing q, k or v and its strides for each row took a
// third of them.  (Four values from each partner instead of eight neighbours save the shuffles but halve the loads' width:
// 357 us for 32,768 rows of 24/4 x 256 where this form's first version took 264.)  Measured: 213 us for those rows, 5.0 TB/s
// (0.75 of the copy rate; issue slots 77 % taken); on the GPU alone 5.8 us for 1-17 rows of 32 sequences of 16 x 128 and 3.3 us for
// one token, whose calls take 9 us of the host.
#include "paged_dev.cuh"

namespace fm {
namespace {

constexpr int kWThreads = 256;
constexpr int kWTokens = 8;        // tokens of a CTA at most
constexpr int kWHeads = 512;       // heads of a CTA at most (their table is 24 KB of shared memory)

// The sequence that holds packed row t, by a look at each, and its numbers (none: those of one without rows).
__device__ __forceinline__ int scan_seqs(const PagedBatch &b, int t, int lane, PagedSeq &q) {
  q = {0, 0, 0};
#pragma unroll 1
  for (int i0 = 0; i0 < b.n_seqs; i0 += 32) {
    PagedSeq r = {0, 0, 0};
    bool ok = false;
    if (i0 + lane < b.n_seqs) r = paged_seq(b, i0 + lane, ok);
    const uint32_t holds = __ballot_sync(0xffffffffu, ok && t >= r.s0 && t - r.s0 < r.n_new);
    if (holds) {
      const int src = __ffs(holds) - 1;
      q.s0 = __shfl_sync(0xffffffffu, r.s0, src);
      q.n_new = __shfl_sync(0xffffffffu, r.n_new, src);
      q.len = __shfl_sync(0xffffffffu, r.len, src);
      return i0 + src;
    }
  }
  return 0;
}
// The sequence of packed row t, and its numbers: the last i with starts[i] <= t (a warp's 32-way search).  Starts outside the batch
// lead the search astray, but then to a sequence that they are the numbers of; the one that holds t is then looked for one by
// one, so that a bad number costs the rows of its own sequences alone.
__device__ __forceinline__ int find_seq(const PagedBatch &b, int t, int lane, PagedSeq &q) {
  int lo = 0, hi = b.n_seqs;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, i < hi && __ldcg(b.starts + i) <= t);
    const int k = below ? 31 - __clz(below) : 0;
    lo += k * step;
    hi = min(hi, lo + step);
  }
  bool ok;
  q = paged_seq(b, lo, ok);
  if (ok) return lo;
  PagedSeq held;
  lo = scan_seqs(b, t, lane, held);
  q = held;
  return lo;
}

// Where a head's rows lie: bytes; dst_ld a token for queries, a row of the pool for keys and values.
struct Head {
  const uint8_t *src;
  uint8_t *dst;
  int64_t src_ld, dst_ld;
  int kind, pad[3];                                 // 0 q, 1 k, 2 v
};

template <int HD, bool BF16, bool F32IN>
__global__ void __launch_bounds__(kWThreads) fm_paged_write_kernel(const __grid_constant__ PagedWriteArgs a) {
  constexpr int kLanes = HD / 8;                    // of a row
  constexpr int kGroups = kWThreads / kLanes;       // rows at a time
  __shared__ float2 turn[kWTokens][HD / 2];         // (cos, sin) times gain
  __shared__ int4 where[kWTokens];                  // the token's row in the pool (first KV head; -1: none), position, done or not
  extern __shared__ __align__(16) uint8_t dyn[];
  Head *heads = reinterpret_cast<Head *>(dyn);      // of this CTA
  const PagedBatch &b = a.b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.tokens, n = min(a.tokens, b.n_tokens - t0);
  pdl_trigger();
  pdl_wait();
  if (warp < n) {
    const int t = t0 + warp;
    PagedSeq q;
    const int seq = find_seq(b, t, lane, q);
    const int pos = q.len - q.n_new + (t - q.s0);
    const bool in = t >= q.s0 && t - q.s0 < q.n_new;   // (rows behind the last sequence are left as they are)
    int64_t row = -1;
    if (in && pos >= 0) {
      const int id = __ldcg(b.table + seq * b.table_ld + (pos >> b.page_log));
      if (id >= 0 && id < b.n_pages)
        row = ((int64_t)(b.page0 + id) * b.n_kv << b.page_log) + (pos & ((1 << b.page_log) - 1));
    }
    if (in && row < 0 && lane == 0 && (a.k.p || pos < 0)) b.err[1] = 1;
    if (lane == 0) where[warp] = make_int4((int)row, pos, in && pos >= 0, 0);
  }
  __syncthreads();
  const int nq = a.q.p ? b.n_kv * b.group : 0, nk = a.k.p ? b.n_kv : 0;
  const int per = (a.slots + a.split - 1) / a.split, h0 = blockIdx.y * per, h1 = min(a.slots, h0 + per);
  for (int h = h0 + threadIdx.x; h < h1; h += kWThreads) {
    const int kind = h < nq ? 0 : h < nq + nk ? 1 : 2, head = h - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk);
    const PagedRows &src = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    Head g;
    g.src = static_cast<const uint8_t *>(src.p) + head * src.hs * (F32IN ? 4 : 2);
    g.src_ld = src.ld * (F32IN ? 4 : 2);
    g.dst = kind == 0 ? static_cast<uint8_t *>(a.qo.p) + head * a.qo.hs * 2
                      : static_cast<uint8_t *>(kind == 1 ? a.k_pool : a.v_pool) + ((int64_t)head << b.page_log) * HD * 2;
    g.dst_ld = kind == 0 ? a.qo.ld * 2 : HD * 2;
    g.kind = kind;
    heads[h - h0] = g;
  }
  const int pairs = a.rot >> 1;
  for (int i = threadIdx.x; i < n * pairs; i += kWThreads) {
    const int t = i / pairs, p = i - t * pairs;
    if (where[t].z) {
      const uint64_t x = (uint64_t)(uint32_t)where[t].y * __ldg(a.freq + p);   // turns, whole ones dropped
      float sn, cs;
      sincospif((float)((int32_t)(x >> 32)) * (1.f / 2147483648.f), &sn, &cs);  // half turns in [-1, 1)
      turn[t][p] = make_float2(cs * a.gain, sn * a.gain);
    }
  }
  __syncthreads();
  const int group = threadIdx.x / kLanes, gl = threadIdx.x % kLanes, d0 = gl * 8;
  const int far = a.half ? a.rot >> 4 : 0;             // half layout: the partner's distance in lanes
  const bool turned = d0 < a.rot, low = gl < far;
  const int partner = (threadIdx.x & 31) + (turned && a.half ? (low ? far : -far) : 0);
  const float sign = low ? -1.f : 1.f;
  // (token, round of heads) one after another, the next rows asked for before these are worked on: a warp has two rows in flight
  const int rounds = (h1 - h0 + kGroups - 1) / kGroups, steps = n * rounds;
  uint4 raw[F32IN ? 2 : 1], next[F32IN ? 2 : 1];
  auto ask = [&](int t, int i, uint4 *to) {
    const int h = i * kGroups + group;
    to[0] = make_uint4(0, 0, 0, 0);
    if constexpr (F32IN) to[1] = to[0];
    if (h < h1 - h0 && where[t].z) {
      const uint4 *p = reinterpret_cast<const uint4 *>(heads[h].src + (int64_t)(t0 + t) * heads[h].src_ld) + gl * (F32IN ? 2 : 1);
      to[0] = __ldcs(p);
      if constexpr (F32IN) to[1] = __ldcs(p + 1);
    }
  };
  if (steps > 0) ask(0, 0, next);
  int t = 0, i = 0;
  for (int step = 0; step < steps; ++step) {
    raw[0] = next[0];
    if constexpr (F32IN) raw[1] = next[1];
    const int tn = i + 1 < rounds ? t : t + 1, in = i + 1 < rounds ? i + 1 : 0;
    if (step + 1 < steps) ask(tn, in, next);
    {
      // this lane's (cos, sin): of its 8 pairs in the half layout, of its 4 otherwise
      const float2 *cs = &turn[t][a.half ? (low ? gl : gl - far) * 8 : gl * 4];
      const int64_t row = where[t].x;
      const int h = i * kGroups + group;
      const bool live = h < h1 - h0 && where[t].z;
      const Head &hd = heads[h < h1 - h0 ? h : 0];
      const int kind = hd.kind;
      uint4 y16 = raw[0];
      if (F32IN || !__all_sync(0xffffffffu, kind == 2)) {   // (V of the pool's type as it is)
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (F32IN) {
            x[e] = __uint_as_float(word(raw[0], e));
            x[4 + e] = __uint_as_float(word(raw[1], e));
          } else {
            const uint32_t w = word(raw[0], e);
            float2 f;
            if constexpr (BF16)
              f = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            else
              f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
            x[2 * e] = f.x;
            x[2 * e + 1] = f.y;
          }
        }
        if (a.q_norm || a.k_norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
          for (int o = kLanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float *nw = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
          if (nw) {
            const float r = rsqrtf(ss * (1.f / HD) + a.eps);
            const float4 u = __ldg(reinterpret_cast<const float4 *>(nw + d0)), v = __ldg(reinterpret_cast<const float4 *>(nw + d0) + 1);
            x[0] *= r * u.x, x[1] *= r * u.y, x[2] *= r * u.z, x[3] *= r * u.w;
            x[4] *= r * v.x, x[5] *= r * v.y, x[6] *= r * v.z, x[7] *= r * v.w;
          }
        }
        if (a.half) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner);
          if (turned && kind != 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 c = reinterpret_cast<const float4 *>(cs)[e];
              x[2 * e] = x[2 * e] * c.x + sign * y[2 * e] * c.y;
              x[2 * e + 1] = x[2 * e + 1] * c.z + sign * y[2 * e + 1] * c.w;
            }
          }
        } else if (turned && kind != 2) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float4 c = reinterpret_cast<const float4 *>(cs)[e];
            const float u0 = x[4 * e], v0 = x[4 * e + 1], u1 = x[4 * e + 2], v1 = x[4 * e + 3];
            x[4 * e] = u0 * c.x - v0 * c.y;
            x[4 * e + 1] = u0 * c.y + v0 * c.x;
            x[4 * e + 2] = u1 * c.z - v1 * c.w;
            x[4 * e + 3] = u1 * c.w + v1 * c.z;
          }
        }
        y16 = make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]), pack2<BF16>(x[6], x[7]));
      }
      if (live && (kind == 0 || row >= 0))              // (row < 0: the table has no page for it)
        *(reinterpret_cast<uint4 *>(hd.dst + (kind == 0 ? (int64_t)(t0 + t) : row) * hd.dst_ld) + gl) = y16;
    }
    t = tn, i = in;
  }
}

template <int HD>
cudaError_t launch_hd(const PagedWriteArgs &a, dim3 grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kWThreads;
  cfg.stream = s;
  cfg.dynamicSmemBytes = (a.slots + a.split - 1) / a.split * sizeof(Head);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.bf16)
    return a.in_f32 ? cudaLaunchKernelEx(&cfg, fm_paged_write_kernel<HD, true, true>, a)
                    : cudaLaunchKernelEx(&cfg, fm_paged_write_kernel<HD, true, false>, a);
  return a.in_f32 ? cudaLaunchKernelEx(&cfg, fm_paged_write_kernel<HD, false, true>, a)
                  : cudaLaunchKernelEx(&cfg, fm_paged_write_kernel<HD, false, false>, a);
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteArgs &args, int n_sm, cudaStream_t s) {
  PagedWriteArgs a = args;
  const int rows = kWThreads / (a.hd / 8);          // (token, head) rows a CTA takes at a time
  // Small batches: a token a CTA and its heads over several CTAs, until the SMs have two CTAs each.  Large ones: as many
  // tokens a CTA as still leave eight a SM.
  a.tokens = 1;
  while (a.tokens < kWTokens && (int64_t)a.b.n_tokens / (2 * a.tokens) >= 8ll * n_sm) a.tokens *= 2;
  a.split = 1;
  while (a.slots > rows * a.split && (int64_t)a.b.n_tokens * 2 * a.split <= 2ll * n_sm) a.split *= 2;
  a.split = a.split > (a.slots + kWHeads - 1) / kWHeads ? a.split : (a.slots + kWHeads - 1) / kWHeads;
  const dim3 grid((a.b.n_tokens + a.tokens - 1) / a.tokens, a.split);
  return a.hd == 64 ? launch_hd<64>(a, grid, s) : a.hd == 128 ? launch_hd<128>(a, grid, s) : launch_hd<256>(a, grid, s);
}

}  // namespace fm
