// kvq_dev.cuh -- device parts of the 4-bit KV cache's attention kernels: the
// query fragments, a strip's scores, the codes' way into f16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dev_common.cuh"
#include "kvq.h"

namespace fm {
namespace kvq {

template <int HD>
struct Dim {
  static constexpr int G = HD / 32;            // groups a row
  static constexpr int GB = G < 4 ? G : 4;     // groups whose scales one shared load fetches
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// ldmatrix x4: four 8 x 16-byte matrices, lane i supplies row i's address
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Eight codes of a word as four f16 pairs (c - 8), pair p = (code p, code p + 4):
// a code put into the low bits of 1024 is the f16 1024 + c (or 1024 + 16 c one
// digit up), and both ways back are exact.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  const __half2 k1032 = __float2half2_rn(1032.f), k16 = __float2half2_rn(0.0625f), k72 = __float2half2_rn(-72.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo = (w & 0x000f000fu) | 0x64006400u, hi = (w & 0x00f000f0u) | 0x64006400u;
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), k1032);
    const __half2 b = __hfma2(*reinterpret_cast<const __half2 *>(&hi), k16, k72);
    h[2 * i] = *reinterpret_cast<const uint32_t *>(&a);
    h[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&b);
    w >>= 8;
  }
}

__device__ __forceinline__ float2 pair_f32(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// GB consecutive 32-bit words from shared memory
template <int GB>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[GB]) {
  if constexpr (GB == 4) {
    const uint4 v = lds128(addr);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = lds64(addr);
    w[0] = v.x, w[1] = v.y;
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = word(v, i);
      if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
        const float2 f = pair_f32(w);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      } else {
        x[2 * i] = __uint_as_float(w << 16), x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
}

// bytes of a query tile's fragments: 16 rows of HD f16 (twice where q is split into hi + lo)
template <int HD, bool QS>
constexpr int q_bytes() {
  return 32 * HD * (QS ? 2 : 1);
}

// Query rows [r0, r0 + 16) of a (sequence, KV head) -- row r is block row r /
// group, head r % group of the group -- into A fragments in shared memory:
// (group of 32 dims, half) -> 32 lanes x 16 bytes.  Inside a group, the k index
// of the matrix product is a permutation of the dims that a word's codes
// dictate: lane column c holds dims 8 c .. 8 c + 7, pair p = dims (p, p + 4) of
// them.  A row is scaled by a power of two that brings its largest value to
// [2^7, 2^8), so any finite q fits f16 (exact for bf16 and f16 inputs down to
// 2^-22 of the row's largest); mult[row] undoes it and carries the softmax scale.
// NT threads, all of which call it; the caller synchronises.
template <int HD, bool QS, int NT, typename T>
__device__ __forceinline__ void load_q(const T *q, int64_t ldq, int group, int r0, int R, float scale_log2, uint8_t *frag,
                                       float *mult, int tid) {
  constexpr int O = HD / 8;
#pragma unroll
  for (int it = tid; it < 16 * O; it += NT) {
    const int r = it / O, o = it % O;
    const int row = r0 + r;
    float x[8];
    if (row < R) {
      const int t = row / group;
      load8(q + (int64_t)t * ldq + (row - t * group) * HD + o * 8, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    float am = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(x[e]));
#pragma unroll
    for (int s = 1; s < O; s <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, s));
    // am in [2^ex, 2^(ex + 1)); the factor 2^(7 - ex), its exponent kept in f32's normal range
    const int ex = am > 0.f && am < INFINITY ? min(126, max(-119, static_cast<int>(__float_as_uint(am) >> 23) - 127)) : 7;
    const float up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23), down = __uint_as_float((uint32_t)(127 + ex - 7) << 23);
    if (o == 0) mult[r] = scale_log2 * down;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= up;
    const int lane = (r & 7) * 4 + (o & 3), g = o >> 2;
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // k halves: registers a0 / a1 then a2 / a3
        const int p = 2 * st + h;
        uint8_t *dst = frag + ((g * 2 + st) * 32 + lane) * 16 + (2 * h + (r >> 3)) * 4;
        if constexpr (QS) {
          uint32_t hi, lo;
          split2_f16(x[p], x[p + 4], hi, lo);
          *reinterpret_cast<uint32_t *>(dst) = hi;
          *reinterpret_cast<uint32_t *>(dst + 32 * HD) = lo;
        } else {
          const __half2 v = __floats2half2_rn(x[p], x[p + 4]);
          *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<const uint32_t *>(&v);
        }
      }
  }
}

// Scores of 16 query rows against the 32 keys of a strip (rows r0 .. r0 + 31 of
// a tile whose K half is at kb): s[j][..] is the accumulator fragment of keys
// 8 j .. 8 j + 7 (rows lane / 4 and + 8, keys 2 (lane % 4) and + 1).  Per group of 32
// dims the product runs over whole codes (exact operands) and the group's scale
// meets the f32 sum.
template <int HD, bool QS>
__device__ __forceinline__ void strip_scores(uint32_t kb, int r0, uint32_t qf, int lane, float (&s)[4][4]) {
  constexpr int G = Dim<HD>::G, GB = Dim<HD>::GB;
  const int c = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
  for (int g0 = 0; g0 < G; g0 += GB) {
    uint32_t sc[4][GB];
#pragma unroll
    for (int j = 0; j < 4; ++j) lds_words<GB>(kb + kvq_scale(r0 + 8 * j + 2 * c, g0, HD), sc[j]);
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const int g = g0 + gi;
      uint32_t w[4], h[4][4];
      ldsm_x4(kb + kvq_unit(r0 + lane, g, HD), w);
#pragma unroll
      for (int j = 0; j < 4; ++j) codes_f16(w[j], h[j]);
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint4 a = lds128(qf + ((g * 2 + st) * 32 + lane) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16(acc[j], a.x, a.y, a.z, a.w, h[j][2 * st], h[j][2 * st + 1]);
        if constexpr (QS) {
          const uint4 l = lds128(qf + 32 * HD + ((g * 2 + st) * 32 + lane) * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(acc[j], l.x, l.y, l.z, l.w, h[j][2 * st], h[j][2 * st + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 d = pair_f32(sc[j][gi]);
        s[j][0] = fmaf(acc[j][0], d.x, s[j][0]);
        s[j][1] = fmaf(acc[j][1], d.y, s[j][1]);
        s[j][2] = fmaf(acc[j][2], d.x, s[j][2]);
        s[j][3] = fmaf(acc[j][3], d.y, s[j][3]);
      }
    }
  }
}

// How P' = p d is brought into f16's range: p carries 2^bias (the sums too, so
// it leaves with the division), d carries 2^shift.  p <= 2^8 (the reference moves
// late) and d <= vmax < 2^e, so that P' < 2^15 with bias = 7 - e - shift.  Split P' is
// formed in f32 and takes the whole factor in p; once-rounded P' has p in f16 as
// well (bias <= 7), and small scales are raised themselves (exactly: f16 times a power of two).
template <bool PS>
struct PRange {
  float bias, undo;      // undo: 2^-shift
  __half2 up;            // 2^shift
  bool shifted;
  __device__ __forceinline__ explicit PRange(uint32_t vmax_bits) {
    const int e = max(-32, static_cast<int>(vmax_bits >> 23) - 126);
    const int shift = PS || e >= -6 ? 0 : min(-e, 15);
    shifted = shift > 0;
    bias = static_cast<float>(PS ? 7 - e : 7 - max(e + shift, 0));
    undo = __uint_as_float((uint32_t)(127 - shift) << 23);
    up = __float2half2_rn(__uint_as_float((uint32_t)(127 + shift) << 23));
  }
};

// O += P V over a strip: p as strip_scores' fragments, o[4 g + i] the
// accumulators of the dims 32 g + 4 n + i (n the fragment's column).  The V
// scale of (key, group) goes into P: P' = p d rounded to f16 once more (PS: split
// into hi + lo, which keeps ~22 bits), and V enters as whole codes.
template <int HD, bool PS>
__device__ __forceinline__ void strip_pv(uint32_t vb, int r0, int lane, const PRange<PS> &range, const float (&p)[4][4],
                                         float (&o)[HD / 8][4]) {
  constexpr int G = Dim<HD>::G, GB = Dim<HD>::GB;
  const int c = lane & 3;
  __half2 ph[4][2];
  if constexpr (!PS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ph[j][0] = __floats2half2_rn(p[j][0], p[j][1]);
      ph[j][1] = __floats2half2_rn(p[j][2], p[j][3]);
    }
  }
#pragma unroll
  for (int g0 = 0; g0 < G; g0 += GB) {
    uint32_t sc[4][GB];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lds_words<GB>(vb + kvq_scale(r0 + 8 * j + 2 * c, g0, HD), sc[j]);
      if (!PS && range.shifted) {
#pragma unroll
        for (int gi = 0; gi < GB; ++gi) {
          const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&sc[j][gi]), range.up);
          sc[j][gi] = *reinterpret_cast<const uint32_t *>(&x);
        }
      }
    }
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const int g = g0 + gi;
      uint32_t w[4], h[4][4];
      ldsm_x4_trans(vb + kvq_unit(r0 + lane, g, HD), w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) codes_f16(w[j], h[j]);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t a[4], l[4];
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {   // keys 16 st + 8 h2 ..
          const int j = 2 * st + h2;
          if constexpr (PS) {
            const float2 d = pair_f32(sc[j][gi]);
            split2_f16(p[j][0] * d.x, p[j][1] * d.y, a[2 * h2], l[2 * h2]);
            split2_f16(p[j][2] * d.x, p[j][3] * d.y, a[2 * h2 + 1], l[2 * h2 + 1]);
          } else {
            const __half2 d = *reinterpret_cast<const __half2 *>(&sc[j][gi]);
            const __half2 x = __hmul2(ph[j][0], d), y = __hmul2(ph[j][1], d);
            a[2 * h2] = *reinterpret_cast<const uint32_t *>(&x);
            a[2 * h2 + 1] = *reinterpret_cast<const uint32_t *>(&y);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_f16(o[4 * g + i], a[0], a[1], a[2], a[3], h[2 * st][i], h[2 * st + 1][i]);
          if constexpr (PS) mma_f16(o[4 * g + i], l[0], l[1], l[2], l[3], h[2 * st][i], h[2 * st + 1][i]);
        }
      }
    }
  }
}

__device__ __forceinline__ int find_seq(const int32_t *pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

}  // namespace kvq
}  // namespace fm
