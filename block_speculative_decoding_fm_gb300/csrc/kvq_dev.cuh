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

// Eight codes of a word as four f16 pairs, pair p = (code p, code p + 4).  A code
// in the low bits of a f16 is the subnormal code * 2^-24, one digit further up
// code * 2^-20: exact, and one AND a pair (the matrix instructions take
// subnormals as they are).  Pairs 0 and 2 come in units of 2^-24, 1 and 3 of 2^-20.
constexpr float kUnitHi = 0x1p-20f, kUnitLo = 0x1p-24f;
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  h[0] = w & 0x000f000fu;
  h[1] = w & 0x00f000f0u;
  w >>= 8;
  h[2] = w & 0x000f000fu;
  h[3] = w & 0x00f000f0u;
}
// the same less 8, in the same units (exact: multiples of 2^-24)
__device__ __forceinline__ void codes_f16_signed(uint32_t w, uint32_t (&h)[4]) {
  codes_f16(w, h);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t k = p & 1 ? 0x80808080u : 0x80088008u;   // -8 in units of 2^-20, 2^-24
    const __half2 x = __hadd2(*reinterpret_cast<const __half2 *>(&h[p]), *reinterpret_cast<const __half2 *>(&k));
    h[p] = *reinterpret_cast<const uint32_t *>(&x);
  }
}

// D = A B + C with D apart from C (C may be the zero register)
__device__ __forceinline__ void mma_f16_c(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1, float c0, float c1,
                                          float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// two f32 at a time
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
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

// A query tile in shared memory: A fragments of 16 rows (hi, and lo where q is
// split), then per group and row the products' start value, then the rows' factors.
template <int HD, bool QS>
struct QTile {
  static constexpr int kLo = 32 * HD;
  static constexpr int kOff = 32 * HD * (QS ? 2 : 1);    // f32 [group][row % 8][row / 8]
  static constexpr int kMult = kOff + HD / 32 * 16 * 4;  // f32 [row % 8][row / 8]
  static constexpr int kBytes = kMult + 16 * 4;
};

// Query rows [r0, r0 + 16) of a (sequence, KV head) -- row r is block row r /
// group, head r % group of the group -- into A fragments: (group of 32 dims,
// half) -> 32 lanes x 16 bytes.  Inside a group, the k index of the matrix
// product is a permutation of the dims that a word's codes dictate: lane column
// c holds dims 8 c .. 8 c + 7, pair p = dims (p, p + 4) of them; the even pairs' codes
// come in units 16 times smaller, which their queries make up for.  A row is
// scaled by a power of two that brings its largest value to [2^7, 2^8), so q up to
// 2^96 fits f16 (exact for bf16 and f16 inputs down to 2^-22 of the row's
// largest); the row's factor undoes it and carries the softmax scale, whose
// sign goes into the queries.  The codes enter the product unsigned, and the start
// value takes their 8 off: -8 sum q over the group.
// NT threads, all of which call it; the caller synchronises.
template <int HD, bool QS, int NT, typename T>
__device__ __forceinline__ void load_q(const T *q, int64_t ldq, int group, int r0, int R, float scale_log2, uint8_t *tile,
                                       int tid) {
  using QT = QTile<HD, QS>;
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
    const int ex = am > 0.f && am < INFINITY ? min(96, max(-119, static_cast<int>(__float_as_uint(am) >> 23) - 127)) : 7;
    const float up = copysignf(__uint_as_float((uint32_t)(127 + 7 - ex) << 23), scale_log2);
    const int rs = (r & 7) * 2 + (r >> 3);
    if (o == 0)   // (2^20: the products' unit)
      reinterpret_cast<float *>(tile + QT::kMult)[rs] =   // (never 0: a masked score is -inf times it)
          fmaxf(fabsf(scale_log2) * __uint_as_float((uint32_t)(127 + ex - 7 + 20) << 23), 1e-37f);
    const int lane = (r & 7) * 4 + (o & 3), g = o >> 2;
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {   // k halves (p & 1): registers a0 / a1, then a2 / a3 of half p / 2
      const float f = p & 1 ? up : 16.f * up;
      uint8_t *dst = tile + ((g * 2 + (p >> 1)) * 32 + lane) * 16 + (2 * (p & 1) + (r >> 3)) * 4;
      uint32_t hi, lo = 0;
      if constexpr (QS) {
        split2_f16(x[p] * f, x[p + 4] * f, hi, lo);
        *reinterpret_cast<uint32_t *>(dst + QT::kLo) = lo;
      } else {
        const __half2 v = __floats2half2_rn(x[p] * f, x[p + 4] * f);
        hi = *reinterpret_cast<const uint32_t *>(&v);
      }
      *reinterpret_cast<uint32_t *>(dst) = hi;
      const float2 h = pair_f32(hi), l = pair_f32(lo);
      sum += (h.x + h.y + (l.x + l.y)) * (p & 1 ? 1.f : 0.0625f);
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if ((o & 3) == 0) reinterpret_cast<float *>(tile + QT::kOff)[g * 16 + rs] = -8.f * kUnitHi * sum;
  }
}

// Where a lane finds its parts of a 32-row strip, relative to the strip's tile:
// its row's codes (the unit of group g: XOR 16 g) and its rows' scales.
template <int HD>
struct LaneAt {
  uint32_t code, scale;
  __device__ __forceinline__ LaneAt(int r0, int lane)
      : code((uint32_t)kvq_unit(r0 + lane, 0, HD)), scale((uint32_t)kvq_scale(r0 + 2 * (lane & 3), 0, HD)) {}
};
constexpr int kPairStep(int hd) { return hd / 32 * 16; }   // scale bytes of eight rows

// Scores of 16 query rows against the 32 keys of a strip: s[j] is the
// accumulator fragment of keys 8 j .. 8 j + 7 (columns 2 (lane % 4) and + 1; s[j][0] packs
// them for row lane / 4, s[j][1] for row lane / 4 + 8).  Per group of 32 dims the product runs
// over whole codes (exact operands) and the group's scale meets the f32 sum.
template <int HD, bool QS>
__device__ __forceinline__ void strip_scores(uint32_t code, uint32_t scale, uint32_t qt, int lane, uint64_t (&s)[4][2]) {
  using QT = QTile<HD, QS>;
  constexpr int G = Dim<HD>::G, GB = Dim<HD>::GB;
#pragma unroll
  for (int g0 = 0; g0 < G; g0 += GB) {
    uint32_t sc[4][GB];
#pragma unroll
    for (int j = 0; j < 4; ++j) lds_words<GB>(scale + j * kPairStep(HD) + g0 * 4, sc[j]);
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const int g = g0 + gi;
      uint32_t w[4], h[4][4];
      ldsm_x4(code ^ (g << 4), w);
      const uint2 off = lds64(qt + QT::kOff + g * 64 + (lane >> 2) * 8);
      const float o0 = __uint_as_float(off.x), o1 = __uint_as_float(off.y);
#pragma unroll
      for (int j = 0; j < 4; ++j) codes_f16(w[j], h[j]);
      float acc[4][4];
      const uint4 a0 = lds128(qt + (g * 64 + lane) * 16), a1 = lds128(qt + (g * 64 + 32 + lane) * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_f16_c(acc[j], a0, h[j][0], h[j][1], o0, o0, o1, o1);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_f16(acc[j], a1.x, a1.y, a1.z, a1.w, h[j][2], h[j][3]);
      if constexpr (QS) {
        const uint4 l0 = lds128(qt + QT::kLo + (g * 64 + lane) * 16), l1 = lds128(qt + QT::kLo + (g * 64 + 32 + lane) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16(acc[j], l0.x, l0.y, l0.z, l0.w, h[j][0], h[j][1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16(acc[j], l1.x, l1.y, l1.z, l1.w, h[j][2], h[j][3]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 d = pair_f32(sc[j][gi]);
        const uint64_t dd = pack2(d.x, d.y);
        if (g == 0) {
          s[j][0] = mul2(pack2(acc[j][0], acc[j][1]), dd);
          s[j][1] = mul2(pack2(acc[j][2], acc[j][3]), dd);
        } else {
          s[j][0] = fma2(pack2(acc[j][0], acc[j][1]), dd, s[j][0]);
          s[j][1] = fma2(pack2(acc[j][2], acc[j][3]), dd, s[j][1]);
        }
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
// accumulators of the dims 32 g + 4 n + i (n the fragment's column), in the code
// pairs' units (i even 2^-24, odd 2^-20).  The V scale of (key, group) goes into P:
// P' = p d rounded to f16 once more (PS: split into hi + lo, which keeps ~22 bits).
// SV: the codes enter with their 8 taken off; else unsigned, and column g of cor
// collects the sum of P' over the keys for group g (a product with a column of
// ones), which the end takes off eight times.
template <int HD, bool PS, bool SV>
__device__ __forceinline__ void strip_pv(uint32_t code, uint32_t scale, int lane, const PRange<PS> &range,
                                         const float (&p)[4][4], float (&o)[HD / 8][4], float (&cor)[4]) {
  constexpr int G = Dim<HD>::G, GB = Dim<HD>::GB;
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
    for (int j = 0; j < 4; ++j) lds_words<GB>(scale + j * kPairStep(HD) + g0 * 4, sc[j]);
    if (!PS && range.shifted) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int gi = 0; gi < GB; ++gi) {
          const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&sc[j][gi]), range.up);
          sc[j][gi] = *reinterpret_cast<const uint32_t *>(&x);
        }
    }
#pragma unroll
    for (int gi = 0; gi < GB; ++gi) {
      const int g = g0 + gi;
      uint32_t w[4], h[4][4];
      ldsm_x4_trans(code ^ (g << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (SV)
          codes_f16_signed(w[j], h[j]);
        else
          codes_f16(w[j], h[j]);
      }
      const uint32_t one = (lane >> 2) == g ? 0x3c003c00u : 0u;
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
        if constexpr (!SV) {
          mma_f16(cor, a[0], a[1], a[2], a[3], one, one);
          if constexpr (PS) mma_f16(cor, l[0], l[1], l[2], l[3], one, one);
        }
      }
    }
  }
}

// The accumulators in the values' own unit: less 8 times the sum of P', times f0 / f1 (rows lane / 4 and + 8).
template <int HD, bool SV>
__device__ __forceinline__ void finish_o(float (&o)[HD / 8][4], const float (&cor)[4], int lane, float f0, float f1) {
#pragma unroll
  for (int g = 0; g < HD / 32; ++g) {
    float c0 = 0.f, c1 = 0.f;
    if constexpr (!SV) {
      const int from = (lane & ~3) | (g >> 1);
      c0 = 8.f * __shfl_sync(0xffffffffu, cor[g & 1], from);
      c1 = 8.f * __shfl_sync(0xffffffffu, cor[2 + (g & 1)], from);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = i & 1 ? 1.f / kUnitHi : 1.f / kUnitLo;
      float(&x)[4] = o[4 * g + i];
      x[0] = fmaf(x[0], u, -c0) * f0;
      x[1] = fmaf(x[1], u, -c0) * f0;
      x[2] = fmaf(x[2], u, -c1) * f1;
      x[3] = fmaf(x[3], u, -c1) * f1;
    }
  }
}

template <typename I>
__device__ __forceinline__ int find_seq(const I *pre, int n, I x) {
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
