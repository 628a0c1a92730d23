// kvq_dev.cuh -- device parts of the 4-bit KV cache's attention kernels: the
// query fragments, a strip's scores, the codes' way into f16.
//
// The products run with the cache as the matrix instructions' first operand:
// S^T = K Q^T over 16 keys at a time and O^T += V^T P^T over 16 dims, with 8 query
// rows a step on the other side, so that few query rows cost few products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "dev_common.cuh"
#include "kvq.h"
#include "kvq_load.cuh"

namespace fm {
namespace kvq {

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
// What that costs is precision: the matrix instructions align their products by the
// operands' exponents, which a subnormal has at 2^-14, so a sum keeps some 2^-17 of its
// largest term (measured: f32 outputs 1e-5 off, 3e-7 to 7e-7 with normal operands).
// f16 and bf16 outputs, rounded to 2^-12 and 2^-9, do not see it, not even with one channel that
// gives every score 100 to 1000: 2.2e-4 and 1.7e-3 off with either operand, as a plain f32 form.
constexpr float kUnitHi = 0x1p-20f, kUnitLo = 0x1p-24f;
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  h[0] = w & 0x000f000fu;
  h[1] = w & 0x00f000f0u;
  w >>= 8;
  h[2] = w & 0x000f000fu;
  h[3] = w & 0x00f000f0u;
}
// The same less 8, as whole numbers, for f32 outputs and for the weights: 1024 + code and 1024 + 16 code by
// one AND-OR, then one exact addition or multiply-add a pair.
__device__ __forceinline__ void codes_f16_signed(uint32_t w, uint32_t (&h)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t x = ((p < 2 ? w : w >> 8) & (p & 1 ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
    const __half2 y = *reinterpret_cast<const __half2 *>(&x);
    const __half2 z = p & 1 ? __hfma2(y, __float2half2_rn(0.0625f), __float2half2_rn(-72.f)) : __hadd2(y, __float2half2_rn(-1032.f));
    h[p] = *reinterpret_cast<const uint32_t *>(&z);
  }
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

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = ldg128f(reinterpret_cast<const float *>(p)), b = ldg128f(reinterpret_cast<const float *>(p) + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = ldg128(p);
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

// What a kernel instance carries: NQ x 8 query rows, strips of KS keys a warp.
template <int HD, typename T, int NQ_>
struct Kind {
  static constexpr int NQ = NQ_, RT = 8 * NQ, G = HD / 32;
  static constexpr bool QS = sizeof(T) == 4;                          // f32 queries: f16 hi + lo
  // P' = p d in f16: rounded twice (p, then the product), which bf16 outputs do not see; once (f16 outputs, whose own
  // rounding is as large); or split into hi + lo (f32 outputs)
  static constexpr int PS = sizeof(T) == 4 ? 2 : std::is_same<T, __half>::value ? 1 : 0;
  static constexpr bool SV = sizeof(T) == 4;                          // f32 outputs: signed V codes (no sums to take off)
  static constexpr int KS = 16 * kvq_stage_tiles(HD), MT = KS / 16;   // a strip, in 16-key products
};

// D = A B + C with D apart from C
__device__ __forceinline__ void mma_f16_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1, const uint4 &c) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c.x), "r"(c.y), "r"(c.z), "r"(c.w));
}

// A query tile in shared memory: B fragments of the group's dims (hi, and lo
// where q is split), the products' start values, the rows' factors.
template <int HD, bool QS, int NQ>
struct QTile {
  static constexpr int kLo = HD * NQ * 16;                      // [group][row / 8][lane] 16 bytes
  static constexpr int kOff = kLo * (QS ? 2 : 1);               // f32 [group][row / 2][the pair, twice] (an accumulator fragment)
  static constexpr int kMult = kOff + HD / 32 * NQ * 8 * 8;     // f32 [row]
  static constexpr int kBytes = kMult + NQ * 8 * 4;
};

// Query rows [r0, r0 + 8 NQ) of a (sequence, KV head) -- row r is block row r /
// group, head r % group of the group -- into B fragments.  Inside a group of 32
// dims the k index of the matrix product is a permutation of the dims that a
// word's codes dictate: lane column c holds dims 8 c .. 8 c + 7, pair p = dims (p, p + 4) of
// them; the even pairs' unsigned codes come in units 16 times smaller, which their
// queries make up for.  A row is scaled by a power of two that brings its
// largest value to [2^7, 2^8), so q up to 2^96 fits f16 (exact for bf16 and f16
// inputs down to 2^-22 of the row's largest); the row's factor undoes it and
// carries the softmax scale, whose sign goes into the queries.  Unless SK the codes enter
// the product unsigned, and the start value takes their 8 off: -8 sum q over the group.
// NT threads, all of which call it; the caller synchronises.
template <int HD, bool QS, bool SK, int NQ, int NT, typename T>
__device__ __forceinline__ void load_q(const T *q, int64_t ldq, int group, int r0, int R, float scale_log2, uint8_t *tile,
                                       int tid) {
  static_assert(!QS || SK, "split queries meet signed codes: the start value has no low part");
  using QT = QTile<HD, QS, NQ>;
  constexpr int O = HD / 8;
  // (the loads of two rounds in flight together)
  constexpr int kItems = 8 * NQ * O, IP = (kItems + NT - 1) / NT, IB = IP < 2 ? 1 : 2;
#pragma unroll 1
  for (int i0 = 0; i0 < IP; i0 += IB) {
    float xs[IB][8];
#pragma unroll
    for (int b = 0; b < IB; ++b) {
      const int it = (i0 + b) * NT + tid, row = r0 + it / O;
      if (it < kItems && row < R) {
        const int t = row / group;
        load8(q + (int64_t)t * ldq + (row - t * group) * HD + it % O * 8, xs[b]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) xs[b][e] = 0.f;
      }
    }
#pragma unroll
    for (int b = 0; b < IB; ++b) {
      const int it = (i0 + b) * NT + tid;
      if (it >= kItems) break;   // (whole warps)
      const int r = it / O, o = it % O;
      float(&x)[8] = xs[b];
      float am = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(x[e]));
#pragma unroll
      for (int s = 1; s < O; s <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, s));
      // am in [2^ex, 2^(ex + 1)); the factor 2^(7 - ex), its exponent kept in f32's normal range
      const int ex = am > 0.f && am < INFINITY ? min(96, max(-119, static_cast<int>(__float_as_uint(am) >> 23) - 127)) : 7;
      const float up = copysignf(__uint_as_float((uint32_t)(127 + 7 - ex) << 23), scale_log2);
      if (o == 0)   // (2^20: the unsigned codes' unit; never 0: a masked score is -inf times it)
        reinterpret_cast<float *>(tile + QT::kMult)[r] =
            fmaxf(fabsf(scale_log2) * __uint_as_float((uint32_t)(127 + ex - 7 + (SK ? 0 : 20)) << 23), 1e-37f);
      const int g = o >> 2, at = ((g * NQ + (r >> 3)) * 32 + (r & 7) * 4 + (o & 3)) * 16;
      float sum = 0.f;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float f = SK || p & 1 ? up : 16.f * up;
        if constexpr (QS) {
          split2_f16(x[p] * f, x[p + 4] * f, hi[p], lo[p]);
        } else {
          const __half2 v = __floats2half2_rn(x[p] * f, x[p + 4] * f);
          hi[p] = *reinterpret_cast<const uint32_t *>(&v);
          lo[p] = 0;
        }
        if constexpr (!SK) {
          const float2 h = pair_f32(hi[p]);
          sum += (h.x + h.y) * (p & 1 ? 1.f : 0.0625f);
        }
      }
      *reinterpret_cast<uint4 *>(tile + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if constexpr (QS) *reinterpret_cast<uint4 *>(tile + QT::kLo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if constexpr (!SK) {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if ((o & 3) == 0) {
          float *off = reinterpret_cast<float *>(tile + QT::kOff) + (g * NQ * 4 + (r >> 1)) * 4 + (r & 1);
          off[0] = off[2] = -8.f * kUnitHi * sum;
        }
      }
    }
  }
}

// Where a lane finds its part of a strip of KS rows from r0 on, relative to the
// tile: the codes that it addresses for ldmatrix (unit of group g: XOR 16 g; a
// strip of 16 rows takes two groups a fetch) and the scales of its rows.
template <int HD, int KS>
struct LaneAt {
  uint32_t code, scale;
  __device__ __forceinline__ LaneAt(int r0, int lane)
      : code((uint32_t)(KS == 32 ? kvq_unit(r0 + lane, 0, HD) : kvq_unit(r0 + (lane & 15), lane >> 4, HD))),
        scale((uint32_t)kvq_kscale(r0 + (lane >> 2), 0, HD)) {}
};

// a row's K scales of 4 groups (2 for head dim 64) as f32
template <int GB>
__device__ __forceinline__ void row_scales(uint32_t addr, float (&d)[GB]) {
  if constexpr (GB == 4) {
    const uint2 v = lds64(addr);
    const float2 a = pair_f32(v.x), b = pair_f32(v.y);
    d[0] = a.x, d[1] = a.y, d[2] = b.x, d[3] = b.y;
  } else {
    const float2 a = pair_f32(lds32(addr));
    d[0] = a.x, d[1] = a.y;
  }
}

// Scores of 8 NQ query rows against the KS keys of a strip: s[m][n] is the
// accumulator fragment of keys 16 m + lane / 4 (first pair) and + 8 (second), query rows
// 8 n + 2 (lane % 4) and + 1.  Per group of 32 dims the product runs over whole codes
// (exact operands) and the row's scale meets the f32 sum.  SK: the codes less 8.
template <int HD, bool QS, bool SK, int NQ, int KS>
__device__ __forceinline__ void strip_scores(uint32_t code, uint32_t scale, uint32_t qt, int lane,
                                             uint64_t (&s)[KS / 16][NQ][2]) {
  using QT = QTile<HD, QS, NQ>;
  constexpr int G = HD / 32, GB = G < 4 ? G : 4, MT = KS / 16, GF = 2 / MT;   // GF groups a fetch
#pragma unroll
  for (int g0 = 0; g0 < G; g0 += GB) {
    float d[MT][2][GB];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) row_scales<GB>(scale + (16 * m + 8 * h) * (G * 2) + g0 * 2, d[m][h]);
#pragma unroll
    for (int gi = 0; gi < GB; gi += GF) {
      uint32_t w[4];
      ldsm_x4(code ^ ((g0 + gi) << 4), w);
#pragma unroll
      for (int f = 0; f < GF; ++f) {
        const int g = g0 + gi + f;
        uint32_t h[2 * MT][4];
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) {
          if constexpr (SK)
            codes_f16_signed(w[2 * f * (GF - 1) + j], h[j]);
          else
            codes_f16(w[2 * f * (GF - 1) + j], h[j]);
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const uint4 off = SK ? make_uint4(0, 0, 0, 0) : lds128(qt + QT::kOff + (g * NQ + n) * 64 + (lane & 3) * 16);
          const uint4 b = lds128(qt + ((g * NQ + n) * 32 + lane) * 16);
          float acc[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
            mma_f16_c(acc[m], h[2 * m][0], h[2 * m + 1][0], h[2 * m][1], h[2 * m + 1][1], b.x, b.y, off);
#pragma unroll
          for (int m = 0; m < MT; ++m) mma_f16(acc[m], h[2 * m][2], h[2 * m + 1][2], h[2 * m][3], h[2 * m + 1][3], b.z, b.w);
          if constexpr (QS) {
            const uint4 l = lds128(qt + QT::kLo + ((g * NQ + n) * 32 + lane) * 16);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_f16(acc[m], h[2 * m][0], h[2 * m + 1][0], h[2 * m][1], h[2 * m + 1][1], l.x, l.y);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_f16(acc[m], h[2 * m][2], h[2 * m + 1][2], h[2 * m][3], h[2 * m + 1][3], l.z, l.w);
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t dd = pack2(d[m][e][gi + f], d[m][e][gi + f]), x = pack2(acc[m][2 * e], acc[m][2 * e + 1]);
              s[m][n][e] = g == 0 ? mul2(x, dd) : fma2(x, dd, s[m][n][e]);
            }
        }
      }
    }
  }
}

// P of a stage of four strips in shared memory as f16, by query row: a row's keys
// together, 16 bytes of padding (eight rows' 16-byte pieces in eight bank groups);
// PS > 0: then what the rounding left of p, in f16 too.
template <int NQ, int PS, int KS>
struct PTile {
  static constexpr int kRow = 4 * KS * 2 + 16;
  static constexpr int kLo = 8 * NQ * kRow;
  static constexpr int kBytes = kLo * (PS ? 2 : 1);
};
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}
__device__ __forceinline__ void stsm_x2_trans(uint32_t addr, uint32_t r0, uint32_t r1) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1,%2};\n" ::"r"(addr), "r"(r0), "r"(r1) : "memory");
}
// this warp's strip (fragments as strip_scores') into columns key0 .. of the tile
template <int NQ, int PS, int KS>
__device__ __forceinline__ void put_p(uint32_t tile, int key0, int lane, const float (&p)[KS / 16][NQ][4]) {
  using PT = PTile<NQ, PS, KS>;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    uint32_t r[KS / 8], l[KS / 8];
#pragma unroll
    for (int m = 0; m < KS / 16; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (PS) {
          split2_f16(p[m][n][2 * e], p[m][n][2 * e + 1], r[2 * m + e], l[2 * m + e]);
        } else {
          const __half2 v = __floats2half2_rn(p[m][n][2 * e], p[m][n][2 * e + 1]);
          r[2 * m + e] = *reinterpret_cast<const uint32_t *>(&v);
        }
      }
    const uint32_t at = tile + (8 * n + (lane & 7)) * PT::kRow + key0 * 2 + (KS == 32 ? lane >> 3 : (lane >> 3) & 1) * 16;
    if constexpr (KS == 32) {
      stsm_x4_trans(at, r[0], r[1], r[2], r[3]);
      if constexpr (PS) stsm_x4_trans(at + PT::kLo, l[0], l[1], l[2], l[3]);
    } else {
      stsm_x2_trans(at, r[0], r[1]);
      if constexpr (PS) stsm_x2_trans(at + PT::kLo, l[0], l[1]);
    }
  }
}

// How P' = p d is brought into f16's range: p carries 2^7 (the sums too, so it leaves
// with the division) and is at most 2^15, as the reference moves when a score beats it
// by 2^8; d carries 2^shift with |d| 2^shift < 2, so P' < 2^16.  Every warp has a shift of
// its own for the scales it multiplies, which begins at 15 and goes down where a scale
// of a row in view asks for it (what the warp holds is brought to the new one): 0 while the
// largest scale is 2^-7 to 2, so that ordinary rows need no multiplication.  Raising a
// scale is exact.  A shift below 0 is halved between d and p, so that neither leaves f16's
// normal range for it while d is 2^-7 at least and p 2^-13; P' keeps 2^-25 of its largest.
constexpr float kBias = 7.f;
// |d| from here on asks for a lower shift (f16 bits of 2^(1 - shift); infinity, which no scale is, for -15)
__device__ __forceinline__ uint32_t shift_limit(int shift) { return (uint32_t)(16 - shift) << 10; }
// the shift that the scale `bits`, at or over the limit, asks for: it lies in [2^(e - 1), 2^e)
__device__ __forceinline__ int shift_for(uint32_t bits) {
  const int e = static_cast<int>(bits >> 10) - 14;
  return e > 1 ? max(-e, -15) : e >= -6 ? 0 : -e;
}
__device__ __forceinline__ __half2 shift_factor(int shift) {
  const uint32_t h = shift > -15 ? (uint32_t)(15 + shift) << 10 : 0x200u;   // (2^-15 is a subnormal)
  const uint32_t w = h * 0x10001u;
  return *reinterpret_cast<const __half2 *>(&w);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ __half2 h2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// O^T += V^T P^T over 32 rows of a tile (code: where the lane fetches their unit of group 0), group g:
// o[t][n] are the accumulators of dims 32 g + 4 (lane / 4) + t (first pair) and + 2 (second), query
// rows 8 n + 2 (lane % 4) and + 1, in the code pairs' units (t = 0: 2^-24, t = 1: 2^-20; SV: 1).
// sc: the V scales of the rows' pairs (kvq_vscale's order).  P' = p d is rounded to
// f16 (PS 1: p's rest joins the product before its only rounding; PS 2: hi + lo, ~22 bits).  SV: the codes enter
// with their 8 taken off; else unsigned, and cor collects the sums of P', which the
// end takes off eight times: a product with ones whose first operand is an octet's P'
// fragments as they are, so that row lane / 4 sums the keys of the first and third
// eight for query row lane / 4 of the octet, and row lane / 4 + 8 the others.
// Low: p is lowered by the factor `low` first (the scales' shift is below 0).
template <int HD, int PS, bool SV, bool Low, int NQ, int KS>
__device__ __forceinline__ void tile_pv(uint32_t code, int g, const uint32_t (&sc)[4], __half2 low, uint32_t pt, int key0, int lane,
                                        float (&o)[2][NQ][4], float (&cor)[NQ][4]) {
  static_assert(PS != 2 || SV, "the sums that unsigned codes need have no second part");
  using PT = PTile<NQ, PS, KS>;
  uint32_t w[4], h[4][4];
  ldsm_x4_trans(code ^ (g << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (SV)
      codes_f16_signed(w[j], h[j]);
    else
      codes_f16(w[j], h[j]);
  }
  uint32_t b[NQ][4], l[NQ][4];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const uint32_t at = pt + (8 * n + (lane & 7)) * PT::kRow + (key0 + (lane >> 3) * 8) * 2;
    ldsm_x4(at, b[n]);
    if constexpr (PS) ldsm_x4(at + PT::kLo, l[n]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (Low) {
        b[n][j] = u32(__hmul2(h2(b[n][j]), low));
        if constexpr (PS) l[n][j] = u32(__hmul2(h2(l[n][j]), low));
      }
      const __half2 p = h2(b[n][j]), d = h2(sc[j]);
      if constexpr (PS == 0) {
        b[n][j] = u32(__hmul2(p, d));
      } else if constexpr (PS == 1) {
        b[n][j] = u32(__hfma2(p, d, __hmul2(h2(l[n][j]), d)));
      } else {   // (the product's rest is exact)
        const __half2 x = __hmul2(p, d);
        b[n][j] = u32(x);
        l[n][j] = u32(__hfma2(h2(l[n][j]), d, __hfma2(p, d, __hneg2(x))));
      }
    }
    if constexpr (PS == 2) {
      // (a sum of its own over the 32 rows: the matrix instructions cut their sums off, which over a long cache adds up:
      // 32768 rows 2.2e-6 off, 3e-7 this way, at 2 % of the time)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float acc[4];
        mma_f16_c(acc, h[0][t], h[0][t + 2], h[1][t], h[1][t + 2], l[n][0], l[n][1], make_uint4(0, 0, 0, 0));
        mma_f16(acc, h[2][t], h[2][t + 2], h[3][t], h[3][t + 2], l[n][2], l[n][3]);
        mma_f16(acc, h[0][t], h[0][t + 2], h[1][t], h[1][t + 2], b[n][0], b[n][1]);
        mma_f16(acc, h[2][t], h[2][t + 2], h[3][t], h[3][t + 2], b[n][2], b[n][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][n][e] += acc[e];
      }
    } else {
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          mma_f16(o[t][n], h[2 * st][t], h[2 * st][t + 2], h[2 * st + 1][t], h[2 * st + 1][t + 2], b[n][2 * st], b[n][2 * st + 1]);
    }
    if constexpr (!SV) {
      constexpr uint32_t kOnes = 0x3c003c00u;
      mma_f16(cor[n], b[n][0], b[n][1], b[n][2], b[n][3], kOnes, kOnes);
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
