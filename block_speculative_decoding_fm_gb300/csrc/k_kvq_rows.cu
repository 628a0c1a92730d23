// k_kvq_rows.cu -- rows into the 4-bit KV cache and back out.
//
// A group of 32 values x gets the f16 scale d = f16(m / -8), m its value of
// largest magnitude (the negative one on a tie), and codes
// c = clamp(rint(x / d) + 8, 0, 15), ties to even, 8 where d = 0; it stands for
// d (c - 8).  NaN counts as 0, infinities saturate (|d| <= 65504).
//
// The codes are exact without a division.  From 16-bit values: a quotient that is
// not itself halfway between two codes is at least 2^-12 away from there (x a multiple of
// d's last place near a border, d an 11-bit number), so x * (1 / d) + 776, rounded by the
// addition to 2^-14, is halfway exactly where x / d is, whatever the reciprocal's
// rounding, and adding 1.5 * 2^23 then rounds to the code, ties to even, in the sum's low byte.
// From f32 values the remainder x - c d, which is exact, tells whether c is off by one.
// A group with NaN, infinities or a scale at the ends of f16 (rare) takes a slower way: c = rint(x * (1 / d))
// corrected against the borders d (c +- 1/2), exact in f32 (an 11-bit d times a 5-bit odd number).
//
// Bound by memory: a row of n values is read once (2 n or 4 n bytes) and
// written as 0.5625 n bytes.  Two lanes share a group, 16 consecutive values each
// (32-byte loads; the lane's codes are half of the group's 16-byte unit), and a
// thread has all its rows' loads in flight.  (Eight values a lane: the scale's and the
// extremes' instructions weigh twice as much, 100 us for 32768 rows of 2 x 16 heads x 128 f16.)  That many rows take 57 us;
// 262144 rows of 8 KV heads of 128, bf16: 226 us, 6.1 TB/s, and 65536 of them back out 55 us, 6.3 TB/s with what L2
// still holds of the writes; 65536 f32 rows of 4 x 256: 127 us, 4.8 TB/s, each way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "dev_common.cuh"
#include "kvq.h"
#include "kvq_load.cuh"

namespace fm {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 floats(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ float2 floats(__nv_bfloat162 v) { return __bfloat1622float2(v); }

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Sixteen consecutive values of a row.
template <typename T>
struct Sixteen {
  static constexpr int W = sizeof(T) * 4;   // 32-bit words
  uint32_t w[W];
  __device__ __forceinline__ void load(const T *p, bool whole) {   // whole: p is on a 32-byte boundary
#pragma unroll
    for (int i = 0; i < W; i += 8) {
      if (whole) {
        uint32_t v[8];
        ldg256(reinterpret_cast<const uint32_t *>(p) + i, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[i + k] = v[k];
      } else {
        const uint4 u = ldg128(reinterpret_cast<const uint4 *>(p) + i / 4), v = ldg128(reinterpret_cast<const uint4 *>(p) + i / 4 + 1);
        w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
        w[i + 4] = v.x, w[i + 5] = v.y, w[i + 6] = v.z, w[i + 7] = v.w;
      }
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[e]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const float2 f = floats(*reinterpret_cast<const __half2 *>(&w[e / 2]));
      return e & 1 ? f.y : f.x;
    } else {
      return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
  }
  // the largest value and the largest negated one; NaN where a value is
  __device__ __forceinline__ void extremes(float &hi, float &nlo) const {
    if constexpr (sizeof(T) == 4) {
      hi = get(0), nlo = -get(0);
#pragma unroll
      for (int e = 1; e < 16; ++e) hi = max_nan(hi, get(e)), nlo = max_nan(nlo, -get(e));
    } else {
      using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      const P *v = reinterpret_cast<const P *>(w);
      P h = v[0], l = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) h = __hmax2_nan(h, v[i]), l = __hmin2_nan(l, v[i]);
      const float2 hf = floats(h), lf = floats(l);
      hi = max_nan(hf.x, hf.y);
      nlo = max_nan(-lf.x, -lf.y);
    }
  }
};

// Eight consecutive values of a row, rounded once each.
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// the sequence whose tiles hold x (n <= 64 prefix sums)
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

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// the codes of a lane's values of a group with scale d, packed: any values, any scale
template <typename T>
__device__ __noinline__ uint2 codes_any(Sixteen<T> v, float d) {
  const float inv = d == 0.f ? 0.f : 1.f / d, ad = fabsf(d);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float f = v.get(e), x = f == f ? f : 0.f;
    float c = rintf(fminf(fmaxf(x * inv, -9.f), 9.f));
    // the borders of code c, in the units of |d|
    const float xs = d < 0.f ? -x : x, up = ad * (c + 0.5f), dn = ad * (c - 0.5f);
    const bool odd = (static_cast<int>(c) & 1) != 0;
    if (xs > up || (xs == up && odd)) c += 1.f;
    else if (xs < dn || (xs == dn && odd)) c -= 1.f;
    w[e >> 3] |= (uint32_t)(d == 0.f ? 8 : min(15, max(0, static_cast<int>(c) + 8))) << (4 * (e & 7));
  }
  return make_uint2(w[0], w[1]);
}

// the low bytes of four words, in order
__device__ __forceinline__ uint32_t low_bytes(const uint32_t (&t)[4]) {
  return __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
}

// the same for finite values and 0 or 2^-14 <= |d| < 65504 (eight values from e0 on)
template <typename T>
__device__ __forceinline__ uint32_t codes_fast(const Sixteen<T> &v, int e0, float d, float inv) {
  uint32_t even[4], odd[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = v.get(e0 + e);
    float t;
    if constexpr (sizeof(T) == 2) {
      t = fminf(fmaf(x, inv, 776.f), 783.f) + 12582912.f;
    } else {
      constexpr float kMagic = 12582912.f;
      const float c = fmaf(x, inv, kMagic) - kMagic, rem = fmaf(-c, d, x);
      const float half = d == 0.f ? INFINITY : 0.5f * fabsf(d);
      const bool off = fabsf(rem) > half || (fabsf(rem) == half && (__float_as_uint(c + kMagic) & 1u));
      const float step = off ? copysignf(1.f, rem) * copysignf(1.f, d) : 0.f;
      t = fminf(fmaxf(c + step, -8.f), 7.f) + (kMagic + 8.f);
    }
    (e & 1 ? odd : even)[e >> 1] = __float_as_uint(t);
  }
  return low_bytes(even) | low_bytes(odd) << 4;
}

// Grid (touched tile, KV head, K or V); thread = (row, 16 values).
template <int HD, typename T>
__global__ void __launch_bounds__(kThreads) kvq_append_kernel(const __grid_constant__ KvqRowsArgs a) {
  constexpr int O = HD / 16;                    // lanes a row
  constexpr int RP = kThreads / O;              // rows a pass of the block
  constexpr int NP = kKvqTile / RP;
  pdl_trigger();
  const int i = find_seq(a.tile0, a.n, blockIdx.x);
  const int at = a.at[i], rows = a.rows[i];
  const int tile = at / kKvqTile + (blockIdx.x - a.tile0[i]);
  const int head = blockIdx.y;
  const bool isv = blockIdx.z != 0;
  const int o = threadIdx.x % O, r0 = threadIdx.x / O, g = o >> 1;
  const size_t plane = (size_t)a.seq[i] * a.c.n_kv + head;
  uint8_t *half_tile = a.c.planes + plane * a.c.plane_bytes + (size_t)tile * kvq_tile_bytes(HD) + (isv ? kvq_k_bytes(HD) : 0);
  const int first = tile * kKvqTile + r0 - at;   // this thread's first row of the sequence's input
  const T *src = static_cast<const T *>(isv ? a.v : a.k) + (a.row0[i] + first) * a.ld + head * HD + o * 16;
  const bool whole = ((reinterpret_cast<uintptr_t>(isv ? a.v : a.k) | (uintptr_t)(a.ld * sizeof(T))) & 31) == 0;
  pdl_wait();
  Sixteen<T> in[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p)
    if (first + p * RP >= 0 && first + p * RP < rows) in[p].load(src + (int64_t)p * RP * a.ld, whole);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int tr = p * RP + r0;
    const bool ok = first + p * RP >= 0 && first + p * RP < rows;
    float hi = 0.f, nlo = 0.f;
    if (ok) in[p].extremes(hi, nlo);
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
    nlo = max_nan(nlo, __shfl_xor_sync(0xffffffffu, nlo, 1));
    const bool nan = !(hi == hi);
    if (__any_sync(0xffffffffu, nan)) {   // (rare) NaN counts for nothing
      float h = 0.f, l = 0.f;
      if (ok && nan) {
        h = l = -INFINITY;
        for (int e = 0; e < 16; ++e) h = fmaxf(h, in[p].get(e)), l = fmaxf(l, -in[p].get(e));
      }
      h = fmaxf(h, __shfl_xor_sync(0xffffffffu, h, 1));
      l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, 1));
      if (nan) hi = h > -INFINITY ? h : 0.f, nlo = h > -INFINITY ? l : 0.f;
    }
    const float m = hi > nlo ? hi : -nlo;
    const __half dh = __float2half_rn(fminf(fmaxf(m * -0.125f, -65504.f), 65504.f));
    const float d = __half2float(dh), ad = fabsf(d);
    if (!ok) continue;
    uint2 w;
    if (!nan && (ad >= 6.103515625e-05f || ad == 0.f) && ad < 65504.f) {
      const float inv = d == 0.f ? 0.f : rcp(d);
      w = make_uint2(codes_fast(in[p], 0, d, inv), codes_fast(in[p], 8, d, inv));
    } else {
      w = codes_any(in[p], d);
    }
    *reinterpret_cast<uint2 *>(half_tile + kvq_unit(tr, g, HD) + (o & 1) * 8) = w;
    if ((o & 1) == 0) *reinterpret_cast<__half *>(half_tile + kvq_scale(tr, g, HD, isv)) = dh;
    if (!isv && o == 0) a.c.weights[plane * a.c.rows_pad + tile * kKvqTile + tr] = 0.f;
  }
}

// The values the codes stand for, d (c - 8), rounded once to T.
template <int HD, typename T>
__global__ void __launch_bounds__(kThreads) kvq_read_kernel(const __grid_constant__ KvqRowsArgs a) {
  constexpr int O = HD / 8, RP = kThreads / O, NP = kKvqTile / RP;
  pdl_trigger();
  const int i = find_seq(a.tile0, a.n, blockIdx.x);
  const int at = a.at[i], rows = a.rows[i];
  const int tile = at / kKvqTile + (blockIdx.x - a.tile0[i]);
  const int head = blockIdx.y;
  const bool isv = blockIdx.z != 0;
  const int o = threadIdx.x % O, r0 = threadIdx.x / O;
  const size_t plane = (size_t)a.seq[i] * a.c.n_kv + head;
  const uint8_t *half_tile =
      a.c.planes + plane * a.c.plane_bytes + (size_t)tile * kvq_tile_bytes(HD) + (isv ? kvq_k_bytes(HD) : 0);
  T *dst = static_cast<T *>(isv ? a.vo : a.ko);
  pdl_wait();
  if (a.wo && !isv && threadIdx.x < kKvqTile) {
    const int r = tile * kKvqTile + threadIdx.x - at;
    if (r >= 0 && r < rows)
      a.wo[((size_t)(a.call0 + i) * a.c.n_kv + head) * a.ldw + r] =
          a.c.weights[plane * a.c.rows_pad + tile * kKvqTile + threadIdx.x];
  }
  if (!dst) return;
  dst += head * HD + o * 8;
  uint32_t w[NP];
  __half d[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int tr = p * RP + r0;
    w[p] = *reinterpret_cast<const uint32_t *>(half_tile + kvq_unit(tr, o >> 2, HD) + (o & 3) * 4);
    d[p] = *reinterpret_cast<const __half *>(half_tile + kvq_scale(tr, o >> 2, HD, isv));
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = tile * kKvqTile + p * RP + r0 - at;
    if (r < 0 || r >= rows) continue;
    const float f = __half2float(d[p]);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f * static_cast<float>(static_cast<int>((w[p] >> (4 * e)) & 15u) - 8);
    store8(dst + (a.row0[i] + r) * a.ld, x);
  }
}

// weights in: cache rows [0, rows[i]) of each sequence
__global__ void __launch_bounds__(kThreads) kvq_set_weights_kernel(const __grid_constant__ KvqRowsArgs a) {
  pdl_trigger();
  const int i = blockIdx.z, head = blockIdx.y;
  const int r = blockIdx.x * kThreads + threadIdx.x;
  pdl_wait();
  if (r < a.rows[i])
    a.c.weights[((size_t)a.seq[i] * a.c.n_kv + head) * a.c.rows_pad + r] =
        a.wi[((size_t)(a.call0 + i) * a.c.n_kv + head) * a.ldw + r];
}

template <int HD>
cudaError_t append_hd(const KvqRowsArgs &a, dim3 grid, cudaStream_t s) {
  if (a.type == KVQ_F32) return kvq_launch(kvq_append_kernel<HD, float>, grid, dim3(kThreads), 0, s, a);
  if (a.type == KVQ_F16) return kvq_launch(kvq_append_kernel<HD, __half>, grid, dim3(kThreads), 0, s, a);
  return kvq_launch(kvq_append_kernel<HD, __nv_bfloat16>, grid, dim3(kThreads), 0, s, a);
}
template <int HD>
cudaError_t read_hd(const KvqRowsArgs &a, dim3 grid, cudaStream_t s) {
  if (a.type == KVQ_F32) return kvq_launch(kvq_read_kernel<HD, float>, grid, dim3(kThreads), 0, s, a);
  if (a.type == KVQ_F16) return kvq_launch(kvq_read_kernel<HD, __half>, grid, dim3(kThreads), 0, s, a);
  return kvq_launch(kvq_read_kernel<HD, __nv_bfloat16>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kvq_append(const KvqRowsArgs &a, int hd, cudaStream_t s) {
  const dim3 grid(a.tiles, a.c.n_kv, 2);
  return hd == 64 ? append_hd<64>(a, grid, s) : hd == 128 ? append_hd<128>(a, grid, s) : append_hd<256>(a, grid, s);
}

cudaError_t launch_kvq_read(const KvqRowsArgs &a, int hd, cudaStream_t s) {
  const dim3 grid(a.tiles, a.c.n_kv, 2);
  return hd == 64 ? read_hd<64>(a, grid, s) : hd == 128 ? read_hd<128>(a, grid, s) : read_hd<256>(a, grid, s);
}

cudaError_t launch_kvq_set_weights(const KvqRowsArgs &a, cudaStream_t s) {
  int most = 0;
  for (int i = 0; i < a.n; ++i) most = a.rows[i] > most ? a.rows[i] : most;
  if (most == 0) return cudaSuccess;
  return kvq_launch(kvq_set_weights_kernel, dim3((most + kThreads - 1) / kThreads, a.c.n_kv, a.n), dim3(kThreads), 0, s, a);
}

}  // namespace fm
