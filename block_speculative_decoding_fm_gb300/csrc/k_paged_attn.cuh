// k_paged_attn.cuh -- launchers of the paged cache's attention, instantiated in a translation unit a head dim.
#pragma once

#include <atomic>

#include "paged_chunk.cuh"
#include "paged_rows.cuh"

namespace fm {
namespace {

// Shared memory above 48 KB has to be asked for once a device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename K, typename... More>
cudaError_t launch_pdl(K kern, dim3 grid, int threads, int smem, cudaStream_t s, const PagedAttnArgs &a, More... more) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, more...);
}

template <int HD, bool BF16>
cudaError_t rows_call(const PagedAttnArgs &a, int n_sm, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(fm_paged_rows_kernel<HD, BF16>, RowsCfg<HD>::kSmem, done);
  const int ctas = n_sm * RowsCfg<HD>::kCtas;
  if (e == cudaSuccess) e = launch_pdl(fm_paged_rows_kernel<HD, BF16>, dim3(ctas), kRowsThreads, RowsCfg<HD>::kSmem, s, a);
  if (e == cudaSuccess) e = launch_pdl(fm_paged_join_kernel<HD, kRowsUnit, true, BF16, 4>, dim3(n_sm, HD / 64, 1), kJoinThreads, 0, s, a, ctas);
  return e;
}

template <int HD, int NT, bool BF16>
cudaError_t chunk_call(const PagedAttnArgs &a, int n_sm, cudaStream_t s) {
  using C = ChunkCfg<HD, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(fm_paged_chunk_kernel<HD, NT, BF16>, C::kSmem, done);
  if (e == cudaSuccess) e = launch_pdl(fm_paged_chunk_kernel<HD, NT, BF16>, dim3(n_sm), C::kThreads, C::kSmem, s, a);
  if (e == cudaSuccess) e = launch_pdl(fm_paged_join_kernel<HD, 128 * NT, false, BF16, 1>, dim3(n_sm, HD / 64, NT), kJoinThreads, 0, s, a, n_sm);
  return e;
}

}  // namespace

template <int HD>
PagedShape paged_attn_shape(int kind, int n_sm) {
  if (kind == 0) return {kRowsUnit, n_sm * RowsCfg<HD>::kCtas};
  return {128 * (kind == 2 && HD < 256 ? 2 : 1), n_sm};
}

template <int HD>
cudaError_t paged_attn_call(const PagedAttnArgs &a, int kind, bool bf16, int n_sm, cudaStream_t s) {
  if (kind == 0) return bf16 ? rows_call<HD, true>(a, n_sm, s) : rows_call<HD, false>(a, n_sm, s);
  if constexpr (HD < 256)
    if (kind == 2) return bf16 ? chunk_call<HD, 2, true>(a, n_sm, s) : chunk_call<HD, 2, false>(a, n_sm, s);
  return bf16 ? chunk_call<HD, 1, true>(a, n_sm, s) : chunk_call<HD, 1, false>(a, n_sm, s);
}

}  // namespace fm
