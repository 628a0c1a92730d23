// k_paged_attn64.cu -- attention over a paged cache, head dim 64.
#include "k_paged_attn.cuh"

namespace fm {
template PagedShape paged_attn_shape<64>(int, int);
template cudaError_t paged_attn_call<64>(const PagedAttnArgs &, int, bool, int, cudaStream_t);
}  // namespace fm
