// k_paged_attn256.cu -- attention over a paged cache, head dim 256.
#include "k_paged_attn.cuh"

namespace fm {
template PagedShape paged_attn_shape<256>(int, int);
template cudaError_t paged_attn_call<256>(const PagedAttnArgs &, int, bool, int, cudaStream_t);
}  // namespace fm
