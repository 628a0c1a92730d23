// k_paged_attn128.cu -- attention over a paged cache, head dim 128.
#include "k_paged_attn.cuh"

namespace fm {
template PagedShape paged_attn_shape<128>(int, int);
template cudaError_t paged_attn_call<128>(const PagedAttnArgs &, int, bool, int, cudaStream_t);
}  // namespace fm
