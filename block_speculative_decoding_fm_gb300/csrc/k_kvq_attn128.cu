// k_kvq_attn128.cu -- kvq_attn.cuh for head dim 128.
#define KVQ_HD 128
#include "kvq_attn.cuh"
