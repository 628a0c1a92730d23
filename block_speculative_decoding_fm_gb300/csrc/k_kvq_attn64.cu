// k_kvq_attn64.cu -- kvq_attn.cuh for head dim 64.
#define KVQ_HD 64
#include "kvq_attn.cuh"
