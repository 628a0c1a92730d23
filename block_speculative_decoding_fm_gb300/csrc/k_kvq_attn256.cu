// k_kvq_attn256.cu -- kvq_attn.cuh for head dim 256.
#define KVQ_HD 256
#include "kvq_attn.cuh"
