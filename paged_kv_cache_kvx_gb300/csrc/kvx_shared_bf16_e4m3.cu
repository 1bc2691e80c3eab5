// kvx_attend_shared for bf16 queries over an 8-bit cache.
#include "kvx_shared.cuh"

template bool kvx::shared::launch<__nv_bfloat16, 1>(const kvx::shared::Args &, cudaStream_t);
