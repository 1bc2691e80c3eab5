// kvx_attend_shared for bf16 queries over a bf16 cache.
#include "kvx_shared.cuh"

template bool kvx::shared::launch<__nv_bfloat16, 2>(const kvx::shared::Args &, cudaStream_t);
