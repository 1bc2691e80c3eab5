// kvx_attend_shared for fp16 queries over an fp16 cache.
#include "kvx_shared.cuh"

template bool kvx::shared::launch<__half, 2>(const kvx::shared::Args &, cudaStream_t);
