// kvx_attend for f16 queries over a f16 cache.
#include "kvx_attend.cuh"

template bool kvx::attend::launch<__half, 2>(kvx::attend::Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);
