// kvx_attend for bf16 queries over a bf16 cache.
#include "kvx_attend.cuh"

template bool kvx::attend::launch<__nv_bfloat16, 2>(kvx::attend::Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);
