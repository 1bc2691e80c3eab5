// kvx_attend for bf16 queries over an e4m3 cache.
#include "kvx_attend.cuh"

template bool kvx::attend::launch<__nv_bfloat16, 1>(kvx::attend::Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);
