// What the cache operators (kvx_append_tokens, kvx_attend, kvx_evict) share:
// the checked kvx_cache as kernels see it, and the 16-bit types' conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvx_common.cuh"

namespace kvx {

// Exact division of n < 2^31 by a fixed 1 <= d < 2^31: with l = ceil(log2 d) and
// m = ceil(2^(31+l) / d), m*d - 2^(31+l) < d <= 2^l, so n*m / 2^(31+l) exceeds
// n/d by less than 1/d and its floor is the quotient.  2^31 <= m < 2^32.
struct FastDiv {
    uint32_t mul, shift, d;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : shift(0), d(div) {
        while ((1ull << shift) < div) shift++;
        mul = (uint32_t)(((1ull << (31 + shift)) - 1) / div + 1);
    }
    __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return (uint32_t)(((uint64_t)(n << 1) * mul) >> 32) >> shift;
    }
};

struct CacheView {
    uint8_t *pool;
    uint64_t pool_bytes;
    const uint64_t *addr;
    uint64_t token_stride;
    uint64_t span;  // bytes from a segment's first row to the end of its last one
    uint32_t B, L, first_lane, heads, dim;
    uint32_t row_bytes;
    FastDiv page;
    float k_scale, v_scale;

    // A segment's pool offset, checked: false leaves it untouched and adds to
    // `bad`.
    __host__ __device__ __forceinline__ bool ok(uint64_t a, uint32_t &bad) const {
        if (a & 15) bad |= KVX_S_ALIGN;
        if (a > pool_bytes || span > pool_bytes - a) bad |= KVX_S_BOUNDS;
        return !(a & 15) && a <= pool_bytes && span <= pool_bytes - a;
    }
    __device__ __forceinline__ const uint64_t *lane_addr(uint32_t block, uint32_t head, uint32_t kv) const {
        return addr + (uint64_t)block * L + first_lane + 2 * head + kv;
    }
};

inline uint32_t elem_size(uint32_t dtype) { return dtype == KVX_E4M3 ? 1 : 2; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The rules of kvx_cache (include/kvx.h).
inline bool cache_ok(const kvx_cache *c) {
    if (!c || !c->pool || !c->addr || !aligned16(c->pool)) return false;
    if (c->dtype != KVX_BF16 && c->dtype != KVX_F16 && c->dtype != KVX_E4M3) return false;
    if (!c->dim || c->dim % 16 || c->dim > 256) return false;
    if (!c->page_tokens || c->page_tokens >= (1u << 31) || !c->heads || !c->B || c->reserved) return false;
    if (c->first_lane > c->L || 2 * (uint64_t)c->heads > c->L - c->first_lane) return false;
    const uint64_t row = (uint64_t)c->dim * elem_size(c->dtype);
    if (c->token_stride % 16 || c->token_stride < row || c->token_stride > (1ull << 31)) return false;
    if (!(c->k_scale > 0 && c->k_scale < INFINITY && c->v_scale > 0 && c->v_scale < INFINITY)) return false;
    if (c->dtype != KVX_E4M3 && (c->k_scale != 1 || c->v_scale != 1)) return false;
    return true;
}

inline CacheView cache_view(const kvx_cache *c) {
    CacheView v;
    v.pool = c->pool;
    v.pool_bytes = c->pool_bytes;
    v.addr = c->addr;
    v.token_stride = c->token_stride;
    v.row_bytes = c->dim * elem_size(c->dtype);
    v.span = (uint64_t)(c->page_tokens - 1) * c->token_stride + v.row_bytes;
    v.B = c->B;
    v.L = c->L;
    v.first_lane = c->first_lane;
    v.heads = c->heads;
    v.dim = c->dim;
    v.page = FastDiv(c->page_tokens);
    v.k_scale = c->k_scale;
    v.v_scale = c->v_scale;
    return v;
}

// Pairs of 16-bit values and floats.
template <class T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    __device__ static __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ static __forceinline__ uint32_t pack(float a, float b) {  // nearest even
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <>
struct Pair<__half> {
    __device__ static __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    __device__ static __forceinline__ uint32_t pack(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

}  // namespace kvx
