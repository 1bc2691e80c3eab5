// kvx_append_tokens: queries and keys normed per head, rotated by their
// positions, keys and values written into their cache pages, in one pass.
//
// Per head x:  y = x / sqrt(sum(x^2)/D + eps) * w, then the pairs (y_a, y_b)
// of the first rot_dim values turn by the token's angles.  A head is one row
// of up to 32 lanes with eight values each, as two runs of four that hold whole
// pairs: a lane turns its own values, and only the sum of squares crosses lanes.
// All in 32 bits, rounded once when stored: a 16-bit norm rounded before the
// rotation would add an error as large as the result's own rounding.
//
// Bound by HBM for prompts (each value read once and written once; the table's
// row of cosines and sines is read once per block of a token's heads) and by
// the launch and a chain of two loads (slot, segment address) for a few tokens.
// A block takes one token, so that the table row and the slot are looked up
// once for all its heads; with fewer tokens than the device has room for, a
// token's heads are spread over several blocks.
#include <cuda_fp8.h>

#include "kvx_cache.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 3;  // rows whose loads a lane has in flight

struct AppendArgs {
    CacheView c;
    const void *q, *k, *v;
    uint64_t q_stride, k_stride, v_stride, q_out_stride;
    const void *q_weight, *k_weight;
    const float *cos_sin;
    const uint32_t *positions;
    const int64_t *slots;
    void *q_out;
    uint32_t *status;
    float eps;
    uint32_t q_heads, rot, max_pos, interleaved;
};

template <class T>
__device__ __forceinline__ void unpack4(const uint2 &r, float *x) {
    const float2 a = Pair<T>::unpack(r.x), b = Pair<T>::unpack(r.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

template <class T>
__device__ __forceinline__ uint2 pack4(const float *x) {
    return make_uint2(Pair<T>::pack(x[0], x[1]), Pair<T>::pack(x[2], x[3]));
}

__device__ __forceinline__ uint32_t e4m3x4(const float *x, float inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// A lane's eight values of a row: four from each of two places.
struct Eight {
    uint2 a, b;
};
template <class T>
__device__ __forceinline__ Eight load8(const T *row, uint32_t da, uint32_t db) {
    return Eight{*reinterpret_cast<const uint2 *>(row + da), *reinterpret_cast<const uint2 *>(row + db)};
}

// Lanes of a row: a power of two with 8 * LANES >= dim.
template <class T, bool FP8, int LANES>
__global__ void __launch_bounds__(kThreads, 4) k_append(const __grid_constant__ AppendArgs a) {
    constexpr uint32_t kRows = kThreads / LANES;
    const uint64_t t = blockIdx.x;
    const uint32_t li = threadIdx.x % LANES;
    // the lanes of this row, whose shuffles other rows take no part in
    const uint32_t mask = LANES == 32 ? 0xFFFFFFFFu : ((1u << LANES % 32) - 1) << (threadIdx.x % 32 / LANES * LANES);
    const uint32_t dim = a.c.dim, heads = a.c.heads, rows = a.q_heads + 2 * heads;
    const bool in = li * 8 < dim;
    uint32_t bad = 0;

    // values da .. da+3 and db .. db+3: rotated halves hold each other's
    // partners, neighbours are partners anyway
    const bool turns = li * 8 < a.rot, halves = turns && !a.interleaved;
    const uint32_t da = halves ? li * 4 : li * 8, db = halves ? da + a.rot / 2 : da + 4;

    const int64_t slot = a.slots[t];
    uint32_t block = 0, place = 0;
    bool write = slot >= 0;
    if (write) {
        const uint64_t b = (uint64_t)slot < (1ull << 31) ? a.c.page.div((uint32_t)slot) : (uint64_t)slot / a.c.page.d;
        place = (uint32_t)((uint64_t)slot - b * a.c.page.d);
        if (b >= a.c.B) {
            bad |= KVX_S_BOUNDS;
            write = false;
        } else {
            block = (uint32_t)b;
        }
    }

    float4 c = make_float4(1, 1, 1, 1), s = make_float4(0, 0, 0, 0);
    if (a.rot) {
        const uint32_t pos = a.positions[t];
        if (pos >= a.max_pos) {  // the same for the whole block
            if (threadIdx.x == 0) raise(a.status, bad | KVX_S_BOUNDS);
            return;
        }
        if (turns) {
            const float *row = a.cos_sin + (uint64_t)pos * a.rot + li * 4;
            c = __ldg(reinterpret_cast<const float4 *>(row));
            s = __ldg(reinterpret_cast<const float4 *>(row + a.rot / 2));
        }
    }
    Eight wq = {}, wk = {};
    if (in && a.q_weight) wq = load8(static_cast<const T *>(a.q_weight), da, db);
    if (in && a.k_weight) wk = load8(static_cast<const T *>(a.k_weight), da, db);

    const T *q = static_cast<const T *>(a.q) + t * a.q_stride;
    const T *k = static_cast<const T *>(a.k) + t * a.k_stride;
    const T *v = static_cast<const T *>(a.v) + t * a.v_stride;
    const uint32_t step = gridDim.y * kRows;
    for (uint32_t r0 = blockIdx.y * kRows + threadIdx.x / LANES; r0 < rows; r0 += kUnroll * step) {
        Eight raw[kUnroll] = {};
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t r = r0 + u * step;
            if (in && r < rows)
                raw[u] = load8(r < a.q_heads           ? q + (uint64_t)r * dim
                               : r < a.q_heads + heads ? k + (uint64_t)(r - a.q_heads) * dim
                                                       : v + (uint64_t)(r - a.q_heads - heads) * dim,
                               da, db);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t r = r0 + u * step;
            if (r >= rows) break;
            const bool is_q = r < a.q_heads, is_v = r >= a.q_heads + heads;
            float x[8];
            unpack4<T>(raw[u].a, x);
            unpack4<T>(raw[u].b, x + 4);
            if (!is_v) {
                if (is_q ? a.q_weight : a.k_weight) {
                    float ss = 0;
#pragma unroll
                    for (int e = 0; e < 8; e++) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
                    const float inv = rsqrtf(ss / (float)dim + a.eps);
                    float w[8];
                    unpack4<T>(is_q ? wq.a : wk.a, w);
                    unpack4<T>(is_q ? wq.b : wk.b, w + 4);
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] = x[e] * inv * w[e];
                }
                if (turns) {
                    const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {  // pair i: values i and i+4, or 2i and 2i+1
                        const float ya = a.interleaved ? x[2 * i] : x[i], yb = a.interleaved ? x[2 * i + 1] : x[i + 4];
                        const float za = fmaf(-yb, sn[i], ya * cc[i]), zb = fmaf(ya, sn[i], yb * cc[i]);
                        if (a.interleaved)
                            x[2 * i] = za, x[2 * i + 1] = zb;
                        else
                            x[i] = za, x[i + 4] = zb;
                    }
                }
            }
            if (!in) continue;
            if (is_q) {
                T *o = static_cast<T *>(a.q_out) + t * a.q_out_stride + (uint64_t)r * dim;
                *reinterpret_cast<uint2 *>(o + da) = pack4<T>(x);
                *reinterpret_cast<uint2 *>(o + db) = pack4<T>(x + 4);
            } else if (write) {
                const uint32_t h = is_v ? r - a.q_heads - heads : r - a.q_heads;
                const uint64_t at = __ldg(a.c.lane_addr(block, h, is_v));
                if (a.c.ok(at, bad)) {
                    uint8_t *o = a.c.pool + at + place * a.c.token_stride;
                    if constexpr (FP8) {
                        const float inv = 1.0f / (is_v ? a.c.v_scale : a.c.k_scale);
                        *reinterpret_cast<uint32_t *>(o + da) = e4m3x4(x, inv);
                        *reinterpret_cast<uint32_t *>(o + db) = e4m3x4(x + 4, inv);
                    } else {
                        *reinterpret_cast<uint2 *>(o + 2 * da) = pack4<T>(x);
                        *reinterpret_cast<uint2 *>(o + 2 * db) = pack4<T>(x + 4);
                    }
                }
            }
        }
    }
    raise(a.status, bad);
}

template <class T, bool FP8>
void launch(const AppendArgs &a, dim3 grid, cudaStream_t s) {
    if (a.c.dim <= 64)
        k_append<T, FP8, 8><<<grid, kThreads, 0, s>>>(a);
    else if (a.c.dim <= 128)
        k_append<T, FP8, 16><<<grid, kThreads, 0, s>>>(a);
    else
        k_append<T, FP8, 32><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace kvx

extern "C" kvx_status kvx_append_tokens(const kvx_cache *cache, const void *q, uint64_t q_stride, const void *k,
                                        uint64_t k_stride, const void *v, uint64_t v_stride, uint32_t dtype,
                                        uint32_t T, uint32_t q_heads, const void *q_weight, const void *k_weight,
                                        float eps, const float *cos_sin, uint32_t rot_dim, uint32_t max_pos,
                                        uint32_t interleaved, const uint32_t *positions, const int64_t *slots,
                                        void *q_out, uint64_t q_out_stride, uint32_t *status, void *stream) {
    using namespace kvx;
    if (!cache_ok(cache) || (dtype != KVX_BF16 && dtype != KVX_F16) || !status) return KVX_EINVAL;
    if (cache->dtype != dtype && cache->dtype != KVX_E4M3) return KVX_EINVAL;
    if (T > 0x7FFFFFFFu || q_heads > 65536u || cache->heads > 65536u) return KVX_EINVAL;
    if (rot_dim % 16 || rot_dim > cache->dim || (rot_dim && (!cos_sin || !positions || !max_pos))) return KVX_EINVAL;
    if (!(eps >= 0 && eps < INFINITY)) return KVX_EINVAL;
    if ((q_stride | k_stride | v_stride | q_out_stride) % 8) return KVX_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(q_weight) ||
        !aligned16(k_weight) || !aligned16(rot_dim ? cos_sin : nullptr))
        return KVX_EINVAL;
    if (!T) return KVX_OK;
    if (!k || !v || !slots || (q_heads && (!q || !q_out))) return KVX_EINVAL;
    AppendArgs a = {cache_view(cache), q, k, v, q_stride, k_stride, v_stride, q_out_stride, q_weight, k_weight,
                    cos_sin, positions, slots, q_out, status, eps, q_heads, rot_dim, max_pos, interleaved};
    const uint32_t lanes = cache->dim <= 64 ? 8 : cache->dim <= 128 ? 16 : 32;
    const uint32_t per_block = kThreads / lanes, rows = q_heads + 2 * cache->heads;
    // A token's rows over several blocks while that fills the device's first wave (8 blocks an SM).
    const uint64_t most = ceil_div(rows, per_block), room = ceil_div(8 * (uint64_t)sm_count(), T);
    const dim3 grid(T, (uint32_t)(most < room ? most : room));
    if (dtype == KVX_BF16)
        cache->dtype == KVX_E4M3 ? launch<__nv_bfloat16, true>(a, grid, as_stream(stream))
                                 : launch<__nv_bfloat16, false>(a, grid, as_stream(stream));
    else
        cache->dtype == KVX_E4M3 ? launch<__half, true>(a, grid, as_stream(stream))
                                 : launch<__half, false>(a, grid, as_stream(stream));
    KVX_LAUNCHED();
    return KVX_OK;
}
