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
// row of cosines and sines is read once per block of a token's heads): 16,000
// tokens of 32 + 8 heads of 128, bf16, in 64 us, 6.2 TB/s.  For a few tokens
// it is the launch and a chain of loads (slot, segment address): 2.8 us.  A
// block is one warp and takes one token, so that the table row and the slot are
// looked up once for all its heads (blocks of 2, 4 and 8 warps took 69, 82 and
// 107 us); with fewer tokens than the device has room for, a token's heads are
// spread over several blocks.
#include <cmath>
#include <cuda_fp8.h>

#include "kvx_cache.cuh"

namespace kvx {
namespace {

constexpr int kThreads = 32;
constexpr int kMinBlocks = 32;  // an SM
constexpr int kUnroll = 2;  // rows that a lane works on at a time, with as many on their way

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
    float eps, inv_dim, inv_k_scale, inv_v_scale;  // of the scales: exact_inverse()
    uint32_t q_heads, rot, max_pos;
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

__device__ __forceinline__ uint32_t e4m3x4(const float *x) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// Eight values over their scale.  A scale of a power of two has an exact
// inverse, by which the quotient is the product; a product with an inverse that
// is rounded would round twice, and turn zeros into NaN where it is infinite.
// A prompt of 16,000 tokens with 8 heads of 128 takes 63 us by the inverse, 72
// with divisions.
__device__ __forceinline__ void divide(float *x, float scale, float inverse) {
    if (inverse != 0) {  // the same for the whole launch
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] *= inverse;
    } else {
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] /= scale;
    }
}

// 1 / scale where that is exact, else 0.
float exact_inverse(float scale) {
    int e;  // scale = 2^(e-1)
    return std::frexp(scale, &e) == 0.5f && e >= -126 && e <= 127 ? std::ldexp(1.0f, 1 - e) : 0.0f;
}

// A lane's eight values of a row: four from each of two places.
struct Eight {
    uint2 a, b;
};

// One token's part that a lane works on.
struct Lane {
    uint32_t da, db;           // its values: da .. da+3 and db .. db+3
    bool in, turns;            // within the head; among the rotated values
    float4 c, s;               // its pairs' angles
    uint32_t first, at, step;  // rows of a section: the warp's first, the lane's among those, to the warp's next
};

enum Kind { kQuery, kKey, kValue };

// All of a token's rows of one kind.  Loads run a round ahead.
template <class T, bool FP8, int LANES, bool NEIGHBOURS, Kind KIND>
struct Section {
    const AppendArgs &a;
    const Lane &l;
    const T *src;
    uint32_t rows;
    Eight raw[kUnroll];
    __device__ __forceinline__ Section(const AppendArgs &args, const Lane &lane, const T *from, uint32_t n)
        : a(args), l(lane), src(from), rows(n) {}
    __device__ __forceinline__ void load(uint32_t r0) {
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t r = r0 + l.at + u * l.step;
            raw[u] = Eight{};
            if (l.in && r < rows) {
                const T *row = src + r * a.c.dim;
                raw[u].a = *reinterpret_cast<const uint2 *>(row + l.da);
                raw[u].b = *reinterpret_cast<const uint2 *>(row + l.db);
            }
        }
    }
    // entry: the block's address-table entries from head 0's K on, or NULL
    __device__ __forceinline__ void run(const void *weight, T *q_out, const uint64_t *entry, uint64_t place, uint64_t room,
                                        uint32_t &bad) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; e++) w[e] = 1.0f;
        if (KIND != kValue && weight && l.in) {
            unpack4<T>(*reinterpret_cast<const uint2 *>(static_cast<const T *>(weight) + l.da), w);
            unpack4<T>(*reinterpret_cast<const uint2 *>(static_cast<const T *>(weight) + l.db), w + 4);
        }
        const bool norm = KIND != kValue && weight;
#pragma unroll 1
        for (uint32_t r0 = l.first; r0 < rows; r0 += kUnroll * l.step) {  // the same turns for a whole warp
            Eight cur[kUnroll];
            uint64_t seg[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; u++) {
                cur[u] = raw[u];
                const uint32_t r = r0 + l.at + u * l.step;
                if (KIND != kQuery && entry && r < rows) seg[u] = __ldg(entry + 2 * r + (KIND == kValue));
            }
            load(r0 + kUnroll * l.step);
#pragma unroll
            for (int u = 0; u < kUnroll; u++) {
                const uint32_t r = r0 + l.at + u * l.step;
                float x[8];
                unpack4<T>(cur[u].a, x);
                unpack4<T>(cur[u].b, x + 4);
                if (norm) {
                    float ss = 0;
#pragma unroll
                    for (int e = 0; e < 8; e++) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float inv = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] *= inv * w[e];
                }
                if (KIND != kValue && l.turns) {
                    const float cc[4] = {l.c.x, l.c.y, l.c.z, l.c.w}, sn[4] = {l.s.x, l.s.y, l.s.z, l.s.w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {  // pair i: values i and i+4, or 2i and 2i+1
                        constexpr int other = NEIGHBOURS ? 1 : 4;
                        const int j = NEIGHBOURS ? 2 * i : i;
                        const float ya = x[j], yb = x[j + other];
                        x[j] = fmaf(-yb, sn[i], ya * cc[i]);
                        x[j + other] = fmaf(ya, sn[i], yb * cc[i]);
                    }
                }
                if (!l.in || r >= rows) continue;
                if constexpr (KIND == kQuery) {
                    T *o = q_out + r * a.c.dim;
                    *reinterpret_cast<uint2 *>(o + l.da) = pack4<T>(x);
                    *reinterpret_cast<uint2 *>(o + l.db) = pack4<T>(x + 4);
                } else if (entry) {
                    if (seg[u] > room || ((uint32_t)seg[u] & 15)) {
                        a.c.ok(seg[u], bad);
                        continue;
                    }
                    uint8_t *o = a.c.pool + (seg[u] + place);
                    if constexpr (FP8) {
                        divide(x, KIND == kValue ? a.c.v_scale : a.c.k_scale, KIND == kValue ? a.inv_v_scale : a.inv_k_scale);
                        *reinterpret_cast<uint32_t *>(o + l.da) = e4m3x4(x);
                        *reinterpret_cast<uint32_t *>(o + l.db) = e4m3x4(x + 4);
                    } else if constexpr (KIND == kValue) {
                        *reinterpret_cast<uint2 *>(o + 2 * l.da) = cur[u].a;
                        *reinterpret_cast<uint2 *>(o + 2 * l.db) = cur[u].b;
                    } else {
                        *reinterpret_cast<uint2 *>(o + 2 * l.da) = pack4<T>(x);
                        *reinterpret_cast<uint2 *>(o + 2 * l.db) = pack4<T>(x + 4);
                    }
                }
            }
        }
    }
};

// Lanes of a row: a power of two with 8 * LANES >= dim.
template <class T, bool FP8, int LANES, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads, kMinBlocks) k_append(const __grid_constant__ AppendArgs a) {
    constexpr uint32_t kRows = kThreads / LANES, kWarpRows = 32 / LANES;
    const uint64_t t = blockIdx.x;
    const uint32_t li = threadIdx.x % LANES, heads = a.c.heads;
    uint32_t bad = 0;
    Lane l;
    l.in = li * 8 < a.c.dim;
    l.turns = li * 8 < a.rot;
    // rotated halves hold each other's partners, neighbours are partners anyway
    const bool halves = l.turns && !NEIGHBOURS;
    l.da = halves ? li * 4 : li * 8;
    l.db = halves ? l.da + a.rot / 2 : l.da + 4;
    l.step = gridDim.y * kRows;
    l.at = threadIdx.x / LANES % kWarpRows;
    l.first = blockIdx.y * kRows + threadIdx.x / LANES - l.at;

    // Two rounds of latency to the first store: the values, the slot and the
    // position, then the angles and the segments' addresses.
    Section<T, FP8, LANES, NEIGHBOURS, kQuery> q(a, l, static_cast<const T *>(a.q) + t * a.q_stride, a.q_heads);
    Section<T, FP8, LANES, NEIGHBOURS, kKey> k(a, l, static_cast<const T *>(a.k) + t * a.k_stride, heads);
    Section<T, FP8, LANES, NEIGHBOURS, kValue> v(a, l, static_cast<const T *>(a.v) + t * a.v_stride, heads);
    q.load(l.first);
    const int64_t slot = a.slots[t];
    const uint32_t pos = a.rot ? a.positions[t] : 0;
    if (a.rot && pos >= a.max_pos) {  // the same for the whole block
        if (threadIdx.x == 0) raise(a.status, KVX_S_BOUNDS);
        return;
    }
    if (l.turns) {
        const float *row = a.cos_sin + (uint64_t)pos * a.rot + li * 4;
        l.c = __ldg(reinterpret_cast<const float4 *>(row));
        l.s = __ldg(reinterpret_cast<const float4 *>(row + a.rot / 2));
    }
    const uint64_t *entry = nullptr;
    uint64_t place = 0;
    if (slot >= 0) {
        const uint64_t b = (uint64_t)slot < (1ull << 31) ? a.c.page.div((uint32_t)slot) : (uint64_t)slot / a.c.page.d;
        place = ((uint64_t)slot - b * a.c.page.d) * a.c.token_stride;
        if (b < a.c.B)
            entry = a.c.lane_addr((uint32_t)b, 0, 0);
        else
            bad |= KVX_S_BOUNDS;
    }
    const uint64_t room = a.c.pool_bytes - a.c.span;  // a segment's largest offset, where any fits
    if (entry && a.c.pool_bytes < a.c.span) {
        bad |= KVX_S_BOUNDS;
        entry = nullptr;
    }
    k.load(l.first);
    q.run(a.q_weight, static_cast<T *>(a.q_out) + t * a.q_out_stride, nullptr, 0, 0, bad);
    v.load(l.first);
    k.run(a.k_weight, nullptr, entry, place, room, bad);
    v.run(nullptr, nullptr, entry, place, room, bad);
    raise(a.status, bad);
}

template <class T, bool FP8, bool NEIGHBOURS>
void launch_one(const AppendArgs &a, dim3 grid, cudaStream_t s) {
    if (a.c.dim <= 64)
        k_append<T, FP8, 8, NEIGHBOURS><<<grid, kThreads, 0, s>>>(a);
    else if (a.c.dim <= 128)
        k_append<T, FP8, 16, NEIGHBOURS><<<grid, kThreads, 0, s>>>(a);
    else
        k_append<T, FP8, 32, NEIGHBOURS><<<grid, kThreads, 0, s>>>(a);
}

template <class T, bool FP8>
void launch(const AppendArgs &a, dim3 grid, bool neighbours, cudaStream_t s) {
    neighbours ? launch_one<T, FP8, true>(a, grid, s) : launch_one<T, FP8, false>(a, grid, s);
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
                    cos_sin, positions, slots, q_out, status, eps, 1.0f / cache->dim,
                    exact_inverse(cache->k_scale), exact_inverse(cache->v_scale), q_heads, rot_dim, max_pos};
    const uint32_t lanes = cache->dim <= 64 ? 8 : cache->dim <= 128 ? 16 : 32;
    const uint32_t per_block = kThreads / lanes, rows = q_heads + 2 * cache->heads;
    // A token's rows go to several blocks while those fit on the device
    // together, and to two up to half a wave beyond that: three waves of halves
    // in place of two of wholes (32 + 8 heads of 128: 4999 tokens 26.9 us in one
    // block each, 24.1 in two; 7000 tokens 31.8 and 30.4; 8000, which stay in
    // one, 34.5 and 35.5, 12,000 49.8 and 50.1).  With eight rounds or fewer a
    // block's start costs as much as that saves (12 + 2 heads: 4865 tokens 11.1
    // and 11.4 us; 16 + 2 heads, ten rounds, 13.0 and 12.2).
    const uint64_t most = ceil_div(rows, per_block), fit = (uint64_t)kMinBlocks * sm_count();
    const bool halves = T > fit && 2 * (uint64_t)T <= 3 * fit && most > 8;
    const uint64_t parts = T < fit ? fit / T : halves ? 2 : 1;
    const dim3 grid(T, (uint32_t)(most < parts ? most : parts));
    if (dtype == KVX_BF16)
        cache->dtype == KVX_E4M3 ? launch<__nv_bfloat16, true>(a, grid, interleaved != 0, as_stream(stream))
                                 : launch<__nv_bfloat16, false>(a, grid, interleaved != 0, as_stream(stream));
    else
        cache->dtype == KVX_E4M3 ? launch<__half, true>(a, grid, interleaved != 0, as_stream(stream))
                                 : launch<__half, false>(a, grid, interleaved != 0, as_stream(stream));
    KVX_LAUNCHED();
    return KVX_OK;
}
