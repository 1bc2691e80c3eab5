// kvx_read_tokens: tokens of a paged cache read back into dense 16-bit tensors.
//
// out[t] = stored * scale, rounded once: 32 bits hold the product of an 8-bit value
// and a power of two, or any scale of up to 20 bits; that with a longer one, up to
// 28 bits, is cut off to 32 so that rounding it to 16 gives what rounding the
// product itself would (scaled_odd).  A warp takes one token, whose sequence, page and
// segment addresses it looks up once for all heads; a lane takes 16 stored bytes
// at a time and writes 16-bit ones as whole sectors.
//
// Bound by HBM, each value read once and written once: eight sequences of 16,000
// tokens, 8 heads of 128, 8-bit rows with scales into bf16, 120 us, 6580 GB/s
// (97 % of a copy's rate); 37 sequences of up to 8000, 6 heads of 96, fp16, 52 us,
// 6085 GB/s.  For one short sequence it is the launch and a chain of four loads:
// 3.5 us.  What it takes is many warps with few loads each (two pieces a lane and
// all 64 warps of an SM 119 us, four pieces and 48 warps 137, 40 warps 132): the
// chain before the first piece is as long as the copy itself.  16-bit rows, whose
// pieces are twice as many, take four at a time (52 us, two 59).
#include "kvx_cache.cuh"

namespace kvx {
namespace {

constexpr int kWarps = 4;   // of a block
constexpr int kBlocks = 16;  // an SM

struct ReadArgs {
    CacheView c;
    const uint32_t *blocks, *first, *starts;
    void *out[2];
    uint64_t stride[2];
    uint32_t *status;
    uint32_t num_seqs, blocks_per_seq, T;
    uint32_t pieces;  // 16-byte pieces of a row
    FastDiv by_pieces;
    uint64_t max_len;
    bool sectors;  // outputs' rows start on multiples of 32 bytes
};

// 32 bytes, a whole sector, by one instruction (by two, which write halves of
// sectors, the eight sequences take 139 us in place of 132).
__device__ __forceinline__ void store_sector(void *to, uint2 a, uint2 b, uint2 c, uint2 d) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(b.x), "r"(b.y),
                 "r"(c.x), "r"(c.y), "r"(d.x), "r"(d.y)
                 : "memory");
}

// How many of starts[0 .. count-1], which do not decrease, are at most t: by the
// whole warp, 32 of them at a time.
__device__ __forceinline__ uint32_t rank_of(const uint32_t *starts, uint32_t count, uint32_t t, uint32_t lane) {
    uint32_t lo = 0;
    while (count > 32) {
        const uint32_t step = (count + 31) / 32;
        const uint32_t i = lane * step;
        const uint32_t below = __popc(__ballot_sync(0xFFFFFFFFu, i < count && __ldg(starts + lo + i) <= t));
        if (!below) return lo;
        const uint32_t at = (below - 1) * step;
        lo += at;
        count = count - at < step ? count - at : step;
    }
    return lo + __popc(__ballot_sync(0xFFFFFFFFu, lane < count && __ldg(starts + lo + lane) <= t));
}

// x * scale cut off, with the last bit set where anything was lost: no border or
// middle of 16-bit values lies between this and the product.  Rounded to 32 bits it
// could become such a middle (1.125 * 0x1.d38e38p-1: 1.03125 in bf16 by way of 32
// bits, 1.0234375 is nearer).  The remainder is exact from 2^-122 on.  For scales that
// need it only: eight sequences of 16,000 tokens take 121 us with such a scale; with row
// scales 120 as they are and 122 this way, heads of 64 66 and 70.
__device__ __forceinline__ float scaled_odd(float x, float scale) {
    const float p = __fmul_rz(x, scale);
    return fmaf(x, scale, -p) == 0 ? p : __uint_as_float(__float_as_uint(p) | 1);
}

// Four stored 8-bit values times a scale, as 16-bit ones.
template <class T, bool LONG>
__device__ __forceinline__ uint2 scaled4(uint32_t four, float scale) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
    const float2 x = Pair<__half>::unpack(lo), y = Pair<__half>::unpack(hi);
    if constexpr (LONG)
        return make_uint2(Pair<T>::pack(scaled_odd(x.x, scale), scaled_odd(x.y, scale)),
                          Pair<T>::pack(scaled_odd(y.x, scale), scaled_odd(y.y, scale)));
    return make_uint2(Pair<T>::pack(x.x * scale, x.y * scale), Pair<T>::pack(y.x * scale, y.y * scale));
}

enum Store { kSame, kScaled, kScaledLong };  // the outputs' type; e4m3; e4m3 with a scale of more than 20 bits

template <class T, Store STORE>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) k_read(const __grid_constant__ ReadArgs a) {
    constexpr bool FP8 = STORE != kSame, LONG = STORE == kScaledLong;
    constexpr int kUnroll = FP8 ? 2 : 4;  // pieces of a lane on their way
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * kWarps + threadIdx.x / 32;
    uint32_t bad = 0;
    if (blockIdx.x == 0)  // the table itself
        for (uint32_t n = threadIdx.x; n < a.num_seqs; n += 32 * kWarps)
            if (a.starts[n] > a.starts[n + 1] || a.starts[n + 1] > a.T) bad |= KVX_S_BOUNDS;
    uint32_t seq = kNone;
    if (t < a.T) seq = rank_of(a.starts, a.num_seqs + 1, t, lane) - 1;  // none: t is before the first start
    if (seq < a.num_seqs) {
        const uint32_t start = __ldg(a.starts + seq);
        const uint64_t pos = (uint64_t)(a.first ? __ldg(a.first + seq) : 0) + (t - start);
        uint32_t id = kNone;
        if (start <= t && pos < a.max_len) {
            const uint32_t page = a.c.page.div((uint32_t)pos);
            id = __ldg(a.blocks + (uint64_t)seq * a.blocks_per_seq + page);
            const uint32_t token = (uint32_t)pos - page * a.c.page.d;
            if (id < a.c.B) {
                const uint64_t *entry = a.c.lane_addr(id, 0, 0);
                const uint32_t total = 2 * a.c.heads * a.pieces;
                const uint64_t place = token * a.c.token_stride;
                for (uint32_t i0 = lane; i0 < total; i0 += 32 * kUnroll) {
                    uint32_t lane_of[kUnroll], piece[kUnroll];
                    bool ok[kUnroll];
                    uint64_t seg[kUnroll];
                    uint4 raw[kUnroll];
                    uint32_t e[kUnroll];
#pragma unroll
                    for (int u = 0; u < kUnroll; u++) {
                        const uint32_t i = i0 + 32 * u;
                        lane_of[u] = a.by_pieces.div(i);
                        piece[u] = i - lane_of[u] * a.pieces;
                        ok[u] = i < total;
                        seg[u] = ok[u] ? __ldg(entry + lane_of[u]) : 0;
                    }
#pragma unroll
                    for (int u = 0; u < kUnroll; u++) {
                        ok[u] = ok[u] && a.c.ok(seg[u], bad);
                        raw[u] = ok[u] ? __ldg(reinterpret_cast<const uint4 *>(a.c.pool + seg[u] + place) + piece[u]) : make_uint4(0, 0, 0, 0);
                        e[u] = FP8 && ok[u] && a.c.scale_offset ? __ldg(a.c.pool + seg[u] + a.c.scale_offset + token) : 127;
                    }
#pragma unroll
                    for (int u = 0; u < kUnroll; u++) {
                        if (!ok[u]) continue;
                        const uint32_t kv = lane_of[u] & 1, head = lane_of[u] >> 1;
                        T *o = static_cast<T *>(a.out[kv]) + t * a.stride[kv] + (uint64_t)head * a.c.dim + piece[u] * (FP8 ? 16 : 8);
                        if constexpr (FP8) {
                            const float scale = a.c.scale_offset ? row_scale(e[u]) : kv ? a.c.v_scale : a.c.k_scale;
                            const uint2 w0 = scaled4<T, LONG>(raw[u].x, scale), w1 = scaled4<T, LONG>(raw[u].y, scale);
                            const uint2 w2 = scaled4<T, LONG>(raw[u].z, scale), w3 = scaled4<T, LONG>(raw[u].w, scale);
                            if (a.sectors) {
                                store_sector(o, w0, w1, w2, w3);
                            } else {
                                reinterpret_cast<uint4 *>(o)[0] = make_uint4(w0.x, w0.y, w1.x, w1.y);
                                reinterpret_cast<uint4 *>(o)[1] = make_uint4(w2.x, w2.y, w3.x, w3.y);
                            }
                        } else {
                            *reinterpret_cast<uint4 *>(o) = raw[u];
                        }
                    }
                }
            } else {
                bad |= KVX_S_BOUNDS;
            }
        } else {
            bad |= KVX_S_BOUNDS;
        }
    }
    raise(a.status, bad);
}

// Whether products with an 8-bit value (4 bits) may take more than the 24 bits of a float.
bool is_long(float scale) {
    int e;
    const float m = frexpf(scale, &e) * 1048576.0f;  // 2^20
    return m != floorf(m);
}

template <class T>
void launch(const ReadArgs &a, Store store, uint32_t grid, cudaStream_t s) {
    store == kSame     ? k_read<T, kSame><<<grid, 32 * kWarps, 0, s>>>(a)
    : store == kScaled ? k_read<T, kScaled><<<grid, 32 * kWarps, 0, s>>>(a)
                       : k_read<T, kScaledLong><<<grid, 32 * kWarps, 0, s>>>(a);
}

}  // namespace
}  // namespace kvx

extern "C" kvx_status kvx_read_tokens(const kvx_cache *cache, const uint32_t *blocks, uint32_t num_seqs,
                                      uint32_t blocks_per_seq, const uint32_t *first, const uint32_t *starts, uint32_t T,
                                      uint32_t dtype, void *k_out, uint64_t k_stride, void *v_out, uint64_t v_stride,
                                      uint32_t *status, void *stream) {
    using namespace kvx;
    if (!cache_ok(cache) || (dtype != KVX_BF16 && dtype != KVX_F16) || !status) return KVX_EINVAL;
    if (cache->dtype != dtype && cache->dtype != KVX_E4M3) return KVX_EINVAL;
    const uint64_t max_len = (uint64_t)blocks_per_seq * cache->page_tokens;
    if (T > 0x7FFFFFFFu || num_seqs > 0x7FFFFFFFu || max_len >= (1ull << 31) || cache->heads > 65536u) return KVX_EINVAL;
    if ((k_stride | v_stride) % 8 || !aligned16(k_out) || !aligned16(v_out)) return KVX_EINVAL;
    if (!T || !num_seqs) return KVX_OK;
    if (!k_out || !v_out || !starts || (max_len && !blocks)) return KVX_EINVAL;
    ReadArgs a = {cache_view(cache), blocks, first, starts, {k_out, v_out}, {k_stride, v_stride}, status, num_seqs,
                  blocks_per_seq, T, 0, FastDiv(1), max_len,
                  ((uintptr_t)k_out | (uintptr_t)v_out | 2 * (k_stride | v_stride)) % 32 == 0};
    a.pieces = a.c.row_bytes / 16;
    a.by_pieces = FastDiv(a.pieces);
    const uint32_t grid = (uint32_t)ceil_div(T, kWarps);
    const cudaStream_t s = as_stream(stream);
    const Store store = cache->dtype != KVX_E4M3 ? kSame : is_long(cache->k_scale) || is_long(cache->v_scale) ? kScaledLong : kScaled;
    if (dtype == KVX_BF16)
        launch<__nv_bfloat16>(a, store, grid, s);
    else
        launch<__half>(a, store, grid, s);
    KVX_LAUNCHED();
    return KVX_OK;
}
