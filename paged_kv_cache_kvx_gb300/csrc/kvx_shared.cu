// kvx_attend_shared: attention of one new token per sequence over a prefix that
// a group of sequences shares, and the sequence's own tokens.
#include "kvx_cache.cuh"

namespace kvx {
namespace shared {
namespace {

constexpr uint32_t kMaxGroup = 128;

struct Args {
    CacheView c;
    const void *q;
    uint64_t q_stride;
    const uint32_t *prefix_blocks, *prefix_lens, *group_first, *blocks, *lens;
    uint32_t blocks_per_prefix, num_groups, blocks_per_seq, num_seqs, q_heads, group;
    uint32_t max_prefix, max_len;
    float scale;
    void *out;
    uint64_t out_stride;
    float *lse;
    uint32_t *status;
};

// One warp for each query head: a lane has eight values of it.
template <class T, int ES>
__global__ void __launch_bounds__(32) k_simple(const __grid_constant__ Args a) {
    const uint32_t n = blockIdx.x, head = blockIdx.y, lane = threadIdx.x, h = head / a.group;
    const bool in = lane * 8 < a.c.dim;
    uint32_t bad = 0;
    float q[8] = {}, o[8] = {}, m = -INFINITY, l = 0;
    if (in)
        for (int i = 0; i < 8; i++)
            q[i] = (float)static_cast<const T *>(a.q)[n * a.q_stride + (uint64_t)head * a.c.dim + lane * 8 + i] * a.scale;
    uint32_t g = kNone;
    for (uint32_t i = 0; i < a.num_groups; i++) {
        const uint32_t from = a.group_first[i], to = a.group_first[i + 1];
        if (from > to || to > a.num_seqs) bad |= KVX_S_BOUNDS;
        if (from <= n && n < to && to <= a.num_seqs) g = i;
    }
    for (int part = 0; part < 2; part++) {
        if (!part && g == kNone) continue;
        uint32_t len = part ? a.lens[n] : a.prefix_lens[g];
        const uint32_t most = part ? a.max_len : a.max_prefix;
        if (len > most) len = most, bad |= KVX_S_BOUNDS;
        const uint32_t *table = part ? a.blocks + (uint64_t)n * a.blocks_per_seq : a.prefix_blocks + (uint64_t)g * a.blocks_per_prefix;
        for (uint32_t j = 0; j < len; j++) {
            const uint32_t page = a.c.page.div(j), id = table[page], token = j - page * a.c.page.d;
            float x[2][8] = {};
            if (id >= a.c.B) {
                bad |= KVX_S_BOUNDS;
            } else {
                for (int kv = 0; kv < 2; kv++) {
                    const uint64_t seg = *a.c.lane_addr(id, h, kv);
                    if (!a.c.ok(seg, bad) || !in) continue;
                    const uint8_t *row = a.c.pool + seg + token * a.c.token_stride + lane * 8 * ES;
                    const uint32_t e = ES == 1 && a.c.scale_offset ? a.c.pool[seg + a.c.scale_offset + token] : 127;
                    const float s = a.c.scale_offset ? __uint_as_float(e == 255 ? 0x7FFFFFFFu : e ? e << 23 : 0x400000u) : kv ? a.c.v_scale : a.c.k_scale;
                    for (int i = 0; i < 8; i++) {
                        if (ES == 1) {
                            uint32_t v;
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"((uint16_t)row[i]));
                            x[kv][i] = Pair<__half>::unpack(v).x * s;
                        } else {
                            x[kv][i] = (float)reinterpret_cast<const T *>(row)[i];
                        }
                    }
                }
            }
            float s = 0;
            for (int i = 0; i < 8; i++) s += q[i] * x[0][i];
            for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
            const float top = fmaxf(m, s);
            if (top == -INFINITY) continue;
            const float r = expf(m - top), p = expf(s - top);
            m = top;
            l = l * r + p;
            for (int i = 0; i < 8; i++) o[i] = o[i] * r + p * x[1][i];
        }
    }
    const float inv = l != 0 ? 1.0f / l : 0.0f;
    if (in)
        for (int i = 0; i < 8; i++)
            static_cast<T *>(a.out)[n * a.out_stride + (uint64_t)head * a.c.dim + lane * 8 + i] = (T)(o[i] * inv);
    if (a.lse && lane == 0) a.lse[(uint64_t)n * a.q_heads + head] = l != 0 ? m + logf(l) : -INFINITY;
    raise(a.status, bad);
}

bool sizes_ok(const kvx_cache *c, uint32_t num_seqs, uint32_t q_heads, uint32_t blocks_per_seq, uint32_t num_groups,
              uint32_t blocks_per_prefix) {
    if (!cache_ok(c) || !q_heads || q_heads % c->heads || q_heads / c->heads > kMaxGroup) return false;
    const uint64_t len = (uint64_t)blocks_per_seq * c->page_tokens, prefix = (uint64_t)blocks_per_prefix * c->page_tokens;
    return len < (1ull << 31) && prefix < (1ull << 31) && num_seqs < (1u << 31) && num_groups < (1u << 31);
}

}  // namespace
}  // namespace shared
}  // namespace kvx

extern "C" size_t kvx_attend_shared_workspace_size(const kvx_cache *cache, uint32_t num_seqs, uint32_t q_heads,
                                                   uint32_t blocks_per_seq, uint32_t num_groups,
                                                   uint32_t blocks_per_prefix) {
    return kvx::shared::sizes_ok(cache, num_seqs, q_heads, blocks_per_seq, num_groups, blocks_per_prefix) ? 256 : 0;
}

extern "C" kvx_status kvx_attend_shared(const kvx_cache *cache, const void *q, uint64_t q_stride, uint32_t dtype,
                                        uint32_t num_seqs, uint32_t q_heads, const uint32_t *prefix_blocks,
                                        uint32_t blocks_per_prefix, const uint32_t *prefix_lens,
                                        const uint32_t *group_first, uint32_t num_groups, const uint32_t *blocks,
                                        uint32_t blocks_per_seq, const uint32_t *lens, float scale, void *out,
                                        uint64_t out_stride, float *lse, uint32_t *status, void *ws, size_t ws_bytes,
                                        void *stream) {
    using namespace kvx;
    using namespace kvx::shared;
    if (!sizes_ok(cache, num_seqs, q_heads, blocks_per_seq, num_groups, blocks_per_prefix)) return KVX_EINVAL;
    if ((dtype != KVX_BF16 && dtype != KVX_F16) || (cache->dtype != dtype && cache->dtype != KVX_E4M3)) return KVX_EINVAL;
    if (!status || !(scale > -INFINITY && scale < INFINITY)) return KVX_EINVAL;
    if ((q_stride | out_stride) % 8 || !aligned16(q) || !aligned16(out)) return KVX_EINVAL;
    if (!num_seqs) return KVX_OK;
    const uint32_t max_len = blocks_per_seq * cache->page_tokens, max_prefix = blocks_per_prefix * cache->page_tokens;
    if (!q || !out || !lens || (max_len && !blocks)) return KVX_EINVAL;
    if (num_groups && (!prefix_lens || !group_first || (max_prefix && !prefix_blocks))) return KVX_EINVAL;
    if (!ws || !aligned16(ws) ||
        ws_bytes < kvx_attend_shared_workspace_size(cache, num_seqs, q_heads, blocks_per_seq, num_groups, blocks_per_prefix))
        return KVX_EINVAL;
    Args a = {cache_view(cache), q, q_stride, prefix_blocks, prefix_lens, group_first, blocks, lens, blocks_per_prefix,
              num_groups, blocks_per_seq, num_seqs, q_heads, q_heads / cache->heads, max_prefix, max_len, scale, out,
              out_stride, lse, status};
    const dim3 grid(num_seqs, q_heads);
    const cudaStream_t s = as_stream(stream);
    if (cache->dtype == KVX_E4M3)
        dtype == KVX_BF16 ? k_simple<__nv_bfloat16, 1><<<grid, 32, 0, s>>>(a) : k_simple<__half, 1><<<grid, 32, 0, s>>>(a);
    else
        dtype == KVX_BF16 ? k_simple<__nv_bfloat16, 2><<<grid, 32, 0, s>>>(a) : k_simple<__half, 2><<<grid, 32, 0, s>>>(a);
    KVX_LAUNCHED();
    return KVX_OK;
}
