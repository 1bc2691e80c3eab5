// kvx_attend: attention of one new token per sequence over a paged cache.
//
// k_attend (kvx_attend.cuh) walks equal shares of all sequences' tiles, one
// per block; a unit (the query heads of one KV head of one sequence) that
// lies in one share is finished there, one that is cut by share borders leaves
// partial outputs with their bases m and sums l.  k_join puts those together,
//     M = max m_c,  L = sum l_c 2^(m_c - M),  out = sum o_c 2^(m_c - M) / L
// in a fixed order.  k_scores adds the attention weights 2^(logit - lse) to the
// scores: a weight needs the sum over all keys, so the logits pass through the
// workspace (4 bytes per key and query head, beside 2*dim*size bytes of key
// and value per KV head).  Each starts beside the last blocks of the kernel
// before it (programmatic dependency) and waits for its results.
#include "kvx_attend.cuh"

namespace kvx {
namespace attend {

// instantiated in kvx_attend_<types>.cu, a file each so that they compile in parallel
extern template bool launch<__nv_bfloat16, 2>(Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);
extern template bool launch<__nv_bfloat16, 1>(Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);
extern template bool launch<__half, 2>(Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);
extern template bool launch<__half, 1>(Args &, uint64_t, uint32_t, uint32_t, cudaStream_t);

namespace {

constexpr uint32_t kMaxGroup = 128;
constexpr int kJoinWarps = 8;
constexpr int kJoinUnroll = 4;  // parts whose loads a warp has in flight
constexpr int kScoreThreads = 128;
constexpr int kScoreUnroll = 8;  // keys of a thread
constexpr uint32_t kScoreKeys = kScoreUnroll * kScoreThreads;  // of a block that adds weights

// Blocks (c, ..) join the query heads of the unit whose first part block c of
// k_attend did; its other parts are the first ones of blocks c+1 .. last.  The
// warps are dealt out to the heads, and those of a head to its parts.  Bound by
// a chain of three loads, about 4 us behind k_attend, and rounds of them where a
// unit has more parts than its blocks have loads in flight for; blocks
// of sixteen warps with eight parts in flight did not fit on the SMs together
// and took 3 us more.
template <class T>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join(const __grid_constant__ Args a, uint32_t dp,
                                                          uint32_t unit_heads) {
    __shared__ float sh_m[kJoinWarps], sh_l[kJoinWarps];
    __shared__ float4 sh_o[kJoinWarps][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t all = a.group < unit_heads ? a.group : unit_heads, each = (all + gridDim.y - 1) / gridDim.y;
    const uint32_t first = blockIdx.y * each;  // this block's heads
    const uint32_t heads = first + each < all ? each : all > first ? all - first : 0;
    const uint32_t deal = heads < kJoinWarps && heads ? kJoinWarps / heads : 1, turn = warp % deal;
    const uint32_t per_head = (a.group + unit_heads - 1) / unit_heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint4 cut = __ldcg(a.cut + blockIdx.x);
    if (!joinable(cut, blockIdx.x, a.num_seqs, a.units, a.grid) || !heads) return;
    const uint32_t n = cut.x, parts = cut.z - blockIdx.x + 1;
    // Four of 128 values a lane, one head after the other where there are more
    // heads than warps; every warp makes the same turns.
    for (uint32_t h0 = 0, d0 = 0; h0 < heads; d0 += 128, h0 += d0 < dp ? 0 : kJoinWarps / deal, d0 = d0 < dp ? d0 : 0) {
        const uint32_t d = d0 + lane * 4, hh = first + h0 + warp / deal;
        const uint32_t in = cut.y % per_head * unit_heads + hh, qh = cut.y / per_head * a.group + in;
        const bool has = hh < first + heads && in < a.group;
        auto slot = [&](uint32_t i) { return (uint64_t)(i ? 2 * (blockIdx.x + i) : cut.w) * unit_heads + hh; };
        float4 v = make_float4(0, 0, 0, 0);
        float top = -INFINITY, sum = 0;
        for (uint32_t i0 = turn; has && i0 < parts; i0 += deal * kJoinUnroll) {
            float2 ml[kJoinUnroll];
            float4 x[kJoinUnroll];
            float higher = top;
#pragma unroll
            for (int u = 0; u < kJoinUnroll; u++) {
                const uint32_t i = i0 + u * deal;
                ml[u] = make_float2(-INFINITY, 0);
                x[u] = make_float4(0, 0, 0, 0);
                if (i < parts) ml[u] = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + slot(i));
                if (i < parts && d < dp) x[u] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot(i) * dp + d));
            }
#pragma unroll
            for (int u = 0; u < kJoinUnroll; u++) higher = fmaxf(higher, ml[u].x);
            float f = top == -INFINITY ? 1.0f : exp2_fast(top - higher);
            top = higher;
            sum *= f, v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
            for (int u = 0; u < kJoinUnroll; u++) {
                f = ml[u].x == -INFINITY ? 1.0f : exp2_fast(ml[u].x - top);  // 1: zeros, or a NaN
                sum += ml[u].y * f;
                v.x += x[u].x * f, v.y += x[u].y * f, v.z += x[u].z * f, v.w += x[u].w * f;
            }
        }
        if (deal > 1) {
            __syncthreads();  // the last round's results have been read
            sh_o[warp][lane] = v;
            if (lane == 0) sh_m[warp] = top, sh_l[warp] = sum;
            __syncthreads();
            if (turn || !has) continue;
            for (uint32_t w = 1; w < deal; w++) top = fmaxf(top, sh_m[warp + w]);
            v = make_float4(0, 0, 0, 0);
            sum = 0;
            for (uint32_t w = 0; w < deal; w++) {
                const float f = sh_m[warp + w] == -INFINITY ? 1.0f : exp2_fast(sh_m[warp + w] - top);
                const float4 x = sh_o[warp + w][lane];
                v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
                sum += sh_l[warp + w] * f;
            }
        }
        if (!has) continue;
        const float inv = sum == 0 ? 0.0f : a.c.v_scale / sum;
        if (d < a.c.dim) {
            T *to = static_cast<T *>(a.out) + (uint64_t)n * a.out_stride + (uint64_t)qh * a.c.dim + d;
            *reinterpret_cast<uint2 *>(to) =
                make_uint2(Pair<T>::pack(v.x * inv, v.y * inv), Pair<T>::pack(v.z * inv, v.w * inv));
        }
        if (d == 0) {
            const float lse2 = sum == 0 ? -INFINITY : top + log2f(sum);
            if (a.lse) a.lse[(uint64_t)n * a.q_heads + qh] = lse2 * 0.6931471805599453f;
            if (a.lse2) a.lse2[(uint64_t)n * a.q_heads + qh] = lse2;
        }
    }
}

// Adds the weights of kScoreKeys keys of a KV head.  Bound by HBM, logits in and
// scores in and out, and by the chain of their loads: 16 sequences of 16,000
// tokens, 4 heads of 5 query heads, take 101 us with weights and 85 without (with
// four keys a thread in place of eight 103).
__global__ void __launch_bounds__(kScoreThreads) k_scores(const __grid_constant__ Args a, uint32_t chunks) {
    __shared__ float sh_lse[kMaxGroup];
    const uint32_t row = blockIdx.x / chunks, n = row / a.c.heads, head = row % a.c.heads;
    const uint32_t i0 = blockIdx.x % chunks * kScoreKeys + threadIdx.x;
    const Seen sv = seen(a, a.lens[n]);
    const uint32_t gp = (a.group + 1) & ~1u;
    float *to = a.scores + (uint64_t)row * a.scores_stride;
    const float2 *x[kScoreUnroll];  // the keys' logits, two query heads a load
    float old[kScoreUnroll], w[kScoreUnroll] = {};
    if (i0 - threadIdx.x >= sv.n) {
        // The grid must not end before those that it depends on, even where no
        // sequence shows a token: one block that waits is enough for that.
        if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
#pragma unroll
    for (int u = 0; u < kScoreUnroll; u++) {
        const uint32_t i = i0 + u * kScoreThreads < sv.n ? i0 + u * kScoreThreads : sv.n - 1;
        x[u] = reinterpret_cast<const float2 *>(a.logits + ((uint64_t)row * a.logits_keys + i) * gp);
        old[u] = to[sv.token(i)];  // (of earlier calls: nothing that runs now writes it)
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float2 next[kScoreUnroll];
#pragma unroll
    for (int u = 0; u < kScoreUnroll; u++) next[u] = x[u][0];
    for (uint32_t i = threadIdx.x; i < gp; i += kScoreThreads) {
        const float lse2 = i < a.group ? a.lse2[(uint64_t)n * a.q_heads + head * a.group + i] : -INFINITY;
        sh_lse[i] = lse2 == -INFINITY ? INFINITY : lse2;  // no finite logit, no weight: 2^(-inf - inf) = 0
    }
    __syncthreads();
    for (uint32_t k = 0; k < a.group; k += 2) {
        const float l0 = sh_lse[k], l1 = sh_lse[k + 1];
        const bool both = k + 1 < a.group;
#pragma unroll
        for (int u = 0; u < kScoreUnroll; u++) {
            const float2 v = next[u];
            if (k + 2 < a.group) next[u] = x[u][k / 2 + 1];
            w[u] += exp2f(v.x - l0);
            if (both) w[u] += exp2f(v.y - l1);
        }
    }
#pragma unroll
    for (int u = 0; u < kScoreUnroll; u++) {
        const uint32_t i = i0 + u * kScoreThreads, pos = sv.token(i);
        if (i < sv.n && (pos < sv.sinks || pos >= sv.recent)) to[pos] = old[u] + w[u];
    }
}

struct Plan {
    uint32_t dp, nt, unit_heads, units, max_len, tile, chunks, align;
    uint64_t max_seen, parts;  // parts: blocks that the workspace has room for
    bool split;
    size_t part_o, part_ml, cut, lse2, logits;  // elements
};

// Sizes that follow from the host's arguments; false where they are refused.
bool plan(const kvx_cache *c, uint32_t num_seqs, uint32_t q_heads, uint32_t blocks_per_seq, uint32_t window,
          uint32_t sinks, bool scores, Plan &p) {
    if (!cache_ok(c) || c->scale_offset || !q_heads || q_heads % c->heads || q_heads / c->heads > kMaxGroup) return false;
    const uint64_t max_len = (uint64_t)blocks_per_seq * c->page_tokens;
    if (q_heads > 65536u || max_len >= (1ull << 31) || num_seqs >= (1u << 24) || (uint64_t)num_seqs * q_heads >= (1ull << 30)) return false;
    const uint32_t group = q_heads / c->heads;
    p.max_len = (uint32_t)max_len;
    p.dp = c->dim <= 64 ? 64 : c->dim <= 128 ? 128 : 256;
    // 16 columns where the group needs them: keys and values are then read
    // once for 16 heads.
    p.nt = group > 8 ? 2 : 1;
    p.unit_heads = 8 * p.nt;
    p.units = c->heads * (uint32_t)ceil_div(group, p.unit_heads);
    p.align = c->page_tokens % 16 ? 1 : 16;
    const uint64_t shown = (uint64_t)window + sinks + 2 * (p.align - 1);  // with what alignment adds
    p.max_seen = window && shown < max_len ? shown : max_len;
    // Up to kWhole keys a unit is left to one block: splitting it would save
    // less than the second launch costs.
    p.tile = p.max_seen <= kWhole ? kWhole : kStep;
    const uint64_t unit_tiles = ceil_div(p.max_seen, p.tile);
    const uint64_t all = unit_tiles * p.units * num_seqs;
    // the kernel counts tiles, and what units cost beside them, in 32 bits
    if ((unit_tiles + kMaxExtra) * p.units * num_seqs >= 1ull << 31) return false;
    p.parts = all < kMaxBlocks ? all : kMaxBlocks;
    p.split = unit_tiles > 1;
    p.part_o = p.split ? 2 * p.parts * p.unit_heads * p.dp : 0;
    p.part_ml = p.split ? 2 * p.parts * p.unit_heads * 2 : 0;
    p.cut = p.split ? p.parts : 0;
    p.lse2 = scores ? (size_t)num_seqs * q_heads : 0;
    p.logits = scores ? (size_t)num_seqs * c->heads * p.max_seen * ((group + 1) & ~1u) : 0;
    p.chunks = scores ? (uint32_t)ceil_div(p.max_seen, kScoreKeys) : 0;
    return (uint64_t)num_seqs * c->heads * p.chunks < (1ull << 31);
}

size_t carve(const Plan &p, void *ws, Args *a) {
    Carver w(ws);
    float *po = w.take<float>(p.part_o), *pm = w.take<float>(p.part_ml);
    uint4 *ct = w.take<uint4>(p.cut);
    float *ls = w.take<float>(p.lse2), *lg = w.take<float>(p.logits);
    if (a) a->part_o = po, a->part_ml = pm, a->cut = p.cut ? ct : nullptr, a->lse2 = p.lse2 ? ls : nullptr, a->logits = p.logits ? lg : nullptr;
    return w.off;
}

}  // namespace
}  // namespace attend
}  // namespace kvx

extern "C" size_t kvx_attend_workspace_size(const kvx_cache *cache, uint32_t num_seqs, uint32_t q_heads,
                                            uint32_t blocks_per_seq, uint32_t window, uint32_t sinks,
                                            uint32_t with_scores) {
    kvx::attend::Plan p;
    if (!kvx::attend::plan(cache, num_seqs, q_heads, blocks_per_seq, window, sinks, with_scores != 0, p)) return 0;
    return kvx::attend::carve(p, nullptr, nullptr);
}

extern "C" kvx_status kvx_attend(const kvx_cache *cache, const void *q, uint64_t q_stride, uint32_t dtype,
                                 uint32_t num_seqs, uint32_t q_heads, const uint32_t *blocks,
                                 uint32_t blocks_per_seq, const uint32_t *lens, float scale, uint32_t window,
                                 uint32_t sinks, void *out, uint64_t out_stride, float *lse, float *scores,
                                 uint64_t scores_stride, uint32_t *status, void *ws, size_t ws_bytes, void *stream) {
    using namespace kvx;
    using namespace kvx::attend;
    Plan p;
    if (!plan(cache, num_seqs, q_heads, blocks_per_seq, window, sinks, scores != nullptr, p)) return KVX_EINVAL;
    if ((dtype != KVX_BF16 && dtype != KVX_F16) || (cache->dtype != dtype && cache->dtype != KVX_E4M3)) return KVX_EINVAL;
    if (!status || !(scale > -INFINITY && scale < INFINITY)) return KVX_EINVAL;
    if ((q_stride | out_stride) % 8 || !aligned16(q) || !aligned16(out)) return KVX_EINVAL;
    if (scores && scores_stride < p.max_len) return KVX_EINVAL;
    if (!num_seqs) return KVX_OK;
    if (!q || !out || !lens || (p.max_len && !blocks)) return KVX_EINVAL;
    if (!ws || !aligned16(ws) || ws_bytes < carve(p, nullptr, nullptr)) return KVX_EINVAL;

    Args a = {};
    a.c = cache_view(cache);
    a.q = q, a.q_stride = q_stride, a.blocks = blocks, a.lens = lens;
    a.out = out, a.out_stride = out_stride, a.lse = lse, a.scores = scores, a.scores_stride = scores_stride;
    a.status = status;
    carve(p, ws, &a);
    a.logits_keys = p.max_seen;
    a.scale2 = scale * cache->k_scale * 1.4426950408889634f;
    a.num_seqs = num_seqs, a.q_heads = q_heads, a.group = q_heads / cache->heads, a.units = p.units;
    a.blocks_per_seq = blocks_per_seq, a.max_len = p.max_len, a.window = window, a.sinks = sinks, a.tile = p.tile, a.align = p.align;
    const cudaStream_t s = as_stream(stream);
    const uint32_t es = elem_size(cache->dtype);
    const bool ok = dtype == KVX_BF16
                        ? (es == 2 ? launch<__nv_bfloat16, 2>(a, p.parts, cache->dim, p.nt, s)
                                   : launch<__nv_bfloat16, 1>(a, p.parts, cache->dim, p.nt, s))
                        : (es == 2 ? launch<__half, 2>(a, p.parts, cache->dim, p.nt, s)
                                   : launch<__half, 1>(a, p.parts, cache->dim, p.nt, s));
    if (!ok) return KVX_ECUDA;
    KVX_LAUNCHED();

    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.split) {
        // A cut unit's heads go to several blocks where it has more parts than
        // one block has loads in flight for: 1 sequence of 16,000 tokens, 32
        // query heads to its KV head 45 us in one, 21 in six; 8 sequences, 4
        // heads, 85.3 in one, 85.9 in two, as blocks without a cut cost too.
        const uint64_t heads = a.group < p.unit_heads ? a.group : p.unit_heads;
        const uint64_t parts = ceil_div(a.grid, (uint64_t)num_seqs * p.units) * heads;
        const uint64_t want = ceil_div(parts, kJoinWarps * kJoinUnroll), fit = 12ull * sm_count() / a.grid;
        const uint64_t y = want < heads ? want : heads;
        cfg.gridDim = dim3(a.grid, (uint32_t)(y < fit ? y : fit ? fit : 1));
        cfg.blockDim = dim3(32 * kJoinWarps);
        const cudaError_t e = dtype == KVX_BF16 ? cudaLaunchKernelEx(&cfg, k_join<__nv_bfloat16>, a, p.dp, p.unit_heads)
                                                : cudaLaunchKernelEx(&cfg, k_join<__half>, a, p.dp, p.unit_heads);
        if (e != cudaSuccess) return KVX_ECUDA;
        KVX_LAUNCHED();
    }
    if (p.chunks) {
        cfg.gridDim = dim3(num_seqs * cache->heads * p.chunks);
        cfg.blockDim = dim3(kScoreThreads);
        if (cudaLaunchKernelEx(&cfg, k_scores, a, p.chunks) != cudaSuccess) return KVX_ECUDA;
        KVX_LAUNCHED();
    }
    return KVX_OK;
}
