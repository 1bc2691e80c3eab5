// kvx_attend: attention of one new token per sequence over a paged cache.
//
// Two launches.  k_attend (kvx_attend.cuh) walks equal shares of all
// sequences' tiles, one per block; a unit (the query heads of one KV head of
// one sequence) that lies in one share is finished there, one that is cut by
// share borders leaves partial outputs with their bases m and sums l.  k_finish
// joins those,
//     M = max m_c,  L = sum l_c 2^(m_c - M),  out = sum o_c 2^(m_c - M) / L
// in the order of the blocks, and adds the attention weights 2^(logit - lse)
// to the scores: a weight needs the sum over all keys, so the logits pass
// through the workspace (4 bytes per key and query head, beside 2*dim*size
// bytes of key and value per KV head).  It starts beside k_attend's last
// blocks (programmatic dependency) and waits for their results.
#include "kvx_attend.cuh"

namespace kvx {
namespace attend {

// instantiated in kvx_attend_<types>.cu, a file each so that they compile in parallel
extern template bool launch<__nv_bfloat16, 2>(const Args &, uint32_t, uint32_t, cudaStream_t);
extern template bool launch<__nv_bfloat16, 1>(const Args &, uint32_t, uint32_t, cudaStream_t);
extern template bool launch<__half, 2>(const Args &, uint32_t, uint32_t, cudaStream_t);
extern template bool launch<__half, 1>(const Args &, uint32_t, uint32_t, cudaStream_t);

namespace {

constexpr uint32_t kMaxGroup = 128;
constexpr uint32_t kScoreKeys = 1024;  // of a block that adds weights

// The blocks of k_attend that hold a unit's parts: first .. last, the first
// one's part in its first or second slot.
struct Parts {
    uint64_t first, last;
    bool second;
    __device__ __forceinline__ uint64_t slot(uint64_t c) const { return 2 * c + (c == first && second); }
};

__device__ __forceinline__ Parts parts_of(uint64_t tile, uint32_t nt, uint64_t share) {
    return Parts{tile / share, (tile + nt - 1) / share, tile % share != 0};
}

// Blocks 0 .. num_seqs*q_heads-1 join a query head each; the others add the
// weights of kScoreKeys keys of a KV head.
template <class T>
__global__ void __launch_bounds__(kThreads) k_finish(const __grid_constant__ Args a, uint32_t dp, uint32_t unit_heads,
                                                     uint32_t chunks) {
    __shared__ uint64_t sh_sum[kWarps];
    __shared__ float sh_lse[kMaxGroup];
    __shared__ float4 sh_o[kWarps][32];
    __shared__ float sh_l[kWarps];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t joins = a.num_seqs * a.q_heads;
    const bool join = blockIdx.x < joins;
    const uint32_t r = join ? 0 : blockIdx.x - joins;
    const uint32_t n = join ? blockIdx.x / a.q_heads : r / chunks / a.c.heads;
    const uint32_t head = join ? blockIdx.x % a.q_heads / a.group : r / chunks % a.c.heads;

    uint64_t mine = 0, mine_before = 0;
    for (uint32_t i = threadIdx.x; i < a.num_seqs; i += kThreads) {
        const uint32_t k = tiles(seen(a, a.lens[i]).n);
        mine += k;
        if (i < n) mine_before += k;
    }
    const uint64_t share = share_of(block_sum(mine, sh_sum) * a.units, a.grid);
    const uint64_t before = block_sum(mine_before, sh_sum) * a.units;
    const Seen sv = seen(a, a.lens[n]);
    const uint32_t nt = tiles(sv.n);
    const uint32_t per_head = (a.group + unit_heads - 1) / unit_heads;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!nt) return;

    if (join) {
        const uint32_t qh = blockIdx.x % a.q_heads, in = qh % a.group;
        const Parts p = parts_of(before + (uint64_t)(head * per_head + in / unit_heads) * nt, nt, share);
        if (p.first == p.last) return;
        const uint32_t hh = in % unit_heads;
        float top = -INFINITY;
        for (uint64_t c = p.first; c <= p.last; c++)
            top = fmaxf(top, __ldcg(a.part_ml + (p.slot(c) * unit_heads + hh) * 2));
        // warp w takes parts w, w+4, ...; a lane four of 128 values at a time
        for (uint32_t d0 = 0; d0 < dp; d0 += 128) {
            const uint32_t d = d0 + lane * 4;
            float4 v = make_float4(0, 0, 0, 0);
            float sum = 0;
#pragma unroll 4
            for (uint64_t c = p.first + warp; c <= p.last; c += kWarps) {
                const uint64_t s = p.slot(c) * unit_heads + hh;
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + s);
                const float4 x = d < dp ? __ldcg(reinterpret_cast<const float4 *>(a.part_o + s * dp + d))
                                        : make_float4(0, 0, 0, 0);
                const float f = ml.x == -INFINITY ? 1.0f : exp2f(ml.x - top);
                sum += ml.y * f;
                v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
            }
            sh_o[warp][lane] = v;
            if (lane == 0) sh_l[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                sum = sh_l[0];
#pragma unroll
                for (int w = 1; w < kWarps; w++) {
                    const float4 x = sh_o[w][lane];
                    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                    sum += sh_l[w];
                }
                const float inv = sum == 0 ? 0.0f : a.c.v_scale / sum;
                if (d < a.c.dim) {
                    T *to = static_cast<T *>(a.out) + (uint64_t)n * a.out_stride + (uint64_t)qh * a.c.dim + d;
                    *reinterpret_cast<uint2 *>(to) =
                        make_uint2(Pair<T>::pack(v.x * inv, v.y * inv), Pair<T>::pack(v.z * inv, v.w * inv));
                }
                if (d == 0 && a.lse)
                    a.lse[(uint64_t)n * a.q_heads + qh] =
                        sum == 0 ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            }
            __syncthreads();
        }
        return;
    }

    const uint32_t i0 = r % chunks * kScoreKeys;
    if (i0 >= sv.n) return;
    for (uint32_t in = warp; in < a.group; in += kWarps) {
        const Parts p = parts_of(before + (uint64_t)(head * per_head + in / unit_heads) * nt, nt, share);
        float lse2;
        if (p.first == p.last) {
            lse2 = __ldcg(a.lse2 + (uint64_t)n * a.q_heads + head * a.group + in);
        } else {
            const uint32_t hh = in % unit_heads;
            float top = -INFINITY, sum = 0;
            for (uint64_t c = p.first + lane; c <= p.last; c += 32)
                top = fmaxf(top, __ldcg(a.part_ml + (p.slot(c) * unit_heads + hh) * 2));
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            for (uint64_t c = p.first + lane; c <= p.last; c += 32) {
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + p.slot(c) * unit_heads + hh);
                sum += ml.y * (ml.x == -INFINITY ? 1.0f : exp2f(ml.x - top));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            lse2 = sum == 0 ? -INFINITY : top + log2f(sum);
        }
        // a head without a finite logit gives no weight: exp2(-inf - inf) = 0
        if (lane == 0) sh_lse[in] = lse2 == -INFINITY ? INFINITY : lse2;
    }
    __syncthreads();
    const uint32_t gp = (a.group + 1) & ~1u;
    const uint64_t row = (uint64_t)n * a.c.heads + head;
    for (uint32_t i = i0 + threadIdx.x; i < sv.n && i < i0 + kScoreKeys; i += kThreads) {
        const float2 *x = reinterpret_cast<const float2 *>(a.logits + (row * a.logits_keys + i) * gp);
        float *to = a.scores + row * a.scores_stride + (i < sv.sinks ? i : i + sv.shift);
        const float old = *to;
        float w = 0;
        for (uint32_t k = 0; k < a.group; k += 2) {
            const float2 v = __ldcg(x + k / 2);
            w += exp2f(v.x - sh_lse[k]);
            if (k + 1 < a.group) w += exp2f(v.y - sh_lse[k + 1]);
        }
        *to = old + w;
    }
}

struct Plan {
    uint32_t dp, nt, unit_heads, units, max_len, grid, chunks;
    uint64_t max_seen, parts;
    bool split;
    size_t part_o, part_ml, lse2, logits;  // elements
};

// Sizes that follow from the host's arguments; false where they are refused.
bool plan(const kvx_cache *c, uint32_t num_seqs, uint32_t q_heads, uint32_t blocks_per_seq, uint32_t window,
          uint32_t sinks, bool scores, Plan &p) {
    if (!cache_ok(c) || !q_heads || q_heads % c->heads || q_heads / c->heads > kMaxGroup) return false;
    const uint64_t max_len = (uint64_t)blocks_per_seq * c->page_tokens;
    if (max_len >= (1ull << 31) || num_seqs >= (1u << 24) || (uint64_t)num_seqs * q_heads >= (1ull << 30)) return false;
    const uint32_t group = q_heads / c->heads;
    p.max_len = (uint32_t)max_len;
    p.dp = c->dim <= 64 ? 64 : c->dim <= 128 ? 128 : 256;
    // 16 columns where the group needs them: keys and values are then read
    // once for 16 heads.  At 256 values a head their accumulators would not
    // leave registers enough, and the heads are taken eight at a time.
    p.nt = group > 8 && p.dp < 256 ? 2 : 1;
    p.unit_heads = 8 * p.nt;
    p.units = c->heads * (uint32_t)ceil_div(group, p.unit_heads);
    p.max_seen = !window ? max_len : (uint64_t)window + sinks < max_len ? (uint64_t)window + sinks : max_len;
    const uint64_t unit_tiles = ceil_div(p.max_seen, kTile);
    const uint64_t all = unit_tiles * p.units * num_seqs;
    p.parts = all < kMaxBlocks ? all : kMaxBlocks;
    p.split = unit_tiles > 1;
    p.part_o = p.split ? 2 * p.parts * p.unit_heads * p.dp : 0;
    p.part_ml = p.split ? 2 * p.parts * p.unit_heads * 2 : 0;
    p.lse2 = scores ? (size_t)num_seqs * q_heads : 0;
    p.logits = scores ? (size_t)num_seqs * c->heads * p.max_seen * ((group + 1) & ~1u) : 0;
    p.chunks = scores ? (uint32_t)ceil_div(p.max_seen, kScoreKeys) : 0;
    return (uint64_t)num_seqs * (q_heads + (uint64_t)c->heads * p.chunks) < (1ull << 31);
}

size_t carve(const Plan &p, void *ws, Args *a) {
    Carver w(ws);
    float *po = w.take<float>(p.part_o), *pm = w.take<float>(p.part_ml);
    float *ls = w.take<float>(p.lse2), *lg = w.take<float>(p.logits);
    if (a) a->part_o = po, a->part_ml = pm, a->lse2 = p.lse2 ? ls : nullptr, a->logits = p.logits ? lg : nullptr;
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
    if (!ws || ws_bytes < carve(p, nullptr, nullptr)) return KVX_EINVAL;

    Args a = {};
    a.c = cache_view(cache);
    a.q = q, a.q_stride = q_stride, a.blocks = blocks, a.lens = lens;
    a.out = out, a.out_stride = out_stride, a.lse = lse, a.scores = scores, a.scores_stride = scores_stride;
    a.status = status;
    carve(p, ws, &a);
    a.logits_keys = p.max_seen;
    a.scale2 = scale * cache->k_scale * 1.4426950408889634f;
    a.num_seqs = num_seqs, a.q_heads = q_heads, a.group = q_heads / cache->heads, a.units = p.units;
    a.blocks_per_seq = blocks_per_seq, a.max_len = p.max_len, a.window = window, a.sinks = sinks;
    const uint64_t room = (uint64_t)sm_count() * 2;
    a.grid = (uint32_t)(p.parts < room ? p.parts : room);
    if (!a.grid) a.grid = 1;  // nothing to see anywhere: the zeros still have to be written
    const cudaStream_t s = as_stream(stream);
    const uint32_t es = elem_size(cache->dtype);
    const bool ok = dtype == KVX_BF16
                        ? (es == 2 ? launch<__nv_bfloat16, 2>(a, cache->dim, p.nt, s)
                                   : launch<__nv_bfloat16, 1>(a, cache->dim, p.nt, s))
                        : (es == 2 ? launch<__half, 2>(a, cache->dim, p.nt, s) : launch<__half, 1>(a, cache->dim, p.nt, s));
    if (!ok) return KVX_ECUDA;
    KVX_LAUNCHED();
    if (!p.split && !scores) return KVX_OK;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_seqs * (q_heads + cache->heads * p.chunks));
    cfg.blockDim = dim3(attend::kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == KVX_BF16
                              ? cudaLaunchKernelEx(&cfg, k_finish<__nv_bfloat16>, a, p.dp, p.unit_heads, p.chunks)
                              : cudaLaunchKernelEx(&cfg, k_finish<__half>, a, p.dp, p.unit_heads, p.chunks);
    if (e != cudaSuccess) return KVX_ECUDA;
    KVX_LAUNCHED();
    return KVX_OK;
}
