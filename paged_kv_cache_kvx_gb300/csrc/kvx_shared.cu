// kvx_attend_shared: attention of one new token per sequence over a prefix that
// a group of sequences shares, and the sequence's own tokens.
//
// k_shared (kvx_shared.cuh) leaves partial results o_c = sum 2^(x_j - m_c) v_j,
// l_c = sum 2^(x_j - m_c) of prefixes and of own tokens, logits x in powers of
// two; k_join puts a query's together,
//     M = max m_c,  L = sum l_c 2^(m_c - M),  out = sum o_c 2^(m_c - M) / L
// in a fixed order.
#include "kvx_shared.cuh"

namespace kvx {
namespace shared {

// instantiated in kvx_shared_<types>.cu, a file each so that they compile in parallel
extern template bool launch<__nv_bfloat16, 2>(const Args &, cudaStream_t);
extern template bool launch<__nv_bfloat16, 1>(const Args &, cudaStream_t);
extern template bool launch<__half, 2>(const Args &, cudaStream_t);
extern template bool launch<__half, 1>(const Args &, cudaStream_t);

namespace {

constexpr uint32_t kJoinWarps = 4;
constexpr int kJoinUnroll = 4;        // parts whose loads a warp has in flight

// A query's parts by WARPS warps, blocks of kJoinWarps.  Bound by the chain of its
// reads (group, lengths, which blocks, bases and sums, outputs), so many warps in
// one wave: 8192 queries of about seven parts by one warp each 16 us, by four 35;
// but 8 queries over 131,071 tokens of one KV head, 300 parts each, in all 67 us by
// one, 41 by four.  For the same reason heads of up to 128 have kernels of their own,
// with 72 registers for 88: 28 warps an SM (8192 queries, 100,000 shared tokens, in all
// 372 us with 88, 368 with 72, 369 with 64, which spills; 32,768 of one piece 84 and 78).
template <class T, uint32_t WARPS, bool WIDE>
__global__ void __launch_bounds__(32 * kJoinWarps, WIDE ? 5 : 7) k_join(const __grid_constant__ Args a) {
    __shared__ float sh_m[WARPS > 1 ? kJoinWarps : 1], sh_l[WARPS > 1 ? kJoinWarps : 1];
    constexpr int kQuads = WIDE ? 2 : 1;  // four outputs that a lane has, and those 128 further
    __shared__ float4 sh_o[WARPS > 1 ? kJoinWarps : 1][WARPS > 1 ? 32 * kQuads : 1];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32, turn = warp % WARPS;
    const uint64_t query = (uint64_t)blockIdx.x * (kJoinWarps / WARPS) + warp / WARPS;
    const bool has = query < (uint64_t)a.num_seqs * a.q_heads;
    const uint32_t n = has ? (uint32_t)(query / a.q_heads) : 0, x = has ? (uint32_t)(query - (uint64_t)n * a.q_heads) : 0;
    const uint32_t head = a.by_group.div(x), in = x - head * a.group;
    // the group: the last that starts at n or before
    uint32_t lo = 0, hi = a.num_groups;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (__ldg(a.group_first + mid) <= n)
            lo = mid + 1;
        else
            hi = mid;
    }
    Parts parts[2] = {};
    uint2 const *where[2] = {};
    Entry entry[2] = {};
    if (lo) {
        const Entry e = entry_of(a, lo - 1);
        if (e.len && n - e.seq0 < e.rows / a.group) {
            entry[0] = e;
            where[0] = a.group_at + lo - 1;
        }
    }
    entry[1] = entry_of(a, a.num_groups + n);
    if (entry[1].len) where[1] = a.own_parts + (uint64_t)n * a.c.heads + head;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint2 w[2] = {};
    for (int k = 0; k < 2; k++)
        if (where[k]) w[k] = __ldcg(where[k]);
    if (where[0] && w[0].y) {
        parts[0] = prefix_parts(a, entry[0], w[0], lo - 1, n, head, in, WIDE);
    }
    if (where[1] && w[1].x <= w[1].y && w[1].y < a.grid) {  // (else left by a block whose wait ran out)
        parts[1] = own_parts(a, w[1], n, head, in, WIDE);
    }
    // A call that ended early, by a table in disorder or a wait that ran out, may
    // leave anything.
    const uint64_t counted = (uint64_t)parts[0].blocks * parts[0].each * parts[0].subs + parts[1].count();
    const uint32_t first = parts[0].count(), all = counted > most_parts(a) ? 0 : (uint32_t)counted;
    const uint32_t most = (uint32_t)(a.rows < kNone ? a.rows : kNone);
    auto at = [&](uint32_t i) {
        const uint32_t row = i < first ? parts[0].at(i) : parts[1].at_own(i - first);
        return row < most ? row : kNone;
    };
    // A warp's share, 32 parts at a time: a lane has one's base and sum; 0 stands
    // for none, whose outputs do not exist.
    float top = -INFINITY, sum = 0;
    float4 o[kQuads] = {};
    for (uint32_t i0 = turn * 32; i0 < all; i0 += 32 * WARPS) {
        const uint32_t here = all - i0 < 32 ? all - i0 : 32;
        float2 ml = make_float2(-INFINITY, 0);
        uint32_t row = 0;  // (rows are below 2^32)
        if (lane < here) row = at(i0 + lane);
        if (lane < here && row != kNone) ml = __ldcg(a.part_ml + row);
        if (ml.y == 0) ml.x = -INFINITY;
        float higher = ml.x;
        for (int d = 16; d; d >>= 1) higher = fmaxf(higher, __shfl_xor_sync(0xFFFFFFFFu, higher, d));
        higher = fmaxf(higher, top);
        const float old = top == -INFINITY ? 0.0f : exp2_fast(top - higher);
        // (an infinite base comes with a NaN sum, which stays one)
        const float weight = ml.y == 0 ? 0.0f : exp2_fast(ml.x - higher);
        top = higher;
        float s = ml.y == 0 ? 0.0f : ml.y * weight;
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        sum = sum * old + s;
#pragma unroll
        for (int k = 0; k < kQuads; k++) o[k].x *= old, o[k].y *= old, o[k].z *= old, o[k].w *= old;
        for (uint32_t i = 0; i < here; i += kJoinUnroll) {
            float4 v[kJoinUnroll][kQuads] = {};
            float f[kJoinUnroll];
#pragma unroll
            for (int u = 0; u < kJoinUnroll; u++) {
                f[u] = __shfl_sync(0xFFFFFFFFu, weight, i + u);  // 0 behind the last
                const float *from = a.part_o + (uint64_t)__shfl_sync(0xFFFFFFFFu, row, i + u) * a.c.dim;
                if (f[u] == 0) continue;  // (a NaN is none)
#pragma unroll
                for (int k = 0; k < kQuads; k++)
                    if (k * 128 + lane * 4 < a.c.dim) v[u][k] = __ldcg(reinterpret_cast<const float4 *>(from + k * 128) + lane);
            }
#pragma unroll
            for (int u = 0; u < kJoinUnroll; u++)
#pragma unroll
                for (int k = 0; k < kQuads; k++) {
                    o[k].x += v[u][k].x * f[u], o[k].y += v[u][k].y * f[u];
                    o[k].z += v[u][k].z * f[u], o[k].w += v[u][k].w * f[u];
                }
        }
    }
    if constexpr (WARPS > 1) {
        if (lane == 0) sh_m[warp] = top, sh_l[warp] = sum;
#pragma unroll
        for (int k = 0; k < kQuads; k++) sh_o[warp][k * 32 + lane] = o[k];
        __syncthreads();
        if (turn) return;
        top = -INFINITY, sum = 0;
        for (uint32_t k = 0; k < WARPS; k++) top = fmaxf(top, sh_m[warp + k]);
#pragma unroll
        for (int h = 0; h < kQuads; h++) o[h] = make_float4(0, 0, 0, 0);
        for (uint32_t k = 0; k < WARPS; k++) {
            const float f = sh_m[warp + k] == -INFINITY ? 0.0f : exp2_fast(sh_m[warp + k] - top);
            if (f == 0) continue;
            sum += sh_l[warp + k] * f;
#pragma unroll
            for (int h = 0; h < kQuads; h++) {
                const float4 v = sh_o[warp + k][h * 32 + lane];
                o[h].x += v.x * f, o[h].y += v.y * f, o[h].z += v.z * f, o[h].w += v.w * f;
            }
        }
    }
    if (!has) return;
    const float inv = sum == 0 ? 0.0f : a.c.v_scale / sum;
#pragma unroll
    for (int k = 0; k < kQuads; k++) {
        const uint32_t d = k * 128 + lane * 4;
        if (d >= a.c.dim) continue;
        T *to = static_cast<T *>(a.out) + (uint64_t)n * a.out_stride + (uint64_t)x * a.c.dim + d;
        *reinterpret_cast<uint2 *>(to) =
            make_uint2(Pair<T>::pack(o[k].x * inv, o[k].y * inv), Pair<T>::pack(o[k].z * inv, o[k].w * inv));
    }
    if (a.lse && lane == 0) a.lse[query] = sum == 0 ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <class T>
cudaError_t launch_join(const cudaLaunchConfig_t &cfg, bool four, bool wide, const Args &a) {
    return wide ? cudaLaunchKernelEx(&cfg, four ? k_join<T, 4, true> : k_join<T, 1, true>, a)
                : cudaLaunchKernelEx(&cfg, four ? k_join<T, 4, false> : k_join<T, 1, false>, a);
}

size_t carve(const Plan &p, const kvx_cache *c, uint32_t num_groups, void *ws, Args *a) {
    Carver w(ws);
    float *o = w.take<float>(p.rows * c->dim);
    float2 *ml = w.take<float2>(p.rows);
    uint2 *groups = w.take<uint2>(num_groups), *own = w.take<uint2>(p.own_units);
    if (a) a->part_o = o, a->part_ml = ml, a->group_at = groups, a->own_parts = own;
    return w.off;
}

}  // namespace
}  // namespace shared
}  // namespace kvx

extern "C" size_t kvx_attend_shared_workspace_size(const kvx_cache *cache, uint32_t num_seqs, uint32_t q_heads,
                                                   uint32_t blocks_per_seq, uint32_t num_groups,
                                                   uint32_t blocks_per_prefix) {
    using namespace kvx::shared;
    Plan p;
    return plan(cache, num_seqs, q_heads, blocks_per_seq, num_groups, blocks_per_prefix, kvx::sm_count(), p) ? carve(p, cache, num_groups, nullptr, nullptr) : 0;
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
    Plan p;
    if (!plan(cache, num_seqs, q_heads, blocks_per_seq, num_groups, blocks_per_prefix, sm_count(), p)) return KVX_EINVAL;
    if ((dtype != KVX_BF16 && dtype != KVX_F16) || (cache->dtype != dtype && cache->dtype != KVX_E4M3)) return KVX_EINVAL;
    if (!status || !(scale > -INFINITY && scale < INFINITY)) return KVX_EINVAL;
    if ((q_stride | out_stride) % 8 || !aligned16(q) || !aligned16(out)) return KVX_EINVAL;
    if (!num_seqs) return KVX_OK;
    if (!q || !out || !lens || (p.max_len && !blocks)) return KVX_EINVAL;
    if (num_groups && (!prefix_lens || !group_first || (p.max_prefix && !prefix_blocks))) return KVX_EINVAL;
    if (!ws || !aligned16(ws) || ws_bytes < carve(p, cache, num_groups, nullptr, nullptr)) return KVX_EINVAL;
    Args a = args_of(cache, num_seqs, q_heads, blocks_per_seq, num_groups, blocks_per_prefix, p);
    a.q = q, a.q_stride = q_stride;
    a.prefix_blocks = prefix_blocks, a.prefix_lens = prefix_lens, a.group_first = group_first;
    a.blocks = blocks, a.lens = lens;
    a.scale2 = fabsf(scale) * cache->k_scale * 1.4426950408889634f;
    if (a.scale2 == 0) a.scale2 = 1.4e-45f;  // the smallest: what is masked by -infinity stays masked
    a.negate = scale < 0;
    a.out = out, a.out_stride = out_stride, a.lse = lse, a.status = status;
    carve(p, cache, num_groups, ws, &a);
    const cudaStream_t s = as_stream(stream);
    const bool ok = dtype == KVX_BF16
                        ? (cache->dtype == KVX_E4M3 ? launch<__nv_bfloat16, 1>(a, s) : launch<__nv_bfloat16, 2>(a, s))
                        : (cache->dtype == KVX_E4M3 ? launch<__half, 1>(a, s) : launch<__half, 2>(a, s));
    if (!ok) return KVX_ECUDA;
    KVX_LAUNCHED();
    cudaLaunchConfig_t cfg = {};
    // four warps a query where that many fit on the device together
    const uint64_t queries = (uint64_t)num_seqs * q_heads;
    const bool four = queries <= 4ull * sm_count();
    cfg.gridDim = dim3((uint32_t)ceil_div(queries, four ? 1 : kJoinWarps));
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == KVX_BF16 ? launch_join<__nv_bfloat16>(cfg, four, cache->dim > 128, a) : launch_join<__half>(cfg, four, cache->dim > 128, a);
    if (e != cudaSuccess) return KVX_ECUDA;
    KVX_LAUNCHED();
    return KVX_OK;
}
