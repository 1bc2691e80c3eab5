// kvx_evict: sequences cut to a budget of tokens per KV head, by the attention
// weight that each token has gathered.
//
// k_select, a block per (sequence, head), finds the M-th largest score among
// the tokens that have to compete with a radix select over order-preserving
// 32-bit keys (digits of 11, 11 and 10 bits from the top: a histogram of the
// scores that share the digits found so far, then the digit in which the M-th
// lies), so the threshold is exact and nothing is sorted.  What is over it, the
// first of its equals, the sinks and the last tokens are then written in order:
// each warp counts its own stretch, a scan over the warps gives their places.
// k_gather copies the kept rows.
#include "kvx_cache.cuh"

namespace kvx {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kRows = 64;  // tokens whose K and V rows a block of k_gather copies
constexpr int kGatherThreads = 256;

struct EvictArgs {
    CacheView c;
    const uint32_t *blocks, *lens;
    const float *scores;
    uint64_t scores_stride;
    const uint32_t *dst_blocks;
    uint32_t *kept;
    float *kept_scores;
    uint32_t *new_lens, *status;
    uint32_t num_seqs, blocks_per_seq, dst_per_seq, max_len, budget, sinks, recent;
};

// Larger key = larger score; -0 = +0, and a NaN ranks with -infinity.
__device__ __forceinline__ uint32_t key_of(float f) {
    uint32_t u = __float_as_uint(f);
    if (f != f) u = 0xFF800000u;
    if (u == 0x80000000u) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) k_select(const __grid_constant__ EvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t sh_scan[33];
    __shared__ uint32_t sh_digit, sh_left;
    __shared__ uint32_t sh_over[kSelWarps], sh_ties[kSelWarps];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t n = blockIdx.x / a.c.heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t len = a.lens[n];
    if (len > a.max_len) {
        if (threadIdx.x == 0) raise(a.status, KVX_S_BOUNDS);
        len = a.max_len;
    }
    const float *x = a.scores + blockIdx.x * a.scores_stride;
    uint32_t *kept = a.kept + (uint64_t)blockIdx.x * a.budget;
    float *ks = a.kept_scores + (uint64_t)blockIdx.x * a.budget;
    const uint32_t keep = len < a.budget ? len : a.budget;
    if (threadIdx.x == 0 && blockIdx.x % a.c.heads == 0) a.new_lens[n] = keep;
    for (uint32_t i = keep + threadIdx.x; i < a.budget; i += kSelThreads) {
        kept[i] = kNone;
        ks[i] = 0.0f;
    }
    if (len <= a.budget) {
        for (uint32_t i = threadIdx.x; i < len; i += kSelThreads) {
            kept[i] = i;
            ks[i] = x[i];
        }
        return;
    }
    const uint32_t lo = a.sinks < a.budget ? a.sinks : a.budget;
    const uint32_t recent = a.recent < a.budget - lo ? a.recent : a.budget - lo;
    const uint32_t hi = len - recent;  // tokens lo .. hi-1 compete for `take` places
    const uint32_t take = a.budget - lo - recent;

    // the threshold: the take-th largest key, and how many of its equals stay
    uint32_t cut = 0, left = take;
    if (take) {
#pragma unroll 1
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bins = pass == 2 ? 1024 : 2048;
            const uint32_t known = pass == 0 ? 0 : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
            for (uint32_t i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (uint32_t i = lo + threadIdx.x; i < hi; i += kSelThreads) {
                const uint32_t k = key_of(__ldg(x + i));
                if ((k & known) == cut) atomicAdd(&hist[k >> shift & (bins - 1)], 1u);
            }
            __syncthreads();
            // two bins a thread, from the largest down
            const uint32_t b1 = kBins - 1 - 2 * threadIdx.x, b0 = b1 - 1;
            const uint32_t h1 = hist[b1], h0 = hist[b0];
            uint32_t total;
            const uint32_t above = block_excl_sum<uint32_t>(h1 + h0, sh_scan, &total);
            if (above < left && above + h1 >= left) {
                sh_digit = b1;
                sh_left = left - above;
            } else if (above + h1 < left && above + h1 + h0 >= left) {
                sh_digit = b0;
                sh_left = left - above - h1;
            }
            __syncthreads();
            cut |= sh_digit << shift;
            left = sh_left;
            __syncthreads();
        }
    }

    // every warp counts its stretch, then writes it at its place
    const uint32_t per = ((len + kSelWarps - 1) / kSelWarps + 31) & ~31u;
    const uint32_t from = warp * per < len ? warp * per : len, to = from + per < len ? from + per : len;
    auto classify = [&](uint32_t i, bool &over, bool &tie) {
        const uint32_t k = i < to ? key_of(__ldg(x + i)) : 0;
        const bool competes = i >= lo && i < hi;
        over = i < to && (!competes || (take && k > cut));
        tie = i < to && competes && take && k == cut;
    };
    uint32_t n_over = 0, n_ties = 0;
    for (uint32_t i0 = from; i0 < to; i0 += 32) {
        bool over, tie;
        classify(i0 + lane, over, tie);
        n_over += __popc(__ballot_sync(0xFFFFFFFFu, over));
        n_ties += __popc(__ballot_sync(0xFFFFFFFFu, tie));
    }
    if (lane == 0) sh_over[warp] = n_over, sh_ties[warp] = n_ties;
    __syncthreads();
    uint32_t over_before = 0, ties_before = 0;
    for (uint32_t w = 0; w < warp; w++) over_before += sh_over[w], ties_before += sh_ties[w];
    for (uint32_t i0 = from; i0 < to; i0 += 32) {
        const uint32_t i = i0 + lane;
        bool over, tie;
        classify(i, over, tie);
        const uint32_t mo = __ballot_sync(0xFFFFFFFFu, over), mt = __ballot_sync(0xFFFFFFFFu, tie);
        const uint32_t below = (1u << lane) - 1;
        const uint32_t ties = ties_before + __popc(mt & below);
        if (over || (tie && ties < left)) {
            const uint32_t at = over_before + __popc(mo & below) + (ties < left ? ties : left);
            kept[at] = i;
            ks[at] = __ldg(x + i);
        }
        over_before += __popc(mo);
        ties_before += __popc(mt);
    }
}

// Copies kRows tokens' K and V rows: a thread looks up each row's two places,
// then all threads move 16-byte pieces.
__global__ void __launch_bounds__(kGatherThreads) k_gather(const __grid_constant__ EvictArgs a, FastDiv pieces) {
    __shared__ uint64_t sh_src[2 * kRows], sh_dst[2 * kRows];
    const uint32_t per = (a.budget + kRows - 1) / kRows;
    const uint32_t nh = blockIdx.x / per, r0 = blockIdx.x % per * kRows;
    const uint32_t n = nh / a.c.heads, h = nh % a.c.heads;
    const uint32_t len = a.lens[n] < a.max_len ? a.lens[n] : a.max_len;
    const uint32_t keep = len < a.budget ? len : a.budget;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (r0 >= keep) return;
    const uint32_t rows = keep - r0 < kRows ? keep - r0 : kRows;
    if (threadIdx.x < 2 * rows) {
        const uint32_t r = r0 + threadIdx.x / 2, kv = threadIdx.x & 1;
        const uint32_t pos = __ldcg(a.kept + (uint64_t)nh * a.budget + r);
        const uint32_t ps = a.c.page.div(pos), pd = a.c.page.div(r);
        const uint32_t bs = __ldg(a.blocks + (uint64_t)n * a.blocks_per_seq + ps);
        const uint32_t bd = __ldg(a.dst_blocks + (uint64_t)n * a.dst_per_seq + pd);
        uint32_t bad = bs < a.c.B && bd < a.c.B ? 0 : KVX_S_BOUNDS;
        uint64_t src = ~0ull, dst = 0;
        if (!bad) {
            const uint64_t s = __ldg(a.c.lane_addr(bs, h, kv)), d = __ldg(a.c.lane_addr(bd, h, kv));
            const bool ok_s = a.c.ok(s, bad), ok_d = a.c.ok(d, bad);
            if (ok_s && ok_d) {
                src = s + (pos - ps * a.c.page.d) * a.c.token_stride;
                dst = d + (r - pd * a.c.page.d) * a.c.token_stride;
            }
        }
        sh_src[threadIdx.x] = src;
        sh_dst[threadIdx.x] = dst;
        raise(a.status, bad);
    }
    __syncthreads();
    const uint32_t items = 2 * rows * pieces.d;
    constexpr int kUnroll = 8;
    for (uint32_t i0 = threadIdx.x; i0 < items; i0 += kUnroll * kGatherThreads) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t i = i0 + u * kGatherThreads;
            if (i >= items) break;
            const uint32_t r = pieces.div(i);
            if (sh_src[r] != ~0ull)
                v[u] = __ldcs(reinterpret_cast<const uint4 *>(a.c.pool + sh_src[r]) + (i - r * pieces.d));
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const uint32_t i = i0 + u * kGatherThreads;
            if (i >= items) break;
            const uint32_t r = pieces.div(i);
            if (sh_src[r] != ~0ull)
                *(reinterpret_cast<uint4 *>(a.c.pool + sh_dst[r]) + (i - r * pieces.d)) = v[u];
        }
    }
}

bool sizes_ok(const kvx_cache *c, uint32_t num_seqs, uint32_t blocks_per_seq, uint32_t budget) {
    if (!cache_ok(c) || !budget || budget >= (1u << 31)) return false;
    if ((uint64_t)blocks_per_seq * c->page_tokens >= (1ull << 31)) return false;
    return ceil_div(budget, kRows) * c->heads * (uint64_t)num_seqs < (1ull << 31);
}

}  // namespace
}  // namespace kvx

extern "C" size_t kvx_evict_workspace_size(const kvx_cache *cache, uint32_t num_seqs, uint32_t blocks_per_seq,
                                           uint32_t budget) {
    return kvx::sizes_ok(cache, num_seqs, blocks_per_seq, budget) ? 256 : 0;
}

extern "C" kvx_status kvx_evict(const kvx_cache *cache, uint32_t num_seqs, const uint32_t *blocks,
                                uint32_t blocks_per_seq, const uint32_t *lens, const float *scores,
                                uint64_t scores_stride, uint32_t budget, uint32_t sinks, uint32_t recent,
                                const uint32_t *dst_blocks, uint32_t dst_per_seq, uint32_t *kept, float *kept_scores,
                                uint32_t *new_lens, uint32_t *status, void *ws, size_t ws_bytes, void *stream) {
    using namespace kvx;
    if (!sizes_ok(cache, num_seqs, blocks_per_seq, budget) || !status) return KVX_EINVAL;
    const uint64_t max_len = (uint64_t)blocks_per_seq * cache->page_tokens;
    if (scores_stride < max_len || (uint64_t)dst_per_seq * cache->page_tokens < budget) return KVX_EINVAL;
    if (!num_seqs) return KVX_OK;
    if (!lens || !kept || !kept_scores || !new_lens || !dst_blocks || (max_len && (!blocks || !scores)))
        return KVX_EINVAL;
    if (!ws || ws_bytes < kvx_evict_workspace_size(cache, num_seqs, blocks_per_seq, budget)) return KVX_EINVAL;
    EvictArgs a = {cache_view(cache), blocks, lens, scores, scores_stride, dst_blocks, kept, kept_scores, new_lens,
                   status, num_seqs, blocks_per_seq, dst_per_seq, (uint32_t)max_len, budget, sinks, recent};
    const cudaStream_t s = as_stream(stream);
    k_select<<<num_seqs * cache->heads, kSelThreads, 0, s>>>(a);
    KVX_LAUNCHED();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((uint32_t)ceil_div(budget, kRows) * cache->heads * num_seqs);
    cfg.blockDim = dim3(kGatherThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_gather, a, FastDiv(a.c.row_bytes / 16)) != cudaSuccess) return KVX_ECUDA;
    KVX_LAUNCHED();
    return KVX_OK;
}
