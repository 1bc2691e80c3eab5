// kvx_evict: sequences cut to a budget of tokens per KV head, by the attention
// weight that each token has gathered.
//
// k_select, a block per (sequence, head) or a cluster of up to eight, finds the
// M-th largest score among the tokens that have to compete with a radix select
// over order-preserving 32-bit keys (digits of 11, 11 and 10 bits from the top:
// a histogram of the scores that share the digits found so far, then the digit
// in which the M-th lies), so the threshold is exact and nothing is sorted.
// Each block keeps its part of the keys in shared memory, so the scores are
// read once; the blocks of a cluster add up each other's histograms through
// distributed shared memory.  What is over the threshold, the first of its
// equals, the sinks and the last tokens are then written in order: each warp
// counts its own stretch, sums over the warps and blocks before it give its
// places.  Bound by the latency of these steps and, with many heads, by their
// instructions: 24 sequences of up to 40,000 tokens, 8 heads, in 23 us.
// k_gather copies the kept rows, 0.8 GB read and written for those in 116 us,
// 6.9 TB/s: at HBM's rate.
#include "kvx_cache.cuh"

namespace kvx {
namespace {

constexpr int kBins = 2048;
constexpr uint32_t kHeld = 49152;  // keys that a block keeps in shared memory
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kShare = 2048;  // tokens for which a block of a cluster pays
constexpr uint32_t kTiny = 2048, kShort = 8192;  // tokens up to which smaller blocks are faster
constexpr int kDigits = 3;
constexpr int kSelUnroll = 2;  // groups of four tokens
// Keys that no score has: a token that is not there, and one that stays in any case.
constexpr uint32_t kAbsent = 0, kStays = 0xFFFFFFFFu;
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
    bool aligned;  // rows of scores to 16 bytes
};

// Larger key = larger score; -0 = +0, and a NaN ranks with -infinity.
__device__ __forceinline__ uint32_t key_of(float f) {
    const float g = f != f ? -INFINITY : f + 0.0f;
    const int u = __float_as_int(g);
    return (uint32_t)(u ^ (u >> 31 | (int)0x80000000));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();  // the whole warp together, whatever came before
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Two words of another block's shared memory, at the place that p has in this one's.
__device__ __forceinline__ uint2 ld_peer(const uint32_t *p, uint32_t rank) {
    uint2 v;
    asm volatile(
        "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.u32 {%0, %1}, [a];\n\t}"
        : "=r"(v.x), "=r"(v.y)
        : "r"(smem_u32(p)), "r"(rank)
        : "memory");
    return v;
}

// Which part of a sequence a block has: tokens first .. first + n - 1.
struct Part {
    uint32_t first, n;
    __device__ __forceinline__ Part(uint32_t len, uint32_t rank, uint32_t size) {
        const uint32_t each = (len + 4 * size - 1) / (4 * size) * 4;  // whole groups of four keys
        first = rank * each < len ? rank * each : len;
        n = len - first < each ? len - first : each;
    }
};

template <int kSelThreads, bool CLUSTER>
__global__ void __launch_bounds__(kSelThreads, kSelThreads == 1024 ? 1 : 1536 / kSelThreads)
k_select(const __grid_constant__ EvictArgs a, uint32_t held) {
    constexpr int kSelWarps = kSelThreads / 32, kHists = CLUSTER ? kDigits : 1;
    extern __shared__ __align__(16) uint32_t keys[];  // [held], of the part's first tokens; held is a multiple of four
    __shared__ __align__(16) uint32_t hist[kHists][kBins];  // one a digit in a cluster: peers may still read the last one
    __shared__ uint32_t sh_scan[33];
    __shared__ uint32_t sh_digit, sh_left;
    __shared__ uint32_t sh_over[kSelWarps], sh_ties[kSelWarps];
    __shared__ __align__(8) uint32_t sh_all[2];  // the block's counts
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = CLUSTER ? cluster_rank() : 0, size = CLUSTER ? cluster_size() : 1;
    const uint32_t row = blockIdx.x / size, n = row / a.c.heads;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint32_t len = a.lens[n];
    if (len > a.max_len) {
        if (threadIdx.x == 0) raise(a.status, KVX_S_BOUNDS);
        len = a.max_len;
    }
    const Part part(len, rank, size);
    const float *x = a.scores + row * a.scores_stride + part.first;  // the part's
    uint32_t *kept = a.kept + (uint64_t)row * a.budget;
    float *ks = a.kept_scores + (uint64_t)row * a.budget;
    const uint32_t keep = len < a.budget ? len : a.budget;
    for (uint32_t i = keep + rank * kSelThreads + threadIdx.x; i < a.budget; i += size * kSelThreads) {
        kept[i] = kNone;
        ks[i] = 0.0f;
    }
    if (len <= a.budget) {  // the same for the whole cluster
        for (uint32_t i = threadIdx.x; i < part.n; i += kSelThreads) {
            kept[part.first + i] = part.first + i;
            ks[part.first + i] = x[i];
        }
        return;
    }
    const uint32_t lo = a.sinks < a.budget ? a.sinks : a.budget;
    const uint32_t recent = a.recent < a.budget - lo ? a.recent : a.budget - lo;
    const uint32_t hi = len - recent;  // tokens lo .. hi-1 compete for `take` places
    const uint32_t take = a.budget - lo - recent;

    // Scores of the part's tokens i .. i+3, i a multiple of four; where rows
    // are aligned what follows the last token is read too, but for nothing.
    auto load = [&](uint32_t i) -> float4 {
        if (a.aligned) return __ldg(reinterpret_cast<const float4 *>(x + i));
        const uint32_t last = part.n - 1;
        return make_float4(__ldg(x + i), __ldg(x + (i + 1 < last ? i + 1 : last)),
                           __ldg(x + (i + 2 < last ? i + 2 : last)), __ldg(x + (i + 3 < last ? i + 3 : last)));
    };
    auto make_key = [&](uint32_t i, float v) -> uint32_t {
        const uint32_t key = part.first + i - lo < hi - lo ? key_of(v) : kStays;
        return i < part.n ? key : kAbsent;
    };
    auto make_keys = [&](uint32_t i, float4 v) {
        return make_uint4(make_key(i, v.x), make_key(i + 1, v.y), make_key(i + 2, v.z), make_key(i + 3, v.w));
    };
    // Keys of the part's tokens i .. i+3, i a multiple of four.
    auto keys_at = [&](uint32_t i) -> uint4 {
        if (i < held) return *reinterpret_cast<const uint4 *>(keys + i);
        return make_keys(i, load(i));
    };

    for (uint32_t i = threadIdx.x; i < kHists * kBins / 4; i += kSelThreads)
        reinterpret_cast<uint4 *>(hist[0])[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const uint32_t padded = (part.n + 3) & ~3u;
    for (uint32_t i0 = 4 * threadIdx.x; i0 < padded; i0 += kSelUnroll * 4 * kSelThreads) {
        float4 v[kSelUnroll];
#pragma unroll
        for (int u = 0; u < kSelUnroll; u++) {
            const uint32_t i = i0 + u * 4 * kSelThreads;
            if (i < padded) v[u] = load(i);
        }
#pragma unroll
        for (int u = 0; u < kSelUnroll; u++) {
            const uint32_t i = i0 + u * 4 * kSelThreads;
            if (i >= padded) break;
            const uint4 k = make_keys(i, v[u]);
            if (i < held) *reinterpret_cast<uint4 *>(keys + i) = k;
            auto add = [&](uint32_t key) {
                if (key - 1 < kStays - 1) atomicAdd(&hist[0][key >> 21], 1u);
            };
            add(k.x), add(k.y), add(k.z), add(k.w);
        }
    }
    __syncthreads();

    // the threshold: what is over `cut` stays, and `left` of what equals it
    uint32_t cut = take ? 0 : kStays - 1, left = take;
    if (take) {
#pragma unroll 1
        for (int pass = 0; pass < kDigits; pass++) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            uint32_t *counts = hist[CLUSTER ? pass : 0];
            if (pass) {
                if (!CLUSTER) {
                    for (uint32_t i = threadIdx.x; i < kBins; i += kSelThreads) counts[i] = 0;
                    __syncthreads();
                }
                const uint32_t rest = pass == 1 ? 1u << 21 : 1u << 10;
                auto add = [&](uint32_t k) {  // (no cut begins like kStays)
                    if ((k ^ cut) < rest) atomicAdd(&counts[(k ^ cut) >> shift], 1u);
                };
#pragma unroll 2
                for (uint32_t i = 4 * threadIdx.x; i < padded; i += 4 * kSelThreads) {
                    const uint4 k = keys_at(i);
                    add(k.x), add(k.y), add(k.z), add(k.w);
                }
            }
            if (CLUSTER) {
                cluster_arrive();
                cluster_wait();
            } else {
                __syncthreads();
            }
            // some bins a thread, from the largest down, of all blocks
            constexpr int kPer = kBins / kSelThreads;
            const uint32_t bin = kBins - kPer * (threadIdx.x + 1);
            uint32_t h[kPer] = {}, sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; i += 2) {
                if (CLUSTER) {
                    for (uint32_t r = 0; r < size; r++) {
                        const uint2 p = ld_peer(counts + bin + i, r);
                        h[i] += p.x, h[i + 1] += p.y;
                    }
                } else {
                    h[i] = counts[bin + i], h[i + 1] = counts[bin + i + 1];
                }
                sum += h[i] + h[i + 1];
            }
            uint32_t total, above = block_excl_sum<uint32_t>(sum, sh_scan, &total);
            if (above < left && above + sum >= left) {
#pragma unroll
                for (int i = kPer - 1; i >= 0; i--) {
                    if (above < left && above + h[i] >= left)
                        sh_digit = bin + i, sh_left = left - above, sh_all[0] = above + h[i] == left;
                    above += h[i];
                }
            }
            __syncthreads();
            cut |= sh_digit << shift;
            left = sh_left;
            const bool all = sh_all[0];
            __syncthreads();
            if (all) {  // all that share these digits stay: the rest does not matter
                cut--, left = 0;
                break;
            }
        }
    }

    // every warp counts its stretch, then writes it at its place
    const uint32_t per = (padded + 128 * kSelWarps - 1) / (128 * kSelWarps) * 128;
    const uint32_t from = warp * per < padded ? warp * per : padded, to = from + per < padded ? from + per : padded;
    uint32_t n_over = 0, n_ties = 0;
#pragma unroll 2
    for (uint32_t i = from + 4 * lane; i < to; i += 128) {
        const uint4 k = keys_at(i);
        n_over += (k.x > cut) + (k.y > cut) + (k.z > cut) + (k.w > cut);
        n_ties += (k.x == cut) + (k.y == cut) + (k.z == cut) + (k.w == cut);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        n_over += __shfl_xor_sync(0xFFFFFFFFu, n_over, o);
        n_ties += __shfl_xor_sync(0xFFFFFFFFu, n_ties, o);
    }
    if (lane == 0) sh_over[warp] = n_over, sh_ties[warp] = n_ties;
    __syncthreads();
    // what comes before the warp: in blocks before this one, and in this one
    uint2 peer = make_uint2(0, 0);
    if constexpr (CLUSTER) {
        if (warp == 0) {
            uint32_t o = lane < kSelWarps ? sh_over[lane] : 0, t = lane < kSelWarps ? sh_ties[lane] : 0;
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                o += __shfl_xor_sync(0xFFFFFFFFu, o, d);
                t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
            }
            if (lane == 0) sh_all[0] = o, sh_all[1] = t;
        }
        cluster_arrive();
        cluster_wait();
        if (lane < rank) peer = ld_peer(sh_all, lane);
    }
    uint32_t over = peer.x + (lane < warp ? sh_over[lane] : 0), ties = peer.y + (lane < warp ? sh_ties[lane] : 0);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        over += __shfl_xor_sync(0xFFFFFFFFu, over, o);
        ties += __shfl_xor_sync(0xFFFFFFFFu, ties, o);
    }
    if (CLUSTER) cluster_arrive();  // done with the peers' memory
    const uint32_t below = (1u << lane) - 1;
    auto write = [&](auto TIES) {
        for (uint32_t i0 = from; i0 < to; i0 += 128) {
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const uint32_t i = i0 + u * 32 + lane;
                uint32_t k = kAbsent;
                if (i < to) k = i < held ? keys[i] : make_key(i, __ldg(x + (i < part.n ? i : part.n - 1)));
                const uint32_t more = __ballot_sync(0xFFFFFFFFu, k > cut);
                uint32_t place = over + __popc(more & below);
                bool stays = k > cut;
                if (TIES.value) {
                    const uint32_t same = __ballot_sync(0xFFFFFFFFu, k == cut);
                    const uint32_t t = ties + __popc(same & below);
                    stays |= k == cut && t < left;
                    place += t < left ? t : left;
                    ties += __popc(same);
                }
                over += __popc(more);
                if (stays) {
                    kept[place] = part.first + i;
                    ks[place] = __ldg(x + i);
                }
            }
        }
    };
    if (left)
        write(std::true_type());
    else
        write(std::false_type());
    if (CLUSTER) cluster_wait();  // no peer reads this block's memory any more
}

// Copies kRows tokens' K and V rows: a thread looks up each row's two places,
// then all threads move 16-byte pieces.
__global__ void __launch_bounds__(kGatherThreads) k_gather(const __grid_constant__ EvictArgs a, FastDiv pieces) {
    __shared__ uint64_t sh_src[2 * kRows], sh_dst[2 * kRows];
    const uint32_t per = (a.budget + kRows - 1) / kRows;
    const uint32_t nh = blockIdx.x / per, r0 = blockIdx.x % per * kRows;
    const uint32_t n = nh / a.c.heads, h = nh % a.c.heads;
    const uint32_t len = a.lens[n];
    uint32_t keep = len < a.max_len ? len : a.max_len;
    if (keep > a.budget) keep = a.budget;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Here, when every block of k_select has read its length, so that lengths
    // may be cut in place: `keep` is the same from the old one and the new one.
    if (threadIdx.x == 0 && h == 0 && r0 == 0) a.new_lens[n] = keep;
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

template <int THREADS, bool CLUSTER>
bool launch_select(const EvictArgs &a, uint32_t rows, uint32_t size, uint32_t held, cudaStream_t s) {
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        if (cudaFuncSetAttribute(k_select<THREADS, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4) !=
            cudaSuccess)
            return false;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    if (!CLUSTER) {
        k_select<THREADS, CLUSTER><<<rows, THREADS, held * 4, s>>>(a, held);
        return true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * size);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = held * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_select<THREADS, CLUSTER>, a, held) == cudaSuccess;
}

bool sizes_ok(const kvx_cache *c, uint32_t num_seqs, uint32_t blocks_per_seq, uint32_t budget) {
    if (!cache_ok(c) || c->scale_offset || !budget || budget >= (1u << 31)) return false;
    if ((uint64_t)blocks_per_seq * c->page_tokens >= (1ull << 31)) return false;
    return (ceil_div(budget, kRows) + kMaxCluster) * c->heads * (uint64_t)num_seqs < (1ull << 31);
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
                   status, num_seqs, blocks_per_seq, dst_per_seq, (uint32_t)max_len, budget, sinks, recent,
                   (uintptr_t)scores % 16 == 0 && scores_stride % 4 == 0};
    const cudaStream_t s = as_stream(stream);
    const uint32_t rows = num_seqs * cache->heads;
    // Where there are fewer (sequence, head) pairs than SMs, blocks share one's
    // tokens, kShare each at the least: 8 sequences of 16,000 tokens, 8 heads 43 us
    // in one block each, 37 us in clusters of two; more blocks than SMs are slower
    // (40 sequences of 20,000 tokens: 145 and 164 us).  Clusters of eight do not
    // all fit at once above half the SMs (2 sequences of 20,000 tokens: 36 us, in
    // fours 26) and want longer shares (1 sequence of 30,000 tokens, 8 heads: 18
    // and 17; of 131,071 tokens: 27 and 30).
    const uint32_t sms = (uint32_t)sm_count();
    uint32_t size = 1;
    while (size < 4 && 2 * size * (uint64_t)rows <= sms && max_len >= 2 * size * (uint64_t)kShare) size *= 2;
    if (size == 4 && 16 * (uint64_t)rows <= sms && max_len >= 32 * (uint64_t)kShare) size = kMaxCluster;
    const uint64_t each = ceil_div(max_len, 4 * size) * 4;
    const uint32_t held = each < kHeld ? (uint32_t)each : kHeld;
    // Threads of a block: 512 and 1024 take 98 and 106 us for 64 sequences of 4000
    // tokens, 8 heads, 67 and 71 for 32 of 8000, 227 and 190 for 32 of 16,000; 256
    // where blocks of 512 would not fit at once: 128 sequences of 1000 tokens 40
    // us, 512 threads 43, but 1 sequence of 1500 tokens 8.7 and 7.6.
    if (!(size > 1                             ? launch_select<1024, true>(a, rows, size, held, s)
          : max_len <= kTiny && rows > 3 * sms ? launch_select<256, false>(a, rows, 1, held, s)
          : max_len <= kShort                  ? launch_select<512, false>(a, rows, 1, held, s)
                                               : launch_select<1024, false>(a, rows, 1, held, s)))
        return KVX_ECUDA;
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
