// The attention kernels of kvx_attend, as templates on the element types and
// the head size; kvx_attend_*.cu instantiate them, kvx_attend.cu has the entry
// point and the joining kernel.
#pragma once

#include <type_traits>

#include "kvx_cache.cuh"

namespace kvx {
namespace attend {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kStep = 16 * kWarps;  // keys of a block's step
constexpr uint32_t kWhole = 256;         // keys up to which no unit is split
constexpr uint32_t kMaxBlocks = 512;     // of the splitting grid: bounds the partial results in the workspace

struct Args {
    CacheView c;
    const void *q;
    uint64_t q_stride;
    const uint32_t *blocks;
    const uint32_t *lens;
    void *out;
    uint64_t out_stride;
    float *lse;
    float *scores;
    uint64_t scores_stride;
    uint32_t *status;
    // workspace
    float *part_o;   // [2 * blocks of the grid][heads of a unit][padded dim]: unnormalised outputs
    float *part_ml;  // [2 * blocks of the grid][heads of a unit][2]: base and sum
    uint4 *cut;      // [blocks of the grid]: the unit whose first part the block did: sequence, unit, last block; or none
    float *lse2;     // [num_seqs][q_heads]: log2 of the sum of the exponentials
    float *logits;   // [num_seqs][heads][visible][group rounded up to even], in powers of two
    uint64_t logits_keys;
    float scale2;    // scale * k_scale * log2(e)
    uint32_t num_seqs, q_heads, group, units;  // units: pieces of a sequence's heads that blocks take
    uint32_t blocks_per_seq, max_len, window, sinks, grid;
    uint32_t tile;   // keys of a tile, in which work is shared out
};

// Visible tokens of a sequence: logical index i is token i below `sinks`, and
// token i + shift from there on.
struct Seen {
    uint32_t n, sinks, shift;
};

__device__ __forceinline__ Seen seen(const Args &a, uint32_t len) {
    Seen v;
    if (len > a.max_len) len = a.max_len;
    v.sinks = a.sinks < len ? a.sinks : len;
    v.shift = 0;
    if (a.window && len - v.sinks > a.window) v.shift = len - a.window - v.sinks;
    v.n = len - v.shift;
    return v;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ----------------------------------------------------------- tensor cores

template <class T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (sizeof(Pair<T>) && std::is_same<T, __nv_bfloat16>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit values held a row of pairs per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The low or the high two of four stored 8-bit values as two fp16 ones, exactly.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t four) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(four));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t four) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(four));
    return r;
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Shapes of the kernel for a stored type of ES bytes, heads padded to DP
// values and NT * 8 query heads at a time.
template <int DP, int ES, int NT>
struct Shape {
    static constexpr int kHeads = 8 * NT;
    static constexpr int kKChunks = DP * ES / 64;                         // 64-byte parts of a K row
    static constexpr int kVBytes = DP * ES / 8 < 16 ? DP * ES / 8 : 16;   // of a V row, per lane and part
    static constexpr int kVParts = DP * ES / 8 / kVBytes;
    static constexpr int kVElems = kVBytes / ES;
    static constexpr int kQVecs = kKChunks * (ES == 1 ? 2 : 1);           // 16-byte vectors of q per lane
    static constexpr int kStage = 2 * 16 * DP * ES;                       // bytes of a warp's 16 keys, K and V
    // Blocks an SM has registers for, and stages that as many rings have room for.
    static constexpr int kBlocks = DP == 256 ? (ES == 1 ? 2 : 1) : NT == 2 && DP == 128 ? 2 : 3;
    static constexpr int kFit = 196608 / kBlocks / (kStage * kWarps);
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static_assert(kStages >= 2, "");
    // A unit's look-ups, first copies, query and output take about as long as
    // a block takes for 32 KB: they count as so many tiles when work is shared out.
    static constexpr uint32_t kExtra = DP * ES >= 256 ? 1 : 256 / (DP * ES);
    static constexpr int kORow = DP + 4;                                  // floats of a row when warps are joined
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kJoin = kWarps * kHeads * kORow * 4;
    static constexpr int kQ = NT * kQVecs * 32 * 16;
    static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQ;
};

// One block walks its share of the tiles.  For 16 keys at a time a warp
// computes, with the KV head's query heads as the columns,
//     S^T = K Q^T   (16 keys x 8 heads per mma.m16n8k16)
//     O^T += V^T P^T
// where P = exp2(S - running maximum).  Contracting over a permuted order of
// the head's values, and of the keys, lets every lane take its operands of
// both products from 16-byte pieces of the rows as they lie in memory: lane
// (g, t) = (lane / 4, lane % 4) holds pieces t, t+4, ... of the rows of keys
// g and g+8 for K, and piece g of the rows of keys 2t, 2t+1, 2t+8, 2t+9 for V
// (whose pairs of keys one byte permutation brings together).  So each lane
// fetches exactly the pieces it will use, with asynchronous copies into its
// own places of a ring in shared memory: no lane waits for another's copies,
// reads are free of bank conflicts, and pages, strides and gaps cost nothing.
//
// Bound by HBM: per key 2*DP*ES bytes for 4*group*DP operations.  mma.sync
// suffices: with 16 columns in use the SMs need well under a fifth of its
// rate to consume the measured bandwidth, and operands come to registers
// without a transposition through shared memory that a larger tile would need.
template <class T, int DP, int ES, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<DP, ES, NT>::kBlocks)) k_attend(const __grid_constant__ Args a) {
    using S = Shape<DP, ES, NT>;
    // the type in which the products are taken: 8-bit values are exact in fp16
    using C = typename std::conditional<ES == 1, __half, T>::type;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t sh_sum[kWarps];
    __shared__ uint64_t sh_first;                   // tiles of the sequences before the first one
    __shared__ uint32_t sh_n;
    __shared__ float sh_ml[kWarps][S::kHeads][2];
    __shared__ float sh_qscale[S::kHeads];          // power of two taken out of a head's query

    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t g = lane >> 2, t4 = lane & 3;
    uint8_t *ring = smem + warp * (S::kStages * S::kStage);
    // A V row's pieces lie together, as they arrive (scattered ones held the
    // copies to three quarters of the bandwidth), in an order that keeps the
    // eight or sixteen lanes that read at a time on different banks.
    const uint32_t vslot = (t4 * 8 + (g ^ (S::kVBytes == 16 ? 2 * t4 : t4 / 2 * 4))) * S::kVBytes;
    uint4 *qs = reinterpret_cast<uint4 *>(smem + (S::kRing > S::kJoin ? S::kRing : S::kJoin));
    uint32_t bad = 0;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the block's share: blocks take equal stretches of the tiles of all
    // units in order, so that a batch of any lengths keeps every SM busy to
    // the end.  Each thread counts the tiles of some sequences in a row.
    const uint32_t per = (a.num_seqs + kThreads - 1) / kThreads;
    const uint32_t n0 = threadIdx.x * per, n1 = n0 + per < a.num_seqs ? n0 + per : a.num_seqs;
    auto unit_tiles = [&](uint32_t keys) { return (keys + a.tile - 1) / a.tile; };
    uint64_t mine = 0;
    bool none = false;
    for (uint32_t n = n0; n < n1; n++) {
        const uint32_t len = a.lens[n], keys = seen(a, len).n;
        if (blockIdx.x == 0 && len > a.max_len) bad |= KVX_S_BOUNDS;
        if (keys)
            mine += unit_tiles(keys) + S::kExtra;
        else
            none |= n % gridDim.x == blockIdx.x;
    }
    uint64_t upto = warp_incl_sum(mine), total = 0;
    if (lane == 31) sh_sum[warp] = upto;
    none = __syncthreads_or(none);
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
        if (w < (int)warp) upto += sh_sum[w];
        total += sh_sum[w];
    }
    total *= a.units;
    const uint64_t share = (total + a.grid - 1) / a.grid;
    uint64_t at = blockIdx.x * share;
    const uint64_t begin = at, end = at + share < total ? at + share : total;
    if (at < end && (upto - mine) * a.units <= at && at < upto * a.units) {  // one thread
        uint64_t before = (upto - mine) * a.units;
        uint32_t n = n0;
        for (;; n++) {
            const uint32_t keys = seen(a, a.lens[n]).n;
            const uint64_t m = keys ? (uint64_t)(unit_tiles(keys) + S::kExtra) * a.units : 0;
            if (at < before + m) break;
            before += m;
        }
        sh_n = n;
        sh_first = before;
    }
    if (none)  // sequences without a visible token
        for (uint32_t n = blockIdx.x; n < a.num_seqs; n += gridDim.x) {
            if (seen(a, a.lens[n]).n) continue;
            for (uint32_t i = threadIdx.x; i < a.q_heads * a.c.dim; i += kThreads)
                static_cast<T *>(a.out)[n * a.out_stride + i] = T(0.0f);
            for (uint32_t i = threadIdx.x; i < a.q_heads; i += kThreads)
                if (a.lse) a.lse[(uint64_t)n * a.q_heads + i] = -INFINITY;
        }
    if (at >= end) {
        if (a.cut && threadIdx.x == 0) a.cut[blockIdx.x].x = kNone;
        raise(a.status, bad);
        return;
    }
    __syncthreads();
    uint32_t n = sh_n;
    uint64_t seq_tile = at - sh_first;  // within the sequence's units
    Seen sv = seen(a, a.lens[n]);
    uint32_t nt = unit_tiles(sv.n), len_u = nt + S::kExtra;
    const uint32_t units_per_head = (a.group + S::kHeads - 1) / S::kHeads;

    // ---- one piece of a unit after the other
    for (uint64_t next; at < end; seq_tile += next - at, at = next) {
        while (seq_tile >= (uint64_t)len_u * a.units) {
            seq_tile -= (uint64_t)len_u * a.units;
            do sv = seen(a, a.lens[++n]);
            while (!sv.n);
            nt = unit_tiles(sv.n);
            len_u = nt + S::kExtra;
        }
        const uint32_t unit = (uint32_t)(seq_tile / len_u), from = (uint32_t)(seq_tile - (uint64_t)unit * len_u);
        const uint32_t to = (uint32_t)(len_u - from < end - at ? len_u : from + (end - at));
        next = at + (to - from);
        // the kExtra that stand for the unit's overhead come first
        const uint32_t tile0 = from > S::kExtra ? from - S::kExtra : 0, tile1 = to > S::kExtra ? to - S::kExtra : 0;
        const bool whole = tile0 == 0 && tile1 == nt;
        if (a.cut && threadIdx.x == 0 && next == end)
            a.cut[blockIdx.x] = make_uint4(tile0 == 0 && tile1 && !whole ? n : kNone, unit,
                                           (uint32_t)((at - from + len_u - 1) / share), at != begin);
        if (tile0 == tile1) continue;
        const uint32_t head = unit / units_per_head, qh0 = unit % units_per_head * S::kHeads;
        const uint32_t nheads = a.group - qh0 < S::kHeads ? a.group - qh0 : S::kHeads;
        const uint32_t q0 = head * a.group + qh0;
        const uint32_t k0 = tile0 * a.tile, k1 = tile1 * a.tile < sv.n ? tile1 * a.tile : sv.n;

        // -- this lane looks up key lane%16's K (lanes 0-15) or V segment
        const uint32_t *seq_blocks = a.blocks + (uint64_t)n * a.blocks_per_seq;
        const uint32_t kv = lane >> 4;
        auto find_block = [&](uint32_t j, uint32_t &place) -> uint32_t {
            const uint32_t i = k0 + (j * kWarps + warp) * 16 + (lane & 15);
            if (i >= k1) return kNone;
            const uint32_t pos = i < sv.sinks ? i : i + sv.shift;
            const uint32_t page = a.c.page.div(pos);
            place = pos - page * a.c.page.d;
            const uint32_t b = __ldg(seq_blocks + page);
            if (b < a.c.B) return b;
            bad |= KVX_S_BOUNDS;
            return kNone;
        };
        auto find_addr = [&](uint32_t b) -> uint64_t {
            return b == kNone ? ~0ull : __ldg(a.c.lane_addr(b, head, kv));
        };
        auto resolve = [&](uint64_t seg, uint32_t place, uint32_t b) -> uint64_t {
            if (b == kNone || !a.c.ok(seg, bad)) return ~0ull;
            return seg + place * a.c.token_stride;
        };
        const uint32_t warp_keys = k1 - k0;
        const uint32_t steps = warp_keys > warp * 16 ? (warp_keys - warp * 16 + kStep - 1) / kStep : 0;
        // -- asynchronous copies of tile j's pieces into its stage: where a row
        // or a piece does not exist, zeros (a copy of no bytes reads nothing)
        auto fetch = [&](uint32_t j, uint64_t row) {
            const uint32_t kdst = smem_u32(ring + (j % S::kStages) * S::kStage + lane * 16);
            const uint32_t vdst = smem_u32(ring + (j % S::kStages) * S::kStage + S::kStage / 2 + vslot);
            const uint8_t *p[6];
            uint32_t n[6];
#pragma unroll
            for (int r = 0; r < 6; r++) {
                const uint32_t from = r < 2 ? g + 8 * r : 16 + 2 * t4 + (r & 1) + 8 * ((r - 2) >> 1);
                const uint64_t src = __shfl_sync(0xFFFFFFFFu, row, from);
                n[r] = src == ~0ull ? 0 : r < 2 ? 16 : S::kVBytes;
                p[r] = a.c.pool + (src == ~0ull ? 0 : src) + (r < 2 ? t4 * 16 : g * S::kVBytes);
            }
            if (a.c.row_bytes == DP * ES) {
#pragma unroll
                for (int r = 0; r < 2; r++)
#pragma unroll
                    for (int c = 0; c < S::kKChunks; c++) copy_async<16>(kdst + (c * 2 + r) * 512, p[r] + c * 64, n[r]);
#pragma unroll
                for (int r = 0; r < 4; r++)
#pragma unroll
                    for (int c = 0; c < S::kVParts; c++)
                        copy_async<S::kVBytes>(vdst + (c * 4 + r) * 32 * S::kVBytes, p[2 + r] + c * 8 * S::kVBytes, n[2 + r]);
            } else {
#pragma unroll
                for (int r = 0; r < 2; r++)
#pragma unroll
                    for (int c = 0; c < S::kKChunks; c++)
                        copy_async<16>(kdst + (c * 2 + r) * 512, p[r] + c * 64,
                                       c * 64 + t4 * 16 < a.c.row_bytes ? n[r] : 0);
#pragma unroll
                for (int r = 0; r < 4; r++)
#pragma unroll
                    for (int c = 0; c < S::kVParts; c++)
                        copy_async<S::kVBytes>(vdst + (c * 4 + r) * 32 * S::kVBytes, p[2 + r] + c * 8 * S::kVBytes,
                                               (c * 8 + g) * S::kVBytes < a.c.row_bytes ? n[2 + r] : 0);
            }
        };

        // look-ups run ahead of the copies: the address of one tile, the block of
        // the next and of the one after, whose address is fetched into L2
        uint32_t b1 = kNone, p1 = 0, b2 = kNone, p2 = 0, b3 = kNone, p3 = 0;
        uint64_t row = ~0ull, seg1 = ~0ull;
        {
            uint32_t b0, p0 = 0;
            b0 = find_block(0, p0);
            b1 = find_block(1, p1);
            b2 = find_block(2, p2);
            b3 = find_block(3, p3);
            const uint64_t seg0 = find_addr(b0);
            seg1 = find_addr(b1);
            row = resolve(seg0, p0, b0);
        }
        auto advance = [&](uint32_t j) {  // after tile j's copies were issued
            row = resolve(seg1, p1, b1);
            b1 = b2;
            p1 = p2;
            seg1 = find_addr(b1);
            b2 = b3;
            p2 = p3;
            if (b2 != kNone) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.lane_addr(b2, head, kv)));
            b3 = find_block(j + 4, p3);
        };
#pragma unroll
        for (int j = 0; j < S::kStages - 1; j++) {
            if (j < steps) {
                fetch(j, row);
                advance(j);
            }
            copies_commit();
        }

        // -- the query heads, as the second operand's lanes hold them
        __syncthreads();  // the last piece's reads of qs and sh_ml are done
        for (uint32_t hh = warp; hh < S::kHeads; hh += kWarps) {
            const uint32_t d0 = lane * 8;
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (hh < nheads && d0 < a.c.dim)
                raw = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) + (uint64_t)n * a.q_stride +
                                                       (uint64_t)(q0 + hh) * a.c.dim + d0);
            float unit2 = 1.0f;
            if constexpr (ES == 1 && std::is_same<T, __nv_bfloat16>::value) {
                // bf16's range does not fit fp16: the head's largest power of
                // two is taken out first (exact, but for values 2^-14 of the
                // largest and below, which lose the bits under 2^-24 of it)
                float x[8], top = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 f = Pair<T>::unpack(word(raw, i));
                    x[2 * i] = f.x, x[2 * i + 1] = f.y;
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                float inv = 1.0f;
                if (top > 0 && top < INFINITY) {
                    int e;
                    frexpf(top, &e);
                    e = e < -120 ? -120 : e > 120 ? 120 : e;
                    unit2 = ldexpf(1.0f, e);
                    inv = ldexpf(1.0f, -e);
                }
                raw = make_uint4(Pair<C>::pack(x[0] * inv, x[1] * inv), Pair<C>::pack(x[2] * inv, x[3] * inv),
                                 Pair<C>::pack(x[4] * inv, x[5] * inv), Pair<C>::pack(x[6] * inv, x[7] * inv));
            }
            if (d0 < DP) {
                // piece (c, t) of a K row is 16 bytes: 8 or 16 values
                constexpr int per = 16 / ES;
                const uint32_t c = d0 / (4 * per), tt = d0 % (4 * per) / per, hf = d0 % per / 8;
                qs[((hh >> 3) * S::kQVecs + c * (per / 8) + hf) * 32 + (hh & 7) * 4 + tt] = raw;
            }
            if (lane == 0) sh_qscale[hh] = unit2;
        }
        __syncthreads();

        // Weights are taken as 2^(logit - base).  The base follows the running
        // maximum only when a logit exceeds it by more than kSlack + kBoost:
        // sums and outputs are divided by the same power in the end, and the
        // few octaves above 1 do not matter to 32-bit sums.  It lies kBoost
        // below that maximum, so that in fp16, whose smallest step is 2^-24,
        // small weights keep some bits more beside a large one.
        constexpr float kSlack = 8.0f, kBoost = std::is_same<C, __half>::value ? 7.0f : 0.0f;
        float scale2[NT][2], limit[NT][2], base[NT][2], l[NT][2];  // limit: base + kBoost + kSlack
        constexpr int kOTiles = DP / 16;
        float o[kOTiles][NT][4];
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                scale2[x][i] = a.scale2 * sh_qscale[x * 8 + 2 * t4 + i];
                limit[x][i] = -INFINITY, base[x][i] = 0, l[x][i] = 0;
            }
#pragma unroll
        for (int j = 0; j < kOTiles; j++)
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < 4; i++) o[j][x][i] = 0;

        for (uint32_t j = 0; j < steps; j++) {
            const uint32_t jf = j + S::kStages - 1;
            if (jf < steps) {
                fetch(jf, row);
                advance(jf);
            }
            copies_commit();
            copies_wait<S::kStages - 1>();
            const uint8_t *st = ring + (j % S::kStages) * S::kStage;

            // S^T = K Q^T
            float s[NT][4] = {}, s2[NT][4] = {};  // two chains of products
#pragma unroll
            for (int c = 0; c < S::kKChunks; c++) {
                const uint4 r0 = *reinterpret_cast<const uint4 *>(st + (c * 2) * 512 + lane * 16);
                const uint4 r1 = *reinterpret_cast<const uint4 *>(st + (c * 2 + 1) * 512 + lane * 16);
                if constexpr (ES == 2) {
#pragma unroll
                    for (int x = 0; x < NT; x++) {
                        const uint4 qv = qs[(x * S::kQVecs + c) * 32 + lane];
                        mma<C>(s[x], r0.x, r1.x, r0.y, r1.y, qv.x, qv.y);
                        mma<C>(s2[x], r0.z, r1.z, r0.w, r1.w, qv.z, qv.w);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        const uint32_t w0 = word(r0, w), w1 = word(r1, w);
                        const uint32_t a0 = e4m3_lo(w0), a1 = e4m3_lo(w1), a2 = e4m3_hi(w0), a3 = e4m3_hi(w1);
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            const uint4 qv = qs[(x * S::kQVecs + c * 2 + w / 2) * 32 + lane];
                            mma<C>(w % 2 ? s2[x] : s[x], a0, a1, a2, a3, w % 2 ? qv.z : qv.x, w % 2 ? qv.w : qv.y);
                        }
                    }
                }
            }

            // logits in powers of two, masked beyond the last key
            const uint32_t i0 = k0 + (j * kWarps + warp) * 16 + g, i1 = i0 + 8;
            bool higher = false;
#pragma unroll
            for (int x = 0; x < NT; x++) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    s[x][i] = (s[x][i] + s2[x][i]) * scale2[x][i & 1];
                    if ((i < 2 ? i0 : i1) >= k1) s[x][i] = -INFINITY;
                    higher |= s[x][i] > limit[x][i & 1];
                }
                if (a.logits) {
                    const uint32_t gp = (a.group + 1) & ~1u, hh = qh0 + x * 8 + 2 * t4;
                    if (hh < a.group) {
                        float *to = a.logits + ((uint64_t)n * a.c.heads + head) * a.logits_keys * gp + hh;
                        if (i0 < k1) *reinterpret_cast<float2 *>(to + (uint64_t)i0 * gp) = make_float2(s[x][0], s[x][1]);
                        if (i1 < k1) *reinterpret_cast<float2 *>(to + (uint64_t)i1 * gp) = make_float2(s[x][2], s[x][3]);
                    }
                }
            }
            if (__any_sync(0xFFFFFFFFu, higher)) {
                float f[NT][2];
#pragma unroll
                for (int x = 0; x < NT; x++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float top = fmaxf(s[x][i], s[x][i + 2]);
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
                        f[x][i] = 1.0f;
                        if (top - kBoost > base[x][i] || (limit[x][i] == -INFINITY && top > -INFINITY)) {
                            if (limit[x][i] > -INFINITY) f[x][i] = exp2_fast(base[x][i] - (top - kBoost));
                            base[x][i] = top - kBoost;
                            limit[x][i] = top + kSlack;
                        }
                        l[x][i] *= f[x][i];
                    }
#pragma unroll
                for (int k = 0; k < kOTiles; k++)
#pragma unroll
                    for (int x = 0; x < NT; x++)
#pragma unroll
                        for (int i = 0; i < 4; i++) o[k][x][i] *= f[x][i & 1];
            }

            // P^T as the sum of two 16-bit values (2^-17 of the weight for
            // bf16): one alone would add an error of the size of the output's
            // own rounding
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const float p0 = exp2_fast(s[x][2 * r] - base[x][0]), p1 = exp2_fast(s[x][2 * r + 1] - base[x][1]);
                    l[x][0] += p0;
                    l[x][1] += p1;
                    const uint32_t hi = Pair<C>::pack(p0, p1);
                    const float2 h = Pair<C>::unpack(hi);
                    ph[x][r] = transpose8(hi);
                    pl[x][r] = transpose8(Pair<C>::pack(p0 - h.x, p1 - h.y));
                }

            // O^T += V^T P^T
            const uint8_t *sv_ = st + S::kStage / 2 + vslot;
#pragma unroll
            for (int c = 0; c < S::kVParts; c++) {
                uint32_t v[4][S::kVBytes / 4];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    if constexpr (S::kVBytes == 16) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(sv_ + (c * 4 + r) * 512);
                        v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(sv_ + (c * 4 + r) * 256);
                        v[r][0] = x.x, v[r][1] = x.y;
                    }
                }
#pragma unroll
                for (int w = 0; w < S::kVBytes / 4; w++) {
                    if constexpr (ES == 2) {
                        const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410);
                        const uint32_t a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
                        const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410);
                        const uint32_t a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            mma<C>(o[c * 4 + w][x], a0, a1, a2, a3, ph[x][0], ph[x][1]);
                            mma<C>(o[c * 4 + w][x], a0, a1, a2, a3, pl[x][0], pl[x][1]);
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 2; y++) {
                            const uint32_t e = __byte_perm(v[0][w], v[1][w], y ? 0x7362 : 0x5140);
                            const uint32_t f = __byte_perm(v[2][w], v[3][w], y ? 0x7362 : 0x5140);
                            const uint32_t a0 = e4m3_lo(e), a1 = e4m3_hi(e), a2 = e4m3_lo(f), a3 = e4m3_hi(f);
                            constexpr int per = S::kVBytes / 2;  // output tiles of a part
#pragma unroll
                            for (int x = 0; x < NT; x++) {
                                mma<C>(o[c * per + 2 * w + y][x], a0, a1, a2, a3, ph[x][0], ph[x][1]);
                                mma<C>(o[c * per + 2 * w + y][x], a0, a1, a2, a3, pl[x][0], pl[x][1]);
                            }
                        }
                    }
                }
            }
        }
        copies_wait<0>();

        // ---- the warps' results joined
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) l[x][i] += __shfl_xor_sync(0xFFFFFFFFu, l[x][i], k);
                if (g == 0) {
                    sh_ml[warp][x * 8 + 2 * t4 + i][0] = limit[x][i] == -INFINITY ? -INFINITY : base[x][i];
                    sh_ml[warp][x * 8 + 2 * t4 + i][1] = l[x][i];
                }
            }
        __syncthreads();  // also: every warp's ring is free
        float *join = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t hh = x * 8 + 2 * t4 + i;
                float top = sh_ml[0][hh][0];
#pragma unroll
                for (int w = 1; w < kWarps; w++) top = fmaxf(top, sh_ml[w][hh][0]);
                const float f = limit[x][i] == -INFINITY ? 1.0f : exp2f(base[x][i] - top);  // 1: zeros, or a NaN
                float *to = join + (warp * S::kHeads + hh) * S::kORow;
#pragma unroll
                for (int c = 0; c < S::kVParts; c++)
#pragma unroll
                    for (int e = 0; e < S::kVElems / 2; e++) {
                        const int k = c * (S::kVElems / 2) + e;
                        *reinterpret_cast<float2 *>(to + (c * 8 + g) * S::kVElems + 2 * e) =
                            make_float2(o[k][x][i] * f, o[k][x][i + 2] * f);
                    }
            }
        __syncthreads();
        const uint32_t slot = 2 * blockIdx.x + (at != begin);
        for (uint32_t i = threadIdx.x * 4; i < nheads * DP; i += kThreads * 4) {
            const uint32_t hh = i / DP, d = i % DP;
            float top = sh_ml[0][hh][0];
#pragma unroll
            for (int w = 1; w < kWarps; w++) top = fmaxf(top, sh_ml[w][hh][0]);
            float sum = 0;
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float mw = sh_ml[w][hh][0];
                // (a NaN among the logits leaves the maximum alone but not the sum)
                sum += sh_ml[w][hh][1] * (mw == -INFINITY ? 1.0f : exp2f(mw - top));
                const float4 x = *reinterpret_cast<const float4 *>(join + (w * S::kHeads + hh) * S::kORow + d);
                v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
            if (!whole) {
                *reinterpret_cast<float4 *>(a.part_o + ((uint64_t)slot * S::kHeads + hh) * DP + d) = v;
                if (d == 0) {
                    a.part_ml[((uint64_t)slot * S::kHeads + hh) * 2] = top;
                    a.part_ml[((uint64_t)slot * S::kHeads + hh) * 2 + 1] = sum;
                }
                continue;
            }
            const float inv = sum == 0 ? 0.0f : a.c.v_scale / sum;
            if (d < a.c.dim) {
                T *to = static_cast<T *>(a.out) + (uint64_t)n * a.out_stride + (uint64_t)(q0 + hh) * a.c.dim + d;
                *reinterpret_cast<uint2 *>(to) =
                    make_uint2(Pair<T>::pack(v.x * inv, v.y * inv), Pair<T>::pack(v.z * inv, v.w * inv));
            }
            if (d == 0) {
                const float lse2 = sum == 0 ? -INFINITY : top + log2f(sum);
                if (a.lse) a.lse[(uint64_t)n * a.q_heads + q0 + hh] = lse2 * 0.6931471805599453f;
                if (a.lse2) a.lse2[(uint64_t)n * a.q_heads + q0 + hh] = lse2;
            }
        }
        __syncthreads();  // the ring takes the next piece's copies
    }
    raise(a.status, bad);
}

// Launches one variant over at most `parts` blocks, and leaves their number in
// a.grid; false where that failed.
template <class T, int DP, int ES, int NT>
bool launch_one(Args &a, uint64_t parts, cudaStream_t s) {
    using S = Shape<DP, ES, NT>;
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        if (cudaFuncSetAttribute(k_attend<T, DP, ES, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
            cudaSuccess)
            return false;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    const uint64_t room = (uint64_t)sm_count() * S::kBlocks;
    a.grid = (uint32_t)(parts < room ? parts : room);
    if (!a.grid) a.grid = 1;  // nothing to see anywhere: the zeros still have to be written
    k_attend<T, DP, ES, NT><<<a.grid, kThreads, S::kSmem, s>>>(a);
    return true;
}

template <class T, int ES>
bool launch(Args &a, uint64_t parts, uint32_t dim, uint32_t nt, cudaStream_t s) {
    if (dim <= 64) return nt == 1 ? launch_one<T, 64, ES, 1>(a, parts, s) : launch_one<T, 64, ES, 2>(a, parts, s);
    if (dim <= 128) return nt == 1 ? launch_one<T, 128, ES, 1>(a, parts, s) : launch_one<T, 128, ES, 2>(a, parts, s);
    return launch_one<T, 256, ES, 1>(a, parts, s);
}

}  // namespace attend
}  // namespace kvx
