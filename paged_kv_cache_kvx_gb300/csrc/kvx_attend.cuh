// The attention kernels of kvx_attend, as templates on the element types and
// the head size; kvx_attend_*.cu instantiate them, kvx_attend.cu has the entry
// point, the joining kernel and the one that adds weights.
#pragma once

#include <type_traits>

#include "kvx_cache.cuh"

namespace kvx {
namespace attend {

constexpr int kWarps = 4;                       // that copy and compute; one more looks pages up
constexpr int kThreads = 32 * (kWarps + 1);
constexpr uint32_t kStep = 16 * kWarps;         // keys of a block's step, and of a tile in which work is shared out
constexpr uint32_t kWhole = 256;                // keys up to which no unit is split
constexpr uint32_t kMaxExtra = 6;               // Shape::kExtra at the most
constexpr uint32_t kFew = 32;                   // sequences that the looking-up warp counts by itself
constexpr uint32_t kMaxBlocks = 512;            // bounds the partial results in the workspace
constexpr int kPieces = 8;                      // descriptors that the looking-up warp may be ahead

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
    float *part_o;   // [2 * blocks][heads of a unit][padded dim]: unnormalised outputs
    float *part_ml;  // [2 * blocks][heads of a unit][2]: base and sum
    uint4 *cut;      // [blocks]: the unit whose first part the block did: sequence (or none), unit, last block, slot
    float *lse2;     // [num_seqs][q_heads]: log2 of the sum of the exponentials
    float *logits;   // [num_seqs][heads][logits_keys][group rounded up to even], in powers of two
    uint64_t logits_keys;
    float scale2;    // scale * k_scale * log2(e)
    uint32_t num_seqs, q_heads, group, units;  // units: pieces of a sequence's heads that blocks take
    uint32_t blocks_per_seq, max_len, window, sinks;
    uint32_t tile;     // keys of a tile, in which work is shared out
    uint32_t grid;     // blocks
    uint32_t align;    // 16 where pages are whole tiles of 16 tokens, else 1
};

// Whether block `block`'s entry of Args::cut names a unit and parts that exist:
// k_join indexes with it, and a block whose wait ran out leaves kNone there.
__host__ __device__ __forceinline__ bool joinable(const uint4 &cut, uint32_t block, uint32_t num_seqs, uint32_t units,
                                                  uint32_t grid) {
    return cut.x < num_seqs && cut.y < units && cut.z >= block && cut.z < grid && cut.w < 2 * grid;
}

// The tokens of a sequence that are looked at: logical index i is token i below
// `turn`, and token i + shift from there on.  With align == 16 both are
// multiples of 16, so that 16 indices from a multiple of 16 on are tokens of
// one page; tokens from `sinks` to `recent`-1 may then be among them, unseen.
struct Seen {
    uint32_t n, turn, shift, sinks, recent;
    __device__ __forceinline__ uint32_t token(uint32_t i) const { return i < turn ? i : i + shift; }
};

__device__ __forceinline__ Seen seen(const Args &a, uint32_t len) {
    Seen v;
    if (len > a.max_len) len = a.max_len;
    v.sinks = a.sinks < len ? a.sinks : len;
    v.recent = a.window && len - v.sinks > a.window ? len - a.window : v.sinks;
    v.turn = (v.sinks + a.align - 1) & ~(a.align - 1);
    const uint32_t from = v.recent & ~(a.align - 1);
    v.shift = v.turn < from ? from - v.turn : 0;
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
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
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

// Two stored 16-bit values, of infinite ones (and of bf16 ones of 2^120 and
// more) that magnitude: what the second parts of weights multiply.
template <class T>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    uint32_t r;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7B807B80u));
    else
        asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7BFF7BFFu));
    return r;
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

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Shapes of the kernel for a stored type of ES bytes, heads padded to DP
// values and NT * 8 query heads at a time.
template <int DP, int ES, int NT, bool PAGED16>
struct Shape {
    static constexpr int kHeads = 8 * NT;
    static constexpr int kKChunks = DP * ES / 64;                         // 64-byte parts of a K row
    static constexpr int kVBytes = DP * ES / 8 < 16 ? DP * ES / 8 : 16;   // of a V row, per lane and part
    static constexpr int kVParts = DP * ES / 8 / kVBytes;
    static constexpr int kVElems = kVBytes / ES;
    static constexpr int kQVecs = kKChunks * (ES == 1 ? 2 : 1);           // 16-byte vectors of q per lane
    // Tiles of 16 keys that a warp takes together.  In 8 bits a tile's bytes are
    // few beside its latencies, which two share: 8 heads of 64 values 118 us in
    // tiles of their own, 103 in pairs (16,000 tokens x 16 KV heads x 16
    // sequences); 16 heads of 128 125 and 110, of 256 81 and 75; but 8 heads of
    // 128 89 and 91, their copies in each other's way.
    static constexpr int kTiles = PAGED16 && ES == 1 && (DP == 64 || NT == 2) ? 2 : 1;
    static constexpr int kTile = 2 * 16 * DP * ES;                        // bytes of a tile, K and V
    static constexpr int kStage = kTiles * kTile;
    // Blocks that an SM has registers for.  Two stages a warp: with more the
    // copies in flight got in each other's way (8-bit, 8 heads of 128: 94 us with
    // three, 96 with four, 89 with two; 16-bit, 8 heads of 64: 90, 91 and 87).
    static constexpr int kBlocks = DP == 256 ? (ES == 1 && NT == 1 ? 2 : 1) : NT == 2 && DP == 128 ? 2 : 3;
    static constexpr int kStages = 2;
    // What a unit costs beside its keys (its query, its output) counts as so
    // many tiles when work is shared out: about 48 KB of copies (96 sequences up
    // to 8192 tokens, 8-bit: 60 us with 32 KB, 56 with 48, 57 with 64, 60 with 96).
    static constexpr uint32_t kExtra = DP * ES >= 384 ? 1 : 384 / (DP * ES);
    static_assert(kExtra <= kMaxExtra);
    static constexpr int kRing = kWarps * kStages * kStage;
    // Where the rings of an SM hold more than 160 KB (16-bit, 128 values, three
    // blocks) the next tile's copies go out when the present one's have
    // arrived: 85 us against 88 at once (16,000 tokens x 8 heads x 8
    // sequences); smaller rings want both on their way (16 heads of 64: 95 us
    // against 99 for 16,000 tokens x 8 KV heads x 8 sequences).
    static constexpr bool kLate = kRing * kBlocks > 160 * 1024;
    static constexpr int kQ = NT * kQVecs * 32 * 16;
    static constexpr int kJoin = (DP / 16 + 1) * NT * 32 * 16;
    static constexpr int kQBufs = kBlocks == 3 ? 2 : 1;
    static constexpr int kSmem = kRing + kQBufs * kQ + kJoin;
};

// a / b, b > 0.  Small quotients go through the reciprocal, a third of a
// division's latency: a < 2^22 is exact as a float, and a * (1/b) is off by
// less than one.
__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t b) {
    if (a >= 1u << 22) return a / b;
    uint32_t q = (uint32_t)__fmul_rz((float)a, __frcp_rz((float)b));
    q += a - q * b >= b;
    return q;
}

// A part of a unit that one block works on.
struct Piece {
    uint32_t n;       // sequence; kNone ends the stream
    uint32_t head;    // KV head
    uint32_t qh0;     // first of the unit's query heads within the group
    uint32_t nheads;
    uint32_t k0, k1;  // visible keys, by logical index
    uint32_t slot;    // of the partial result; kNone: the piece is the whole unit
    uint32_t turn, shift, sinks, recent;  // of the sequence's Seen
};

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Arrives when this thread's copies so far are complete.
__device__ __forceinline__ void mbar_arrive_copies(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Loads into a register that is not touched again before its use: a branch or
// a copy around them would wait for them.
__device__ __forceinline__ void load_early(uint32_t &v, const uint32_t *p, bool go) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                 : "+r"(v)
                 : "l"(p), "r"((uint32_t)go));
}
__device__ __forceinline__ void load_early(uint64_t &v, const uint64_t *p, bool go) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u64 %0, [%1];\n\t}"
                 : "+l"(v)
                 : "l"(p), "r"((uint32_t)go));
}

// The looking-up warp.  It runs ahead of the computing warps, over pieces
// without a pause: the block ids of one step are loaded while the segment
// addresses of the step before are, and the rows of the one before that are
// handed to the warps.
template <class T, int DP, int ES, int NT, bool PAGED16>
__device__ __forceinline__ void look_up(const Args &a, uint32_t per, uint32_t len, uint32_t lane,
                                        uint4 *qbuf, const uint32_t *upto, uint64_t (*rows)[32], uint64_t (*ready)[2],
                                        uint64_t (*taken)[2], uint64_t *pfull, uint64_t *pempty, Piece *pieces,
                                        uint32_t &bad) {
    using S = Shape<DP, ES, NT, PAGED16>;
    const uint32_t g = lane >> 2, t4 = lane & 3;
    const uint32_t units_per_head = (a.group + S::kHeads - 1) / S::kHeads;
    auto unit_len = [&](uint32_t keys) { return keys ? (keys + a.tile - 1) / a.tile + S::kExtra : 0; };
    bool alive = true;  // no wait has run out

    // tiles of the sequences up to this lane's, or of those up to its threads'
    const bool few = a.num_seqs <= kFew;
    uint32_t mine = 0, sum = 0;
    if (few) {
        if (len > a.max_len) bad |= KVX_S_BOUNDS;
        mine = unit_len(seen(a, len).n);
        sum = warp_incl_sum(mine);
    } else {
        sum = upto[lane];
    }
    const uint32_t total = __shfl_sync(0xFFFFFFFFu, sum, 31) * a.units;
    // -- where the walk is: tiles at .. end-1 are still to come
    const uint32_t share = quotient(total + a.grid - 1, a.grid);
    const uint32_t begin = blockIdx.x * share < total ? blockIdx.x * share : total;
    const uint32_t end = total - begin > share ? begin + share : total;
    uint32_t at = begin, seq_tile = 0;  // seq_tile: within the sequence
    uint32_t n = 0, len_u = 0;
    Seen sv = {};
    uint32_t np = 0;                   // pieces so far
    uint32_t k = 0, k1 = 0, head = 0;  // the piece's keys still to come
    bool fresh = false;                // its first step is still to come
    if (a.cut && lane == 0) a.cut[blockIdx.x].x = kNone;  // before any wait: one that runs out leaves it so
    if (at < end) {
        // the first sequence: a lane's, or by the threads' counts and then one by one
        const uint32_t i = __popc(__ballot_sync(0xFFFFFFFFu, sum * a.units <= at));
        uint32_t before = __shfl_sync(0xFFFFFFFFu, sum - mine, i) * a.units;
        if (few) {
            n = i;
            sv = seen(a, __shfl_sync(0xFFFFFFFFu, len, i));
            len_u = unit_len(sv.n);
        } else {
            before = i ? upto[i - 1] * a.units : 0;
            for (n = i * kWarps * per;; n++) {
                sv = seen(a, a.lens[n]);
                len_u = unit_len(sv.n);
                if (at - before < len_u * a.units) break;
                before += len_u * a.units;
            }
        }
        seq_tile = at - before;
    }

    // Moves on to the next piece with keys; false at the end of all work.
    auto next_piece = [&]() -> bool {
        while (at < end) {
            while (seq_tile >= len_u * a.units) {
                seq_tile -= len_u * a.units;
                do sv = seen(a, a.lens[++n]);
                while (!sv.n);
                len_u = unit_len(sv.n);
            }
            const uint32_t unit = quotient(seq_tile, len_u), from = seq_tile - unit * len_u;
            const uint32_t to = len_u - from < end - at ? len_u : from + (end - at);
            // the kExtra that stand for the unit's overhead come first
            const uint32_t nt = len_u - S::kExtra;
            const uint32_t tile0 = from > S::kExtra ? from - S::kExtra : 0, tile1 = to > S::kExtra ? to - S::kExtra : 0;
            const bool whole = tile0 == 0 && tile1 == nt;
            // of a block's pieces at most the first and the last are parts
            const uint32_t slot = 2 * blockIdx.x + (at != begin);
            if (a.cut && lane == 0 && at + (to - from) == end)
                a.cut[blockIdx.x] = make_uint4(tile0 == 0 && tile1 && !whole ? n : kNone, unit,
                                               quotient(at - from + len_u - 1, share), slot);
            at += to - from;
            seq_tile += to - from;
            if (tile0 == tile1) continue;
            head = unit / units_per_head;
            k = tile0 * a.tile;
            k1 = tile1 * a.tile < sv.n ? tile1 * a.tile : sv.n;
            fresh = true;
            if (np >= kPieces && !mbar_wait(&pempty[np % kPieces], (np / kPieces & 1) ^ 1)) return alive = false;
            if (lane == 0) {
                const uint32_t qh0 = unit % units_per_head * S::kHeads;
                const uint32_t nheads = a.group - qh0 < S::kHeads ? a.group - qh0 : S::kHeads;
                pieces[np % kPieces] = Piece{n,  head, qh0, nheads, k, k1, whole ? kNone : slot,
                                             sv.turn, sv.shift, sv.sinks, sv.recent};
            }
            np++;
            __syncwarp();
            return true;
        }
        return false;
    };

    // Three steps on their way: the block ids of one are loaded, the table
    // entries of the one before brought into L2, the segment addresses of the
    // one before that loaded.  Loaded registers are used up where they are (a
    // copy of one would wait for it).
    //   PAGED16: 16 tiles of 16 keys; lane 2*i + kv has tile i's K or V segment.
    //   Otherwise 4 tiles; a lane has both segments of keys `lane` and `lane` + 32.
    constexpr int kKeys = PAGED16 ? 1 : 2, kSegs = PAGED16 ? 1 : 2;
    constexpr uint32_t kReach = PAGED16 ? 16 * 16 : kStep;  // keys of a step
    struct Step {
        uint32_t place[kKeys], valid;  // place in the page; a bit per key: its block exists
        uint32_t mask, left;           // PAGED16: rows of the tile that are seen; a bit per tile with keys
        uint32_t table, piece, warps;  // lane of the address table; warps with keys, 0 at the end
        bool fresh;                    // the piece's first step
    };
    uint32_t ids[kKeys] = {};
    const uint64_t *entry[kKeys];
    uint64_t segs[kKeys][kSegs] = {};
    auto find_blocks = [&]() -> Step {
        Step s = {};
        if (k >= k1 && !next_piece()) return s;
        s.warps = k1 - k < kStep ? (k1 - k + 15) / 16 : kWarps;
        s.piece = np - 1;
        s.fresh = fresh;
        s.table = a.c.first_lane + 2 * head + (PAGED16 ? lane & 1 : 0);
        const uint32_t *seq_blocks = a.blocks + (uint64_t)n * a.blocks_per_seq;
#pragma unroll
        for (int u = 0; u < kKeys; u++) {
            const uint32_t i = k + (PAGED16 ? lane / 2 * 16 : u * 32 + lane);
            const uint32_t pos = sv.token(i), page = a.c.page.div(pos);
            s.place[u] = pos - page * a.c.page.d;
            s.valid |= (uint32_t)(i < k1) << u;
            load_early(ids[u], seq_blocks + page, i < k1);
            if constexpr (PAGED16) {
                auto bits = [](uint32_t count) { return count < 16 ? (1u << count) - 1 : 0xFFFFu; };
                s.mask = bits(i < k1 ? k1 - i : 0);
                if (sv.recent > sv.sinks)
                    s.mask &= ~bits(sv.recent > pos ? sv.recent - pos : 0) | bits(sv.sinks > pos ? sv.sinks - pos : 0);
            }
        }
        s.left = k1 - k < kReach ? (1u << (k1 - k + 15) / 16) - 1 : 0xFFFFu;
        fresh = false;
        k = k1 - k < kReach ? k1 : k + kReach;
        return s;
    };
    auto find_entries = [&](Step &s) {
#pragma unroll
        for (int u = 0; u < kKeys; u++) {
            const uint32_t id = ids[u], there = s.valid >> u & 1, known = id < a.c.B;
            entry[u] = a.c.addr + (there & known ? (uint64_t)id * a.c.L + s.table : 0);
            bad |= there & ~known ? KVX_S_BOUNDS : 0;
            s.valid &= ~((known ^ 1) << u);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(entry[u]));
        }
    };
    auto find_addrs = [&](const Step &s) {
#pragma unroll
        for (int u = 0; u < kKeys; u++)
#pragma unroll
            for (int kv = 0; kv < kSegs; kv++) load_early(segs[u][kv], entry[u] + kv, s.valid >> u & 1);
    };

    const uint64_t no_row = reinterpret_cast<uint64_t>(a.c.pool) | 1;
    const uint64_t room = a.c.pool_bytes - a.c.span;  // a segment's largest offset, where any fits
    const bool fits = a.c.pool_bytes >= a.c.span;
    const uint32_t stride = (uint32_t)a.c.token_stride;
    uint32_t handed = 0;  // hand-overs to warp lane%4 so far
    auto announce = [&](uint32_t p) {
        mbar_arrive_copies(&pfull[p % kPieces]);
        if (lane == 0) mbar_arrive(&pfull[p % kPieces]);
    };
    auto issue = [&](const Step &s, const uint64_t (&row)[kKeys][kSegs]) {
        if (s.fresh) {  // the piece's query heads, as the second operand's lanes hold them
            const uint32_t p = s.piece;
            const uint32_t q_of = p - S::kQBufs;  // the piece whose query was there before
            if (p >= S::kQBufs && !mbar_wait(&pempty[q_of % kPieces], q_of / kPieces & 1)) {
                alive = false;
                return;
            }
            const Piece pc = pieces[p % kPieces];
            const T *q = static_cast<const T *>(a.q) + (uint64_t)pc.n * a.q_stride +
                         (uint64_t)(pc.head * a.group + pc.qh0) * a.c.dim;
            const uint32_t dst = smem_u32(qbuf + p % S::kQBufs * (S::kQ / 16) + lane);
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < S::kQVecs; i++) {
                    const uint32_t d = ES == 2 ? i * 32 + t4 * 8 : (i / 2) * 64 + t4 * 16 + (i & 1) * 8;
                    const bool in = x * 8 + g < pc.nheads && d < a.c.dim;
                    copy_async<16>(dst + (x * S::kQVecs + i) * 512, in ? q + (uint64_t)(x * 8 + g) * a.c.dim + d : q,
                                   in ? 16 : 0);
                }
            announce(p);
        }
        // one buffer of rows a warp, or two of up to four tiles each
        const uint32_t w = lane % kWarps, buffer = PAGED16 ? handed & 1 : 0;
        const uint32_t turn = PAGED16 ? handed >> 1 : handed;
        const bool mine = w < s.warps;
        const bool free = !mine || !turn || mbar_wait(&taken[w][buffer], (turn & 1) ^ 1);
        if (!__all_sync(0xFFFFFFFFu, free)) {
            alive = false;
            return;
        }
        handed += mine;
        if constexpr (PAGED16) {
            const uint32_t i = lane / 2, to = __shfl_sync(0xFFFFFFFFu, buffer, i % kWarps);
            const bool last = i / kWarps == 3 || !(s.left >> (i + kWarps) & 1);
            if (s.left >> i & 1)
                reinterpret_cast<uint4 *>(rows[i % kWarps])[(to * 4 + i / kWarps) * 2 + (lane & 1)] =
                    make_uint4((uint32_t)row[0][0], (uint32_t)(row[0][0] >> 32), row[0][0] & 1 ? 0 : s.mask, last);
        } else {
#pragma unroll
            for (int u = 0; u < kKeys; u++) {
                if (2 * u + lane / 16 >= s.warps) continue;
                rows[2 * u + lane / 16][lane % 16] = row[u][0];
                rows[2 * u + lane / 16][16 + lane % 16] = row[u][kSegs - 1];
            }
        }
        __syncwarp();
        if (lane < s.warps) mbar_arrive(&ready[lane][buffer]);
    };

    // (find_blocks() is not asked again after it has said that there is no
    // more; the first step's rows are handed over before the third is looked for)
    Step now = find_blocks(), held = {}, next = {};
    find_entries(now);
    find_addrs(now);
    if (now.warps) held = find_blocks();
    find_entries(held);
    bool first = true;
    while (alive && now.warps) {
        uint64_t row[kKeys][kSegs];
#pragma unroll
        for (int u = 0; u < kKeys; u++)
#pragma unroll
            for (int kv = 0; kv < kSegs; kv++) {
                const uint64_t seg = segs[u][kv];
                const bool there = now.valid >> u & 1, good = fits && seg <= room && !((uint32_t)seg & 15);
                row[u][kv] = no_row;
                if (there && good) row[u][kv] = no_row - 1 + seg + (uint64_t)now.place[u] * stride;
                if (there && !good) a.c.ok(seg, bad);
            }
        const Step s = now;
        now = held;
        find_addrs(now);
        issue(s, row);
        if (first && now.warps) next = find_blocks();
        first = false;
        held = next;
        find_entries(held);
        if (held.warps) next = find_blocks();
    }
    if (alive) {  // the end of the stream
        if (np >= kPieces && !mbar_wait(&pempty[np % kPieces], (np / kPieces & 1) ^ 1)) alive = false;
        if (lane == 0) pieces[np % kPieces].n = kNone;
        __syncwarp();
        if (alive) announce(np);
    }
    if (!alive) bad |= KVX_S_TIMEOUT;

    // the sequences without a visible token
    for (uint32_t i = blockIdx.x; i < a.num_seqs; i += gridDim.x)
        if (!seen(a, a.lens[i]).n) {
            for (uint32_t d = lane; d < a.q_heads * a.c.dim; d += 32)
                static_cast<T *>(a.out)[i * a.out_stride + d] = T(0.0f);
            for (uint32_t d = lane; d < a.q_heads; d += 32)
                if (a.lse) a.lse[(uint64_t)i * a.q_heads + d] = -INFINITY;
        }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The tiles of all units, in order, are shared out equally, one share a block.
// A block's last warp walks the share and looks the pages up; the others copy
// keys and values into rings of their own and compute, 16 keys of a step each.
// For those a warp computes, with the KV head's query heads as the columns,
//     S^T = K Q^T   (16 keys x 8 heads per mma.m16n8k16)
//     O^T += V^T P^T
// where P = 2^(S - base).  Contracting over a permuted order of the head's
// values, and of the keys, lets every lane take its operands of both products
// from 16-byte pieces of the rows as they lie in memory: lane (g, t) =
// (lane / 4, lane % 4) holds pieces t, t+4, ... of the rows of keys g and g+8
// for K, and piece g of the rows of keys 2t, 2t+1, 2t+8, 2t+9 for V (whose
// pairs of keys one byte permutation brings together).  So rows are copied
// piece by piece to where their lanes read them, free of bank conflicts, and
// pages, strides and gaps cost nothing.  A unit's four partial results pass
// from warp to warp through a buffer of the same lanes' places, so that no
// warp waits for a slower one before it goes on to the next piece.
//
// Bound by HBM: per key 2*DP*ES bytes for 4*group*DP operations.  One sequence
// of 131,071 tokens, 8 KV heads of 128 values, bf16: 85 us at 6.3 TB/s (7.1
// between the first and the last copy) with 12 % of the tensor pipe's cycles
// in use; 8-bit with 8 query heads to a KV head: 20 %.  So mma.sync suffices:
// its operands come to registers from rows as they lie, where a larger tile of
// the tensor cores' would want them transposed and regrouped first, for 4 to 16
// query heads that fill a fraction of it.
template <class T, int DP, int ES, int NT, bool PAGED16>
__global__ void __launch_bounds__(kThreads, (Shape<DP, ES, NT, PAGED16>::kBlocks)) k_attend(const __grid_constant__ Args a) {
    using S = Shape<DP, ES, NT, PAGED16>;
    // the type in which the products are taken: 8-bit values are exact in fp16
    using C = typename std::conditional<ES == 1, __half, T>::type;
    constexpr bool kConvertQ = !std::is_same<C, T>::value;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t sh_sum[kWarps + 1], sh_upto[32];
    __shared__ uint64_t full[kWarps][S::kStages];   // a warp's tiles
    // Where its next ones' rows are.  PAGED16: two buffers of four tiles, for
    // each the first row's address, which rows are seen, and whether the tile
    // is the buffer's last, for K and for V.  Otherwise one tile: addresses of
    // its 16 rows of K and of V, with bit 0 set where there is none.
    __shared__ __align__(16) uint64_t rows[kWarps][32];
    __shared__ uint64_t ready[kWarps][2], taken[kWarps][2];
    __shared__ uint64_t pfull[kPieces], pempty[kPieces];                      // pieces
    __shared__ uint64_t passed[kWarps], converted[2];
    __shared__ uint64_t joined[kPieces];  // the first warp has the piece's results: the join buffer is free again
    __shared__ Piece pieces[kPieces];
    __shared__ float sh_qscale[2][S::kHeads];  // power of two taken out of a head's query

    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t g = lane >> 2, t4 = lane & 3;
    uint4 *qbuf = reinterpret_cast<uint4 *>(smem + S::kRing);
    // A V row's pieces lie together, as they arrive (scattered ones held the
    // copies to three quarters of the bandwidth), in an order that keeps the
    // eight or sixteen lanes that read at a time on different banks.
    const uint32_t vslot = (t4 * 8 + (g ^ (S::kVBytes == 16 ? 2 * t4 : t4 / 2 * 4))) * S::kVBytes;
    uint32_t bad = 0;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the tiles of all units: each thread counts those of some sequences in
    // a row, or the looking-up warp by itself where a lane has one at most (one
    // sequence of 77 tokens: 6.9 and 6.7 us; of 1000: 10.2 and 9.7).
    const bool few = a.num_seqs <= kFew;
    const uint32_t per = (a.num_seqs + kWarps * 32 - 1) / (kWarps * 32);
    auto unit_len = [&](uint32_t keys) { return keys ? (keys + a.tile - 1) / a.tile + S::kExtra : 0; };
    uint32_t mine = 0, own_len = 0;
    if (warp < kWarps) {
        const uint32_t n0 = threadIdx.x * per, n1 = few ? n0 : n0 + per < a.num_seqs ? n0 + per : a.num_seqs;
        for (uint32_t n = n0; n < n1; n++) {
            const uint32_t len = a.lens[n];
            if (len > a.max_len) bad |= KVX_S_BOUNDS;
            mine += unit_len(seen(a, len).n);
        }
    } else {
        if (few && lane < a.num_seqs) own_len = a.lens[lane];
        if (lane == 0) {
            for (int w = 0; w < kWarps; w++) {
                for (int i = 0; i < S::kStages; i++) mbar_init(&full[w][i], 32);
                for (int i = 0; i < 2; i++) {
                    mbar_init(&ready[w][i], 1);
                    mbar_init(&taken[w][i], 1);
                }
                mbar_init(&passed[w], 1);
            }
            for (int i = 0; i < kPieces; i++) {
                mbar_init(&pfull[i], 33);
                mbar_init(&pempty[i], kWarps);
                mbar_init(&joined[i], 1);
            }
            mbar_init(&converted[0], NT);
            mbar_init(&converted[1], NT);
        }
    }
    if (!few) {
        uint32_t upto = warp_incl_sum(mine);
        if (lane == 31) sh_sum[warp] = upto;
        __syncthreads();
        for (uint32_t w = 0; w < warp && w < kWarps; w++) upto += sh_sum[w];
        if (warp < kWarps && threadIdx.x % kWarps == kWarps - 1) sh_upto[threadIdx.x / kWarps] = upto;
    }
    __syncthreads();

    if (warp == kWarps) {
        look_up<T, DP, ES, NT, PAGED16>(a, per, own_len, lane, qbuf, sh_upto, rows, ready, taken, pfull, pempty, pieces, bad);
        raise(a.status, bad);
        return;
    }
    raise(a.status, bad);

    // ---- a computing warp: one piece after the other
    uint8_t *ring = smem + warp * (S::kStages * S::kStage);
    uint32_t copied = 0;   // tiles whose copies this warp has issued: up to kStages ahead, of later pieces too
    uint32_t buffers = 0, in_buffer = 0;  // buffers of rows used up, tiles of the present one taken
    const bool cover = a.c.row_bytes == DP * ES;
    const uint32_t stride = (uint32_t)a.c.token_stride;
    // Takes the next tiles' rows and copies this lane's pieces of them: where a
    // row, a piece or the second tile does not exist, zeros (a copy of no bytes
    // reads nothing).
    auto copy_tiles = [&]() {
        uint8_t *st = ring + copied % S::kStages * S::kStage;
        bool done = false;
#pragma unroll
        for (int h = 0; h < S::kTiles; h++, st += S::kTile) {
            const uint8_t *row[6];
            uint32_t there[6];
            const bool none = done;  // the buffer has no second tile
            if constexpr (PAGED16) {
                const uint4 *from = reinterpret_cast<const uint4 *>(rows[warp]) + ((buffers & 1) * 4 + in_buffer) * 2;
                uint4 kr = make_uint4((uint32_t)(uintptr_t)a.c.pool, (uint32_t)((uintptr_t)a.c.pool >> 32), 0, 0), vr = kr;
                if (!none) kr = from[0], vr = from[1];
                const uint8_t *kp = reinterpret_cast<const uint8_t *>(((uint64_t)kr.y << 32 | kr.x) & ~1ull);
                const uint8_t *vp = reinterpret_cast<const uint8_t *>(((uint64_t)vr.y << 32 | vr.x) & ~1ull);
                row[0] = kp + (uint64_t)g * stride;
                row[1] = row[0] + 8ull * stride;
                row[2] = vp + 2ull * t4 * stride;
                row[3] = row[2] + stride;
                row[4] = row[2] + 8ull * stride;
                row[5] = row[3] + 8ull * stride;
#pragma unroll
                for (int r = 0; r < 6; r++)
                    there[r] = r < 2 ? kr.z >> (g + 8 * r) & 1 : vr.z >> (2 * t4 + (r & 1) + 8 * ((r - 2) >> 1)) & 1;
                done = kr.w;
            } else {
                const uint64_t *from = rows[warp];
                const ulonglong2 v0 = *reinterpret_cast<const ulonglong2 *>(from + 16 + 2 * t4);
                const ulonglong2 v1 = *reinterpret_cast<const ulonglong2 *>(from + 24 + 2 * t4);
                const uint64_t at[6] = {from[g], from[g + 8], v0.x, v0.y, v1.x, v1.y};
#pragma unroll
                for (int r = 0; r < 6; r++) {
                    row[r] = reinterpret_cast<const uint8_t *>(at[r] & ~1ull);
                    there[r] = ~(uint32_t)at[r] & 1;
                }
                done = true;
            }
            if (!none) in_buffer++;
            if (done && !none) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&taken[warp][PAGED16 ? buffers & 1 : 0]);
                buffers++;
                in_buffer = 0;
            }
            done |= none;
            const uint32_t kdst = smem_u32(st + lane * 16), vdst = smem_u32(st + S::kTile / 2 + vslot);
#pragma unroll
            for (int r = 0; r < 6; r++) {
                if (r < 2) {
#pragma unroll
                    for (int c = 0; c < S::kKChunks; c++)
                        copy_async<16>(kdst + (c * 2 + r) * 512, row[r] + t4 * 16 + c * 64,
                                       there[r] && (cover || c * 64 + t4 * 16 < a.c.row_bytes) ? 16 : 0);
                } else {
#pragma unroll
                    for (int c = 0; c < S::kVParts; c++)
                        copy_async<S::kVBytes>(vdst + (c * 4 + r - 2) * 32 * S::kVBytes, row[r] + (c * 8 + g) * S::kVBytes,
                                               there[r] && (cover || (c * 8 + g) * S::kVBytes < a.c.row_bytes) ? S::kVBytes : 0);
                }
            }
        }
        mbar_arrive_copies(&full[warp][copied % S::kStages]);
        copied++;
    };
    // Whether the next tile's rows are there; the barrier is asked once a buffer.
    auto rows_there = [&]() {
        const uint32_t parity = (PAGED16 ? buffers >> 1 : buffers) & 1;
        return in_buffer || __all_sync(0xFFFFFFFFu, mbar_test(&ready[warp][PAGED16 ? buffers & 1 : 0], parity));
    };
    float4 *join = reinterpret_cast<float4 *>(smem + S::kRing + S::kQBufs * S::kQ) + lane;
    uint32_t tile = 0, passes = 0;  // tiles taken, and results taken over so far
    for (uint32_t p = 0;; p++) {
        if (!mbar_wait(&pfull[p % kPieces], p / kPieces & 1)) break;
        const Piece pc = pieces[p % kPieces];
        if (pc.n == kNone) return;
        uint4 *qs = qbuf + p % S::kQBufs * (S::kQ / 16);
        if constexpr (kConvertQ) {
            // bf16's range does not fit fp16: a head's largest power of two is
            // taken out first (exact, but for values 2^-14 of the largest and
            // below, which lose the bits under 2^-24 of it)
            if (warp < NT) {
                uint4 *mine_q = qs + warp * S::kQVecs * 32 + lane;
                float top = 0;
#pragma unroll
                for (int i = 0; i < S::kQVecs; i++) {
                    const uint4 raw = mine_q[i * 32];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 f = Pair<T>::unpack(word(raw, k));
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                int e = 0;
                if (top > 0 && top < INFINITY) frexpf(top, &e);
                e = e < -120 ? -120 : e > 120 ? 120 : e;
                const float inv = ldexpf(1.0f, -e);
#pragma unroll
                for (int i = 0; i < S::kQVecs; i++) {
                    const uint4 raw = mine_q[i * 32];
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 f = Pair<T>::unpack(word(raw, k));
                        w[k] = Pair<C>::pack(f.x * inv, f.y * inv);
                    }
                    mine_q[i * 32] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (t4 == 0) sh_qscale[p & 1][warp * 8 + g] = ldexpf(1.0f, e);
                __syncwarp();
                if (lane == 0) mbar_arrive(&converted[p & 1]);
            }
            if (!mbar_wait(&converted[p & 1], p / 2 & 1)) break;
        }

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
                scale2[x][i] = a.scale2;
                if constexpr (kConvertQ) scale2[x][i] *= sh_qscale[p & 1][x * 8 + 2 * t4 + i];
                limit[x][i] = -INFINITY, base[x][i] = 0, l[x][i] = 0;
            }
#pragma unroll
        for (int j = 0; j < kOTiles; j++)
#pragma unroll
            for (int x = 0; x < NT; x++)
#pragma unroll
                for (int i = 0; i < 4; i++) o[j][x][i] = 0;
        float *logits = nullptr;
        const uint32_t gp = (a.group + 1) & ~1u;
        if (a.logits)
            logits = a.logits + ((uint64_t)pc.n * a.c.heads + pc.head) * a.logits_keys * gp + pc.qh0 + 2 * t4;

        bool ok = true;
        for (uint32_t k = pc.k0 + warp * 16; k < pc.k1; k += S::kTiles * kStep, tile++) {
            if (copied == tile) {
                const uint32_t parity = (PAGED16 ? buffers >> 1 : buffers) & 1;
                if (!in_buffer && !mbar_wait(&ready[warp][PAGED16 ? buffers & 1 : 0], parity)) {
                    ok = false;
                    break;
                }
                copy_tiles();
            }
            if (!S::kLate)
                while (copied < tile + S::kStages && rows_there()) copy_tiles();
            const uint32_t stage = tile % S::kStages;
            if (!mbar_wait(&full[warp][stage], tile / S::kStages & 1)) {
                ok = false;
                break;
            }
            if (S::kLate)
                while (copied < tile + S::kStages && rows_there()) copy_tiles();
            const uint8_t *st = ring + stage * S::kStage;

            // S^T = K Q^T, in two chains of products at the least
            constexpr int KT = S::kTiles;
            float s[KT][NT][4] = {}, s2[NT][4] = {};
#pragma unroll
            for (int c = 0; c < S::kKChunks; c++) {
                uint4 r0[KT], r1[KT];
#pragma unroll
                for (int h = 0; h < KT; h++) {
                    r0[h] = *reinterpret_cast<const uint4 *>(st + h * S::kTile + (c * 2) * 512 + lane * 16);
                    r1[h] = *reinterpret_cast<const uint4 *>(st + h * S::kTile + (c * 2 + 1) * 512 + lane * 16);
                }
                if constexpr (ES == 2) {
#pragma unroll
                    for (int x = 0; x < NT; x++) {
                        const uint4 qv = qs[(x * S::kQVecs + c) * 32 + lane];
#pragma unroll
                        for (int h = 0; h < KT; h++) {
                            mma<C>(s[h][x], r0[h].x, r1[h].x, r0[h].y, r1[h].y, qv.x, qv.y);
                            mma<C>(KT > 1 ? s[h][x] : s2[x], r0[h].z, r1[h].z, r0[h].w, r1[h].w, qv.z, qv.w);
                        }
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        uint32_t k0[KT], k1[KT], k2[KT], k3[KT];
#pragma unroll
                        for (int h = 0; h < KT; h++) {
                            const uint32_t w0 = word(r0[h], w), w1 = word(r1[h], w);
                            k0[h] = e4m3_lo(w0), k1[h] = e4m3_lo(w1), k2[h] = e4m3_hi(w0), k3[h] = e4m3_hi(w1);
                        }
#pragma unroll
                        for (int x = 0; x < NT; x++) {
                            const uint4 qv = qs[(x * S::kQVecs + c * 2 + w / 2) * 32 + lane];
#pragma unroll
                            for (int h = 0; h < KT; h++)
                                mma<C>(KT == 1 && w % 2 ? s2[x] : s[h][x], k0[h], k1[h], k2[h], k3[h], w % 2 ? qv.z : qv.x,
                                       w % 2 ? qv.w : qv.y);
                        }
                    }
                }
            }

            // logits in powers of two, masked beyond the last key
            bool higher = false;
#pragma unroll
            for (int h = 0; h < KT; h++) {
                const uint32_t i0 = k + h * kStep + g, i1 = i0 + 8;
                bool hide0 = i0 >= pc.k1, hide1 = i1 >= pc.k1;
                if (PAGED16 && a.window) {
                    const uint32_t p0 = i0 < pc.turn ? i0 : i0 + pc.shift, p1 = p0 + 8;  // in one page
                    hide0 |= p0 >= pc.sinks && p0 < pc.recent;
                    hide1 |= p1 >= pc.sinks && p1 < pc.recent;
                }
#pragma unroll
                for (int x = 0; x < NT; x++) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (KT == 1) s[h][x][i] += s2[x][i];
                        s[h][x][i] *= scale2[x][i & 1];
                        if (i < 2 ? hide0 : hide1) s[h][x][i] = -INFINITY;
                        higher |= s[h][x][i] > limit[x][i & 1];
                    }
                    if (logits && x * 8 + 2 * t4 < pc.nheads) {
                        float2 *to = reinterpret_cast<float2 *>(logits + x * 8 + (uint64_t)i0 * gp);
                        if (i0 < pc.k1) to[0] = make_float2(s[h][x][0], s[h][x][1]);
                        if (i1 < pc.k1) to[4 * gp] = make_float2(s[h][x][2], s[h][x][3]);
                    }
                }
            }
            if (__any_sync(0xFFFFFFFFu, higher)) {
                float f[NT][2];
#pragma unroll
                for (int x = 0; x < NT; x++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        float top = fmaxf(s[0][x][i], s[0][x][i + 2]);
#pragma unroll
                        for (int h = 1; h < KT; h++) top = fmaxf(top, fmaxf(s[h][x][i], s[h][x][i + 2]));
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
            uint32_t ph[KT][NT][2], pl[KT][NT][2];
#pragma unroll
            for (int h = 0; h < KT; h++)
#pragma unroll
                for (int x = 0; x < NT; x++)
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const float p0 = exp2_fast(s[h][x][2 * r] - base[x][0]), p1 = exp2_fast(s[h][x][2 * r + 1] - base[x][1]);
                        l[x][0] += p0;
                        l[x][1] += p1;
                        const uint32_t hi = Pair<C>::pack(p0, p1);
                        const float2 f = Pair<C>::unpack(hi);
                        ph[h][x][r] = transpose8(hi);
                        pl[h][x][r] = transpose8(Pair<C>::pack(p0 - f.x, p1 - f.y));
                    }

            // O^T += V^T P^T
#pragma unroll
            for (int h = 0; h < KT; h++) {
                const uint8_t *sv = st + h * S::kTile + S::kTile / 2 + vslot;
#pragma unroll
                for (int c = 0; c < S::kVParts; c++) {
                    uint32_t v[4][S::kVBytes / 4];
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        if constexpr (S::kVBytes == 16) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(sv + (c * 4 + r) * 512);
                            v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(sv + (c * 4 + r) * 256);
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
                            // A weight's second part may be zero or negative:
                            // times an infinite value it would turn the
                            // infinity of the first into NaN.
                            const uint32_t f0 = finite2<C>(a0), f1 = finite2<C>(a1), f2 = finite2<C>(a2), f3 = finite2<C>(a3);
#pragma unroll
                            for (int x = 0; x < NT; x++) {
                                mma<C>(o[c * 4 + w][x], a0, a1, a2, a3, ph[h][x][0], ph[h][x][1]);
                                mma<C>(o[c * 4 + w][x], f0, f1, f2, f3, pl[h][x][0], pl[h][x][1]);
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
                                    mma<C>(o[c * per + 2 * w + y][x], a0, a1, a2, a3, ph[h][x][0], ph[h][x][1]);
                                    mma<C>(o[c * per + 2 * w + y][x], a0, a1, a2, a3, pl[h][x][0], pl[h][x][1]);
                                }
                            }
                        }
                    }
                }
            }
        }
        if (!ok) break;
        __syncwarp();  // a lane without keys may still be reading the descriptor
        if (lane == 0) mbar_arrive(&pempty[p % kPieces]);  // its query and descriptor are done with

        // ---- the warps' results: each adds its own to the next one's
        const uint32_t active = pc.k1 - pc.k0 < kStep ? (pc.k1 - pc.k0 + 15) / 16 : kWarps;
        if (warp >= active) continue;
        float m[NT][2];
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) l[x][i] += __shfl_xor_sync(0xFFFFFFFFu, l[x][i], k);
                m[x][i] = limit[x][i] == -INFINITY ? -INFINITY : base[x][i];
            }
        if (warp + 1 < active) {
            if (!mbar_wait(&passed[warp + 1], passes++ & 1)) break;
#pragma unroll
            for (int x = 0; x < NT; x++) {
                const float4 ml = join[(kOTiles * NT + x) * 32];
                float f[2], fj[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float mj = i ? ml.y : ml.x, top = fmaxf(m[x][i], mj);
                    f[i] = m[x][i] == -INFINITY ? 1.0f : exp2f(m[x][i] - top);  // 1: zeros, or a NaN
                    fj[i] = mj == -INFINITY ? 1.0f : exp2f(mj - top);
                    l[x][i] = l[x][i] * f[i] + (i ? ml.w : ml.z) * fj[i];
                    m[x][i] = top;
                }
#pragma unroll
                for (int k = 0; k < kOTiles; k++) {
                    const float4 v = join[(k * NT + x) * 32];
                    o[k][x][0] = o[k][x][0] * f[0] + v.x * fj[0];
                    o[k][x][1] = o[k][x][1] * f[1] + v.y * fj[1];
                    o[k][x][2] = o[k][x][2] * f[0] + v.z * fj[0];
                    o[k][x][3] = o[k][x][3] * f[1] + v.w * fj[1];
                }
            }
        } else if (active > 1 && p) {
            // The first to write: the last piece's results have been read.  A
            // barrier for each place of `pieces`, for warps without keys pass a
            // piece by and may be two ahead of the first one, or behind it: a
            // single barrier's parity would stand for two phases.  Of one place
            // the last phase but this is over, as the first warp has handed
            // back the descriptor that was here before this piece's, and the
            // next one is after this piece.
            if (!mbar_wait(&joined[(p - 1) % kPieces], (p - 1) / kPieces & 1)) break;
        }
        if (warp > 0) {
#pragma unroll
            for (int x = 0; x < NT; x++) {
                join[(kOTiles * NT + x) * 32] = make_float4(m[x][0], m[x][1], l[x][0], l[x][1]);
#pragma unroll
                for (int k = 0; k < kOTiles; k++)
                    join[(k * NT + x) * 32] = make_float4(o[k][x][0], o[k][x][1], o[k][x][2], o[k][x][3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&passed[warp]);
            continue;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[p % kPieces]);

        // ---- the unit's output, or its part for k_join
#pragma unroll
        for (int x = 0; x < NT; x++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t hh = x * 8 + 2 * t4 + i;
                if (hh >= pc.nheads) continue;
                const uint32_t qh = pc.head * a.group + pc.qh0 + hh;
                if (pc.slot != kNone) {
                    float *to = a.part_o + ((uint64_t)pc.slot * S::kHeads + hh) * DP;
#pragma unroll
                    for (int c = 0; c < S::kVParts; c++)
#pragma unroll
                        for (int e = 0; e < S::kVElems; e += 4) {
                            const int k = (c * S::kVElems + e) / 2;
                            *reinterpret_cast<float4 *>(to + (c * 8 + g) * S::kVElems + e) =
                                make_float4(o[k][x][i], o[k][x][i + 2], o[k + 1][x][i], o[k + 1][x][i + 2]);
                        }
                    if (g == 0)
                        *reinterpret_cast<float2 *>(a.part_ml + ((uint64_t)pc.slot * S::kHeads + hh) * 2) =
                            make_float2(m[x][i], l[x][i]);
                    continue;
                }
                const float inv = l[x][i] == 0 ? 0.0f : a.c.v_scale / l[x][i];
                T *to = static_cast<T *>(a.out) + (uint64_t)pc.n * a.out_stride + (uint64_t)qh * a.c.dim;
#pragma unroll
                for (int c = 0; c < S::kVParts; c++)
#pragma unroll
                    for (int e = 0; e < S::kVElems; e += 8) {
                        const int k = (c * S::kVElems + e) / 2;
                        const uint32_t d = (c * 8 + g) * S::kVElems + e;
                        if (d < a.c.dim)
                            *reinterpret_cast<uint4 *>(to + d) =
                                make_uint4(Pair<T>::pack(o[k][x][i] * inv, o[k][x][i + 2] * inv),
                                           Pair<T>::pack(o[k + 1][x][i] * inv, o[k + 1][x][i + 2] * inv),
                                           Pair<T>::pack(o[k + 2][x][i] * inv, o[k + 2][x][i + 2] * inv),
                                           Pair<T>::pack(o[k + 3][x][i] * inv, o[k + 3][x][i + 2] * inv));
                    }
                if (g == 0) {
                    const float lse2 = l[x][i] == 0 ? -INFINITY : m[x][i] + log2f(l[x][i]);
                    if (a.lse) a.lse[(uint64_t)pc.n * a.q_heads + qh] = lse2 * 0.6931471805599453f;
                    if (a.lse2) a.lse2[(uint64_t)pc.n * a.q_heads + qh] = lse2;
                }
            }
    }
    raise(a.status, KVX_S_TIMEOUT);  // a wait ran out
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Launches one variant over at most `most` blocks and leaves their number in
// a.grid; false where that failed.
template <class T, int DP, int ES, int NT, bool PAGED16>
bool launch_kernel(Args &a, uint64_t most, cudaStream_t s) {
    using S = Shape<DP, ES, NT, PAGED16>;
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        if (cudaFuncSetAttribute(k_attend<T, DP, ES, NT, PAGED16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::kSmem) != cudaSuccess)
            return false;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    uint64_t room = (uint64_t)sm_count() * S::kBlocks;
    if (room > kMaxBlocks) room = kMaxBlocks;
    a.grid = (uint32_t)(most < room ? most : room);
    if (!a.grid) a.grid = 1;  // nothing to see anywhere: the zeros still have to be written
    k_attend<T, DP, ES, NT, PAGED16><<<a.grid, kThreads, S::kSmem, s>>>(a);
    return true;
}

template <class T, int DP, int ES, int NT>
bool launch_one(Args &a, uint64_t most, cudaStream_t s) {
    return a.align == 16 ? launch_kernel<T, DP, ES, NT, true>(a, most, s) : launch_kernel<T, DP, ES, NT, false>(a, most, s);
}

template <class T, int ES>
bool launch(Args &a, uint64_t most, uint32_t dim, uint32_t nt, cudaStream_t s) {
    if (dim <= 64) return nt == 1 ? launch_one<T, 64, ES, 1>(a, most, s) : launch_one<T, 64, ES, 2>(a, most, s);
    if (dim <= 128) return nt == 1 ? launch_one<T, 128, ES, 1>(a, most, s) : launch_one<T, 128, ES, 2>(a, most, s);
    return nt == 1 ? launch_one<T, 256, ES, 1>(a, most, s) : launch_one<T, 256, ES, 2>(a, most, s);
}

}  // namespace attend
}  // namespace kvx
