// The attention kernel of kvx_attend_shared, as a template on the element types
// and the head size; kvx_shared_*.cu instantiate it, kvx_shared.cu has the entry
// point and the joining kernel.
#pragma once

#include <type_traits>

#include "kvx_cache.cuh"

namespace kvx {
namespace shared {

// Warps of a block: 0-3 and 4-7 take softmaxes, each thread one row of a slot;
// 8-15 copy; one for each slot issues the tensor cores' instructions; one walks the
// schedule; one looks up pages of whole groups of 16 tokens (of others each
// copying warp looks up its own).
constexpr int kSoftWarps = 8, kCopyWarps = 8, kMmaWarp = 16, kWalkWarp = 18, kLookWarp = 19, kWarps = 20;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kKindWarps = kCopyWarps / 2;  // that copy keys; the others copy values
constexpr uint32_t kKindThreads = 32 * kKindWarps;
constexpr int kPieces = 8;  // descriptors that the walking warp may be ahead
constexpr uint32_t kFewRows = 16;  // up to so many, four lanes share a row of logits (soften_few)
constexpr uint32_t kHalf = 64;  // keys that a slot's softmax takes at a time
constexpr uint32_t kRows = 128;  // of a slot: the tensor cores' M, a query row for each lane of tensor memory
constexpr uint32_t kExtra = 2;   // columns (Region) that a head's own overhead counts as
constexpr uint32_t kMinShare = 2;
constexpr uint32_t kMaxGroup = 128;  // query heads of a KV head
// Keys of a tile and query rows of a unit, of heads wider than 128 and of others.
__host__ __device__ __forceinline__ constexpr uint32_t keys_of(bool wide) { return wide ? 64 : 128; }
__host__ __device__ __forceinline__ constexpr uint32_t tile_rows_of(bool wide) { return wide ? 128 : 256; }

struct Args {
    CacheView c;
    const void *q;
    uint64_t q_stride;
    const uint32_t *prefix_blocks, *prefix_lens, *group_first, *blocks, *lens;
    uint32_t blocks_per_prefix, num_groups, blocks_per_seq, num_seqs, q_heads, group;
    uint32_t max_prefix, max_len;
    FastDiv by_group;
    float scale2;     // |scale| * k_scale * log2(e)
    uint32_t negate;  // scale < 0
    uint32_t paged16; // pages are whole groups of 16 tokens
    void *out;
    uint64_t out_stride;
    float *lse;
    uint32_t *status;
    // workspace
    float *part_o;        // [rows of parts][dim]: unnormalised outputs
    float2 *part_ml;      // [rows of parts]: base (of powers of two) and sum
    uint2 *group_at;      // [num_groups]: where a group's columns start, and a block's share
    uint2 *own_parts;     // [num_seqs * heads]: the first and the last block with a part
    uint32_t tile_rows;                          // query rows of a unit of a prefix
    uint32_t prefix_cap, prefix_off_b;           // rows of a part of a prefix; where those of slot B start
    uint32_t own_cap, own_off_b, own_first_row;  // of a sequence's own tokens; the first such part's first row
    uint32_t grid;
    uint64_t rows;  // of all parts
};

// What is shared out: a group's prefix, or a sequence's own tokens.
struct Entry {
    uint32_t seq0, rows, len;
    bool disorder, beyond;  // a group whose sequences do not exist; more tokens than pages
};
__host__ __device__ __forceinline__ uint32_t load(const uint32_t *p) {
#ifdef __CUDA_ARCH__
    return __ldg(p);
#else
    return *p;
#endif
}
__host__ __device__ __forceinline__ Entry entry_of(const Args &a, uint32_t i) {
    Entry e = {};
    uint32_t most;
    if (i < a.num_groups) {
        const uint32_t from = load(a.group_first + i), to = load(a.group_first + i + 1);
        e.len = load(a.prefix_lens + i);
        most = a.max_prefix;
        e.seq0 = from;
        if (from > to || to > a.num_seqs)
            e.disorder = true;
        else
            e.rows = (to - from) * a.group;
    } else {
        e.seq0 = i - a.num_groups;
        e.rows = a.group;
        e.len = load(a.lens + e.seq0);
        most = a.max_len;
    }
    if (e.len > most) e.len = most, e.beyond = true;
    if (!e.rows) e.len = 0;
    return e;
}

// How an entry's work is shared out.  It has heads * len columns, `keys` keys in
// one head each (kExtra at a head's start stand for what a part costs beside its
// keys), and tile_rows query rows at a time make `rows` rows of them.  Where both
// slots work on a tile it takes twice the time of one, and makes two columns (128
// sequences with 2000 shared tokens and one of their own: 76 us with one column,
// 62 with two).  Blocks of
// `block` columns, a share each where there are several rows, are gone through row
// by row: so the blocks that work on different rows of the same columns do so at
// the same time, and keys and values come from memory once (100,000 tokens, 8
// heads, 4 rows: 1.71 GB of DRAM reads with the rows one after the other, 0.4 GB
// so; 382 us and 370).
struct Region {
    uint32_t keys, len, width, rows, block;
    __host__ __device__ __forceinline__ uint32_t columns(uint32_t b) const {  // of block b
        return width - b * block < block ? width - b * block : block;
    }
    // Number of the parts of a row's columns of one head in a block, by which parts
    // are laid out: it grows in the order in which these are gone through.
    __host__ __device__ __forceinline__ uint32_t rank(uint32_t b, uint32_t row, uint32_t head) const {
        const uint32_t first = b * block / len, last = (b * block + columns(b) - 1) / len;
        return rows * (b + first) + row * (last - first + 1) + head - first;
    }
};
__host__ __device__ __forceinline__ Region region_of(const Args &a, const Entry &e, uint32_t share, uint32_t keys) {
    Region r;
    r.keys = keys > kHalf && e.rows > kRows ? keys / 2 : keys;
    r.len = e.len ? (e.len + r.keys - 1) / r.keys + kExtra : 0;
    r.width = a.c.heads * r.len;
    r.rows = (e.rows + a.tile_rows - 1) / a.tile_rows;
    r.block = r.rows > 1 ? share : r.width;
    return r;
}
// The first part of a group's, by number.  Its parts are at most rows * (blocks + heads),
// and one for each border of a share: blocks * rows is its columns over the share,
// and tiles of query rows of all groups before it, g for rounding, count the rest.
__host__ __device__ __forceinline__ uint32_t group_parts(const Args &a, uint32_t start, uint32_t share, uint32_t first_seq, uint32_t g) {
    return start / share + ((uint32_t)((uint64_t)first_seq * a.group / a.tile_rows) + g) * (a.c.heads + 2);
}

// a / b for b > 0; small quotients go through the reciprocal: a < 2^22 is exact
// as a float, and a * (1/b) is off by less than one.
__host__ __device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t b) {
#ifdef __CUDA_ARCH__
    if (a < 1u << 22) {
        uint32_t q = (uint32_t)__fmul_rz((float)a, __frcp_rz((float)b));
        q += a - q * b >= b;
        return q;
    }
#endif
    return a / b;
}

// What a block does next: columns from .. to-1 of a head's, in a row of a block of columns,
// from the place `off` of an entry's on, at most `left` of them.
struct Cut {
    uint32_t block, row, head, from, to;
};
__host__ __device__ __forceinline__ Cut cut(const Region &r, uint32_t off, uint32_t left) {
    Cut c;
    c.block = quotient(off, r.block * r.rows);
    const uint32_t in_block = off - c.block * r.block * r.rows, columns = r.columns(c.block);
    c.row = quotient(in_block, columns);
    const uint32_t in_row = in_block - c.row * columns, column = c.block * r.block + in_row;
    c.head = quotient(column, r.len), c.from = column - c.head * r.len;
    c.to = c.from + (columns - in_row);
    if (c.to > r.len) c.to = r.len;
    if (c.to - c.from > left) c.to = c.from + left;
    return c;
}
// A block's share of all columns.
__host__ __device__ __forceinline__ uint32_t share_of(const Args &a, uint32_t total) {
    const uint32_t share = (total + a.grid - 1) / a.grid;
    return share < kMinShare ? kMinShare : share;
}
// The first rows of partial results: of a prefix, of own tokens; and the blocks that
// have the latter, of a head whose columns start at `first`.
__host__ __device__ __forceinline__ uint32_t prefix_row(const Args &a, const Region &r, const Cut &c, uint32_t start, uint32_t share,
                                                        uint32_t first_seq, uint32_t g, uint32_t block) {
    return (group_parts(a, start, share, first_seq, g) + r.rank(c.block, c.row, c.head) + block) * a.prefix_cap;
}
__host__ __device__ __forceinline__ uint32_t own_row(const Args &a, uint32_t unit, uint32_t block) {
    return a.own_first_row + (unit + block) * a.own_cap;
}
__host__ __device__ __forceinline__ uint2 own_blocks(const Region &r, uint32_t first, uint32_t share) {
    return make_uint2((first + kExtra) / share, (first + r.len - 1) / share);
}

// The parts of a query's results over one set of keys, by number 0 .. count()-1:
// `subs` rows for each pair of a block of columns and a block of k_shared that
// works on it, of which there may be fewer than `each`.
struct Parts {
    Region r;
    uint32_t row, head, c0, c1;     // the columns c0 .. c1-1 of a row
    uint32_t start, share;          // of the entry; of a block
    uint32_t first_row, cap, off_b, subs;
    uint32_t b0, blocks, each;
    __host__ __device__ __forceinline__ void find() {
        b0 = c0 / r.block;
        blocks = (c1 - 1) / r.block - b0 + 1;
        uint32_t from, to;
        span(b0, from, to);
        each = blocks > 1 || r.rows > 1 ? 2 : to / share - from / share + 1;
    }
    // First and last place of the columns in a block.
    __host__ __device__ __forceinline__ void span(uint32_t b, uint32_t &from, uint32_t &to) const {
        const uint32_t n = r.columns(b), begin = b * r.block, at = start + begin * r.rows + row * n;
        from = at + (c0 > begin ? c0 - begin : 0);
        to = at + (c1 - begin < n ? c1 - begin : n) - 1;
    }
    __host__ __device__ __forceinline__ uint32_t count() const { return blocks * each * subs; }
    // The row of a part, kNone where there is none.
    __host__ __device__ __forceinline__ uint32_t at(uint32_t i) const {
        const uint32_t sub = subs == 2 ? i & 1 : 0, k = subs == 2 ? i >> 1 : i, b = k / each;
        uint32_t from, to;
        span(b0 + b, from, to);
        const uint32_t c = from / share + (k - b * each);
        if (c > to / share) return kNone;
        return first_row + (r.rank(b0 + b, row, head) + c) * cap + sub * off_b;
    }
    // The same of own tokens' parts: one column a block of k_shared.
    __host__ __device__ __forceinline__ uint32_t at_own(uint32_t i) const {
        return first_row + (c0 + i / subs) * cap + i % subs * off_b;
    }
};

// The parts over the prefix of a group g, e, of the query head `in` of sequence n's KV
// head; w: what the walking warps left in group_at.
__host__ __device__ __forceinline__ Parts prefix_parts(const Args &a, const Entry &e, uint2 w, uint32_t g, uint32_t n, uint32_t head,
                                                       uint32_t in, bool wide) {
    Parts p = {};
    p.start = w.x, p.share = w.y;
    p.r = region_of(a, e, p.share, keys_of(wide));
    const uint32_t query_row = (n - e.seq0) * a.group + in;
    p.row = query_row / a.tile_rows, p.head = head;
    p.c0 = head * p.r.len + kExtra, p.c1 = (head + 1) * p.r.len;
    const uint32_t at = query_row - p.row * a.tile_rows, rows = e.rows - p.row * a.tile_rows;
    p.first_row = group_parts(a, p.start, p.share, e.seq0, g) * a.prefix_cap + at;
    p.cap = a.prefix_cap, p.off_b = a.prefix_off_b;
    p.subs = wide || rows > kRows ? 1 : 2;
    p.find();
    return p;
}
// Those over its own tokens; w: from own_parts.
__host__ __device__ __forceinline__ Parts own_parts(const Args &a, uint2 w, uint32_t n, uint32_t head, uint32_t in, bool wide) {
    Parts p = {};
    p.r.len = p.r.rows = p.r.block = 1, p.r.width = w.y + 1;
    p.share = 1, p.c0 = w.x, p.c1 = w.y + 1;
    p.first_row = a.own_first_row + (n * a.c.heads + head) * a.own_cap + in;
    p.cap = a.own_cap, p.off_b = a.own_off_b, p.subs = wide ? 1 : 2;
    p.b0 = w.x, p.blocks = w.y - w.x + 1, p.each = 1;
    return p;
}


// A query's parts are at most 2 * (grid + 2) pairs over a prefix, and a pair for each
// block over own tokens.
__host__ __device__ __forceinline__ uint64_t most_parts(const Args &a) { return 8ull * (a.grid + 2); }

// Sizes of the call, known on the host: the lengths are not, so every bound is the tables'.
struct Plan {
    uint32_t max_len, max_prefix, grid;
    uint32_t tile_rows, prefix_cap, prefix_off_b, own_cap, own_off_b;
    uint64_t own_units, own_first_row, rows;
};

inline bool plan(const kvx_cache *c, uint32_t num_seqs, uint32_t q_heads, uint32_t blocks_per_seq, uint32_t num_groups,
                 uint32_t blocks_per_prefix, uint32_t sms, Plan &p) {
    if (!cache_ok(c) || !q_heads || q_heads % c->heads || q_heads / c->heads > kMaxGroup) return false;
    const uint64_t len = (uint64_t)blocks_per_seq * c->page_tokens, prefix = (uint64_t)blocks_per_prefix * c->page_tokens;
    if (len >= (1ull << 31) || prefix >= (1ull << 31)) return false;
    if (num_seqs >= (1u << 30) || num_groups >= (1u << 30) || (uint64_t)num_seqs * q_heads >= (1ull << 31)) return false;
    const bool wide = c->dim > 128;
    const uint32_t group = q_heads / c->heads, keys = keys_of(wide);
    const uint64_t queries = (uint64_t)num_seqs * group;
    p.max_len = (uint32_t)len, p.max_prefix = (uint32_t)prefix;
    p.tile_rows = tile_rows_of(wide);
    // a part's rows: both slots', where they have the same ones
    const uint32_t few = queries < kRows ? (uint32_t)queries : kRows;
    p.prefix_off_b = wide ? 0 : few;
    p.prefix_cap = wide ? few : 2 * few;
    p.own_off_b = wide ? 0 : group;
    p.own_cap = wide ? group : 2 * group;
    const uint64_t tiles = num_groups ? queries / p.tile_rows + num_groups : 0;
    p.own_units = (uint64_t)num_seqs * c->heads;
    const uint64_t most = tiles * c->heads * (ceil_div(prefix, kHalf) + kExtra) + p.own_units * (ceil_div(len, keys) + kExtra);
    if (tiles * (c->heads + 2) >= (1ull << 31) || most >= (1ull << 31)) return false;
    const uint64_t want = ceil_div(most, kMinShare);
    p.grid = want < sms ? (want ? (uint32_t)want : 1) : sms;
    p.own_first_row = num_groups ? (tiles * (c->heads + 2) + 2 * p.grid) * p.prefix_cap : 0;
    p.rows = p.own_first_row + (p.own_units + p.grid) * p.own_cap;
    return p.rows < (1ull << 32);
}

// What kernels and the join take of it.
inline Args args_of(const kvx_cache *c, uint32_t num_seqs, uint32_t q_heads, uint32_t blocks_per_seq, uint32_t num_groups,
                    uint32_t blocks_per_prefix, const Plan &p) {
    Args a = {};
    a.c = cache_view(c);
    a.blocks_per_prefix = blocks_per_prefix, a.num_groups = num_groups;
    a.blocks_per_seq = blocks_per_seq, a.num_seqs = num_seqs;
    a.q_heads = q_heads, a.group = q_heads / c->heads;
    a.max_prefix = p.max_prefix, a.max_len = p.max_len;
    a.by_group = FastDiv(a.group);
    a.paged16 = c->page_tokens % 16 == 0;
    a.tile_rows = p.tile_rows;
    a.prefix_cap = p.prefix_cap, a.prefix_off_b = p.prefix_off_b;
    a.own_cap = p.own_cap, a.own_off_b = p.own_off_b, a.own_first_row = (uint32_t)p.own_first_row;
    a.grid = p.grid, a.rows = p.rows;
    return a;
}

// Where among the 128 rows a slot's few ones lie, which says which of its warps works:
// the two slots' not on the same scheduler (59 us on one, 56 on two, neither an
// issuing warp's).
__host__ __device__ __forceinline__ constexpr uint32_t few_at(uint32_t slot) { return 64 + 32 * slot; }

// A part of a unit that one block works on.
struct Piece {
    const uint32_t *table;                    // its pages
    uint32_t seq0, row0, rows, head, k0, k1;  // query rows row0 .. row0 + rows-1 of seq0's group on; 0 rows end the stream
    uint32_t both, event;                     // both slots take every tile, or tiles in turn: slot `event` & 1 the first
    uint32_t few;                             // no more than kFewRows rows
    uint32_t part_row, off_b;                 // of the partial result
};

template <int DP, int ES>
struct Shape {
    static constexpr uint32_t kKeys = keys_of(DP == 256);
    // A slot has room for the logits of 128 keys: of a tile's two halves, or of
    // two tiles.  (Two halves that the tensor cores fill one by one, the next
    // while the softmax works on the other, keep the tensor cores longer: a product
    // with 64 keys reads as many bytes of the queries as one with 128, and is bound
    // by shared memory's bandwidth.  100,000 tokens, 4 x 256 rows, the products
    // alone: 327 us and 233.)
    static constexpr uint32_t kHalves = kKeys / kHalf, kPlaces = 2 / kHalves;
    static constexpr uint32_t kStage = kKeys * DP * 2;  // bytes of a tile of keys or values in 16 bits
    static constexpr uint32_t kQ = kRows * DP * 2;
    static constexpr uint32_t kQBufs = DP == 256 ? 1 : 2;
    static constexpr uint32_t kStages = ES == 2 ? (DP == 64 ? 11 : 5) : (DP == 64 ? 6 : 3);
    static constexpr uint32_t kHeld = ES == 2 ? 0 : DP == 64 ? 8 : 4;  // 8-bit tiles on their way
    static constexpr uint32_t kTiles = kQ * kQBufs + kStages * kStage + kHeld * (kStage / 2);
    static constexpr uint32_t kGroups = kKeys / 16;        // of 16 tokens in a tile
    static constexpr uint32_t kFound = 64 / (2 * kGroups);  // tiles whose look-ups may be ahead
};

// 16 tokens' rows of keys or values: where the first is, and its scale from there.
struct alignas(16) Group {
    uint64_t row;
    uint32_t scale, count;  // rows that exist
};

struct alignas(16) Shared {  // behind the tiles
    uint64_t kv_full[11], kv_empty[11];
    uint64_t q_empty[2];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // by slot and place (s_full: the tile's)
    uint64_t o_free[2];
    uint64_t pc_full[kPieces], pc_empty[kPieces];
    uint64_t found[8], taken[8];
    uint64_t turn[2];
    uint32_t begun[2];  // tiles of keys and of values whose copies to their places have begun
    uint64_t drained;
    Piece pieces[kPieces];
    Group groups[64];        // [tile][group][keys, values]
    uint32_t sums[kWarps];
    uint32_t tmem;
};
constexpr uint32_t kTileScales = 128;  // bytes of an 8-bit tile on its way, behind Shared: [row]
template <int DP, int ES>
constexpr uint32_t kSmem = Shape<DP, ES>::kTiles + sizeof(Shared) + Shape<DP, ES>::kHeld * kTileScales;

// ------------------------------------------------------------- instructions

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
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
// A word of shared memory that says how far its writer is.  (Relaxed: a release
// would wait for the writer's copies on their way.  What a reader does next, it
// asks of a barrier that the writer had seen pass.)
__device__ __forceinline__ uint32_t progress(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.relaxed.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)) : "memory");
    return v;
}
__device__ __forceinline__ void set_progress(uint32_t *p, uint32_t v) {
    asm volatile("st.relaxed.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}
// mbar_wait by a whole warp, which goes on together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity));
}
__device__ __forceinline__ bool warp_test(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, mbar_test(bar, parity));
}
// 16 bytes, or zeros where there is nothing to read.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Arrives when this thread's copies so far are complete.
__device__ __forceinline__ void mbar_arrive_copies(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait(uint32_t most) {  // until at most that many groups are on their way
    switch (most) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}
// What this thread wrote to shared memory, or has seen others write, is there for
// the tensor cores.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Until loads so far are in their registers; nothing that uses these comes before it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                     "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Arrives when the tensor instructions issued so far are complete.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// One of a warp's threads issues; all of them go the same way.
__device__ __forceinline__ bool elected() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// 16 rows of 8 * N columns: a lane has columns 2 * (lane % 4) and the next, of every
// eight, of rows lane / 4 (the first two of four values) and lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_rows64(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void tmem_ld_rows16(uint32_t (&r)[8], uint32_t at) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_st_rows16(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 16 rows of 32 columns: a lane has column lane % 4 of every four, of rows lane / 4
// and lane / 4 + 8.
__device__ __forceinline__ void tmem_st_rows32(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Operands by the low words of their descriptors (Operand); d += or, without
// `add`, d = a b.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high, uint32_t idesc,
                                       uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %6, 0;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(b_high), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Shared-memory operands lie in rows of 128 bytes whose 16-byte pieces are
// exchanged within groups of eight rows (the 128-byte swizzle).  Descriptor:
// bits 0-13 the address / 16, 16-29 and 32-45 the leading and the stride byte
// offsets / 16, 46 the version, 61-63 the swizzle.
__device__ __forceinline__ constexpr uint32_t operand_low(uint32_t addr, uint32_t leading) {
    return (addr & 0x3FFFF) >> 4 | (leading >> 4) << 16;
}
constexpr uint32_t kOperandHigh = 1024 >> 4 | 1u << 14 | 2u << 29;  // a stride of 1024 bytes from eight rows to the next
// M = 128; both operands bf16 or fp16, results 32 bits.
template <class T>
__device__ __forceinline__ uint32_t instruction(uint32_t n, bool b_by_columns, bool negate) {
    constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | (uint32_t)negate << 13 | (uint32_t)b_by_columns << 16 | n / 8 << 17 |
           kRows / 16 << 24;
}

// ------------------------------------------------------------- the schedule

// The walking warp: the block's share of all units' tiles, piece by piece.
template <int DP, int ES>
__device__ __forceinline__ bool walk(const Args &a, Shared &sh, const uint32_t *cum, uint32_t total, uint32_t per,
                                     uint32_t lane) {
    using S = Shape<DP, ES>;
    const uint32_t entries = a.num_groups + a.num_seqs;
    const uint32_t share = share_of(a, total);
    const uint64_t begin64 = (uint64_t)blockIdx.x * share;
    uint32_t at = begin64 < total ? (uint32_t)begin64 : total;
    const uint32_t end = total - at > share ? at + share : total;
    uint32_t i = 0, off = 0, np = 0, event = 0;
    Entry e = {};
    if (at < end) {
        // the thread that counted the first entry: the first whose sum passes `at`
        uint32_t t = 0;
        for (uint32_t j = 0; j < kThreads; j += 32) t += __popc(__ballot_sync(0xFFFFFFFFu, cum[j + lane] <= at));
        uint32_t before = t ? cum[t - 1] : 0;
        for (i = t * per; i < entries; i++) {
            e = entry_of(a, i);
            const Region r = region_of(a, e, share, S::kKeys);
            const uint32_t n = r.width * r.rows;
            if (at - before < n) break;
            before += n;
        }
        off = at - before;
        if (i >= entries) at = end;  // (only where lengths changed since they were counted)
    }
    __syncthreads();  // cum's place is the copies' from here on
    Entry next = {};
    if (at < end && i + 1 < entries) next = entry_of(a, i + 1);
    while (at < end) {
        const Region r = region_of(a, e, share, S::kKeys);
        if (off >= r.width * r.rows) {
            off -= r.width * r.rows;
            e = next;
            i++;
            // Those without columns, the free places of a batch, 32 at a time: one by
            // one they take 235 ns each (5 million between two sequences outlast a wait).
            if (!e.len) {
                do {
                    Entry x = {};
                    if (i + 1 + lane < entries) x = entry_of(a, i + 1 + lane);
                    const uint32_t some = __ballot_sync(0xFFFFFFFFu, x.len != 0);
                    i += some ? __ffs(some) : 32;
                    if (some) break;
                } while (i < entries);
                if (i >= entries) break;  // (as above)
                e = entry_of(a, i);
            }
            next = Entry{};
            if (i + 1 < entries) next = entry_of(a, i + 1);
            continue;
        }
        const Cut c = cut(r, off, end - at);
        const uint32_t start = at - off;  // the entry's
        at += c.to - c.from;
        off += c.to - c.from;
        if (c.to <= kExtra) continue;
        const uint32_t t0 = c.from > kExtra ? c.from - kExtra : 0, t1 = c.to - kExtra;
        if (np >= kPieces && !warp_wait(&sh.pc_empty[np % kPieces], (np / kPieces & 1) ^ 1)) return false;
        if (lane == 0) {
            Piece p;
            p.seq0 = e.seq0;
            p.row0 = c.row * a.tile_rows;
            p.rows = e.rows - p.row0 < a.tile_rows ? e.rows - p.row0 : a.tile_rows;
            p.head = c.head;
            p.k0 = t0 * r.keys;
            p.k1 = t1 * r.keys < e.len ? t1 * r.keys : e.len;
            p.both = DP == 256 || p.rows > kRows;
            p.few = p.rows <= kFewRows;
            p.event = event;
            if (i < a.num_groups) {
                p.table = a.prefix_blocks + (uint64_t)i * a.blocks_per_prefix;
                p.part_row = prefix_row(a, r, c, start, share, e.seq0, i, blockIdx.x);
                p.off_b = a.prefix_off_b;
                a.group_at[i] = make_uint2(start, share);  // the same from all blocks
            } else {
                const uint32_t u = e.seq0 * a.c.heads + c.head;
                p.table = a.blocks + (uint64_t)e.seq0 * a.blocks_per_seq;
                p.part_row = own_row(a, u, blockIdx.x);
                p.off_b = a.own_off_b;
                if (!t0) a.own_parts[u] = own_blocks(r, start + c.head * r.len, share);
            }
            sh.pieces[np % kPieces] = p;
            mbar_arrive(&sh.pc_full[np % kPieces]);
        }
        __syncwarp();
        np++;
        event += ((t1 - t0) * r.keys + S::kKeys - 1) / S::kKeys;
    }
    if (np >= kPieces && !warp_wait(&sh.pc_empty[np % kPieces], (np / kPieces & 1) ^ 1)) return false;
    if (lane == 0) {
        sh.pieces[np % kPieces].rows = 0;
        mbar_arrive(&sh.pc_full[np % kPieces]);
    }
    return true;
}

// --------------------------------------------------------------- the copies

// Stored 8-bit values times a power of two (1 in a cache with one scale, which
// enters with the logits and the sums), as 16-bit ones.  bf16, exactly: an e4m3
// value's bits, moved to a bf16's, are the value times 2^-120, normal and
// subnormal numbers alike; one product brings the scale as well.  A NaN, whose
// bits would be 480's, and scales above 2^7, whose factor bf16 does not hold, take
// the way through 32 bits (any()).
__device__ __forceinline__ void halves(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
template <class T>
struct Widen;
template <>
struct Widen<__nv_bfloat16> {
    uint32_t e, factor;
    __device__ __forceinline__ explicit Widen(uint32_t exponent) : e(exponent), factor((exponent + 120) * 0x00800080u) {}
    __device__ __forceinline__ bool simple() const { return e - 1 <= 133; }
    __device__ __forceinline__ static uint32_t check(const uint4 &v) {  // bits 7, 15, ...: there is a NaN
        auto nan = [](uint32_t w) {
            uint32_t r;
            asm("mad.lo.u32 %0, %1, 1, %2;" : "=r"(r) : "r"(w & 0x7F7F7F7Fu), "r"(0x01010101u));
            return r;
        };
        return nan(v.x) | nan(v.y) | nan(v.z) | nan(v.w);
    }
    // Bytes 0 and 2, by products that shift them by four places and their signs by
    // four more: the units for logic have half the rate and the most to do (a tile's
    // keys and values 2040 clocks so, 2320 with shifts and masks).
    __device__ __forceinline__ uint32_t two(uint32_t w) const {
        uint32_t v, r;
        asm("mul.lo.u32 %0, %1, 16;" : "=r"(v) : "r"(w));
        asm("mad.lo.u32 %0, %1, 240, %2;" : "=r"(v) : "r"(w & 0x00800080u), "r"(v));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(factor));
        return r;
    }
    __device__ __forceinline__ uint2 four(uint32_t v) const {
        return make_uint2(two(__byte_perm(v, 0, 0x4140)), two(__byte_perm(v, 0, 0x4342)));
    }
    __device__ __forceinline__ uint2 any(uint32_t v) const {
        uint32_t lo, hi;
        halves(v, lo, hi);
        const float s = row_scale(e);
        const float2 x = Pair<__half>::unpack(lo), y = Pair<__half>::unpack(hi);
        return make_uint2(Pair<__nv_bfloat16>::pack(x.x * s, x.y * s), Pair<__nv_bfloat16>::pack(y.x * s, y.y * s));
    }
};
// fp16: the conversion is exact, and a product by 2^-12 to 2^15 is as exact as
// fp16 can be; others come in two steps, of which the first is exact (an 8-bit
// value's last bit is 2^-9 or more).
template <>
struct Widen<__half> {
    uint32_t e, a;
    __device__ __forceinline__ explicit Widen(uint32_t exponent) : e(exponent) {
        const int k = (int)e - 127, ka = k < -12 ? -12 : k > 15 ? 15 : k;
        a = (uint32_t)(ka + 15) * 0x04000400u;
    }
    __device__ __forceinline__ bool simple() const { return e - 115 <= 27; }
    __device__ __forceinline__ static uint32_t check(const uint4 &) { return 0; }  // a NaN stays one
    __device__ __forceinline__ static uint32_t times(uint32_t x, uint32_t y) {
        const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    __device__ __forceinline__ uint2 four(uint32_t v) const {
        uint32_t lo, hi;
        halves(v, lo, hi);
        return make_uint2(times(lo, a), times(hi, a));
    }
    __device__ __forceinline__ uint2 any(uint32_t v) const {
        const int k = (int)e - 127, kb = k < -12 ? k + 12 : k > 15 ? k - 15 : 0;
        const uint32_t b = e == 255 ? 0x7FFF7FFFu : kb < -24 ? 0u : kb < -14 ? 0x00010001u << (kb + 24)
                                                 : (uint32_t)((kb > 15 ? 15 : kb) + 15) * 0x04000400u;
        const uint2 w = four(v);
        return make_uint2(times(w.x, b), times(w.y, b));
    }
};

// Whether a copy has begun.  A barrier's parity tells a tile from the one before in
// its place, but not from earlier ones, which may be another warp's business: so
// its copy has to have begun before the barrier is asked, for which the tile
// before must have come and gone.  `known`: what was read last.
__device__ __forceinline__ bool has_begun(const Shared &sh, uint32_t &known, uint32_t copy) {
    if (known <= copy / 2) known = progress(&sh.begun[copy & 1]);
    return known > copy / 2;
}
__device__ __forceinline__ bool await_begun(const Shared &sh, uint32_t &known, uint32_t copy) {
    if (has_begun(sh, known, copy)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < kSpinLimit; i++) {
        if (has_begun(sh, known, copy)) return true;
        if (global_ns() - t0 > kWaitNs) return false;
    }
    return false;
}

// The copying warps: four for keys, four for values, a quarter of a tile's rows
// each.  Copies are numbered 2 * tile and 2 * tile + 1 and take their places in
// turn.  Without groups of 16 tokens a lane looks up one token's segment, which
// the copying lanes take from it.
template <class T, int DP, int ES>
__device__ __forceinline__ bool copy_tiles(const Args &a, Shared &sh, uint8_t *q_smem, uint8_t *ring, uint8_t *held, uint32_t thread,
                                           uint32_t &bad) {
    using S = Shape<DP, ES>;
    constexpr uint32_t kWarpKeys = S::kKeys / kKindWarps;
    constexpr uint32_t kParts = DP * ES / 16;  // 16-byte pieces of a row
    constexpr uint32_t kAtOnce = 32 / kParts;  // rows that a warp copies with one instruction
    constexpr uint32_t kCopies = kWarpKeys / kAtOnce;
    constexpr uint32_t kHeld = S::kHeld ? S::kHeld / 2 : 1;  // of a kind
    const uint32_t kind = thread / kKindThreads, lane = thread & 31;
    thread %= kKindThreads;
    const uint32_t warp = thread / 32;
    const uint32_t key = warp * kWarpKeys + lane % kWarpKeys;  // whose address this lane looks up, within the tile
    // What it copies: that piece of rows row0 + kAtOnce * i.  Eight lanes that write
    // 8-bit rows' pieces in 16 bits, two pieces each, do so to four of a row and
    // four of the next, whose places in 128 bytes differ.
    const uint32_t part = ES == 2 ? lane % kParts : (lane & 3) | ((lane >> 3 << 2) & (kParts - 1));
    const uint32_t row0 = ES == 2 ? lane / kParts : kParts == 4 ? lane >> 2 : (lane >> 2 & 1) | (kParts == 8 ? lane >> 4 << 1 : 0);
    const bool in = part < a.c.row_bytes / 16;
    // Where those go: the pattern of the swizzle comes again after eight rows.
    constexpr uint32_t kPeriod = 8 / kAtOnce ? 8 / kAtOnce : 1;
    uint32_t place[kPeriod];
#pragma unroll
    for (uint32_t i = 0; i < kPeriod; i++) {
        const uint32_t r = i * kAtOnce + row0, p16 = ES == 2 ? part : 2 * part;  // piece in 16 bits
        place[i] = p16 / 8 * (S::kKeys * 128) + (warp * kWarpKeys + r) * 128 + ((p16 % 8 ^ (r & 7)) * 16);
    }
    auto place_of = [&](uint32_t c) { return place[c % kPeriod] + c / kPeriod * 1024; };
    const uint64_t room = a.c.pool_bytes - a.c.span;
    const bool fits = a.c.pool_bytes >= a.c.span, row_scales = ES == 1 && a.c.scale_offset;
    uint8_t *scales = reinterpret_cast<uint8_t *>(&sh + 1);

    // 16-bit tiles are copied to where the tensor cores take them, and count as
    // there when the copies arrive.  8-bit ones come to a place of the thread's own
    // first and are handed over as 16-bit ones.
    uint32_t issued = 0, done = 0;  // of this kind
    uint64_t exist = 0;             // 16 bits for each of the last four tiles: a bit less than 17 for each group, rows that exist
    auto held_at = [&](uint32_t n) { return held + (n % kHeld * 2 + kind) * (S::kStage / 2); };
    auto scales_at = [&](uint32_t n) { return scales + (n % kHeld * 2 + kind) * kTileScales + warp * kWarpKeys; };
    // Waits for room for copy n of this kind, and says that it begins.  (The copy
    // before in its place has to have begun, too, before its barrier is asked: see
    // has_begun.  With an odd number of places that is one of the other kind.)
    uint32_t others = 0;
    auto begin = [&](uint32_t n) -> bool {
        const uint32_t t = 2 * n + kind, use = t / S::kStages;
        if (use && S::kStages % 2 && !await_begun(sh, others, t - S::kStages)) return false;
        if (use && !warp_wait(&sh.kv_empty[t % S::kStages], (use & 1) ^ 1)) return false;
        if (thread == 0) set_progress(&sh.begun[kind], n + 1);
        return true;
    };
    auto hand_over = [&]() -> bool {
        const uint32_t n = done, stage = (2 * n + kind) % S::kStages;
        if (!begin(n)) return false;
        if constexpr (ES == 1) {
            const uint4 *from = reinterpret_cast<const uint4 *>(held_at(n)) + thread;
            uint8_t *to = ring + stage * S::kStage;
            const uint8_t *exponents = scales_at(n);
            __syncwarp();  // each lane has waited for its copies
            const uint32_t groups = (uint32_t)(exist >> (n % 4 * 16)) & 0xFFFF;
            auto exists = [&](uint32_t r) { return r % 16 < (groups >> (r / 16 * 8) & 0xFF); };
            uint32_t odd = 0, check = 0;
            constexpr uint32_t kBatch = kCopies < 4 ? kCopies : 4;
#pragma unroll
            for (uint32_t c0 = 0; c0 < kCopies; c0 += kBatch) {
                uint32_t e[kBatch];
                uint4 v[kBatch];
#pragma unroll
                for (uint32_t i = 0; i < kBatch; i++) {  // all reads before the first write, which they could not pass
                    const uint32_t r = (c0 + i) * kAtOnce + row0;
                    v[i] = from[(c0 + i) * kKindThreads];
                    e[i] = row_scales ? exponents[r] : 127;
                    if (row_scales && !exists(r)) e[i] = 127;  // zeros, whatever its scale says
                }
#pragma unroll
                for (uint32_t i = 0; i < kBatch; i++) {
                    const Widen<T> w(e[i]);
                    check |= Widen<T>::check(v[i]);
                    odd |= !w.simple();
                    const uint2 x0 = w.four(v[i].x), x1 = w.four(v[i].y), x2 = w.four(v[i].z), x3 = w.four(v[i].w);
                    const uint32_t at = place_of(c0 + i);
                    *reinterpret_cast<uint4 *>(to + at) = make_uint4(x0.x, x0.y, x1.x, x1.y);
                    *reinterpret_cast<uint4 *>(to + (at ^ 16)) = make_uint4(x2.x, x2.y, x3.x, x3.y);
                }
            }
            if (in && (odd | (check & 0x80808080u))) {  // (pieces behind a row's end are whatever was there)
#pragma unroll 1
                for (uint32_t c = 0; c < kCopies; c++) {
                    const uint4 raw = from[c * kKindThreads];
                    const uint32_t r = c * kAtOnce + row0, p0 = 2 * part;
                    const Widen<T> w(row_scales && exists(r) ? exponents[r] : 127);
                    const uint2 x0 = w.any(raw.x), x1 = w.any(raw.y), x2 = w.any(raw.z), x3 = w.any(raw.w);
                    const uint32_t at = p0 / 8 * (S::kKeys * 128) + (warp * kWarpKeys + r) * 128 + ((p0 % 8 ^ (r & 7)) * 16);
                    *reinterpret_cast<uint4 *>(to + at) = make_uint4(x0.x, x0.y, x1.x, x1.y);
                    *reinterpret_cast<uint4 *>(to + (at ^ 16)) = make_uint4(x2.x, x2.y, x3.x, x3.y);
                }
            }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kv_full[stage]);
        done++;
        return true;
    };
    // Hands over all that is held back, before a wait for another warp.
    auto drain = [&]() -> bool {
        if (ES == 2) return true;
        copies_wait(0);
        while (done < issued)
            if (!hand_over()) return false;
        return true;
    };
    // Room for the next tile.
    auto make_room = [&]() -> bool {
        if (ES == 2) return begin(issued);
        if (issued - done < kHeld) return true;
        copies_wait(kHeld - 1);
        return hand_over();
    };
    auto set_rows = [&](uint32_t first, uint32_t second) {
        if (ES == 1) exist = (exist & ~(0xFFFFull << (issued % 4 * 16))) | (uint64_t)(first | second << 8) << (issued % 4 * 16);
    };
    auto set_scale = [&](uint32_t exponent) {
        set_rows(16, 16);
        if (row_scales && lane < kWarpKeys) scales_at(issued)[lane] = (uint8_t)exponent;
    };
    auto issued_one = [&]() {
        if (ES == 2)
            mbar_arrive_copies(&sh.kv_full[(2 * issued + kind) % S::kStages]);
        else
            copies_commit();
        issued++;
    };
    auto place_now = [&]() {  // where the next copy's pieces go
        return smem_u32(ES == 2 ? ring + (2 * issued + kind) % S::kStages * S::kStage : held_at(issued) + thread * 16);
    };
    auto issue = [&](uint64_t row) {  // this lane's row; odd: there is none
        const uint32_t base = place_now();
        const uint32_t rows = __ballot_sync(0xFFFFFFFFu, !(row & 1)) >> row0;
        const uint64_t shift = (uint64_t)part * 16;
        if (__all_sync(0xFFFFFFFFu, !(row & 1))) {
#pragma unroll
            for (uint32_t c = 0; c < kCopies; c++) {
                const uint64_t from = __shfl_sync(0xFFFFFFFFu, row, c * kAtOnce + row0) + shift;
                if (in) copy16(base + (ES == 2 ? place_of(c) : c * (kKindThreads * 16)), reinterpret_cast<const void *>(from), true);
            }
        } else {
#pragma unroll 1
            for (uint32_t c = 0; c < kCopies; c++) {
                const uint64_t from = (__shfl_sync(0xFFFFFFFFu, row, c * kAtOnce + row0) & ~1ull) + shift;
                const uint32_t r = c * kAtOnce + row0;
                const uint32_t at = part / 8 * (S::kKeys * 128) + (warp * kWarpKeys + r) * 128 + ((part % 8 ^ (r & 7)) * 16);
                if (in) copy16(base + (ES == 2 ? at : c * (kKindThreads * 16)), reinterpret_cast<const void *>(from), rows >> (c * kAtOnce) & 1);
            }
        }
        issued_one();
    };
    uint32_t q_used[2] = {};
    auto issue_q = [&](uint32_t b, uint32_t piece) -> bool {  // rows of a piece into buffer b: they come with its first keys
        if (kind) return true;
        const Piece p = sh.pieces[piece % kPieces];
        const uint32_t r0 = DP != 256 && p.both ? b * kRows : 0;
        const uint32_t rows = p.rows - r0 < kRows ? p.rows - r0 : kRows;
        const uint32_t parity = (q_used[b] & 1) ^ 1;
        if (q_used[b] && !warp_test(&sh.q_empty[b], parity) && !(drain() && warp_wait(&sh.q_empty[b], parity))) return false;
        q_used[b]++;
        constexpr uint32_t kQParts = DP / 8;
        const uint32_t base = smem_u32(q_smem + b * S::kQ), q_parts = a.c.dim / 8;
        for (uint32_t j = thread; j < rows * kQParts; j += kKindThreads) {
            const uint32_t r = j / kQParts, part = j % kQParts;
            const uint32_t rr = p.row0 + r0 + r, s = a.by_group.div(rr);
            const uint64_t from = (uint64_t)(p.seq0 + s) * a.q_stride + (uint64_t)(p.head * a.group + rr - s * a.group) * a.c.dim;
            const uint32_t to = base + (part / 8) * (kRows * 128) + r * 128 + ((part % 8 ^ (r & 7)) * 16);
            if (part < q_parts) {
                copy16(to + (p.few ? few_at(0) * 128 : 0), static_cast<const T *>(a.q) + from + part * 8, true);
                if (p.few) copy16(to + few_at(1) * 128, static_cast<const T *>(a.q) + from + part * 8, true);
            }
        }
        return true;
    };

    if (a.paged16) {
        constexpr uint32_t kWarpGroups = kWarpKeys / 16;
        static_assert(kWarpKeys % 16 == 0 && kWarpGroups <= 2 && 16 % kAtOnce == 0);
        const uint64_t stride = a.c.token_stride, shift = row0 * stride + part * 16;
        auto issue_groups = [&](const Group (&g)[kWarpGroups]) {
            const uint32_t base = place_now();
            const bool whole = g[0].count == 16 && g[kWarpGroups - 1].count == 16;
#pragma unroll
            for (uint32_t k = 0; k < kWarpGroups; k++) {
                const uint8_t *from = reinterpret_cast<const uint8_t *>(g[k].row + shift);
#pragma unroll
                for (uint32_t i = 0; i < 16 / kAtOnce; i++, from += kAtOnce * stride) {
                    const uint32_t c = k * (16 / kAtOnce) + i, to = base + (ES == 2 ? place_of(c) : c * (kKindThreads * 16));
                    const bool there = whole || row0 + i * kAtOnce < g[k].count;
                    if (in) copy16(to, there ? from : a.c.pool, there);
                }
            }
            set_rows(g[0].count, g[kWarpGroups - 1].count);
            if (row_scales && lane < kWarpGroups) {  // a group's 16 scales lie together
                const Group &last = g[kWarpGroups - 1];
                const uint64_t from = lane ? last.row + last.scale : g[0].row + g[0].scale;
                copy16(smem_u32(scales_at(issued) + lane * 16), reinterpret_cast<const uint8_t *>(from), (lane ? last.count : g[0].count) > 0);
            }
            issued_one();
        };
        uint32_t tile = 0;
        for (uint32_t np = 0;; np++) {
            uint64_t *bar = &sh.pc_full[np % kPieces];
            if (!warp_test(bar, np / kPieces & 1) && !(drain() && warp_wait(bar, np / kPieces & 1))) return false;
            const Piece &p = sh.pieces[np % kPieces];
            if (!p.rows) return drain();
            const uint32_t nt = (p.k1 - p.k0 + S::kKeys - 1) / S::kKeys, both = p.both;
            for (uint32_t b = 0; b < S::kQBufs; b++)
                if ((DP == 256 || both || b == (np & 1)) && !issue_q(b, np)) return false;
            for (uint32_t t = 0; t < nt; t++, tile++) {
                const uint32_t slot = tile % S::kFound, parity = tile / S::kFound & 1;
                if (!warp_test(&sh.found[slot], parity) && !(drain() && warp_wait(&sh.found[slot], parity))) return false;
                Group g[kWarpGroups];
#pragma unroll
                for (uint32_t k = 0; k < kWarpGroups; k++) g[k] = sh.groups[(slot * S::kGroups + warp * kWarpGroups + k) * 2 + kind];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.taken[slot]);
                if (!make_room()) return false;
                issue_groups(g);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pc_empty[np % kPieces]);
        }
    }

    // A tile on its way through the look-up: its block ids, then its segments'
    // addresses, then its rows' scales are loaded, each while the tile before
    // is a step further.
    struct Look {
        uint32_t any, first, last, piece;
        uint32_t valid, token, head;
    };
    uint32_t np = 0, k = 0, k1 = 0, head = 0;  // where the look-up is
    const uint32_t *table = nullptr;
    bool over = false, alive = true;
    uint32_t id = 0;
    uint64_t seg = 0;
    auto find = [&]() -> Look {
        Look l = {};
        if (over || !alive) return l;
        if (k >= k1) {
            uint64_t *bar = &sh.pc_full[np % kPieces];
            if (!warp_test(bar, np / kPieces & 1) && !(drain() && warp_wait(bar, np / kPieces & 1))) {
                alive = false;
                return l;
            }
            const Piece &p = sh.pieces[np % kPieces];
            if (!p.rows) {
                over = true;
                return l;
            }
            k = p.k0, k1 = p.k1, head = p.head, table = p.table;
            l.first = 1;
            np++;
        }
        l.any = 1;
        l.piece = np - 1;
        l.head = head;
        const uint32_t pos = k + key;
        l.valid = pos < k1;
        const uint32_t page = a.c.page.div(l.valid ? pos : k);
        l.token = pos - page * a.c.page.d;
        id = 0;
        if (l.valid) id = __ldg(table + page);
        k += S::kKeys;
        l.last = k >= k1;
        return l;
    };
    auto find_segments = [&](Look &l) {
        if (l.valid && id >= a.c.B) bad |= KVX_S_BOUNDS, l.valid = 0;
        if (l.valid) seg = __ldg(a.c.lane_addr(id, l.head, kind));
    };

    // The row of the tile after a look-up's, with its scale on its way.
    struct Row {
        uint64_t row;
        uint32_t exponent;
        uint32_t any, first, last, piece;
    };
    auto find_row = [&](const Look &l) -> Row {
        Row r = {};
        r.any = l.any, r.first = l.first, r.last = l.last, r.piece = l.piece;
        if (!l.any) return r;
        const bool good = l.valid && fits && seg <= room && !((uint32_t)seg & 15);
        if (l.valid && !good) a.c.ok(seg, bad);
        r.row = reinterpret_cast<uint64_t>(a.c.pool) + (good ? seg + l.token * a.c.token_stride : 1);
        r.exponent = 127;
        if (row_scales && good) r.exponent = __ldg(a.c.pool + seg + a.c.scale_offset + l.token);
        return r;
    };
    Look one = find();
    find_segments(one);
    Look two = one.any ? find() : Look{};
    Row next = find_row(one);
    one = two;
    find_segments(one);
    two = one.any ? find() : Look{};
    while (next.any && alive) {
        // the next tile's scales, the addresses of the one after and the block ids
        // of the one after that are loaded meanwhile
        const Row now = next;
        next = find_row(one);
        one = two;
        find_segments(one);
        two = one.any ? find() : Look{};
        if (!alive || !make_room()) return false;
        if (now.first) {
            const uint32_t both = sh.pieces[now.piece % kPieces].both;
            for (uint32_t b = 0; b < S::kQBufs; b++)
                if ((DP == 256 || both || b == (now.piece & 1)) && !issue_q(b, now.piece)) return false;
        }
        set_scale(now.exponent);
        issue(now.row);
        if (now.last) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pc_empty[now.piece % kPieces]);
        }
    }
    return alive && drain();
}

// The looking-up warp, for pages of whole groups of 16 tokens: a lane has the keys'
// or the values' segment of one group; several tiles at a time.  Block ids of a
// step are loaded while the segment addresses of the step before are.
template <int DP, int ES>
__device__ __forceinline__ bool look_up(const Args &a, Shared &sh, uint32_t lane, uint32_t &bad) {
    using S = Shape<DP, ES>;
    constexpr uint32_t kLanes = 2 * S::kGroups, kTilesAtOnce = 32 / kLanes;
    const uint32_t which = lane / kLanes, group = lane % kLanes / 2, kv = lane & 1;
    const uint64_t room = a.c.pool_bytes - a.c.span;
    const bool fits = a.c.pool_bytes >= a.c.span;
    uint32_t np = 0, k = 0, k1 = 0, head = 0;
    const uint32_t *table = nullptr;
    bool over = false, alive = true;
    struct Step {
        uint32_t tiles, count, token, head;
    };
    uint32_t id = 0;
    uint64_t seg = 0;
    auto find = [&]() -> Step {
        Step s = {};
        if (over || !alive) return s;
        if (k >= k1) {
            alive = warp_wait(&sh.pc_full[np % kPieces], np / kPieces & 1);
            if (!alive) return s;
            const Piece p = sh.pieces[np % kPieces];
            __syncwarp();
            if (!p.rows) {
                over = true;
                return s;
            }
            if (lane == 0) mbar_arrive(&sh.pc_empty[np % kPieces]);
            k = p.k0, k1 = p.k1, head = p.head, table = p.table;
            np++;
        }
        const uint32_t left = (k1 - k + S::kKeys - 1) / S::kKeys, pos = k + which * S::kKeys + group * 16;
        s.tiles = left < kTilesAtOnce ? left : kTilesAtOnce;
        s.head = head;
        s.count = pos < k1 ? (k1 - pos < 16 ? k1 - pos : 16) : 0;
        const uint32_t page = a.c.page.div(s.count ? pos : k);
        s.token = pos - page * a.c.page.d;
        id = __ldg(table + page);
        k += s.tiles * S::kKeys;
        return s;
    };
    auto find_segment = [&](Step &s) {
        if (s.count && id >= a.c.B) bad |= KVX_S_BOUNDS, s.count = 0;
        seg = 0;
        if (s.count) seg = __ldg(a.c.lane_addr(id, s.head, kv));
    };
    Step one = find();
    find_segment(one);
    Step two = one.tiles ? find() : Step{};
    uint32_t tile = 0;
    while (one.tiles && alive) {
        Group g;
        const bool good = fits && seg <= room && !((uint32_t)seg & 15);
        if (one.count && !good) a.c.ok(seg, bad);
        g.count = good ? one.count : 0;
        g.row = reinterpret_cast<uint64_t>(a.c.pool) + (g.count ? seg + one.token * a.c.token_stride : 0);
        g.scale = (uint32_t)(a.c.scale_offset + one.token - one.token * a.c.token_stride);
        const Step now = one;
        find_segment(two);
        one = two;
        for (uint32_t t = 0; t < now.tiles; t++) {
            const uint32_t slot = (tile + t) % S::kFound, use = (tile + t) / S::kFound;
            if (use && !warp_wait(&sh.taken[slot], (use & 1) ^ 1)) return false;
        }
        if (which < now.tiles) sh.groups[((tile + which) % S::kFound * S::kGroups + group) * 2 + kv] = g;
        __syncwarp();
        if (lane < now.tiles) mbar_arrive(&sh.found[(tile + lane) % S::kFound]);
        tile += now.tiles;
        two = one.tiles ? find() : Step{};
    }
    return alive;
}

// --------------------------------------------------------- the tensor cores

// One warp a slot, of which one thread does it all: without votes and branches
// that a warp would have to come together after.  It takes the next product Q K^T
// as soon as there is room for its logits and keys are there, else the oldest
// product with V.
template <class T, int DP, int ES>
__device__ __forceinline__ bool multiply(const Args &a, Shared &sh, const uint8_t *q_smem, const uint8_t *ring, uint32_t tmem,
                                         uint32_t slot) {
    using S = Shape<DP, ES>;
    const uint32_t steps = a.c.dim / 16;
    const uint32_t qk = instruction<T>(S::kKeys, false, a.negate), qk_half = instruction<T>(kHalf, false, a.negate);
    const uint32_t pv = instruction<T>(DP == 256 ? (slot ? a.c.dim - 128 : 128) : a.c.dim, true, false);
    const uint32_t q0 = operand_low(smem_u32(q_smem), 16), k0 = operand_low(smem_u32(ring), 16);
    const uint32_t v0 = operand_low(smem_u32(ring) + (DP == 256 ? slot * 2 * (S::kKeys * 128) : 0), S::kKeys * 128);
    const uint32_t s_at = tmem + slot * 128, o_at = tmem + 256 + slot * 128;
    uint32_t tile = 0;                         // its keys are the copies' number 2 * tile, its values the next
    uint32_t started = 0, done = 0, outs = 0;  // this slot's tiles, and pieces with one
    struct Due {    // a product with V
        uint32_t v;  // the values' number
        bool fresh, second, twice;  // the piece's first; the tile has a second half; lets go of the values for both slots
    };
    Due due = {}, then = {};
    uint32_t keys_begun = 0, values_begun = 0;
    auto there = [&](uint32_t &known, uint32_t copy) -> bool {
        return has_begun(sh, known, copy) && mbar_test(&sh.kv_full[copy % S::kStages], copy / S::kStages & 1);
    };
    auto await = [&](uint32_t &known, uint32_t copy) -> bool {
        return await_begun(sh, known, copy) && mbar_wait(&sh.kv_full[copy % S::kStages], copy / S::kStages & 1);
    };
    auto times_v = [&](uint32_t h) -> bool {  // with the values of a half
        const uint32_t stage = due.v % S::kStages, place = S::kHalves == 2 ? h : done & 1;
        if (!mbar_wait(&sh.p_full[slot][place], (S::kHalves == 2 ? done : done >> 1) & 1)) return false;
        tmem_after();
        if (!h) fence_async();  // the copies' writes, too, are before what follows
        if (!h || due.second) {
            const uint32_t low = v0 + stage * (S::kStage / 16);
#pragma unroll
            for (uint32_t i = 0; i < kHalf / 16; i++)
                mma_ts(o_at, s_at + place * kHalf + i * 8, low + (h * kHalf / 16 + i) * 128, kOperandHigh, pv, h || i ? 1 : !due.fresh);
        }
        mma_commit(&sh.pv_done[slot][place]);
        return true;
    };
    auto finish_most = [&]() -> bool {  // but for the last half
        if (!await(values_begun, due.v)) return false;
        if (due.fresh) {
            if (outs && !mbar_wait(&sh.o_free[slot], (outs & 1) ^ 1)) return false;
            outs++;
        }
        return S::kHalves == 1 || times_v(0);
    };
    auto finish_rest = [&]() -> bool {
        if (!times_v(S::kHalves - 1)) return false;
        mma_commit(&sh.kv_empty[due.v % S::kStages]);
        if (due.twice) mma_commit(&sh.kv_empty[due.v % S::kStages]);
        due = then;
        done++;
        return true;
    };
    auto finish = [&]() -> bool { return finish_most() && finish_rest(); };
    // Where both slots take every tile they take turns: what one gives the tensor
    // cores at a time, the rest of a tile and the next one's logits, is not mixed
    // with the other's.  Mixed, both end together, and both softmaxes want the same
    // units at the same time while the tensor cores wait (100,000
    // tokens, 4 x 256 rows: 425 us and 368).
    uint32_t turns = 0;
    auto take_turn = [&]() -> bool { return slot ? mbar_wait(&sh.turn[1], turns & 1) : !turns || mbar_wait(&sh.turn[0], (turns & 1) ^ 1); };
    for (uint32_t np = 0;; np++) {
        if (!mbar_test(&sh.pc_full[np % kPieces], np / kPieces & 1)) {
            while (done != started)  // nothing waits for the next piece
                if (!finish()) return false;
            if (!mbar_wait(&sh.pc_full[np % kPieces], np / kPieces & 1)) return false;
        }
        const Piece &p = sh.pieces[np % kPieces];
        if (!p.rows) break;
        const uint32_t keys = p.k1 - p.k0, nt = (keys + S::kKeys - 1) / S::kKeys;
        const bool both = p.both;
        uint32_t t = both ? 0 : (p.event & 1) ^ slot;
        const bool any = t < nt;
        const uint32_t q = q0 + (DP == 256 ? 0 : both ? slot : np & 1) * (S::kQ / 16);
        for (bool fresh = true; t < nt; t += both ? 1 : 2, fresh = false) {
            const uint32_t k = 2 * (tile + t), stage = k % S::kStages;
            // (a piece's queries come with its first keys)
            if (started - done == S::kPlaces) {
                if (!finish_most()) return false;
                const bool now = both && there(keys_begun, k);
                if (now && !take_turn()) return false;
                if (!finish_rest()) return false;
                if (!now) {
                    while (done != started && !there(keys_begun, k))
                        if (!finish()) return false;
                    if (!await(keys_begun, k)) return false;
                    if (both && !take_turn()) return false;
                }
            } else {
                while (done != started && !there(keys_begun, k))
                    if (!finish()) return false;
                if (!await(keys_begun, k)) return false;
                if (both && !take_turn()) return false;
            }
            tmem_after();
            fence_async();
            const bool second = S::kHalves == 2 && keys - t * S::kKeys > kHalf;
            const uint32_t kk = k0 + stage * (S::kStage / 16), place = S::kPlaces == 2 ? started & 1 : 0, d = s_at + place * kHalf;
            const uint32_t what = S::kHalves == 1 || second ? qk : qk_half;
#pragma unroll
            for (uint32_t i = 0; i < DP / 16; i++)
                if (i < steps)
                    mma_ss(d, q + i / 4 * (kRows * 8) + i % 4 * 2, kOperandHigh, kk + i / 4 * (S::kKeys * 8) + i % 4 * 2,
                           kOperandHigh, what, i > 0);
            if (both) mbar_arrive(&sh.turn[slot ^ 1]), turns++;
            mma_commit(&sh.s_full[slot][place]);
            mma_commit(&sh.kv_empty[stage]);
            if (!both) mma_commit(&sh.kv_empty[stage]);
            const Due r = {k + 1, fresh, second, !both};
            if (started == done)
                due = r;
            else
                then = r;
            started++;
        }
        tile += nt;
        // both slots let go of a query, or the only one that took it twice
        if (any)
            for (int i = 0; i < (both || nt > 1 ? 1 : 2); i++) {
                if (DP == 256 || both || !(np & 1)) mma_commit(&sh.q_empty[0]);
                if (DP != 256 && (both || (np & 1))) mma_commit(&sh.q_empty[1]);
            }
        mbar_arrive(&sh.pc_empty[np % kPieces]);
    }
    while (done != started)
        if (!finish()) return false;
    return true;
}

// -------------------------------------------------------------- the softmax

// Pairs of floats: two results an instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Weights are 2^(logit - base).  The base follows the running maximum only when
// a logit exceeds it by more than kSlack + kBoost: sums and outputs are
// divided by the same power in the end.  It lies kBoost below that maximum,
// so that in fp16, whose smallest step is 2^-24, small weights keep some
// bits more beside a large one.
constexpr float kSlack = 8.0f;
template <class T>
constexpr float kBoost = std::is_same<T, __half>::value ? 7.0f : 0.0f;
struct Running {  // a row's
    float base, limit, sum;
    // What sums and outputs are to be multiplied by where a larger maximum has come.
    __device__ __forceinline__ float follow(float top, float boost) {
        const float to = top - boost, factor = limit == -INFINITY ? 0.0f : exp2_fast(base - to);  // 0: nothing was added so far
        base = to;
        limit = top + kSlack;
        sum *= factor;
        return factor;
    }
};

// soften's part for a piece of at most kFewRows rows.  One warp of a slot has them all,
// and a lane 32 logits of a row (of a tile with 128 keys) and, with more than eight
// rows, of another: its four lanes are of one mind.  With a row a lane, as in soften,
// 24 lanes of 32 idle over eight rows (48 sequences of up to 8000 tokens, 8-bit rows,
// 8 heads of 64: 72 us, and 53 so).  A loop of its own, whose registers soften's does
// not spill (100,000 tokens behind 4 x 256 rows 386 us in one loop, 373 in two).
template <class T, int DP, int ES>
__device__ __forceinline__ bool soften_few(Shared &sh, uint32_t s_at, uint32_t o_at, uint32_t slot, bool mine, uint32_t t, uint32_t tiles,
                                        uint32_t keys, uint32_t step, uint32_t rows, uint32_t cols, float scale2, float *part_o,
                                        float2 *part_ml, uint32_t dim) {
    using S = Shape<DP, ES>;
    constexpr int kN = S::kKeys / kHalf;
    const uint32_t lane = threadIdx.x & 31, nt = (keys + S::kKeys - 1) / S::kKeys;
    const uint64_t scale = pair(scale2, scale2);
    const bool more = rows > 8, any = t < nt;
    Running run[2] = {{0, -INFINITY, 0}, {0, -INFINITY, 0}};
    bool fresh = true;
    for (; t < nt; t += step, tiles++) {
        const uint32_t left_tile = keys - t * S::kKeys, tile_place = S::kPlaces == 2 ? tiles & 1 : 0;
        if (!warp_wait(&sh.s_full[slot][tile_place], (S::kPlaces == 2 ? tiles >> 1 : tiles) & 1)) return false;
        if (mine) {
            const uint32_t s = s_at + (S::kPlaces == 2 ? tile_place * kHalf : 0);
            uint32_t x[kN][32];
            tmem_after();
#pragma unroll
            for (int n = 0; n < kN; n++) tmem_ld_rows64(x[n], s + n * kHalf);
#pragma unroll
            for (int n = 0; n < kN; n++) tmem_wait_ld(x[n]);
            if (left_tile < S::kKeys) {
#pragma unroll
                for (int n = 0; n < kN; n++)
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        if (n * kHalf + i / 4 * 8 + lane % 4 * 2 + i % 2 >= left_tile) x[n][i] = 0xFF800000u;
            }
            float factor[2] = {1.0f, 1.0f};
            bool over = false;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                if (k && !more) break;
                float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < kN; n++)
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        tops[i % 4] = fmaxf(tops[i % 4], fmaxf(__uint_as_float(x[n][4 * i + 2 * k]), __uint_as_float(x[n][4 * i + 2 * k + 1])));
                float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2)) * scale2;
                if (lane / 4 + 8 * k < rows && top > run[k].limit) factor[k] = run[k].follow(top, kBoost<T>), over = true;
            }
            if (__any_sync(0xFFFFFFFFu, over) && !fresh) {
                // the product before has to be in the outputs: with one place for
                // logits it came before this tile's first one
                if (S::kPlaces == 2 && !warp_wait(&sh.pv_done[slot][tile_place ^ 1], (tiles - 1) >> 1 & 1)) return false;
                tmem_after();
#pragma unroll 1
                for (uint32_t c = 0; c < cols; c += 16) {
                    uint32_t y[8];
                    tmem_ld_rows16(y, o_at + c);
                    tmem_wait_ld(y);
#pragma unroll
                    for (int i = 0; i < 8; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) * factor[i / 2 % 2]);
                    tmem_st_rows16(o_at + c, y);
                }
                tmem_wait_st();
            }
            uint32_t w[kN][16] = {};
#pragma unroll
            for (int k = 0; k < 2; k++) {
                if (k && !more) break;
                const uint64_t shift = pair(-run[k].base, -run[k].base);
                uint64_t sums[2] = {};
#pragma unroll
                for (int n = 0; n < kN; n++)
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        float e0, e1;
                        unpair(fma2(pair(__uint_as_float(x[n][4 * i + 2 * k]), __uint_as_float(x[n][4 * i + 2 * k + 1])), scale, shift), e0, e1);
                        e0 = exp2_fast(e0), e1 = exp2_fast(e1);
                        sums[i & 1] = add2(sums[i & 1], pair(e0, e1));
                        w[n][2 * i + k] = Pair<T>::pack(e0, e1);
                    }
                float s0, s1;
                unpair(add2(sums[0], sums[1]), s0, s1);
                run[k].sum += s0 + s1;
            }
#pragma unroll
            for (int n = 0; n < kN; n++) tmem_st_rows32(s + n * kHalf, w[n]);
            tmem_wait_st();
            tmem_before();
        }
        __syncwarp();
        if (lane < S::kHalves) mbar_arrive(&sh.p_full[slot][S::kHalves == 2 ? lane : tile_place]);
        fresh = false;
    }
    if (any) {
        const uint32_t last = tiles - 1;
        if (!warp_wait(&sh.pv_done[slot][S::kHalves == 2 ? 1 : last & 1], (S::kHalves == 2 ? last : last >> 1) & 1)) return false;
        if (mine) {
            tmem_after();
#pragma unroll 1
            for (uint32_t c = 0; c < cols; c += 16) {
                uint32_t y[8];
                tmem_ld_rows16(y, o_at + c);
                tmem_wait_ld(y);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const uint32_t x = lane / 4 + i / 2 % 2 * 8;
                    if (x < rows)
                        *reinterpret_cast<uint2 *>(part_o + (uint64_t)x * dim + c + i / 4 * 8 + lane % 4 * 2) = make_uint2(y[i], y[i + 1]);
                }
            }
            tmem_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_free[slot]);
    }
    if (mine && part_ml) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            float l = any ? run[k].sum : 0.0f;
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
            const uint32_t x = lane / 4 + 8 * k;
            if (lane % 4 == 0 && x < rows) part_ml[x] = make_float2(run[k].base, l);
        }
    }
    return true;
}

template <class T, int DP, int ES>
__device__ __forceinline__ bool soften(const Args &a, Shared &sh, uint32_t tmem, uint32_t slot, uint32_t warp, uint32_t lane) {
    using S = Shape<DP, ES>;
    const uint32_t r = warp * 32 + lane;  // row of the slot
    const uint32_t lanes = (warp * 32) << 16;
    const uint32_t s_at = tmem + lanes + slot * 128, o_at = tmem + lanes + 256 + slot * 128;
    const uint32_t col = DP == 256 ? slot * 128 : 0;
    const uint32_t cols = DP == 256 ? (slot ? a.c.dim - 128 : 128) : a.c.dim;  // of the output, a multiple of 16
    const uint64_t scale = pair(a.scale2, a.scale2);
    uint32_t tiles = 0;  // of this slot
    for (uint32_t np = 0;; np++) {
        if (!warp_wait(&sh.pc_full[np % kPieces], np / kPieces & 1)) return false;
        const Piece &p = sh.pieces[np % kPieces];
        if (!p.rows) return true;
        const uint32_t keys = p.k1 - p.k0, nt = (keys + S::kKeys - 1) / S::kKeys;
        const bool both = p.both;
        const uint32_t first_row = DP != 256 && both ? slot * kRows : 0;
        const bool busy = first_row + warp * 32 < p.rows, mine = first_row + r < p.rows;
        uint32_t t = both ? 0 : (p.event & 1) ^ slot;
        const bool any = t < nt;
        if (p.few) {
            const uint32_t step = both ? 1 : 2;
            const uint64_t row = p.part_row + (slot && DP != 256 ? p.off_b : 0);
            if (!soften_few<T, DP, ES>(sh, s_at, o_at, slot, warp == few_at(slot) / 32, t, tiles, keys, step, p.rows, cols, a.scale2,
                                       a.part_o + row * a.c.dim + col, DP == 256 && slot ? nullptr : a.part_ml + row, a.c.dim))
                return false;
            if (any) tiles += (nt - t + step - 1) / step;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pc_empty[np % kPieces]);
            continue;
        }
        bool fresh = true;
        Running run = {0, -INFINITY, 0};
        for (; t < nt; t += both ? 1 : 2, tiles++) {
            const uint32_t left_tile = keys - t * S::kKeys, tile_place = S::kPlaces == 2 ? tiles & 1 : 0;
            if (!warp_wait(&sh.s_full[slot][tile_place], (S::kPlaces == 2 ? tiles >> 1 : tiles) & 1)) return false;
#pragma unroll 1
            for (uint32_t h = 0; h < S::kHalves; h++) {
                const uint32_t place = S::kHalves == 2 ? h : tiles & 1;
                const uint32_t left = left_tile > h * kHalf ? left_tile - h * kHalf : 0;
                if (busy && left) {
                    tmem_after();
                    const uint32_t s = s_at + place * kHalf;
                    if (left < kHalf) {  // what lies behind the last key weighs nothing
#pragma unroll 1
                        for (uint32_t c = left & ~15u; c < kHalf; c += 16) {
                            uint32_t y[16];
                            tmem_ld16(y, s + c);
                            tmem_wait_ld(y);
#pragma unroll
                            for (int i = 0; i < 16; i++) y[i] = c + i < left ? y[i] : 0xFF800000u;
                            tmem_st16(s + c, y);
                        }
                        tmem_wait_st();
                    }
                    uint32_t x[2][32];
                    tmem_ld32(x[0], s);
                    tmem_ld32(x[1], s + 32);
                    tmem_wait_ld(x[0]);
                    tmem_wait_ld(x[1]);
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 64; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            top[k] = fmaxf(top[k], fmaxf(__uint_as_float(x[i / 32][i % 32 + 2 * k]), __uint_as_float(x[i / 32][i % 32 + 2 * k + 1])));
                    top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale2;
                    const bool over = top[0] > run.limit;
                    if (__any_sync(0xFFFFFFFFu, over)) {
                        const float factor = over ? run.follow(top[0], kBoost<T>) : 1.0f;
                        if (!fresh) {
                            // the product before has to be in the outputs
                            const uint32_t use = S::kHalves == 2 ? (h ? tiles : tiles - 1) : (tiles - 1) >> 1;
                            if (!warp_wait(&sh.pv_done[slot][place ^ 1], use & 1)) return false;
                            tmem_after();
#pragma unroll 1
                            for (uint32_t c = 0; c < cols; c += 16) {
                                uint32_t y[16];
                                tmem_ld16(y, o_at + c);
                                tmem_wait_ld(y);
#pragma unroll
                                for (int i = 0; i < 16; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) * factor);
                                tmem_st16(o_at + c, y);
                            }
                            tmem_wait_st();
                        }
                    }
                    const uint64_t shift = pair(-run.base, -run.base);
                    uint64_t sums[2] = {};
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            float e0, e1;
                            unpair(fma2(pair(__uint_as_float(x[h][2 * i]), __uint_as_float(x[h][2 * i + 1])), scale, shift), e0, e1);
                            e0 = exp2_fast(e0), e1 = exp2_fast(e1);
                            sums[i & 1] = add2(sums[i & 1], pair(e0, e1));
                            w[i] = Pair<T>::pack(e0, e1);
                        }
                        tmem_st16(s + h * 16, w);
                    }
                    float s0, s1;
                    unpair(add2(sums[0], sums[1]), s0, s1);
                    run.sum += s0 + s1;
                    tmem_wait_st();
                    tmem_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[slot][place]);
                fresh = false;
            }
        }
        const uint64_t row = p.part_row + (slot && DP != 256 ? p.off_b : 0) + r;
        if (any) {
            const uint32_t last = tiles - 1;
            if (!warp_wait(&sh.pv_done[slot][S::kHalves == 2 ? 1 : last & 1], (S::kHalves == 2 ? last : last >> 1) & 1)) return false;
            if (busy) {
                tmem_after();
#pragma unroll 1
                for (uint32_t c = 0; c < cols; c += 16) {
                    uint32_t y[16];
                    tmem_ld16(y, o_at + c);
                    tmem_wait_ld(y);
                    if (mine) {
                        uint4 *to = reinterpret_cast<uint4 *>(a.part_o + row * a.c.dim + col + c);
#pragma unroll
                        for (int i = 0; i < 4; i++) to[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    }
                }
                tmem_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.o_free[slot]);
        }
        if (mine && (DP != 256 || !slot)) a.part_ml[row] = make_float2(run.base, any ? run.sum : 0.0f);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pc_empty[np % kPieces]);
    }
}

// Units are a KV head's query rows of a group (128 or 256 at a time) over the
// group's prefix, and a sequence's query heads over its own tokens; a block goes
// through an equal share of all units' columns, piece by piece (Region). For a tile
// of keys and the 128 rows of a slot
//     S = Q K^T          128 x keys, in tensor memory
//     P = 2^(S - base)   in 16 bits, in place of S
//     O += P V           128 x dim, in tensor memory
// with tcgen05.mma: queries and tiles come from shared memory (128-byte swizzle), P
// from tensor memory.  A block has two slots, each with its softmax warps and its
// issuing thread, so that one's products run beside the other's softmax: of more
// than 128 rows both take every tile, else they take tiles in turn.  Of heads wider
// than 128, whose outputs one slot's part of tensor memory does not hold, both slots
// take the same rows and tiles, half of V's columns each: Q K^T and its exponentials
// are done twice.  Bases, sums and outputs go to k_join, a row of floats each.
//
// Weights are rounded to 16 bits for the second product (as V and the output are):
// beside the output's own rounding that adds as much again, 1.4 times the error
// (kvx_attend, bound by its copies, multiplies the sum of two 16-bit weights; here
// that would be half as many products again).  Their sums are of the unrounded ones.
//
// Keys and values are copied by cp.async, 16 bytes at a time, to where the swizzle has
// them, from rows at any multiple of 16 bytes; copies by tensor map were not tried.
// 8-bit rows come to a place of their own and are widened with their scale on the way
// to the tile.
//
// Bound, for many rows, by the softmax and the latency from product to product (a
// tile takes two slots 2050 clocks of the tensor cores and 3900 in all): 128 x
// 64 heads over 100,000 tokens of 8 KV heads of 128, bf16, 368 us, 1140 TFLOP/s, 59 %
// of the measured rate of matrix products, with 490 MB of DRAM reads for 433 MB of
// cache.  For few rows by the copies: 8 x 16,000 own tokens, bf16, 91 us at 5.8 TB/s;
// in 8 bits by their widening, 62 instructions per 16 values, and a tile's chain:
// 106 us at 2.5 TB/s.  Heads of 256, four KV heads: 8 x 16,000 own tokens 93 us, 64 x 16
// heads over 16,000 shared ones 61 (128, eight: 90 and 57).  Threads have 96 registers,
// of which every variant spills some (28 to 124 bytes stored, 80 to 116 loaded).
template <class T, int DP, int ES>
__global__ void __launch_bounds__(kThreads, 1) k_shared(const __grid_constant__ Args a) {
    using S = Shape<DP, ES>;
    extern __shared__ __align__(1024) uint8_t smem[];  // (without others it starts on a multiple of 1024)
    uint8_t *ring = smem, *q_smem = smem + S::kStages * S::kStage, *held = q_smem + S::kQBufs * S::kQ;
    Shared &sh = *reinterpret_cast<Shared *>(smem + S::kTiles);
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- count all tiles
    const uint32_t entries = a.num_groups + a.num_seqs, per = (entries + kThreads - 1) / kThreads;
    uint32_t *cum = reinterpret_cast<uint32_t *>(smem);
    uint32_t mine = 0, bad = 0;
    bool disorder = false;
    for (uint32_t i = threadIdx.x * per; i < (threadIdx.x + 1) * per && i < entries; i++) {
        const Entry e = entry_of(a, i);
        if (e.disorder || e.beyond) bad |= KVX_S_BOUNDS;
        disorder |= e.disorder;
        const Region r = region_of(a, e, 1, S::kKeys);
        mine += r.width * r.rows;
    }
    uint32_t upto = warp_incl_sum(mine);
    if (lane == 31) sh.sums[warp] = upto;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S::kStages; i++) mbar_init(&sh.kv_full[i], ES == 2 ? kKindThreads : kKindWarps), mbar_init(&sh.kv_empty[i], 2);
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.q_empty[i], 2);
            for (int k = 0; k < 2; k++) mbar_init(&sh.s_full[i][k], 1), mbar_init(&sh.p_full[i][k], 4), mbar_init(&sh.pv_done[i][k], 1);
            mbar_init(&sh.o_free[i], 4);
        }
        for (int i = 0; i < kPieces; i++)
            mbar_init(&sh.pc_full[i], 1), mbar_init(&sh.pc_empty[i], kSoftWarps + kCopyWarps + 2 + (a.paged16 ? 1 : 0));
        for (int i = 0; i < 8; i++) mbar_init(&sh.found[i], 1), mbar_init(&sh.taken[i], kCopyWarps);
        mbar_init(&sh.drained, 2);
        mbar_init(&sh.turn[0], 1), mbar_init(&sh.turn[1], 1);
        sh.begun[0] = sh.begun[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (__syncthreads_or(disorder)) {  // (groups may overlap: their parts, and all tiles, would be more than there is room for)
        raise(a.status, bad);
        return;
    }
    uint32_t total = 0;
    for (uint32_t w = 0; w < kWarps; w++) {
        if (w < warp) upto += sh.sums[w];
        total += sh.sums[w];
    }
    cum[threadIdx.x] = upto;
    raise(a.status, bad);
    bad = 0;
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tmem_before();
    }
    __syncthreads();
    tmem_after();
    const uint32_t tmem = sh.tmem;
    bool ok = true;
    if (warp == kWalkWarp) {
        ok = walk<DP, ES>(a, sh, cum, total, per, lane);
    } else {
        __syncthreads();  // the walking warp has found its first entry
        if (warp < kSoftWarps) {
            ok = soften<T, DP, ES>(a, sh, tmem, warp / 4, warp % 4, lane);
        } else if (warp < kSoftWarps + kCopyWarps) {
            ok = copy_tiles<T, DP, ES>(a, sh, q_smem, ring, held, threadIdx.x - 32 * kSoftWarps, bad);
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == kLookWarp) {
            if (a.paged16) ok = look_up<DP, ES>(a, sh, lane, bad);
        } else {
            if (elected()) {
                ok = multiply<T, DP, ES>(a, sh, q_smem, ring, tmem, warp - kMmaWarp);
                mma_commit(&sh.drained);  // no instruction outlives its operands
                if (!mbar_wait(&sh.drained, 0)) ok = false;
            }
            __syncwarp();
        }
    }
    if (!ok) bad |= KVX_S_TIMEOUT;
    raise(a.status, bad);
    tmem_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Launches one variant on a.grid blocks; false where that failed.
template <class T, int DP, int ES>
bool launch_kernel(const Args &a, cudaStream_t s) {
    using S = Shape<DP, ES>;
    static bool done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        if (cudaFuncSetAttribute(k_shared<T, DP, ES>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<DP, ES>) != cudaSuccess)
            return false;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    k_shared<T, DP, ES><<<a.grid, kThreads, kSmem<DP, ES>, s>>>(a);
    return true;
}

template <class T, int ES>
bool launch(const Args &a, cudaStream_t s) {
    return a.c.dim <= 64 ? launch_kernel<T, 64, ES>(a, s) : a.c.dim <= 128 ? launch_kernel<T, 128, ES>(a, s)
                                                                            : launch_kernel<T, 256, ES>(a, s);
}

}  // namespace shared
}  // namespace kvx
