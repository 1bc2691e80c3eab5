"""kvx_attend_shared's schedule and its join against each other, on the host: the same functions that the kernels call."""
import os
import subprocess

from conftest import ROOT
from paged_kv_cache_kvx_gb300 import build

CHECK = r"""
#include <cstdio>
#include <map>
#include <random>
#include <unordered_map>
#include <vector>
#include "kvx_shared.cuh"
using namespace kvx;
using namespace kvx::shared;
#define NEED(x) do { if (!(x)) { printf("line %d: %s (round %d)\n", __LINE__, #x, round); return 1; } } while (0)

struct Row { uint32_t entry, head, query_row, keys; };  // of partial results: whose, and how many keys its piece has
struct Want { uint32_t rows, keys; };

// Goes through all blocks' shares as the walking warp does and writes down which rows of partial results the softmax
// warps write; then looks every query's parts up as the join does.  Each row is written once and lies in the workspace;
// the join finds those of its query, each once, and all of them; their keys are all keys there are.
int main() {
    std::mt19937 r(11);
    uint64_t queries = 0, found = 0;
    for (int round = 0; round < 1200; round++) {
        kvx_cache c = {};
        c.pool = (uint8_t *)16, c.addr = (const uint64_t *)16, c.B = 1, c.k_scale = c.v_scale = 1;
        c.dim = r() % 3 ? 16 * (1 + r() % 8) : 16 * (9 + r() % 8);
        c.heads = 1 + r() % 5, c.L = 2 * c.heads, c.dtype = KVX_BF16, c.token_stride = 2 * c.dim;
        c.page_tokens = 1 + r() % 40;
        const bool wide = c.dim > 128;
        const uint32_t group = r() % 8 ? 1 + r() % 16 : 1 + r() % 128, q_heads = group * c.heads;
        const uint32_t groups = r() % 4 ? r() % 6 : r() % 40, seqs = 1 + (r() % 3 ? r() % 40 : r() % 300);
        const uint32_t per = r() % 8 ? r() % 12 : r() % 200, pper = groups ? r() % 3 ? r() % 40 : r() % 300 : 0;
        const uint32_t sms = r() % 2 ? 152 : 1 + r() % 152;
        std::vector<uint32_t> first(groups + 1), plens(groups), lens(seqs);
        for (auto &x : first) x = r() % (seqs + 1);
        std::sort(first.begin(), first.end());
        for (auto &x : plens) x = r() % 4 ? r() % (pper * c.page_tokens + 1) : 0;
        for (auto &x : lens) x = r() % 3 ? r() % (per * c.page_tokens + 1) : r() % 2 ? 0 : per ? 1 : 0;
        Plan p;
        NEED(plan(&c, seqs, q_heads, per, groups, pper, sms, p));
        Args a = args_of(&c, seqs, q_heads, per, groups, pper, p);
        a.group_first = first.data(), a.prefix_lens = plens.data(), a.lens = lens.data();
        const uint32_t keys = keys_of(wide), entries = groups + seqs;
        std::vector<Entry> e(entries);
        uint64_t total = 0;
        for (uint32_t i = 0; i < entries; i++) {
            e[i] = entry_of(a, i);
            NEED(!e[i].disorder && !e[i].beyond);
            const Region g = region_of(a, e[i], 1, keys);
            total += (uint64_t)g.width * g.rows;
        }
        NEED(total < 1ull << 31);
        const uint32_t share = share_of(a, (uint32_t)total);
        NEED((uint64_t)share * p.grid >= total);
        std::vector<uint2> group_at(groups, make_uint2(0, 0)), own_at((size_t)seqs * c.heads, make_uint2(1, 0));
        std::unordered_map<uint64_t, Row> rows;
        std::map<std::vector<uint32_t>, Want> want;  // by entry, head, query row
        for (uint32_t block = 0; block < p.grid; block++) {
            uint64_t at = (uint64_t)block * share, end = at + share < total ? at + share : total;
            uint64_t before = 0;
            uint32_t i = 0;
            while (at < end) {
                const Region g = region_of(a, e[i], share, keys);
                const uint64_t size = (uint64_t)g.width * g.rows;
                if (at - before >= size) { before += size, i++; NEED(i < entries); continue; }
                const Cut k = cut(g, (uint32_t)(at - before), (uint32_t)(end - at));
                NEED(k.to > k.from && k.to <= g.len && k.row < g.rows && k.head < c.heads);
                at += k.to - k.from;
                if (k.to <= kExtra) continue;
                const uint32_t t0 = k.from > kExtra ? k.from - kExtra : 0, t1 = k.to - kExtra;
                const uint32_t k0 = t0 * g.keys, k1 = t1 * g.keys < e[i].len ? t1 * g.keys : e[i].len;
                NEED(k0 < k1);
                const uint32_t row0 = k.row * a.tile_rows, n = e[i].rows - row0 < a.tile_rows ? e[i].rows - row0 : a.tile_rows;
                const bool both = wide || n > kRows;
                uint32_t part, off_b;
                if (i < groups) {
                    part = prefix_row(a, g, k, (uint32_t)before, share, e[i].seq0, i, block), off_b = a.prefix_off_b;
                    group_at[i] = make_uint2((uint32_t)before, share);
                } else {
                    const uint32_t unit = e[i].seq0 * c.heads + k.head;
                    part = own_row(a, unit, block), off_b = a.own_off_b;
                    if (!t0) own_at[unit] = own_blocks(g, (uint32_t)before + k.head * g.len, share);
                }
                // The softmax warps' rows: a slot has 128, its own where both take every tile, else the same ones.  Of
                // heads wider than 128 both slots have the same rows, and half of each one's values.
                for (uint32_t slot = 0; slot < (wide ? 1 : 2); slot++)
                    for (uint32_t x = 0; x < kRows; x++) {
                        const uint32_t of_piece = (both && !wide ? slot * kRows : 0) + x;
                        if (of_piece >= n) continue;
                        const uint64_t row = (uint64_t)part + slot * off_b + x;
                        NEED(row < p.rows && (i < groups) == (row < p.own_first_row));
                        NEED(rows.emplace(row, Row{i, k.head, row0 + of_piece, k1 - k0}).second);
                        Want &w = want[{i, k.head, row0 + of_piece}];
                        w.rows++;
                        if (both || !slot) w.keys += k1 - k0;
                    }
            }
        }
        for (uint32_t n = 0; n < seqs; n++)
            for (uint32_t x = 0; x < q_heads; x++) {
                const uint32_t head = a.by_group.div(x), in = x - head * group;
                uint32_t g = groups;  // the last that starts here or before
                for (uint32_t k = 0; k < groups; k++)
                    if (first[k] <= n) g = k;
                queries++;
                uint64_t counted = 0;
                for (int own = 0; own < 2; own++) {
                    const uint32_t i = own ? groups + n : g;
                    if (!own && (g == groups || n - e[g].seq0 >= e[g].rows / group)) continue;
                    if (!e[i].len) continue;
                    const uint32_t query_row = own ? in : (n - e[i].seq0) * group + in;
                    const uint2 w = own ? own_at[n * c.heads + head] : group_at[g];
                    NEED(own ? w.x <= w.y && w.y < p.grid : w.y == share);
                    const Parts parts = own ? own_parts(a, w, n, head, in, wide) : prefix_parts(a, e[i], w, g, n, head, in, wide);
                    counted += parts.count();
                    uint32_t count = 0;
                    uint64_t last = 0;
                    for (uint32_t k = 0; k < parts.count(); k++) {
                        const uint32_t row = own ? parts.at_own(k) : parts.at(k);
                        if (row == kNone) continue;
                        const auto it = rows.find(row);
                        NEED(it != rows.end());
                        NEED(it->second.entry == i && it->second.head == head && it->second.query_row == query_row);
                        NEED(!count || row != last);
                        it->second.entry = kNone;  // taken
                        last = row, count++;
                    }
                    const Want all = want[{i, head, query_row}];
                    NEED(count == all.rows && all.keys == e[i].len);
                    found += count;
                }
                NEED(counted <= most_parts(a));
            }
        for (const auto &x : rows) NEED(x.second.entry == kNone);  // nothing that nobody looks for
    }
    printf("ok %llu queries %llu parts\n", (unsigned long long)queries, (unsigned long long)found);
}
"""


def compiled(tmp_path, csrc=build.CSRC):
    src = tmp_path / "join_check.cu"
    src.write_text("#include <algorithm>\n#include <cstdint>\n" + CHECK)
    exe = tmp_path / "join_check"
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-o", str(exe),
                    str(src)], check=True, capture_output=True, text=True)
    return exe


def test_the_join_finds_every_part(tmp_path):
    out = subprocess.run([str(compiled(tmp_path))], capture_output=True, text=True)
    assert out.stdout.startswith("ok "), out.stdout
