"""Argument checks of row-scaled caches, kvx_read_tokens and kvx_attend_shared: they return before any CUDA call, so they run
without a GPU.  Pointers are dummy addresses that are never dereferenced."""
import math
import os
import subprocess

import pytest
import torch

from conftest import ROOT
from paged_kv_cache_kvx_gb300 import kvx
from test_cache_args import BAD_CACHES, EINVAL, OK, P, append, attend, cache, evict


def rows_cache(**kw):
    """A cache of 8-bit rows of 128 with scales behind them: 16 tokens a page."""
    return cache(**(dict(dtype=kvx.KVX_E4M3, token_stride=128, reserved=16 * 128) | kw))


def read(c=None, **kw):
    a = dict(cache=c if c is not None else cache(), blocks=P, n=1, per=100, first=P, starts=P, T=0, dtype=kvx.KVX_BF16, k=P,
             ks=1024, v=P, vs=1024, status=P, stream=None)
    a |= kw
    a["cache"] = kvx.ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return kvx.lib().kvx_read_tokens(*a.values())


def shared(c=None, **kw):
    a = dict(cache=c if c is not None else cache(), q=P, qs=4096, dtype=kvx.KVX_BF16, n=0, hq=32, pblocks=P, pper=100, plens=P,
             first=P, groups=4, blocks=P, per=100, lens=P, scale=0.1, out=P, os=4096, lse=None, status=P, ws=P, wsb=1 << 40,
             stream=None)
    a |= kw
    a["cache"] = kvx.ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return kvx.lib().kvx_attend_shared(*a.values())


def size(c, n=4, hq=32, per=100, groups=2, pper=50):
    return kvx.kvx_attend_shared_workspace_size(c, n, hq, per, groups, pper)


def test_nothing_to_do_is_accepted():
    for c in (cache(), rows_cache()):
        assert append(c) == OK and read(c) == OK and read(c, n=0, T=5) == OK and shared(c) == OK
    assert read(first=None) == OK and shared(groups=0, pblocks=None, plens=None, first=None, pper=0) == OK
    assert shared(rows_cache(), dtype=kvx.KVX_F16) == OK and read(rows_cache(), dtype=kvx.KVX_F16) == OK


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    c = cache(**bad)
    assert read(c) == EINVAL and shared(c) == EINVAL and size(c) == 0


@pytest.mark.parametrize("bad", [dict(reserved=16 * 128 - 16), dict(reserved=8), dict(reserved=16 * 128 + 8), dict(k_scale=2.0),
                                 dict(v_scale=0.5), dict(token_stride=256), dict(dtype=kvx.KVX_BF16, token_stride=256),
                                 dict(dtype=kvx.KVX_F16, reserved=16 * 256, token_stride=256), dict(page_tokens=17)], ids=str)
def test_bad_row_scales(bad):
    c = rows_cache(**bad)
    assert append(c) == EINVAL and read(c) == EINVAL and shared(c) == EINVAL and size(c) == 0


def test_row_scales_behind_the_rows():
    for ok in (dict(), dict(reserved=16 * 128 + 16), dict(reserved=2 ** 32 - 16), dict(token_stride=1024, reserved=16 * 1024),
               dict(token_stride=1024, reserved=15 * 1024 + 128), dict(page_tokens=1, reserved=128)):
        c = rows_cache(**ok)
        assert append(c) == OK and read(c) == OK and shared(c) == OK and size(c) > 0
    # the operators that take no row scales
    c = rows_cache()
    assert attend(c) == EINVAL and evict(c) == EINVAL
    assert kvx.kvx_attend_workspace_size(c, 4, 32, 100) == 0 and kvx.kvx_evict_workspace_size(c, 4, 100, 10) == 0


@pytest.mark.parametrize("bad", [dict(status=None), dict(dtype=kvx.KVX_F32), dict(dtype=kvx.KVX_E4M3), dict(dtype=kvx.KVX_F16),
                                 dict(T=2 ** 31), dict(n=2 ** 31), dict(per=2 ** 27), dict(ks=1028), dict(vs=4), dict(k=P + 8),
                                 dict(v=P + 2), dict(T=1, k=None), dict(T=1, v=None), dict(T=1, starts=None), dict(T=1, blocks=None),
                                 dict(cache=None)], ids=str)
def test_read_refuses(bad):
    assert read(**bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(status=None), dict(dtype=kvx.KVX_F32), dict(dtype=kvx.KVX_E4M3), dict(dtype=kvx.KVX_F16),
                                 dict(hq=0), dict(hq=33), dict(hq=8 * 129), dict(per=2 ** 27), dict(pper=2 ** 27),
                                 dict(n=2 ** 30), dict(groups=2 ** 30), dict(n=2 ** 26, hq=64), dict(scale=math.nan),
                                 dict(scale=math.inf), dict(scale=-math.inf), dict(qs=4092), dict(os=4100), dict(q=P + 8),
                                 dict(out=P + 2), dict(n=1, q=None), dict(n=1, out=None), dict(n=1, lens=None), dict(n=1, blocks=None),
                                 dict(n=1, pblocks=None), dict(n=1, plens=None), dict(n=1, first=None), dict(n=1, ws=None),
                                 dict(n=1, ws=P + 8), dict(n=1, wsb=0), dict(n=1, wsb="less"), dict(cache=None)], ids=str)
def test_attend_shared_refuses(bad):
    if bad.get("wsb") == "less":
        bad = dict(n=1, wsb=size(cache(), 1, 32, 100, 4, 100) - 1)
    assert shared(**bad) == EINVAL


def test_workspace_sizes():
    assert kvx.lib().kvx_attend_shared_workspace_size(None, 4, 32, 100, 1, 100) == 0
    base = size(cache())
    assert 0 < base < 1 << 30
    assert size(cache(), n=400) > base and size(cache(), groups=40) > base
    assert size(cache(), n=0, groups=0, pper=0, per=0) > 0
    # it grows with the sequences and groups, not with their lengths
    assert size(cache(), per=100_000) - base < 64 << 20
    for refused in (dict(hq=7), dict(hq=0), dict(n=2 ** 30), dict(groups=2 ** 30), dict(per=2 ** 27), dict(n=2 ** 20, per=2 ** 20)):
        assert size(cache(), **refused) == 0


def call_args(dev):
    T, D = 3, 64
    q, k = torch.zeros(T, 4, D, dtype=torch.bfloat16, device=dev), torch.zeros(T, 2, D, dtype=torch.bfloat16, device=dev)
    ids = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    # (a workspace of whatever size a device wants)
    attend_shared = dict(q=q, prefix_blocks=ids(2, 5), prefix_lens=ids(2), group_first=ids(3), blocks=ids(T, 5), lens=ids(T),
                         out=q.clone(), ws=torch.empty(1 << 24, dtype=torch.uint8, device=dev), lse=torch.zeros(T, 4, device=dev))
    read = dict(blocks=ids(T, 5), starts=ids(T + 1), k_out=k, v_out=k.clone(), first=ids(T))
    return dict(attend_shared=attend_shared, read=read)


def make_cache(dev):
    pool, addr = torch.zeros(1 << 16, dtype=torch.uint8, device=dev), torch.zeros(4, 4, dtype=torch.int64, device=dev)
    return kvx.Cache(pool, addr, heads=2, dim=64, dtype=torch.bfloat16, page_tokens=4)


@pytest.mark.parametrize("name", ["attend_shared", "read"])
def test_binding_checks_its_tensors(name):
    c, ok = make_cache("cpu"), call_args("cpu")[name]
    with pytest.raises(kvx.KvxError, match="on a GPU"):
        getattr(c, name)(**ok)
    for arg, t in ok.items():
        wrong = [t.double()] + ([t[:, :1]] if t.dim() > 1 else [t[:-1]] if arg != "ws" else [t[::2]])
        for x in wrong:
            # (another number of pages, or of rows to read into, is not a mistake by itself)
            if (arg, x.dtype) in (("blocks", torch.int32), ("prefix_blocks", torch.int32)):
                continue
            with pytest.raises(kvx.KvxError):
                getattr(c, name)(**(ok | {arg: x}))
    c._device = 0  # as if the pool were on the first GPU
    with pytest.raises(kvx.KvxError, match="on cuda:0"):
        getattr(c, name)(**ok)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["attend_shared", "read"])
def test_binding_refuses_each_host_tensor(name):
    c, args = make_cache("cuda"), call_args("cuda")[name]
    getattr(c, name)(**args)
    before = kvx.kvx_launch_count()
    for arg, t in args.items():
        with pytest.raises(kvx.KvxError, match="^%s: .*on cuda:0" % arg):
            getattr(c, name)(**(args | {arg: t.cpu()}))
    assert kvx.kvx_launch_count() == before
    torch.cuda.synchronize()
    assert c.read_status() == 0


def test_python_struct_has_the_scales_place():
    c = kvx.Cache(torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.int64), heads=2, dim=64,
                  dtype=torch.float8_e4m3fn, page_tokens=16, scale_offset=1024)
    assert c.c.reserved == 1024 and append(c.c, cs=None, rot=0) in (OK, EINVAL)
    src = open(os.path.join(ROOT, "include", "kvx.h")).read()
    body = src[src.index("typedef struct kvx_cache {"):src.index("} kvx_cache;")]
    assert body.index("page_tokens;") < body.index("scale_offset;") < body.index("token_stride;")


SCHEDULE_CHECK = r"""
#include <cstdio>
#include <random>
#include <set>
#include "kvx_shared.cuh"
using namespace kvx;
using namespace kvx::shared;
#define NEED(x) do { if (!(x)) { printf("line %d: %s (round %d)\n", __LINE__, #x, round); return 1; } } while (0)
// Goes through groups' columns as the kernel's blocks do: every tile of every row is done once, parts have numbers of their
// own below their bound, and a row's parts of a head are where the join looks for them.
int main() {
    std::mt19937 r(7);
    for (int round = 0; round < 3000; round++) {
        Args a = {};
        a.c.heads = 1 + r() % 9;
        a.group = 1 + r() % 16;
        a.tile_rows = r() % 2 ? 256 : 128;
        const uint32_t keys = a.tile_rows == 256 ? 128 : 64, groups = 1 + r() % 5, grid = 1 + r() % 152;
        std::vector<Entry> e(groups);
        uint32_t seqs = 0;
        uint64_t total = 0;
        for (auto &x : e) {
            const uint32_t n = r() % 4 ? r() % 200 : r() % 3;
            x.seq0 = seqs, seqs += n;
            x.rows = n * a.group;
            x.len = x.rows ? (r() % 5 ? r() % 5000 : r() % 100) : 0;
        }
        a.num_seqs = seqs;
        for (auto &x : e) { const Region g = region_of(a, x, 1, keys); total += (uint64_t)g.width * g.rows; }
        uint32_t share = (uint32_t)((total + grid - 1) / grid);
        if (share < kMinShare) share = kMinShare;
        std::set<uint64_t> numbers;
        uint64_t start = 0, bound = (uint64_t)((uint64_t)seqs * a.group / a.tile_rows + groups) * (a.c.heads + 2) + 2 * grid;
        int64_t last = -1;
        for (uint32_t i = 0; i < groups; i++) {
            const Region g = region_of(a, e[i], share, keys);
            const uint64_t size = (uint64_t)g.width * g.rows;
            std::vector<uint32_t> seen(size, 0);
            for (uint64_t off = 0; off < size;) {
                const uint64_t at = start + off, c = at / share;
                const uint32_t b = quotient_host(off, (uint64_t)g.block * g.rows), in_block = off - (uint64_t)b * g.block * g.rows;
                const uint32_t columns = g.columns(b), row = in_block / columns, column = b * g.block + in_block % columns;
                const uint32_t head = column / g.len;
                uint64_t n = columns - in_block % columns;
                if (n > (uint64_t)(head + 1) * g.len - column) n = (uint64_t)(head + 1) * g.len - column;
                if (n > (c + 1) * share - at) n = (c + 1) * share - at;
                NEED(n > 0 && c < grid && row < g.rows && head < a.c.heads);
                for (uint64_t k = 0; k < n; k++) NEED(++seen[(uint64_t)row * g.width + column + k] == 1);
                if (column + n > head * g.len + kExtra) {
                    const uint64_t part = (uint64_t)group_parts(a, (uint32_t)start, share, e[i].seq0, i) + g.rank(b, row, head) + c;
                    NEED(part < bound && (int64_t)part > last && numbers.insert(part).second);
                    last = part;
                }
                off += n;
            }
            for (uint32_t x : seen) NEED(x == 1);
            start += size;
        }
    }
    puts("ok");
}
"""


def test_every_tile_is_done_once(tmp_path):
    """How prefixes' columns are shared out, and how their parts are numbered."""
    from paged_kv_cache_kvx_gb300 import build
    src = tmp_path / "schedule_check.cu"
    src.write_text("#include <cstdint>\n#include <vector>\nstatic inline uint32_t quotient_host(uint64_t a, uint64_t b) { return (uint32_t)(a / b); }\n"
                   + SCHEDULE_CHECK)
    exe = tmp_path / "schedule_check"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I" + os.path.join(ROOT, "include"), "-I" + build.CSRC,
                    "-o", str(exe), str(src)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stdout
