"""Argument checks of the cache operators: they return before any CUDA call, so they run without a GPU.  Pointers are
dummy addresses that are never dereferenced."""
import math
import os
import subprocess

import pytest
import torch

from conftest import ROOT
from paged_kv_cache_kvx_gb300 import kvx

OK, EINVAL = 0, 1
P = 0x1000


def cache(**kw):
    c = dict(pool=P, pool_bytes=1 << 30, addr=P, B=100, L=64, first_lane=16, heads=8, dim=128, dtype=kvx.KVX_BF16,
             page_tokens=16, reserved=0, token_stride=256, k_scale=1.0, v_scale=1.0)
    return kvx.CacheStruct(**(c | kw))


BAD_CACHES = [dict(pool=None), dict(pool=P + 8), dict(addr=None), dict(B=0), dict(first_lane=49), dict(first_lane=65),
              dict(first_lane=2 ** 32 - 1), dict(heads=0), dict(heads=25), dict(dim=0), dict(dim=72), dict(dim=272),
              dict(dtype=0), dict(dtype=4), dict(page_tokens=0), dict(page_tokens=2 ** 31), dict(reserved=1),
              dict(token_stride=240), dict(token_stride=264), dict(token_stride=0), dict(k_scale=0.0),
              dict(dtype=kvx.KVX_E4M3, k_scale=-1.0), dict(v_scale=math.nan), dict(dtype=kvx.KVX_E4M3, v_scale=math.inf),
              dict(k_scale=2.0), dict(v_scale=0.5)]


def append(c=None, **kw):
    a = dict(cache=c if c is not None else cache(), q=P, qs=4096, k=P, ks=1024, v=P, vs=1024, dtype=kvx.KVX_BF16, T=0, hq=32,
             wq=P, wk=P, eps=1e-6, cs=P, rot=128, mp=1000, il=0, pos=P, slots=P, out=P, os=4096, status=P, stream=None)
    a |= kw
    a["cache"] = kvx.ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return kvx.lib().kvx_append_tokens(*a.values())


def attend(c=None, **kw):
    a = dict(cache=c if c is not None else cache(), q=P, qs=4096, dtype=kvx.KVX_BF16, n=0, hq=32, blocks=P, per=100, lens=P,
             scale=0.1, window=0, sinks=0, out=P, os=4096, lse=None, scores=None, ss=0, status=P, ws=P, wsb=1 << 40,
             stream=None)
    a |= kw
    a["cache"] = kvx.ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return kvx.lib().kvx_attend(*a.values())


def evict(c=None, **kw):
    a = dict(cache=c if c is not None else cache(), n=0, blocks=P, per=100, lens=P, scores=P, ss=1600, budget=160, sinks=4,
             recent=16, dst=P, dper=10, kept=P, ksc=P, nl=P, status=P, ws=P, wsb=1 << 40, stream=None)
    a |= kw
    a["cache"] = kvx.ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return kvx.lib().kvx_evict(*a.values())


def test_nothing_to_do_is_accepted():
    assert append() == OK and attend() == OK and evict() == OK


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    c = cache(**bad)
    assert append(c) == EINVAL and attend(c) == EINVAL and evict(c) == EINVAL
    assert kvx.kvx_attend_workspace_size(c, 4, 32, 100) == 0 and kvx.kvx_evict_workspace_size(c, 4, 100, 10) == 0


@pytest.mark.parametrize("bad", [dict(dtype=kvx.KVX_F32), dict(dtype=kvx.KVX_E4M3), dict(dtype=kvx.KVX_F16), dict(status=None),
                                 dict(rot=8), dict(rot=144), dict(cs=None), dict(pos=None), dict(mp=0), dict(eps=-1.0),
                                 dict(eps=math.nan), dict(qs=4100), dict(ks=1), dict(vs=4), dict(os=12), dict(q=P + 2),
                                 dict(k=P + 8), dict(v=P + 8), dict(out=P + 8), dict(wq=P + 8), dict(wk=P + 4), dict(cs=P + 4),
                                 dict(T=1, k=None), dict(T=1, v=None), dict(T=1, slots=None), dict(T=1, q=None),
                                 dict(T=1, out=None), dict(T=2 ** 31), dict(hq=70000)], ids=str)
def test_append_refuses(bad):
    assert append(**bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(dtype=kvx.KVX_F32), dict(dtype=kvx.KVX_F16), dict(status=None), dict(hq=0), dict(hq=31),
                                 dict(hq=8 * 129), dict(per=2 ** 27), dict(scale=math.nan), dict(scale=math.inf), dict(qs=4),
                                 dict(os=4), dict(q=P + 8), dict(out=P + 8), dict(scores=P, ss=1599), dict(n=1, q=None),
                                 dict(n=1, out=None), dict(n=1, lens=None), dict(n=1, blocks=None), dict(n=1, ws=None),
                                 dict(n=1, wsb=0), dict(n=2 ** 24)], ids=str)
def test_attend_refuses(bad):
    assert attend(**bad) == EINVAL


@pytest.mark.parametrize("ws", [P + 1, P + 4, P + 8])
def test_attend_refuses_an_unaligned_workspace(ws):
    """It is cut into arrays of 16-byte vectors."""
    assert attend(n=1, ws=ws) == EINVAL


def test_attend_workspace_is_checked_to_the_byte():
    c = cache()
    for scores in (0, 1):
        need = kvx.kvx_attend_workspace_size(c, 4, 32, 100, 0, 0, scores)
        assert need > 0
        assert attend(c, n=4, wsb=need - 1, scores=P if scores else None, ss=1600) == EINVAL
    # a window bounds the logits that are kept
    assert kvx.kvx_attend_workspace_size(c, 4, 32, 10000, 256, 4, True) < kvx.kvx_attend_workspace_size(c, 4, 32, 10000, 0, 0, True)


@pytest.mark.parametrize("bad", [dict(status=None), dict(budget=0), dict(budget=2 ** 31), dict(ss=1599), dict(dper=9),
                                 dict(per=2 ** 27), dict(n=1, blocks=None), dict(n=1, lens=None), dict(n=1, scores=None),
                                 dict(n=1, dst=None), dict(n=1, kept=None), dict(n=1, ksc=None), dict(n=1, nl=None),
                                 dict(n=1, ws=None), dict(n=1, wsb=0)], ids=str)
def test_evict_refuses(bad):
    assert evict(**bad) == EINVAL


def test_null_cache():
    L = kvx.lib()
    assert L.kvx_attend_workspace_size(None, 4, 32, 100, 0, 0, 0) == 0
    assert L.kvx_evict_workspace_size(None, 4, 100, 10) == 0


def test_struct_matches_the_header():
    src = open(os.path.join(ROOT, "include", "kvx.h")).read()
    body = src[src.index("typedef struct kvx_cache {"):src.index("} kvx_cache;")]
    at = [body.index(f) for f in ("pool;", "pool_bytes", "addr;", "B, L", "first_lane", "heads", "dim;", "dtype", "page_tokens",
                                  "reserved", "token_stride", "k_scale", "v_scale")]
    assert at == sorted(at)


def test_cache_checks_its_tensors():
    pool, addr = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.int64)
    make = lambda p=pool, a=addr, dt=torch.bfloat16: kvx.Cache(p, a, heads=2, dim=64, dtype=dt, page_tokens=4)  # noqa: E731
    c = make()
    for bad in (dict(p=pool.float()), dict(a=addr.int()), dict(a=addr[:, ::2]), dict(a=addr[0]), dict(dt=torch.float32)):
        with pytest.raises(kvx.KvxError):
            make(**bad)
    T = 3
    q, k = torch.zeros(T, 4, 64, dtype=torch.bfloat16), torch.zeros(T, 2, 64, dtype=torch.bfloat16)
    slots, pos = torch.zeros(T, dtype=torch.int64), torch.zeros(T, dtype=torch.int32)
    table = torch.zeros(8, 64)
    ok = dict(q=q, k=k, v=k, positions=pos, slots=slots, q_out=q, cos_sin=table)
    for bad in (dict(q=q.float()), dict(k=k[:2]), dict(v=k.half()), dict(k=k.transpose(1, 2)), dict(slots=slots.int()),
                dict(positions=pos.long()), dict(q_out=q[:2]), dict(cos_sin=table.double()), dict(q_weight=torch.ones(64)),
                dict(k_weight=torch.ones(32, dtype=torch.bfloat16)), dict(q=torch.zeros(T, 4, 128, dtype=torch.bfloat16)),
                dict(q=torch.zeros(T, 8, 64, dtype=torch.bfloat16)[:, ::2])):
        with pytest.raises(kvx.KvxError):
            c.append(**(ok | bad))
    blocks, lens = torch.zeros(T, 5, dtype=torch.int32), torch.zeros(T, dtype=torch.int32)
    ws = torch.empty(8, dtype=torch.uint8)
    ok = dict(q=q, blocks=blocks, lens=lens, out=q, ws=ws)
    for bad in (dict(out=q[:2]), dict(blocks=blocks.long()), dict(lens=lens[:2]), dict(blocks=blocks[0]),
                dict(lse=torch.zeros(T, 3)), dict(scores=torch.zeros(T, 4, 20)), dict(blocks=blocks.t().contiguous())):
        with pytest.raises(kvx.KvxError):
            c.attend(**(ok | bad))
    with pytest.raises(kvx.KvxError):
        c.attend_workspace(4, 5, 100)
    with pytest.raises(kvx.KvxError):
        c.evict_workspace(4, 100, 0)
    kept, ksc, nl = torch.zeros(T, 2, 8, dtype=torch.int32), torch.zeros(T, 2, 8), torch.zeros(T, dtype=torch.int32)
    ok = dict(blocks=blocks, lens=lens, scores=torch.zeros(T, 2, 20), dst_blocks=blocks, kept=kept, kept_scores=ksc,
              new_lens=nl, ws=ws)
    for bad in (dict(scores=torch.zeros(T, 3, 20)), dict(kept=kept[:, :1]), dict(kept_scores=ksc[..., :7]), dict(new_lens=nl.long()),
                dict(dst_blocks=blocks[:2]), dict(kept=kept[0])):
        with pytest.raises(kvx.KvxError):
            c.evict(**(ok | bad))


def call_args(dev):
    """Valid arguments of the three calls, on a device, and the cache's own."""
    T, D = 3, 64
    pool, addr = torch.zeros(1 << 16, dtype=torch.uint8, device=dev), torch.zeros(4, 4, dtype=torch.int64, device=dev)
    q, k = torch.zeros(T, 4, D, dtype=torch.bfloat16, device=dev), torch.zeros(T, 2, D, dtype=torch.bfloat16, device=dev)
    ids = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    z = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    append = dict(q=q, k=k, v=k.clone(), positions=ids(T), slots=ids(T).long() - 1, q_out=q.clone(), cos_sin=z(8, D),
                  q_weight=q[0, 0].clone(), k_weight=q[0, 0].clone())
    attend = dict(q=q, blocks=ids(T, 5), lens=ids(T), out=q.clone(), ws=ws, lse=z(T, 4), scores=z(T, 2, 20))
    evict = dict(blocks=ids(T, 5), lens=ids(T), scores=z(T, 2, 20), dst_blocks=ids(T, 5), kept=ids(T, 2, 8),
                 kept_scores=z(T, 2, 8), new_lens=ids(T), ws=ws)
    return pool, addr, dict(append=append, attend=attend, evict=evict)


def make_cache(pool, addr):
    return kvx.Cache(pool, addr, heads=2, dim=64, dtype=torch.bfloat16, page_tokens=4)


def test_cache_wants_a_gpu():
    """Valid arguments in host memory are refused by the binding, before the library sees their pointers."""
    pool, addr, calls = call_args("cpu")
    c, before = make_cache(pool, addr), kvx.kvx_launch_count()
    for name, args in calls.items():
        with pytest.raises(kvx.KvxError, match="on a GPU"):
            getattr(c, name)(**args)
    assert kvx.kvx_launch_count() == before


def test_cache_refuses_tensors_of_another_device():
    """A cache whose pool is on another device than the call's tensors: each is named."""
    pool, addr, calls = call_args("cpu")
    c = make_cache(pool, addr)
    c._device = 0  # as if the pool were on the first GPU
    for name, first in (("append", "q"), ("attend", "lse"), ("evict", "blocks")):
        with pytest.raises(kvx.KvxError, match=r"^%s: .*on cuda:0" % first):
            getattr(c, name)(**calls[name])


@pytest.mark.parametrize("name", ["attend", "evict"])
def test_cache_checks_its_workspace(name):
    pool, addr, calls = call_args("cpu")
    c, ws = make_cache(pool, addr), calls[name]["ws"]
    for bad in (ws.view(torch.float32), ws[::2], ws.view(torch.int8)):
        with pytest.raises(kvx.KvxError, match="^ws: "):
            getattr(c, name)(**(calls[name] | dict(ws=bad)))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["append", "attend", "evict"])
def test_cache_refuses_each_host_tensor(name):
    pool, addr, calls = call_args("cuda")
    c, args = make_cache(pool, addr), calls[name]
    getattr(c, name)(**args)
    before = kvx.kvx_launch_count()
    for arg, t in args.items():
        with pytest.raises(kvx.KvxError, match="^%s: .*on cuda:0" % arg):
            getattr(c, name)(**(args | {arg: t.cpu()}))
    with pytest.raises(kvx.KvxError, match="^addr: "):
        make_cache(pool, addr.cpu())
    assert kvx.kvx_launch_count() == before
    torch.cuda.synchronize()
    assert c.read_status() == 0


HOST_CHECK = r"""
#include <cstdio>
#include <random>
#include "kvx_cache.cuh"
using namespace kvx;
#define NEED(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
    std::mt19937_64 r(1);
    for (int i = 0; i < 200000; i++) {
        uint32_t d = 1 + (uint32_t)(r() >> (33 + r() % 31)), n = (uint32_t)(r() >> (33 + r() % 31));
        if (i < 4096) d = 1 + i % 64, n = i / 64;
        if (i % 7 == 0) n = (uint32_t)((uint64_t)(n / d) * d), n -= n > 0 && i % 2;
        if (d >= (1u << 31)) d = (1u << 31) - 1;
        NEED(FastDiv(d).div(n) == n / d);
        NEED(FastDiv(d).div(0x7FFFFFFFu) == 0x7FFFFFFFu / d);
    }
    kvx_cache c = {(uint8_t *)0x1000, 10000, (const uint64_t *)0x1000, 4, 4, 0, 2, 64, KVX_BF16, 16, 0, 256, 1, 1};
    NEED(cache_ok(&c));
    CacheView v = cache_view(&c);
    NEED(v.span == 15 * 256 + 128 && v.row_bytes == 128);
    uint32_t bad = 0;
    NEED(v.ok(0, bad) && v.ok(10000 - v.span - (10000 - v.span) % 16, bad) && bad == 0);
    NEED(!v.ok(10000 - v.span + 16 - (10000 - v.span) % 16, bad) && bad == KVX_S_BOUNDS);
    bad = 0;
    NEED(!v.ok(8, bad) && bad == KVX_S_ALIGN);
    bad = 0;
    for (uint64_t a : {10000ull / 16 * 16 + 16, 1ull << 40, ~0ull - 15, (~0ull - 15) - 16 * 300}) {
        bad = 0;
        NEED(!v.ok(a, bad) && bad == KVX_S_BOUNDS);
    }
    c.pool_bytes = 100;  // smaller than a segment
    v = cache_view(&c);
    bad = 0;
    NEED(!v.ok(0, bad) && bad == KVX_S_BOUNDS);
    puts("ok");
}
"""


def test_address_arithmetic_on_the_host(tmp_path):
    """The segment check and the exact division that every kernel indexes with."""
    from paged_kv_cache_kvx_gb300 import build
    src = tmp_path / "host_check.cu"
    src.write_text(HOST_CHECK)
    exe = tmp_path / "host_check"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I" + os.path.join(ROOT, "include"), "-I" + build.CSRC,
                    "-o", str(exe), str(src)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stdout


JOIN_CHECK = r"""
#include <cstdio>
#include <random>
#include "kvx_attend.cuh"
using namespace kvx;
using namespace kvx::attend;
#define NEED(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
    std::mt19937_64 r(1);
    const uint32_t seqs = 5, units = 8, grid = 456;
    NEED(joinable(make_uint4(4, 7, 455, 911), 0, seqs, units, grid));
    NEED(joinable(make_uint4(0, 0, 8, 14), 7, seqs, units, grid));
    // what a workspace holds before its first use, and what a call with other sizes leaves there
    NEED(!joinable(make_uint4(kNone, 0, 8, 14), 7, seqs, units, grid));
    NEED(!joinable(make_uint4(kNone, kNone, kNone, kNone), 7, seqs, units, grid));
    NEED(!joinable(make_uint4(0, 0, 0, 0), 7, seqs, units, grid));
    NEED(!joinable(make_uint4(5, 0, 8, 14), 7, seqs, units, grid));
    NEED(!joinable(make_uint4(0, 8, 8, 14), 7, seqs, units, grid));
    NEED(!joinable(make_uint4(0, 0, 456, 14), 7, seqs, units, grid));
    NEED(!joinable(make_uint4(0, 0, 8, 912), 7, seqs, units, grid));
    for (int i = 0; i < 1000000; i++) {
        const uint32_t block = r() % grid;
        uint32_t w[4];
        for (uint32_t &x : w) x = (uint32_t)(r() >> (32 + r() % 32));
        const uint4 cut = make_uint4(w[0], w[1], w[2], w[3]);
        if (!joinable(cut, block, seqs, units, grid)) continue;
        const uint64_t parts = (uint64_t)cut.z - block + 1;
        NEED(cut.x < seqs && cut.y < units && parts <= grid - block && cut.w < 2 * grid && 2 * (block + parts - 1) < 2 * grid);
    }
    puts("ok");
}
"""


def test_join_entries_are_checked_on_the_host(tmp_path):
    """The entries by which a cut unit's parts are joined are indexed with only where they name parts that exist."""
    from paged_kv_cache_kvx_gb300 import build
    src = tmp_path / "join_check.cu"
    src.write_text(JOIN_CHECK)
    exe = tmp_path / "join_check"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-I" + os.path.join(ROOT, "include"), "-I" + build.CSRC,
                    "-o", str(exe), str(src)], check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.stdout.strip() == "ok", out.stdout
