"""Row-scaled caches through a transfer: the scales lie in their segments, so a receiver has them with the rows."""
import numpy as np
import pytest
import torch

from paged_kv_cache_kvx_gb300 import kvx, workloads as W

pytestmark = pytest.mark.gpu
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.mark.parametrize("act,dim,page,layers,heads,seg", [
    (BF, 128, 16, 2, 3, 16 * 128 + 16),
    (FP, 64, 24, 1, 2, 24 * 64 + 32),          # 24 scales in 32 bytes
    (BF, 96, 256, 2, 1, 256 * 96 + 256),
    (BF, 128, 1, 1, 4, 128 + 16 + 32),         # a gap behind the scale
])
def test_quantised_prefix_is_transferred(act, dim, page, layers, heads, seg):
    """A prompt quantised at the holder, packed, and (a) unpacked into a pool of the holder's layout, (b) sealed into pages of
    the receiver's own: read back and attended over, each gives the holder's bits."""
    blocks, group, seqs = 23, 4, 5
    tokens = blocks * page - page // 2
    wl = W.bump("prompt", blocks, layers * heads, seg, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(dim)
    holder = torch.zeros(wl.pool_bytes, dtype=torch.uint8, device="cuda")
    table = torch.from_numpy(wl.addr.astype(np.int64)).cuda()

    def caches(pool, addr):
        return [kvx.Cache(pool, addr, heads, dim, E4, page, first_lane=2 * heads * i, scale_offset=page * dim) for i in range(layers)]

    for cache in caches(holder, table):
        q, k, v = (torch.randn(tokens, n, dim, generator=gen, device="cuda") for n in (heads * group, heads, heads))
        size = torch.randn(tokens, 1, 1, generator=gen, device="cuda").exp()  # rows of different size
        q, k, v = (x.to(act) for x in (q, k * size, v * size))
        cache.append(q, k, v, None, torch.arange(tokens, device="cuda"), torch.empty_like(q))
        assert cache.read_status() == 0

    tr = kvx.Transfer(wl.blocks, wl.seg_len, wl.numa, wl.pool_bytes)
    tr.set_addr(wl.addr)
    slab = torch.empty(tr.slab_bytes, dtype=torch.uint8, device="cuda")
    tr.encode()
    tr.plan()
    tr.pack(holder, slab)
    same = torch.full((wl.pool_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
    tr.unpack(slab, same)
    # the receiver's pages: as many more, shuffled, segments 48 bytes apart
    place = np.random.default_rng(4).permutation(2 * blocks).astype(np.int64)[:blocks]
    own = torch.from_numpy(place[:, None] * (wl.lanes * (seg + 48)) + 16 + np.arange(wl.lanes) * (seg + 48)).cuda()
    pool = torch.full((2 * blocks * wl.lanes * (seg + 48) + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    tr.seal(slab, own, pool)
    torch.cuda.synchronize()
    assert tr.read_status() == 0

    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ids = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    q = torch.randn(seqs, heads * group, dim, generator=gen, device="cuda").to(act)

    def results(cache):
        k, v = (torch.empty(tokens, heads, dim, dtype=act, device="cuda") for _ in range(2))
        cache.read(ids, i(0, tokens), k, v)
        out, lse = torch.empty_like(q), torch.empty(seqs, heads * group, device="cuda")
        cache.attend_shared(q, ids, i(tokens), i(0, seqs), ids[:, :0].expand(seqs, 0), i(*[0] * seqs), out,
                            cache.attend_shared_workspace(seqs, heads * group, 0, 1, blocks), lse=lse)
        assert cache.read_status() == 0
        return k, v, out, lse

    for at_holder, unpacked, sealed in zip(caches(holder, table), caches(same, table), caches(pool, own)):
        want = results(at_holder)
        assert all(torch.isfinite(x).all() for x in want) and want[0].float().std() > 0.5
        for cache in (unpacked, sealed):
            for x, y in zip(want, results(cache)):
                assert torch.equal(x, y)
