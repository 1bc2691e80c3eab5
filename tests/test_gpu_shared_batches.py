"""kvx_attend_shared over batches with free places: sequences and groups of no tokens between those that have some."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_kvx_gb300 import kvx
from test_gpu_shared import BF, FP, Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,store", [(BF, BF), (FP, "rows")])
@pytest.mark.parametrize("gap", [0, 1, 30, 31, 32, 33, 63, 64, 65, 200])
def test_free_places_between_sequences(act, store, gap):
    """Long and short sequences, `gap` free places before, between and behind them."""
    lens = [0] * gap
    for n in (300, 1, 70, 16, 900):
        lens += [n] + [0] * gap
    p = Problem(act, store, [0, 0], [50], lens, 4, 2, 64, 16)
    p.check(*p.run())


def test_free_places_among_groups():
    """Groups of no tokens, of no sequences, and sequences that see their group's tokens alone."""
    gen = np.random.default_rng(5)
    N, groups = 700, 330
    sizes = np.where(gen.random(groups) < 0.1, gen.integers(0, 30, groups), 0)
    firsts = np.minimum(np.cumsum(np.concatenate([[40], sizes])), N).tolist()
    prefixes = np.where(gen.random(groups) < 0.3, gen.integers(1, 200, groups), 0).tolist()
    lens = np.where(gen.random(N) < 0.05, gen.integers(1, 100, N), 0).tolist()
    p = Problem(BF, BF, firsts, prefixes, lens, 2, 2, 64, 16)
    p.check(*p.run())
    p = Problem(BF, "rows", [0, 0], [100], [0] * 500, 2, 2, 64, 16)  # nobody there at all
    out, lse = p.run()
    assert p.cache.read_status() == 0 and (out == 0).all() and (lse == -math.inf).all()


def test_millions_of_free_places():
    """Two sequences of one token at both ends of five million: nothing waits so long that it gives up."""
    N = 5_000_000
    pool = torch.ones(1 << 12, dtype=BF, device="cuda").view(torch.uint8)
    cache = kvx.Cache(pool, torch.zeros(4, 2, dtype=torch.int64, device="cuda"), heads=1, dim=16, dtype=BF, page_tokens=16)
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    lens[0] = lens[-1] = 1
    q, blocks = torch.ones(N, 1, 16, dtype=BF, device="cuda"), torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    cache.attend_shared(q, i().view(0, 0), i(), i(0), blocks, lens, out, cache.attend_shared_workspace(N, 1, 1, 0, 0))
    assert cache.read_status() == 0
    assert (out[0] == 1).all() and (out[-1] == 1).all() and not out[1:-1].any()


def test_lengths_to_the_end_of_31_bits():
    """A history of 2^31 - 2^20 - 5 tokens, one page again and again and another at its end: own, as a prefix, and read back.
    All logits are 0 but the last token's, 25; the one behind it, which nobody sees, would outweigh all."""
    page, per, dim = 1 << 20, 2047, 16
    length = per * page - 5
    kv = torch.zeros(2, 2, page, dim, dtype=BF, device="cuda")  # [block][K, V]
    kv[:, 1, 1::2, 3] = 1
    kv[1, :, page - 6, 0] = 25
    kv[1, :, page - 5, 0] = 100
    cache = kvx.Cache(kv.view(-1).view(torch.uint8), torch.arange(4, device="cuda").view(2, 2) * (2 * dim * page), heads=1, dim=dim, dtype=BF,
                      page_tokens=page)
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    table = i(*[0] * (per - 1), 1)[None]
    q, out, lse = torch.zeros(3, 2, dim, dtype=BF, device="cuda"), torch.empty(3, 2, dim, dtype=BF, device="cuda"), torch.empty(3, 2, device="cuda")
    q[:, :, 0] = 1
    for prefix in (False, True):
        if prefix:
            args = table, i(length), i(0, 3), table[:, :0].expand(3, 0), i(0, 0, 0), out, cache.attend_shared_workspace(3, 2, 0, 1, per)
        else:
            args = table[:0], i(), i(0), table.expand(3, per).contiguous(), i(*[length] * 3), out, cache.attend_shared_workspace(3, 2, per, 0, per)
        cache.attend_shared(q, *args, scale=1.0, lse=lse)
        assert cache.read_status() == 0
        total = math.exp(25) + (length - 1)
        # sums of a block's 220,000 tiles in 32 bits, and bf16's rounding of weights and outputs
        near = 250_000 * 2.0 ** -24 + 2.0 ** -7
        assert (lse - math.log(total)).abs().max() <= near
        assert (out[..., 0].double() - 25 * math.exp(25) / total).abs().max() <= 25 * near
        assert (out[..., 3].double() - (length // 2) / total).abs().max() <= near
        assert not out[..., 4:].any()
    k, v = torch.full((2, 9, 1, dim), 7.0, dtype=BF, device="cuda")
    cache.read(table, i(1, 8), k, v, first=i(length - 7))
    assert cache.read_status() == 0 and (k[[0, 8]] == 7).all() and (v[[0, 8]] == 7).all()
    for got, x in ((k, kv[1, 0]), (v, kv[1, 1])):
        assert torch.equal(got[1:8, 0], x[page - 12:page - 5])


@pytest.mark.parametrize("store", [BF, "rows"])
def test_read_in_a_graph_and_at_once(store):
    """Captured once and replayed with other tables; two streams at once into rows of their own of one tensor."""
    p = Problem(BF, store, [0, 0], [50], [40, 0, 100, 7], 4, 2, 64, 16)
    k, v = p.c.values()

    def want(x, lens, firsts):
        return torch.cat([x[p.blocks[n].long()[(torch.arange(m) + f) // 16], :, (torch.arange(m) + f) % 16] for n, (m, f) in enumerate(zip(lens, firsts))])

    i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    blocks, starts, first = p.blocks.cuda(), i([0, 40, 40, 140, 147]), i([0, 0, 0, 0])
    outs = [torch.zeros(160, 2, 64, dtype=BF, device="cuda") for _ in range(2)]
    p.cache.read(blocks, starts, *outs, first=first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.cache.read(blocks, starts, *outs, first=first)
    for lens, firsts in (([40, 0, 100, 7], [0, 0, 0, 0]), ([1, 0, 60, 7], [39, 5, 40, 0]), ([0, 0, 100, 0], [3, 0, 0, 0])):
        starts.copy_(torch.tensor([0, *lens]).cumsum(0).int())
        first.copy_(torch.tensor(firsts).int())
        for o in outs:
            o.fill_(5.0)
        g.replay()
        m = sum(lens)
        for o, x in zip(outs, (k, v)):
            assert torch.equal(o[:m].cpu(), want(x, lens, firsts).to(BF)) and (o[m:] == 5).all()
    streams = [torch.cuda.Stream() for _ in range(2)]
    halves = [i([0, 40, 40, 40, 40]), i([40, 40, 40, 140, 147])]
    torch.cuda.synchronize()
    for o in outs:
        o.fill_(5.0)
    torch.cuda.synchronize()
    for s, h in zip(streams, halves):
        p.cache.read(blocks, h, *outs, stream=s)
    torch.cuda.synchronize()
    for o, x in zip(outs, (k, v)):
        assert torch.equal(o[:147].cpu(), want(x, [40, 0, 100, 7], [0] * 4).to(BF)) and (o[147:] == 5).all()
    assert p.cache.read_status() == 0


def test_pages_that_many_tables_name():
    """Groups whose prefixes are the same pages, own pages that are a prefix's too, a page twice in one table."""
    p = Problem(BF, BF, [0, 3, 7], [96, 96], [64, 0, 33, 64, 5, 64, 64, 20], 4, 2, 128, 16)
    p.prefix_blocks[1] = p.prefix_blocks[0]
    p.prefix_blocks[:, 3] = p.prefix_blocks[0, 1]
    p.blocks[0] = p.prefix_blocks[0, :4]
    p.blocks[3] = p.blocks[5]
    p.check(*p.run())


def test_graphs_that_share_a_workspace():
    """Two captured calls of other shapes, one after the other on one workspace, replayed in turn."""
    a = Problem(BF, BF, [0, 20], [300], [40] * 21, 8, 2, 128, 16)
    b = Problem(FP, "rows", [0, 2], [30], [40] * 3, 3, 2, 64, 16)
    ws = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda")
    calls = []
    for p in (a, b):
        want = [x.clone() for x in p.run()]
        q, args, out = p.q.cuda(), p.args(), torch.zeros_like(want[0])
        p.run(q=q, args=args, out=out, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _, lse = p.run(q=q, args=args, out=out, ws=ws)
        calls.append((g, out, lse, want, q, args))
    for _ in range(5):
        for g, out, lse, want, _, _ in calls:
            out.zero_(), lse.zero_()
            g.replay()
            g.replay()
        for g, out, lse, want, _, _ in calls:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
