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
