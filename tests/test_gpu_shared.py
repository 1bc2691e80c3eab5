"""Row-scaled caches, reading tokens back and attention over shared prefixes on the GPU, against plain 64-bit statements of
them (shared_ref.py).  Tolerances are half a step of the output's type plus bounds on what the 32-bit steps before it, and
the weights' rounding to 16 bits, can add up to."""
import math

import numpy as np
import pytest
import torch

import cache_ref as R
import shared_ref as S
from paged_kv_cache_kvx_gb300 import kvx
from test_gpu_cache import near

pytestmark = pytest.mark.gpu
BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
NAME = {BF: "bf16", FP: "fp16", E4: "e4m3"}


def label(case):
    return str(tuple(x if isinstance(x, list) else NAME.get(x, x) for x in case))[:100]


# ------------------------------------------------------------------ writing

APPEND = [  # act, T, q_heads, heads, dim, page, rot, interleaved, token_major, norm
    (BF, 1, 8, 2, 128, 16, 128, False, False, True),
    (BF, 37, 32, 8, 128, 16, 128, False, False, True),
    (BF, 37, 6, 3, 128, 7, 64, False, True, True),
    (FP, 50, 4, 4, 96, 24, 64, True, True, True),
    (FP, 9, 5, 1, 256, 1, 256, False, False, True),
    (BF, 11, 12, 2, 64, 4, 16, True, False, True),
    (FP, 5, 1, 1, 16, 2, 16, False, False, True),
    (BF, 5, 3, 1, 80, 16, 0, False, False, True),
    (BF, 6, 0, 2, 112, 16, 112, False, False, False),
    (FP, 700, 16, 16, 128, 256, 32, False, False, False),
    (BF, 5001, 2, 2, 64, 32, 64, False, True, True),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_write(case):
    act, T, HQ, H, D, page, rot, interleaved, token_major, norm = case
    gen = torch.Generator().manual_seed(T)
    blocks = -(-T // page) + 2
    old = S.Caches("rows", blocks, H, D, page, T, token_major)
    lay, host = old.lay, old.pool()
    pool = host.cuda()
    cache = old.cache(pool)
    qkv = R.randn((T, (HQ + 2 * H) * D), torch.float32, gen, 1.7)
    qkv = (qkv * torch.randn(T, 1, generator=gen).exp()).to(act)  # rows of different size
    cut = lambda x: [y.unflatten(1, (-1, D)) if y.numel() else y.view(T, 0, D) for y in  # noqa: E731
                     x.split([HQ * D, H * D, H * D], dim=1)]
    q, k, v = cut(qkv)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=gen)).to(act) for _ in range(2)) if norm else (None, None)
    most, table = 500, None
    pos = torch.randint(0, most, (T,), generator=gen, dtype=torch.int32)
    if rot:
        ang = torch.arange(most).double()[:, None] * 100.0 ** (-torch.arange(rot // 2).double() / rot)
        table = torch.cat([ang.cos(), ang.sin()], 1).float()
    slots = torch.randperm(blocks * page, generator=gen)[:T].clone()
    if T > 4:
        slots[T // 2] = -1
    dq, dk, dv = cut(qkv.cuda())
    out = torch.empty(T, HQ, D, dtype=act, device="cuda")
    cu = lambda x: None if x is None else x.cuda()  # noqa: E731
    cache.append(dq, dk, dv, pos.cuda(), slots.cuda(), out, q_weight=cu(wq), k_weight=cu(wk), eps=1e-5, cos_sin=cu(table),
                 interleaved=interleaved)
    torch.cuda.synchronize()
    assert cache.read_status() == 0
    steps = (D / 8 + 24) * R.U
    want, size = R.norm_rotate(q, wq, 1e-5, table, pos, interleaved)
    near(out, want, act, steps * size)
    got, exps = lay.values(pool.cpu()), lay.exponents(pool.cpu())
    has = slots >= 0
    b, o = slots[has] // page, slots[has] % page
    want_k, size_k = R.norm_rotate(k, wk, 1e-5, table, pos, interleaved)
    for i, (want, off) in enumerate(((want_k[has], steps * size_k[has]), (v.double()[has], torch.zeros(()).double()))):
        e = exps[i][b, :, o].int()
        # the row's largest magnitude is known to `off`: its exponent is that of a value within
        slack = off.amax(-1) if off.dim() else 0
        top = want.abs().amax(-1)
        low, high = (S.exponent_of((top + s * slack)[..., None]) for s in (-1, 1))
        assert ((e >= low) & (e <= high)).all()
        scale = S.power(e)[..., None]
        near(got[i].float()[b, :, o], (want / scale).clamp(-448, 448), E4, off / scale)
    untouched = torch.ones((blocks, H, page), dtype=torch.bool)
    untouched[b, :, o] = False
    for i in range(2):
        assert torch.equal(got[i].float()[untouched], old.stored[i][untouched])
        assert torch.equal(exps[i].int()[untouched], old.exps[i][untouched])
    assert torch.equal(lay.pool(*got, *exps), pool.cpu())  # nothing outside the rows and their scales


def test_write_special_values():
    """Exponents at both ends and next to the border, infinities limited, NaN kept, a row of zeros."""
    big = torch.finfo(BF).max
    rows = [[1.0], [448.0], [450.0], [0.0], [2.0 ** -133, -2.0 ** -130], [big, 1.0], [math.inf, 1.0], [-math.inf, math.nan, 7.0],
            [math.nan], [2.0 ** -126 * 448], [2.0 ** -126 * 450], [-2.0 ** -140]]
    x = torch.zeros(len(rows), 1, 64, dtype=BF)
    for i, r in enumerate(rows):
        x[i, 0, :len(r)] = torch.tensor(r)
    lay = S.ScaledLayout(2, 1, 64, 8, 3)
    zero = torch.zeros(2, 1, 8, 64).to(E4)
    pool = lay.pool(zero, zero).cuda()
    cache = lay.cache(pool)
    q = torch.ones(len(rows), 1, 64, dtype=BF, device="cuda")
    cache.append(q, x.cuda(), x.cuda(), None, torch.arange(len(rows)).cuda(), torch.empty_like(q))
    got, exps = lay.values(pool.cpu()), lay.exponents(pool.cpu())
    assert cache.read_status() == 0
    want_e = S.exponent_of(x[:, 0].double())
    for i in range(2):
        e = exps[i].permute(0, 2, 1).reshape(-1)[:len(rows)].int()
        assert torch.equal(e, want_e)
        assert (e >= 1).all() and (e <= 247).all()
        y = got[i].permute(0, 2, 1, 3).reshape(-1, 64)[:len(rows)]
        want = (x[:, 0].double() / S.power(e)[:, None]).clamp(-448, 448).float().to(E4)
        nan = torch.isnan(x[:, 0])
        assert torch.isnan(y.float())[nan].all()
        assert torch.equal(y.float()[~nan], want.float()[~nan])


def test_write_beyond_the_cache():
    lay = S.ScaledLayout(2, 2, 64, 4, 5)
    zero = torch.zeros(2, 2, 4, 64).to(E4)
    host = lay.pool(zero, zero)
    pool = host.cuda()
    cache = lay.cache(pool)
    x = torch.ones(1, 2, 64, dtype=BF, device="cuda")
    for slot in (8, 2 ** 40):
        cache.append(x, x, x, None, torch.tensor([slot]).cuda(), torch.empty_like(x))
    assert cache.read_status() == kvx.S_BOUNDS and torch.equal(pool.cpu(), host)
    # a pool that ends before the last page's scales do: that page is not written
    for cut, bits in ((0, 0), (1, kvx.S_BOUNDS)):
        end = int(lay.scale_bytes().max()) + 1
        short = host[:end - cut].cuda()
        cache = lay.cache(short)
        cache.append(x, x, x, None, torch.arange(8).cuda()[:1] + int(np.argmax(lay.addr[:, lay.first_lane])) * 4, torch.empty_like(x))
        assert cache.read_status() == bits


# ------------------------------------------------------------------ reading

READ = [  # act, store, lens, first, heads, dim, page, token_major, spare rows
    (BF, BF, [77], None, 8, 128, 16, False, 0),
    (BF, "rows", [77], None, 8, 128, 16, False, 3),
    (FP, FP, [5, 0, 33, 1, 0], [2, 0, 7, 0, 9], 3, 96, 7, True, 40),
    (BF, E4, [64, 1, 17], [0, 3, 40], 2, 256, 24, True, 1),
    (FP, E4, [200, 13], None, 1, 16, 1, False, 0),
    (FP, "rows", [200, 13, 64], [100, 1, 0], 5, 80, 32, True, 5),
    (BF, "rows", [1] * 300, None, 2, 64, 16, False, 2),
    (BF, BF, [3] * 33, [1] * 33, 4, 48, 2, False, 0),
    (BF, "rows", [0, 0, 0], None, 2, 64, 16, False, 7),
    (FP, "rows", [2000], [31], 4, 128, 256, False, 0),
]


@pytest.mark.parametrize("case", READ, ids=label)
@pytest.mark.parametrize("strided", [False, True])
def test_read(case, strided):
    act, store, lens, first, H, D, page, token_major, spare = case
    gen = torch.Generator().manual_seed(len(lens))
    firsts = first or [0] * len(lens)
    per = max(1, max(-(-(f + n) // page) for f, n in zip(firsts, lens))) + 1
    c = S.Caches(store, per * len(lens) + 1, H, D, page, 3, token_major)
    pool = c.pool().cuda()
    cache = c.cache(pool)
    blocks = torch.randperm(c.lay.blocks, generator=gen).int()[:per * len(lens)].view(-1, per)
    before = 3 if spare else 0  # rows that no sequence has, before and after
    starts = np.cumsum([before] + lens)
    T = int(starts[-1]) + spare
    wide = H * D + (8 if strided else 0)
    outs = [torch.randn(T, wide, generator=gen).to(act).cuda() for _ in range(2)]
    old = [o.cpu().clone() for o in outs]
    views = [o[:, :H * D].unflatten(1, (H, D)) for o in outs]
    cache.read(blocks.cuda(), torch.from_numpy(starts).int().cuda(), *views, first=None if first is None else torch.tensor(first).int().cuda())
    torch.cuda.synchronize()
    assert cache.read_status() == 0
    for got, was, x in zip(outs, old, c.values()):
        got = got.cpu()
        want = was[:, :H * D].double().unflatten(1, (H, D)).clone()
        for n, m in enumerate(lens):
            pos = torch.arange(m) + firsts[n]
            want[starts[n]:starts[n + 1]] = x[blocks[n].long()[pos // page], :, pos % page]
        # exactly the nearest: products of 8-bit values and powers of two, or 32-bit products of two short factors
        want = want.float().to(act) if store == E4 else want.to(act)
        assert torch.equal(got[:, :H * D].unflatten(1, (H, D)), want)
        assert torch.equal(got[:, H * D:], was[:, H * D:])


def test_read_exponents():
    """Every scale byte, and every 8-bit value with one of them, in both types."""
    for act in (BF, FP):
        lay = S.ScaledLayout(1, 1, 256, 256, 1)
        v = torch.arange(256).to(torch.uint8).view(E4).expand(1, 1, 256, 256).contiguous()
        e = torch.arange(256).view(1, 1, 256)
        pool = lay.pool(v, v, e, e).cuda()
        cache = lay.cache(pool)
        outs = [torch.empty(256, 1, 256, dtype=act, device="cuda") for _ in range(2)]
        cache.read(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 256]).int().cuda(), *outs)
        want = (v[0, 0].double() * S.power(e[0, 0])[:, None])
        # (through 32 bits, in which all of these are exact or beyond the type; by numpy where torch converts twice)
        want = want.float().to(act)
        for o in outs:
            got = o.cpu()[:, 0]
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])


def test_read_bad_pages():
    c = S.Caches("rows", 6, 2, 64, 4, 1)
    pool = c.pool().cuda()
    k, _ = c.values()
    blocks = torch.tensor([[0, 1, 99], [2, 3, 4]], dtype=torch.int32)

    def read(cache, starts, first=None, T=40):
        outs = [torch.full((T, 2, 64), 7.0, dtype=BF, device="cuda") for _ in range(2)]
        cache.read(blocks.cuda(), torch.tensor(starts).int().cuda(), *outs, first=None if first is None else torch.tensor(first).int().cuda())
        torch.cuda.synchronize()
        return outs[0].cpu(), cache.read_status()

    got, bits = read(c.cache(pool), [0, 12, 24])  # block 99 does not exist: its tokens' rows stay
    assert bits == kvx.S_BOUNDS
    assert torch.equal(got[:4].double(), k[0].permute(1, 0, 2).to(BF).double()) and (got[8:12] == 7).all() and (got[24:] == 7).all()
    assert torch.equal(got[12:16].double(), k[2].permute(1, 0, 2).to(BF).double())
    got, bits = read(c.cache(pool), [0, 0, 5], [0, 10])  # tokens 10 .. 14 of 12
    assert bits == kvx.S_BOUNDS and (got[2:] == 7).all() and (got[:2] != 7).any()
    got, bits = read(c.cache(pool), [0, 0, 3], [0, 2 ** 31 - 2])
    assert bits == kvx.S_BOUNDS and (got == 7).all()
    for starts in ([0, 12, 3], [0, 41, 44], [30, 2, 1]):  # no table of rows
        got, bits = read(c.cache(pool), starts)
        assert bits & kvx.S_BOUNDS
    assert torch.equal(pool.cpu(), c.pool())


def test_read_nothing():
    c = S.Caches(BF, 2, 1, 64, 4, 1)
    cache = c.cache(c.pool().cuda())
    out = torch.empty(0, 1, 64, dtype=BF, device="cuda")
    before = kvx.kvx_launch_count()
    cache.read(torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), out, out)
    out = torch.empty(3, 1, 64, dtype=BF, device="cuda")
    cache.read(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), out, out)
    assert kvx.kvx_launch_count() == before


# ------------------------------------------------------------------ attending

class Problem:
    def __init__(self, act, store, firsts, prefixes, lens, G, H, D, page, token_major=False, seed=1, scale=None, spread=2.0, **kw):
        gen = torch.Generator().manual_seed(seed)
        self.act, self.firsts, self.prefixes, self.lens, self.scale = act, firsts, prefixes, lens, scale
        N, groups = len(lens), len(prefixes)
        need = lambda x: -(-x // page)  # noqa: E731
        per, pper = max([need(x) for x in lens] + [1]), max([need(x) for x in prefixes] + [1])
        total = sum(need(x) for x in list(lens) + list(prefixes)) + 1
        self.c = S.Caches(store, total, H, D, page, seed, token_major, **kw)
        ids = torch.randperm(total, generator=gen).int()
        at = 0

        def table(xs, width):
            nonlocal at
            t = torch.full((len(xs), width), 2 ** 31 - 1, dtype=torch.int32)  # entries that are not to be read
            for i, x in enumerate(xs):
                t[i, :need(x)] = ids[at:at + need(x)]
                at += need(x)
            return t

        self.blocks, self.prefix_blocks = table(lens, per), table(prefixes, pper)
        self.q = R.randn((N, G * H, D), act, gen, spread / (self.c.scales[0] if store == E4 else 1.0))
        self.N, self.HQ, self.D, self.H = N, G * H, D, H
        self.pool = self.c.pool().cuda()
        self.cache = self.c.cache(self.pool)
        self.ws = self.cache.attend_shared_workspace(N, G * H, per, groups, pper)
        self.ws.fill_(0xFF)

    def args(self):
        i = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        return (self.prefix_blocks.cuda(), i(self.prefixes), i(self.firsts), self.blocks.cuda(), i(self.lens))

    def run(self, stream=None, lse=True, q=None, out=None, args=None, ws=None):
        out = torch.full((self.N, self.HQ, self.D), 9.0, dtype=self.act, device="cuda") if out is None else out
        sums = torch.full((self.N, self.HQ), 9.0, device="cuda") if lse else None
        self.cache.attend_shared(self.q.cuda() if q is None else q, *(args or self.args()), out, self.ws if ws is None else ws,
                                 scale=self.scale, lse=sums, stream=stream)
        return out, sums

    def check(self, out, lse):
        assert self.cache.read_status() == 0
        k, v = self.c.values()
        scale = self.D ** -0.5 if self.scale is None else self.scale
        want, want_lse, off, off_lse = S.attend(self.q, k, v, self.prefix_blocks, self.prefixes, self.firsts, self.blocks, self.lens,
                                                scale, self.act, rounded=self.act == FP and self.c.store == "rows")
        near(out, want, self.act, off)
        lse = lse.double().cpu()
        dead = want_lse == -math.inf
        assert (lse[dead] == -math.inf).all() and (out.cpu()[dead] == 0).all()
        assert ((lse - want_lse)[~dead].abs() <= off_lse[~dead]).all()


ATTEND = [  # act, store, firsts, prefixes, lens, group, heads, dim, page, token_major
    (BF, BF, [0, 1], [1], [0], 1, 1, 64, 16, False),
    (BF, BF, [0, 1], [0], [1], 1, 1, 64, 16, False),
    (BF, BF, [0, 2], [40], [0, 3], 4, 2, 128, 16, False),
    (BF, BF, [0], [], [63, 64, 65, 127, 128, 129, 0, 300], 4, 2, 128, 16, False),
    (BF, BF, [0, 40], [700], list(range(40)), 8, 2, 128, 16, False),
    (BF, BF, [0, 3, 3, 20], [130, 500, 257], [1, 0, 9, 70] * 5 + [200, 0], 5, 3, 128, 16, True),
    (BF, BF, [2, 9, 50], [64, 1000], [5] * 60, 7, 1, 128, 24, False),
    (FP, FP, [0, 17], [333], [30] * 17, 16, 2, 96, 7, True),
    (FP, FP, [0, 5], [200], [3, 500, 0, 64, 65], 128, 1, 64, 32, False),
    (BF, BF, [0, 33], [450], [17] * 33, 9, 2, 256, 16, False),
    (FP, FP, [0, 2, 5], [100, 65], [200, 1, 0, 63, 64], 3, 2, 160, 1, False),
    (BF, BF, [0, 6], [150], [20] * 6, 2, 2, 16, 16, False),
    (FP, FP, [1, 4], [129], [31] * 6, 1, 4, 48, 2, False),
    (BF, E4, [0, 30], [600], [40] * 32, 8, 2, 128, 64, False),
    (FP, E4, [0, 4, 9], [257, 64], [129] * 10, 8, 2, 64, 5, True),
    (BF, E4, [0, 6], [300], [70] * 6, 4, 2, 256, 16, True),
    (FP, E4, [0, 20], [300], [7] * 20, 7, 1, 80, 16, False),
    (BF, "rows", [0, 40, 44], [513, 200], [33] * 48, 8, 2, 128, 16, False),
    (BF, "rows", [0, 2], [90], [300, 1], 8, 2, 128, 16, True),
    (FP, "rows", [0, 9, 12], [260, 70], [140] * 14, 4, 3, 64, 32, False),
    (BF, "rows", [0, 5], [140], [64] * 6, 6, 2, 256, 48, False),
    (FP, "rows", [0, 5], [140], [64] * 6, 6, 2, 256, 3, False),
    (BF, "rows", [0], [], [1, 2, 15, 16, 17, 130, 500], 8, 1, 96, 24, True),
    (BF, "rows", [0, 3], [100], [5] * 3, 1, 1, 32, 256, False),
]


@pytest.mark.parametrize("case", ATTEND, ids=label)
def test_attend(case):
    act, store, firsts, prefixes, lens, G, H, D, page, token_major = case
    p = Problem(act, store, firsts, prefixes, lens, G, H, D, page, token_major)
    out, lse = p.run()
    p.check(out, lse)
    again, sums = p.run()
    assert torch.equal(out, again) and torch.equal(lse, sums)
    assert torch.equal(p.run(lse=False)[0], out)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.9])
def test_attend_scales(scale):
    p = Problem(BF, BF, [0, 20], [300], [40] * 21, 8, 2, 128, 16, scale=scale, spread=1.0)
    p.check(*p.run())
    p = Problem(FP, "rows", [0, 2], [30], [40] * 3, 3, 2, 64, 16, scale=scale, spread=1.0)
    p.check(*p.run())


def test_attend_rising_logits():
    """Logits that rise along the keys, so that the base moves on again and again, and one key that outweighs all."""
    for act, store in ((BF, BF), (FP, FP), (FP, "rows")):
        p = Problem(act, store, [0, 24], [900], [300] * 24, 8, 1, 128, 16, v_mean=0.5)
        k = p.c.stored[0]
        for table, length in [(p.prefix_blocks[0], 900)] + [(p.blocks[n], 300) for n in range(24)]:
            pos = torch.arange(length)
            b = table.long()[pos // 16]
            rise = torch.linspace(0, 30, length)[:, None]
            k[b, 0, pos % 16] = k[b, 0, pos % 16] * 0.2 + rise * (4 if store == "rows" else 1)
        p.q = p.q.abs()
        p.pool.copy_(p.c.pool())
        p.check(*p.run())


@pytest.mark.parametrize("act,store,G,D,n", [(BF, BF, 1, 128, 48), (BF, "rows", 8, 128, 48), (FP, FP, 9, 64, 48), (BF, E4, 16, 64, 48),
                                             (FP, "rows", 17, 64, 48), (BF, BF, 8, 256, 24), (FP, FP, 16, 160, 24)])
def test_attend_rising_logits_of_few_rows(act, store, G, D, n):
    """Up to 16 rows, and 17, over many tiles of a piece, the last of every kind; every other row rises, the others fall."""
    lens = [2500 - 37 * i for i in range(n)]
    p = Problem(act, store, [0], [], lens, G, 1, D, 16, v_mean=0.0 if store == "rows" else 0.5)
    k = p.c.stored[0]
    for i, length in enumerate(lens):
        pos = torch.arange(length)
        b = p.blocks[i].long()[pos // 16]
        rise = torch.linspace(0, 20, length)[:, None]
        k[b, 0, pos % 16] = k[b, 0, pos % 16] * 0.2 + rise * (1 if store in (BF, FP) else 4)
    p.q = p.q.abs()
    p.q[:, 1::2] *= -1
    p.pool.copy_(p.c.pool())
    p.check(*p.run())


def test_attend_many_small_weights():
    """One key with all but a little of the weight and many with the rest: 20,000 keys of 2^-22 of the largest."""
    for act in (BF, FP):
        p = Problem(act, act, [0, 2], [20000], [1, 1], 1, 1, 64, 16, scale=1.0)
        p.c.stored[0].zero_(), p.c.stored[1].fill_(1.0)
        p.q.zero_()
        p.q[:, :, 0] = 1.0
        b, o = p.prefix_blocks[0, 0].long(), 0
        p.c.stored[0][b, 0, o, 0] = 15.25  # e^-15.25 = 2^-22
        p.c.stored[1][b, 0, o] = -1.0
        p.pool.copy_(p.c.pool())
        p.check(*p.run())


def test_attend_infinities_and_nan():
    base = dict(firsts=[0, 3], prefixes=[70], lens=[40, 0, 5], G=4, H=2, D=64, page=16)
    # keys that no head sees: logits of -infinity everywhere
    p = Problem(BF, BF, **base)
    p.c.stored[0][:, 0] = -math.inf
    p.q[:, :4] = p.q[:, :4].abs() + 0.1
    p.pool.copy_(p.c.pool())
    out, lse = p.run()
    assert (lse[:, :4] == -math.inf).all() and (out[:, :4] == 0).all() and torch.isfinite(out[:, 4:]).all()
    # some keys of -infinity weigh nothing
    p = Problem(BF, BF, **base)
    p.q = p.q.abs() + 0.1
    b = p.prefix_blocks[0].long()
    p.c.stored[0][b[1], :, 3] = -math.inf
    p.c.stored[0][b[0], :, 0] = -math.inf
    p.pool.copy_(p.c.pool())
    out, lse = p.run()
    p.check(out, lse)
    # a NaN in a key makes its heads' outputs NaN, in a value its column, an infinity in a value its column infinite
    for act, store in ((BF, BF), (FP, FP), (BF, E4), (FP, E4), (BF, "rows"), (FP, "rows")):
        p = Problem(act, store, **base, spread=0.3)
        b = p.prefix_blocks[0].long()
        p.c.stored[0][b[2], 0, 1, 7] = math.nan
        p.c.stored[1][b[2], 1, 1, 9] = math.nan
        if store in (BF, FP):
            p.c.stored[1][b[3], 1, 2, 11] = -math.inf
        p.pool.copy_(p.c.pool())
        out, lse = (x.cpu() for x in p.run())
        assert torch.isnan(out[:, :4]).all() and torch.isnan(lse[:, :4]).all()
        assert torch.isnan(out[:, 4:, 9]).all()
        rest = [i for i in range(64) if i not in (9, 11)]
        assert torch.isfinite(out[:, 4:, rest]).all() and torch.isfinite(lse[:, 4:]).all()
        if store in (BF, FP):
            assert (out[:, 4:, 11] == -math.inf).all()
    # what lies behind a sequence's last token, in pages it has, is not seen
    for store in (BF, "rows", E4):
        p = Problem(BF, store, **base)
        want = [x.clone() for x in p.run()]
        for n, m in ((0, 40), (2, 5)):
            b = p.blocks[n].long()[m // 16]
            p.c.stored[0][b, :, m % 16:], p.c.stored[1][b, :, m % 16:] = math.nan, math.nan
        b = p.prefix_blocks[0].long()[70 // 16]
        p.c.stored[0][b, :, 70 % 16:], p.c.stored[1][b, :, 70 % 16:] = math.nan, math.nan
        if p.c.exps is not None:
            for e in p.c.exps:
                e[b, :, 70 % 16:] = 255
        p.pool.copy_(p.c.pool())
        for x, y in zip(want, p.run()):
            assert torch.equal(x, y)


def test_attend_row_exponents():
    """Rows of very different scales, and scales that 16 bits do not hold in one factor."""
    for act, far in ((BF, 60), (FP, 6)):
        p = Problem(act, "rows", [0, 20], [300], [40] * 20, 8, 1, 128, 16)
        gen = torch.Generator().manual_seed(2)
        p.c.exps[1] = torch.randint(121 - far, 121 + far, p.c.exps[1].shape, generator=gen, dtype=torch.int32)
        p.c.exps[1][p.prefix_blocks[0].long()[2], 0, 3] = 121 + far + 1
        p.pool.copy_(p.c.pool())
        p.check(*p.run())
    p = Problem(BF, "rows", [0, 3], [50], [10] * 3, 2, 1, 64, 16, scale=2.0 ** 70)
    p.c.exps[0].fill_(121 - 70)
    p.c.exps[1].fill_(121 + 100)
    p.pool.copy_(p.c.pool())
    p.check(*p.run())
    # a row whose scale is NaN
    p.c.exps[1][p.prefix_blocks[0].long()[0], 0, 3] = 255
    p.pool.copy_(p.c.pool())
    assert torch.isnan(p.run()[0]).all()


def test_attend_strides_and_streams():
    p = Problem(BF, BF, [0, 20], [300], [40] * 21, 8, 2, 128, 16)
    want, want_lse = p.run()
    N, HQ, D = p.q.shape
    wide = torch.zeros(N, HQ * D + 24, dtype=BF, device="cuda")
    wide[:, 8:8 + HQ * D] = p.q.cuda().flatten(1)
    out = torch.full((N, HQ * D + 8), 3.0, dtype=BF, device="cuda")
    got, lse = p.run(q=wide[:, 8:8 + HQ * D].unflatten(1, (HQ, D)), out=out[:, :HQ * D].unflatten(1, (HQ, D)))
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and (out[:, HQ * D:] == 3).all()
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces, args, q = [p.ws, torch.empty_like(p.ws)], p.args(), p.q.cuda()
    torch.cuda.synchronize()
    results = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 2]):
            results.append(p.run(q=q, args=args, ws=spaces[i % 2]))
    torch.cuda.synchronize()
    for out, lse in results:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert p.cache.read_status() == 0


def test_attend_in_a_graph():
    """Captured once, replayed with other lengths, groups and pages: nothing of them is kept on the host."""
    p = Problem(BF, "rows", [0, 30, 40], [400, 100], [60] * 44, 8, 2, 128, 16)
    q, args = p.q.cuda(), p.args()
    out, lse = torch.empty(44, 16, 128, dtype=BF, device="cuda"), torch.empty(44, 16, device="cuda")
    p.cache.attend_shared(q, *args, out, p.ws, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.cache.attend_shared(q, *args, out, p.ws, lse=lse)
    g.replay()
    p.check(out, lse)
    for firsts, prefixes, lens in (([0, 44, 44], [400, 3], [7] * 44), ([5, 6, 9], [1, 100], [0, 60] * 22), ([0, 0, 0], [0, 0], [33] * 44)):
        p.firsts, p.prefixes, p.lens = firsts, prefixes, lens
        for t, x in zip((args[1], args[2], args[4]), (prefixes, firsts, lens)):
            t.copy_(torch.tensor(x, dtype=torch.int32))
        g.replay()
        p.check(out, lse)


def test_attend_many():
    """More sequences than threads, more groups than blocks, and all of the card for one sequence."""
    gen = np.random.default_rng(3)
    N = 1500
    sizes = gen.integers(0, 9, 400)
    firsts = np.minimum(np.cumsum(np.concatenate([[3], sizes])), N).tolist()
    p = Problem(BF, BF, firsts, gen.integers(0, 60, 400).tolist(), gen.integers(0, 40, N).tolist(), 2, 1, 64, 16)
    p.check(*p.run())
    p = Problem(BF, "rows", [0, 1], [150000], [70000], 4, 1, 64, 16, scale=0.2)
    p.check(*p.run())


@pytest.mark.parametrize("store,dim,G,n", [("rows", 128, 8, 300), (BF, 128, 4, 700), (BF, 256, 8, 200), (FP, 64, 16, 150)])
def test_attend_long_prefix(store, dim, G, n):
    """Many rows of queries over one prefix, which blocks of columns cut anywhere, against 64-bit products on the GPU."""
    act = FP if store == FP else BF
    P, page, H = 20011, 16, 2
    p = Problem(act, store, [0, n], [P], [3] * n, G, H, dim, page)
    out, lse = p.run()
    assert p.cache.read_status() == 0
    k, v = (x.cuda() for x in p.c.values())
    pos = torch.arange(P, device="cuda")
    b = p.prefix_blocks.cuda().long()[0][pos // page]
    own = torch.arange(3, device="cuda")
    for h in range(H):
        pk, pv = k[b, h, pos % page], v[b, h, pos % page]
        ob = p.blocks.cuda().long()[:, 0]
        ok, ov = k[ob, h][:, own], v[ob, h][:, own]  # [n, 3, dim]
        q = p.q.cuda().double()[:, h * G:(h + 1) * G]
        x = torch.cat([q @ pk.T, torch.einsum("ngd,ntd->ngt", q, ok)], -1) * dim ** -0.5
        size = (q.abs() @ pk.abs().T).amax() * dim ** -0.5
        s = torch.logsumexp(x, -1)
        w = (x - s[..., None]).exp()
        want = w[..., :P] @ pv + torch.einsum("ngt,ntd->ngd", w[..., P:], ov)
        bound = w[..., :P] @ pv.abs() + torch.einsum("ngt,ntd->ngd", w[..., P:], ov.abs())
        d = (2 * dim + 16) * R.U * size + 8 * R.U * x.abs().amax() + 16 * R.U
        off = bound * (2 * d + R.HALF[act] + (P / 8 + 64) * R.U)
        if act == FP:
            off = off + P * 2.0 ** -32 * w.amax(-1, keepdim=True) * pv.abs().amax()
        near(out[:, h * G:(h + 1) * G], want.cpu(), act, off.cpu())
        assert ((lse.double()[:, h * G:(h + 1) * G] - s).abs() <= 2 * d + (P / 8 + 64) * R.U + 4 * R.U * s.abs()).all()


def test_attend_bad_tables():
    base = dict(firsts=[0, 4, 8], prefixes=[100, 40], lens=[20] * 10, G=4, H=2, D=64, page=16)
    p = Problem(BF, BF, **base)
    good, good_lse = (x.clone() for x in p.run())
    # lengths beyond the tables count as full pages (the tables are full here)
    full = Problem(BF, BF, firsts=[0, 4, 8], prefixes=[112, 112], lens=[32] * 10, G=4, H=2, D=64, page=16)
    want = [x.clone() for x in full.run()]
    args = list(full.args())
    args[1], args[4] = torch.tensor([113, -1]).int().cuda(), torch.tensor([33, 2 ** 31 - 1, -1, 32, 99] * 2).int().cuda()
    got = full.run(args=args)
    assert full.cache.read_status() == kvx.S_BOUNDS
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    # tables of groups that decrease or reach beyond the sequences: refused on the device, and the next call is right
    for firsts in ([0, 4, 11], [4, 0, 8], [0, 8, 4], [-1, 4, 8], [0, -1, 8], [9, 2 ** 31 - 1, 2 ** 31 - 1]):
        args = list(p.args())
        args[2] = torch.tensor(firsts).int().cuda()
        p.cache.status.zero_()
        p.run(args=args)
        torch.cuda.synchronize()
        assert p.cache.read_status() == kvx.S_BOUNDS
    p.cache.status.zero_()
    out, lse = p.run()
    assert torch.equal(out, good) and torch.equal(lse, good_lse) and p.cache.read_status() == 0
    # a page that does not exist, a segment that is not aligned or leaves the pool
    for page in (16, 7):
        p = Problem(BF, "rows", **(base | dict(page=page)))
        args = list(p.args())
        args[0] = args[0].clone()
        args[0][0, 1] = 2 ** 31 - 1
        p.run(args=args)
        assert p.cache.read_status() == kvx.S_BOUNDS
        for bad, bits in ((8, kvx.S_ALIGN), (2 ** 40, kvx.S_BOUNDS), (p.pool.numel() // 16 * 16 - 16, kvx.S_BOUNDS)):
            p.cache.status.zero_()
            lane = p.c.lay.first_lane + 1
            block = int(p.blocks[3, 0])
            was = int(p.cache.addr[block, lane])
            p.cache.addr[block, lane] = bad if bad > 100 else was + bad
            p.run()
            assert p.cache.read_status() == bits
            p.cache.addr[block, lane] = was
        p.cache.status.zero_()
        p.check(*p.run())


@pytest.mark.parametrize("act,store", [(BF, BF), (BF, "rows"), (FP, E4)])
@pytest.mark.parametrize("page", [16, 7])
def test_attend_bad_pages_are_zeros(act, store, page):
    p = Problem(act, store, firsts=[0, 3], prefixes=[100], lens=[40, 5, 0, 70], G=4, H=2, D=80, page=page)
    own, prefix = int(p.blocks[3, 1]), int(p.prefix_blocks[0, 2])
    args = list(p.args())
    args[0], args[3] = args[0].clone(), args[3].clone()
    args[0][0, 2], args[3][3, 1] = p.cache.addr.shape[0], 2 ** 31 - 1
    got = [x.clone() for x in p.run(args=args)]
    assert p.cache.read_status() == kvx.S_BOUNDS
    p.cache.status.zero_()
    for b in (own, prefix):
        for x in p.c.stored:
            x[b] = 0
    p.pool.copy_(p.c.pool())
    want = p.run()
    assert p.cache.read_status() == 0
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dim", [48, 80, 96, 160])
def test_attend_what_lies_behind_rows_of_odd_widths(dim):
    """Nothing of it enters: NaN and large values between the rows."""
    p = Problem(BF, "rows", firsts=[0, 3], prefixes=[300], lens=[40, 5, 0, 270], G=4, H=2, D=dim, page=16)
    want = [x.clone() for x in p.run()]
    p.check(*want)
    # the same call behind one that leaves NaN in all that shared memory may keep
    other = Problem(BF, "rows", firsts=[0, 3], prefixes=[4000], lens=[400] * 4, G=4, H=2, D=256 if dim > 128 else 128, page=16)
    for x in other.c.stored:
        x.fill_(math.nan)
    other.pool.copy_(other.c.pool())
    for _ in range(3):
        other.run()
        for x, y in zip(want, p.run()):
            assert torch.equal(x, y)


def test_attend_beyond_32_bits():
    """A pool of more than 4 GB, the pages at its end."""
    for store in (BF, "rows"):
        p = Problem(BF, store, [0, 3], [100], [40] * 4, 4, 2, 64, 16)
        shift = (5 << 30) // 16 * 16
        big = torch.zeros(shift + p.pool.numel(), dtype=torch.uint8, device="cuda")
        big[shift:] = p.pool
        lay = p.c.lay
        lanes = slice(lay.first_lane, lay.first_lane + 2 * lay.heads)
        lay.addr[:, lanes] += shift
        p.cache, p.pool = p.c.cache(big), big
        p.check(*p.run())
        x = torch.empty(100, 2, 64, dtype=BF, device="cuda"), torch.empty(100, 2, 64, dtype=BF, device="cuda")
        p.cache.read(p.prefix_blocks.cuda(), torch.tensor([0, 100]).int().cuda(), *x)
        pos = torch.arange(100)
        for got, v in zip(x, p.c.values()):
            assert torch.equal(got.cpu(), v[p.prefix_blocks[0].long()[pos // 16], :, pos % 16].to(BF))
        del big


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("act", [BF, FP])
def test_together(act):
    """A prompt is written into a quantised cache, its first part shared; it is read back, sequences decode behind it, and
    attention is the one over what was read back."""
    gen = torch.Generator().manual_seed(4)
    H, G, D, page, prompt, N, steps = 2, 4, 128, 16, 203, 5, 3
    shared, per = -(-prompt // page), 1
    c = S.Caches("rows", shared + N * per, H, D, page, 9)
    pool = c.pool().cuda()
    cache = c.cache(pool)
    ids = torch.randperm(c.lay.blocks, generator=gen).int()
    prefix, blocks = ids[:shared][None], ids[shared:].view(N, per)
    ang = torch.arange(prompt + steps).double()[:, None] * 10000.0 ** (-torch.arange(D // 2).double() * 2 / D)
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    wq, wk = (torch.ones(D, dtype=act, device="cuda") for _ in range(2))

    def write(T, positions, slots):
        qkv = R.randn((T, (G * H + 2 * H) * D), act, gen).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([G * H * D, H * D, H * D], dim=1))
        out = torch.empty(T, G * H, D, dtype=act, device="cuda")
        cache.append(q, k, v, positions.int().cuda(), slots.long().cuda(), out, q_weight=wq, k_weight=wk, cos_sin=cos_sin)
        return out

    pos = torch.arange(prompt)
    write(prompt, pos, prefix[0].long()[pos // page] * page + pos % page)
    ws = cache.attend_shared_workspace(N, G * H, per, 1, shared)
    for step in range(steps):
        q = write(N, torch.full((N,), prompt + step), blocks[:, 0].long() * page + step)
        out, lse = torch.empty_like(q), torch.empty(N, G * H, device="cuda")
        lens = torch.full((N,), step + 1, dtype=torch.int32, device="cuda")
        cache.attend_shared(q, prefix.cuda(), torch.tensor([prompt]).int().cuda(), torch.tensor([0, N]).int().cuda(), blocks.cuda(),
                            lens, out, ws, lse=lse)
        k, v = (torch.empty(prompt + N * (step + 1), H, D, dtype=act, device="cuda") for _ in range(2))
        cache.read(prefix.cuda(), torch.tensor([0, prompt]).int().cuda(), k[:prompt], v[:prompt])
        cache.read(blocks.cuda(), torch.arange(N + 1).int().cuda() * (step + 1), k[prompt:], v[prompt:])
        torch.cuda.synchronize()
        assert cache.read_status() == 0
        # the same by its definition, over dense keys and values laid out as a cache of one-token pages
        dense = [x.double().cpu()[:, :, None] for x in (k, v)]
        want, want_lse, off, off_lse = S.attend(q.cpu(), *dense, torch.arange(prompt)[None], [prompt], [0, N],
                                                prompt + torch.arange(N * (step + 1)).view(N, -1), [step + 1] * N, D ** -0.5, act)
        near(out, want, act, off)
        assert ((lse.double().cpu() - want_lse).abs() <= off_lse).all()
