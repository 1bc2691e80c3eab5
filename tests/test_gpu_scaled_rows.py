"""8-bit caches at the borders of the 16-bit types: what is read back and attended over where a product lies next to the
middle of two values, or a row's largest value beyond fp16."""
import math

import numpy as np
import pytest
import torch

import cache_ref as R
import shared_ref as S
from test_gpu_cache import near

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
BITS = {BF: (8, -125), FP: (11, -13)}  # of a significand; the exponent (as frexp has it) of the smallest normal number
EVERY = torch.arange(256).to(torch.uint8).view(E4)


def nearest(x, act):
    """x in 64 bits rounded once to act, to the nearest even.  (Tensor.to() goes through 32 bits.)"""
    bits, least = BITS[act]
    e = torch.frexp(x)[1].clamp(min=least)
    step = torch.ldexp(torch.ones_like(x), e - bits)
    y = torch.round(x / step) * step
    y = torch.where(torch.isfinite(x), y, x)
    return torch.where(y.abs() > torch.finfo(act).max, torch.copysign(torch.tensor(math.inf, dtype=x.dtype), y), y)


def scales_near_middles(act):
    """Scales in 32 bits whose product with some 8-bit value is next to a middle of two values of act, on either side, so
    near that 32 bits take it for the middle."""
    bits = BITS[act][0]
    gen = np.random.default_rng(bits)
    found = []
    while len(found) < 24:
        m = float(gen.choice([9, 11, 13, 15]))  # 1.125, 1.375, ...: an odd significand of 4 bits
        middle = (2 * int(gen.integers(2 ** (bits - 1), 2 ** bits)) + 1) * 2.0 ** int(gen.integers(-14, 3) - bits)
        s = float(np.float32(middle / m))
        if s * m != middle and float(np.float32(s * m)) == middle:
            found.append(s)
    return found


@pytest.mark.parametrize("act", [BF, FP], ids=["bf16", "fp16"])
def test_the_scales_tell_one_rounding_from_two(act):
    """(And nearest() is the rounding of numpy, which converts from 64 bits to fp16 at once.)"""
    x = EVERY.double()
    x = x[~torch.isnan(x)]
    differ = 0
    for s in scales_near_middles(act):
        exact = x * s  # 28 bits
        if act == FP:
            with np.errstate(over="ignore"):
                assert np.array_equal(nearest(exact, FP).numpy(), exact.numpy().astype(np.float16).astype(np.float64))
        differ += int((nearest(exact, act) != nearest(exact.float().double(), act)).any())
    assert differ >= 8
    assert float(nearest(torch.tensor(1.125 * float.fromhex("0x1.d38e38p-1"), dtype=torch.float64), BF)) == 1.0234375


@pytest.mark.gpu
@pytest.mark.parametrize("act", [BF, FP], ids=["bf16", "fp16"])
def test_read_rounds_a_product_once(act):
    """Every 8-bit value with scales of 24 bits, of 20 and of one: equal, not near."""
    lay = R.Layout(1, 1, 256, 1, E4, 1)
    host = lay.pool(EVERY.view(1, 1, 1, 256), EVERY.view(1, 1, 1, 256))
    pool = host.cuda()
    near = scales_near_middles(act) + [float.fromhex("0x1.d38e38p-1"), float(np.float32(0.21)), 3.0e38, 1e-33, 448.0]
    short = [1.0, 0.1875, float.fromhex("0x1.fffffp-3"), 2.0 ** -100, 1.5 * 2.0 ** 20]
    for k_scale, v_scale in list(zip(near, near[1:] + near[:1])) + list(zip(short, short[1:] + near[:1])):
        cache = lay.cache(pool, k_scale=k_scale, v_scale=v_scale)
        outs = [torch.empty(1, 1, 256, dtype=act, device="cuda") for _ in range(2)]
        cache.read(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 1]).int().cuda(), *outs)
        for out, scale in zip(outs, (k_scale, v_scale)):
            want, got = nearest(EVERY.double() * float(np.float32(scale)), act), out.cpu().double().view(256)
            nan = torch.isnan(want)
            assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan]), scale
        assert cache.read_status() == 0


def stored_rows(x, act):
    """Row-scaled 8-bit rows of x [tokens, dim] (64 bits): (stored values, exponents)."""
    e = S.exponent_of(x)
    y = x / S.power(e)[:, None]
    if act == FP:  # what fp16 holds stays finite in it
        y = torch.where((e == 135)[:, None] & (x.abs() < 65520), y.clamp(-240, 240), y)
    return y.clamp(-448, 448).float().to(E4), e


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 96, 256])
def test_what_fp16_holds_stays_finite(dim):
    """Keys and values up to fp16's largest, written, read back and attended over."""
    gen = torch.Generator().manual_seed(dim)
    x = 65504 * (2 * torch.rand(61, dim, generator=gen) - 1) * torch.rand(61, 1, generator=gen).sqrt()
    x[0, :8] = torch.tensor([65504.0, -65504.0, 63488.0, 63456.0, -63520.0, 61440.0, 57344.0, 57376.0])
    x[1] = torch.linspace(57000, 65504, dim)
    x[2] = torch.linspace(-65504, 57344, dim)
    x[3] = 57344.0  # 448 * 2^7
    x[4], x[4, 3] = 1.0, 57376.0
    x = x.to(FP)
    lay = S.ScaledLayout(4, 1, dim, 16, 5)
    zero = torch.zeros(4, 1, 16, dim).to(E4)
    pool = lay.pool(zero, zero).cuda()
    cache = lay.cache(pool)
    kv = x[:, None].cuda()
    cache.append(kv, kv, kv, None, torch.arange(61).cuda(), torch.empty_like(kv))
    want, e = stored_rows(x.double(), FP)
    got, exps = lay.values(pool.cpu()), lay.exponents(pool.cpu())
    for i in range(2):
        assert torch.equal(exps[i].reshape(-1)[:61].int(), e.int())
        assert torch.equal(got[i].float().reshape(-1, dim)[:61], want.float())
    back = want.double() * S.power(e)[:, None]
    assert ((back - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + (2.0 ** -10 * S.power(e))[:, None]).all()
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    ids = i(0, 1, 2, 3)[None]
    outs = [torch.empty(61, 1, dim, dtype=FP, device="cuda") for _ in range(2)]
    cache.read(ids, i(0, 61), *outs)
    for o in outs:
        assert torch.equal(o.cpu()[:, 0].double(), nearest(back, FP)) and torch.isfinite(o).all()
    q, lse = torch.full((2, 1, dim), 2.0 ** -16, dtype=FP, device="cuda"), torch.empty(2, 1, device="cuda")
    q[1] *= -1
    out = torch.empty_like(q)
    cache.attend_shared(q, ids, i(61), i(0, 2), ids[:, :0].expand(2, 0), i(0, 0), out, cache.attend_shared_workspace(2, 1, 0, 1, 4), lse=lse)
    assert cache.read_status() == 0
    w, w_lse, off, off_lse = S.attend(q.cpu(), back[:, None, None], back[:, None, None], torch.arange(61)[None], [61], [0, 2],
                                      torch.zeros(2, 0, dtype=torch.int32), [0, 0], dim ** -0.5, FP, rounded=True)
    near(out, w, FP, off)
    assert ((lse.double().cpu() - w_lse).abs() <= off_lse).all()


@pytest.mark.gpu
def test_bf16_rows_are_stored_as_the_nearest():
    """(Only fp16 limits its largest values: the same ones in bf16, and what fp16 does not hold.)"""
    for act in (BF, FP):
        x = torch.ones(6, 64)
        x[:, 0] = torch.tensor([63488.0, 65280.0, 61440.0, 57344.0, math.inf, math.nan])
        x[4:, 1] = 64000.0
        x = x.to(act)
        lay = S.ScaledLayout(1, 1, 64, 16, 5)
        pool = lay.pool(*[torch.zeros(1, 1, 16, 64).to(E4)] * 2).cuda()
        kv = x[:, None].cuda()
        lay.cache(pool).append(kv, kv, kv, None, torch.arange(6).cuda(), torch.empty_like(kv))
        want, e = stored_rows(x.double(), act)
        for got, exps in zip(lay.values(pool.cpu()), lay.exponents(pool.cpu())):
            got = got.float().view(16, 64)[:6]
            nan = torch.isnan(x)
            assert torch.isnan(got[nan]).all() and torch.equal(got[~nan], want.float()[~nan]) and torch.equal(exps.view(16)[:6].int(), e.int())
        assert float(want[0, 0].float()) == (240 if act == FP else 256)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("act", [BF, FP], ids=["bf16", "fp16"])
def test_attend_every_exponent(act, page):
    """256 sequences of one token, whose weight is 1: outputs are the values themselves, every 8-bit one with every scale that
    the type holds without subnormal numbers (in fp16 every one)."""
    lay = S.ScaledLayout(256, 1, 256, page, 3)
    zero = torch.zeros(256, 1, page, 256).to(E4)
    v = EVERY.expand(256, 1, page, 256).contiguous()
    e = torch.arange(256).view(256, 1, 1).expand(256, 1, page)
    cache = lay.cache(lay.pool(zero, v, torch.full_like(e, 127), e).cuda())
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    out = torch.empty(256, 2, 256, dtype=act, device="cuda")
    cache.attend_shared(torch.ones_like(out), i().view(0, 0), i(), i(0), torch.arange(256).int().cuda()[:, None], i(*[1] * 256), out,
                        cache.attend_shared_workspace(256, 2, 1, 0, 0))
    assert cache.read_status() == 0
    want = nearest(EVERY.double() * S.power(torch.arange(256))[:, None], act)
    some = slice(0, 256) if act == FP else slice(16, 247)
    for x in range(2):
        got, w = out[some, x].double().cpu(), want[some]
        assert torch.equal(torch.isnan(got), torch.isnan(w)) and torch.equal(got.nan_to_num(7.0, math.inf, -math.inf), w.nan_to_num(7.0, math.inf, -math.inf))
