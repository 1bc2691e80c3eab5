"""8-bit caches at the borders of the 16-bit types: what is read back and attended over where a product lies next to the
middle of two values, or a row's largest value beyond fp16."""
import math

import numpy as np
import pytest
import torch

import cache_ref as R
import shared_ref as S
from test_gpu_shared import Problem

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


def in_fp16(x):
    """How row-scaled values enter products in fp16: 65536 as 65504, the rest rounded."""
    y = nearest(x, FP)
    return torch.where(x.abs() == 65536, torch.copysign(torch.tensor(65504.0, dtype=x.dtype), x), y)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 3])
@pytest.mark.parametrize("act", [BF, FP], ids=["bf16", "fp16"])
def test_attend_every_exponent(act, page):
    """256 sequences of one token, whose weight is 1: outputs are the values themselves, every 8-bit one with every scale that
    the type holds without subnormal numbers (in fp16 every one), 65536 as 65504."""
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
    exact = EVERY.double() * S.power(torch.arange(256))[:, None]
    want = in_fp16(exact) if act == FP else nearest(exact, act)
    some = slice(0, 256) if act == FP else slice(16, 247)
    for x in range(2):
        got, w = out[some, x].double().cpu(), want[some]
        assert torch.equal(torch.isnan(got), torch.isnan(w)) and torch.equal(got.nan_to_num(7.0, math.inf, -math.inf), w.nan_to_num(7.0, math.inf, -math.inf))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 7])
def test_attend_values_next_to_the_end_of_fp16(page):
    """Keys and values that 8 bits round up to 65536, among smaller ones, behind a prefix and in it."""
    p = Problem(FP, "rows", [0, 4], [100], [40, 5, 0, 70], 4, 2, 64, page)
    for kind in range(2):
        for b in (int(p.prefix_blocks[0, 1]), int(p.blocks[3, 0])):
            p.c.stored[kind][b, :, 2, 5] = 256.0
            p.c.stored[kind][b, :, 2, 6] = -256.0
            p.c.exps[kind][b, :, 2] = 135
    p.q *= 2.0 ** -14
    p.pool.copy_(p.c.pool())
    k, v = p.c.values()
    assert (k.abs() == 65536).sum() == 8 and (v.abs() == 65536).sum() == 8
    p.c.values = lambda: [torch.where(x.abs() == 65536, torch.copysign(torch.full_like(x, 65504.0), x), x) for x in (k, v)]
    out, lse = p.run()
    p.check(out, lse)
    assert torch.isfinite(out).all() and out.abs().max() > 100


@pytest.mark.gpu
def test_large_fp16_values_written_and_attended_over():
    """What a cache of 16 bits takes, one of row scales takes too."""
    lay = S.ScaledLayout(2, 1, 64, 16, 5)
    zero = torch.zeros(2, 1, 16, 64).to(E4)
    cache = lay.cache(lay.pool(zero, zero).cuda())
    x = torch.linspace(-65504, 65504, 32 * 64).view(32, 1, 64).to(FP).cuda()
    cache.append(x, x, x, None, torch.arange(32).cuda(), torch.empty_like(x))
    i = lambda *x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q, out, lse = torch.full((2, 1, 64), 2.0 ** -16, dtype=FP, device="cuda"), torch.empty(2, 1, 64, dtype=FP, device="cuda"), torch.empty(2, 1, device="cuda")
    cache.attend_shared(q, i(0, 1).view(1, 2), i(32), i(0, 2), i().view(2, 0), i(0, 0), out, cache.attend_shared_workspace(2, 1, 0, 1, 2), lse=lse)
    assert cache.read_status() == 0 and torch.isfinite(out).all() and torch.isfinite(lse).all()
