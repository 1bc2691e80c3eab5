"""8-bit caches at the borders of the 16-bit types: what is read back and attended over where a product lies next to the
middle of two values, or a row's largest value beyond fp16."""
import math

import numpy as np
import pytest
import torch

import cache_ref as R

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
