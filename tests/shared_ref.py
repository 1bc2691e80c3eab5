"""Plain 64-bit statements of row-scaled caches, of reading tokens back, and of attention over shared prefixes."""
import math

import numpy as np
import torch

import cache_ref as R
from paged_kv_cache_kvx_gb300 import kvx

U = R.U


class ScaledLayout(R.Layout):
    """Pages of 8-bit rows whose scale exponents lie behind the rows of their segment: for head-major pages `page` bytes
    rounded up to 16, for token-major ones a place for one token more that holds the scales of all heads."""

    def __init__(self, blocks, heads, dim, page, seed, layer=1, token_major=False, gap=48):
        super().__init__(blocks, heads, dim, page, R.E4M3, seed, layer, token_major, gap)
        rng = np.random.default_rng(seed)
        if token_major:
            assert page <= dim
            self.scale_offset, seg = page * heads * dim, None
            per_block = 2 * heads * (page + 1) * dim + gap
        else:
            self.scale_offset = page * dim
            seg = page * dim + -(-page // 16) * 16
            per_block = 2 * heads * seg + gap
        place = rng.permutation(blocks).astype(np.int64) * per_block + 16
        for h in range(heads):
            for kv in range(2):
                off = kv * heads * (page + 1) * dim + h * dim if token_major else (2 * h + kv) * seg
                self.addr[:, self.first_lane + 2 * h + kv] = place + off
        self.pool_bytes = int(blocks * per_block + 16)

    def scale_bytes(self):
        """Byte offsets [blocks, heads, 2, page] of every row's exponent."""
        a = self.addr[:, self.first_lane:self.first_lane + 2 * self.heads].reshape(self.blocks, self.heads, 2)
        return a[..., None] + self.scale_offset + np.arange(self.page)

    def pool(self, k, v, ek=None, ev=None, fill=0xA5):
        out = super().pool(k, v, fill)
        if ek is not None:
            out[torch.from_numpy(self.scale_bytes())] = torch.stack([ek, ev], dim=2).to(torch.uint8)
        return out

    def exponents(self, pool):
        x = pool[torch.from_numpy(self.scale_bytes())]
        return x[:, :, 0], x[:, :, 1]

    def cache(self, pool, **kw):
        return super().cache(pool, scale_offset=self.scale_offset, **kw)


def power(exponents):
    """What scale bytes stand for: float8_e8m0fnu, in 64 bits."""
    e = exponents.to(torch.uint8)
    return torch.where(e == 255, math.nan, torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e.int() - 127))


def exponent_of(rows):
    """The biased exponent of the smallest power of two, from 2^-126 on, over which the rows' largest finite magnitude is
    at most 448 (rows [..., dim] in 64 bits)."""
    x = rows.abs()
    top = torch.where(torch.isfinite(x), x, 0).amax(-1)
    mantissa, e = torch.frexp(top)  # top = mantissa * 2^e, 448 = 0.875 * 2^9
    k = torch.where(top > 0, e - 9 + (mantissa > 0.875).int(), -126)
    return k.clamp(min=-126) + 127


class Caches:
    """Random caches of every kind: `stored` [blocks, heads, page, dim] are the stored values in 32 bits, values() what they
    stand for in 64."""

    def __init__(self, store, blocks, heads, dim, page, seed, token_major=False, spread=0.7, v_mean=0.0):
        gen = torch.Generator().manual_seed(seed)
        shape = (blocks, heads, page, dim)
        self.store = store
        if store == "rows":
            self.lay = ScaledLayout(blocks, heads, dim, page, seed, token_major=token_major)
            self.stored = [R.randn(shape, torch.float32, gen, 60.0).clamp(-448, 448).to(R.E4M3).float() for _ in range(2)]
            self.exps = [(spread * torch.randn(shape[:3], generator=gen)).round().int() + 121 for _ in range(2)]
            self.scales = (1.0, 1.0)
        else:
            self.lay = R.Layout(blocks, heads, dim, page, store, seed, token_major=token_major)
            self.stored = [(R.randn(shape, torch.float32, gen) + (v_mean if i else 0)).to(store).float() for i in range(2)]
            self.exps, self.scales = None, (0.21, 0.037) if store == R.E4M3 else (1.0, 1.0)

    def values(self):
        x = [s.to(self.lay.dtype).double() for s in self.stored]
        if self.exps is not None:
            return [y * power(e)[..., None] for y, e in zip(x, self.exps)]
        return [y * float(np.float32(s)) for y, s in zip(x, self.scales)]

    def pool(self):
        x = [s.to(self.lay.dtype) for s in self.stored]
        return self.lay.pool(*x) if self.exps is None else self.lay.pool(*x, *self.exps)

    def cache(self, pool):
        return self.lay.cache(pool) if self.exps is not None else self.lay.cache(pool, k_scale=self.scales[0], v_scale=self.scales[1])


def group_of(n, firsts):
    for g in range(len(firsts) - 1):
        if firsts[g] <= n < firsts[g + 1]:
            return g
    return None


def attend(q, k, v, prefix_blocks, prefix_lens, firsts, blocks, lens, scale, act, rounded=False):
    """q [N, q_heads, dim], k and v in 64 bits [blocks, heads, page, dim].  (out, lse, a bound on the kernel's error in out
    before its last rounding, one on lse's); `rounded`: values were rounded to fp16 on their way."""
    N, HQ, D = q.shape
    H, page = k.shape[1], k.shape[2]
    G = HQ // H
    out, off = (torch.zeros(N, HQ, D, dtype=torch.float64) for _ in range(2))
    lse, off_lse = torch.full((N, HQ), -math.inf, dtype=torch.float64), torch.zeros(N, HQ, dtype=torch.float64)
    for n in range(N):
        parts = []
        g = group_of(n, firsts)
        for table, length in ([] if g is None else [(prefix_blocks[g], int(prefix_lens[g]))]) + [(blocks[n], int(lens[n]))]:
            pos = torch.arange(length)
            b = table.long()[pos // page]
            parts.append((k[b, :, pos % page], v[b, :, pos % page]))  # [tokens, heads, dim]
        kk, vv = (torch.cat([p[i] for p in parts]) for i in range(2))
        m = len(kk)
        if not m:
            continue
        for h in range(H):
            x = q[n, h * G:(h + 1) * G].double()
            logits = scale * (x @ kk[:, h].T)
            # products of D terms in 32 bits, by 16 at a time, truncated or rounded; the exponential and its argument
            d = ((2 * D + 16) * U * abs(scale) * (x.abs() @ kk[:, h].abs().T) + 8 * U * logits.abs()).amax(1) + 16 * U
            if rounded:
                d = d + abs(scale) * 2.0 ** -25 * x.abs().sum(1)
            top = logits.amax(1)
            some = top > -math.inf
            s = torch.logsumexp(logits, 1)
            w = torch.where(some[:, None], (logits - s[:, None]).exp(), 0)
            rows = slice(h * G, (h + 1) * G)
            lse[n, rows] = s
            out[n, rows] = w @ vv[:, h]
            # weights rounded to the type of V: half a step of each, and in fp16 2^-32 of the largest where they are small;
            # sums of any length of positive terms
            size = w @ vv[:, h].abs()
            off[n, rows] = size * (2 * d[:, None] + R.HALF[act] + (m / 8 + 64) * U)
            if act == torch.float16:
                off[n, rows] += m * 2.0 ** -32 * w.amax(1)[:, None] * vv[:, h].abs().amax(0) + (2.0 ** -25 if rounded else 0)
            off_lse[n, rows] = torch.where(some, 2 * d + (m / 8 + 64) * U + 4 * U * s.abs(), 0)
    return out, lse, off, off_lse
