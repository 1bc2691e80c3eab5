"""Plain 64-bit statements of the cache operators on the host, and small caches to run them on.

A cache is held as values K, V [blocks, heads, page, dim]; `Layout` places them in a pool of bytes."""
import math

import numpy as np
import torch

from paged_kv_cache_kvx_gb300 import kvx

E4M3 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, E4M3: 2.0 ** -4}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, E4M3: 2.0 ** -10}  # half the smallest step
U = 2.0 ** -24


class Layout:
    """Shuffled pages in a pool with gaps; head-major or token-major segments."""

    def __init__(self, blocks, heads, dim, page, dtype, seed, layer=1, token_major=False, gap=48):
        rng = np.random.default_rng(seed)
        self.blocks, self.heads, self.dim, self.page, self.dtype = blocks, heads, dim, page, dtype
        row = dim * dtype.itemsize
        per_block = 2 * heads * page * row + gap
        place = rng.permutation(blocks).astype(np.int64) * per_block + 16
        self.L, self.first_lane = 2 * heads * (layer + 2), 2 * heads * layer  # the middle one of three or more layers
        self.addr = np.full((blocks, self.L), 2 ** 62, dtype=np.int64)       # other layers' lanes: not to be touched
        for h in range(heads):
            for kv in range(2):
                if token_major:
                    off = kv * heads * page * row + h * row
                else:
                    off = (2 * h + kv) * page * row
                self.addr[:, self.first_lane + 2 * h + kv] = place + off
        self.token_stride = heads * row if token_major else row
        self.pool_bytes = int(blocks * per_block + 16)
        self.row = row

    def rows(self):
        """Byte offsets [blocks, heads, 2, page] of every token's row."""
        a = self.addr[:, self.first_lane:self.first_lane + 2 * self.heads].reshape(self.blocks, self.heads, 2)
        return a[..., None] + np.arange(self.page) * self.token_stride

    def pool(self, k, v, fill=0xA5):
        """Bytes of the pool holding stored values k, v [blocks, heads, page, dim] (torch, of the cache's type)."""
        out = torch.full((self.pool_bytes,), fill, dtype=torch.uint8)
        kv = torch.stack([k, v], dim=2).contiguous().view(torch.uint8).view(-1, self.row)
        at = torch.from_numpy(self.rows().reshape(-1, 1)) + torch.arange(self.row)
        out[at.reshape(-1)] = kv.reshape(-1)
        return out

    def values(self, pool):
        """(k, v) [blocks, heads, page, dim] as stored, from the pool's bytes."""
        at = torch.from_numpy(self.rows().reshape(-1, 1)) + torch.arange(self.row)
        x = pool[at.reshape(-1)].view(self.dtype).view(self.blocks, self.heads, 2, self.page, self.dim)
        return x[:, :, 0], x[:, :, 1]

    def cache(self, pool, **kw):
        return kvx.Cache(pool, torch.from_numpy(self.addr).to(pool.device), heads=self.heads, dim=self.dim, dtype=self.dtype,
                         page_tokens=self.page, first_lane=self.first_lane, token_stride=self.token_stride, **kw)


def randn(shape, dtype, gen, scale=1.0):
    return (scale * torch.randn(shape, generator=gen)).to(dtype)


def norm_rotate(x, weight, eps, cos_sin, positions, interleaved):
    """x [T, heads, dim] -> (result, sum of the magnitudes that it adds up) in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    y, size = x.clone(), x.abs()
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        cs = cos_sin.double()[positions.long()]
        c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
        ib = ia + 1 if interleaved else ia + rot // 2
        y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
        size[..., ia] = (x[..., ia] * c).abs() + (x[..., ib] * s).abs()
        size[..., ib] = (x[..., ib] * c).abs() + (x[..., ia] * s).abs()
    return y, size


def seen(length, window, sinks):
    pos = np.arange(length)
    return pos[(pos >= length - window) | (pos < sinks)] if window else pos


def attend(q, k, v, blocks, lens, scale, window, sinks, k_scale=1.0, v_scale=1.0):
    """q [N, q_heads, dim]; k, v as stored.  Per sequence and head, in 64 bits: out, lse, weights (a list per sequence of
    (positions, [q_heads, visible])), and a bound on the kernel's error in out before its last rounding and in lse."""
    N, HQ, D = q.shape
    H, page = k.shape[1], k.shape[2]
    G = HQ // H
    out = torch.zeros(N, HQ, D, dtype=torch.float64)
    lse = torch.full((N, HQ), -math.inf, dtype=torch.float64)
    off, off_lse, weights = torch.zeros_like(out), torch.zeros(N, HQ, dtype=torch.float64), []
    for n in range(N):
        pos = torch.from_numpy(seen(int(lens[n]), window, sinks))
        w = torch.zeros(HQ, len(pos), dtype=torch.float64)
        if len(pos):
            b = blocks[n].long()[pos // page]
            for h in range(H):
                kk, vv = k[b, h, pos % page].double() * k_scale, v[b, h, pos % page].double() * v_scale
                for x in range(h * G, (h + 1) * G):
                    logit = scale * (kk @ q[n, x].double())
                    # dot products of D terms in 32 bits, in any order, then a few more roundings; exp of it
                    d = ((D + 8) * U * abs(scale) * (kk.abs() @ q[n, x].double().abs()) + 8 * U * logit.abs()).max() + 16 * U
                    top = logit.max()
                    if top == -math.inf:
                        continue
                    lse[n, x] = torch.logsumexp(logit, 0)
                    w[x] = (logit - lse[n, x]).exp()
                    out[n, x] = w[x] @ vv
                    # weights as two 16-bit parts: 2^-17 of each; sums of any length of positive terms: n/16 steps and more
                    off[n, x] = (w[x] @ vv.abs()) * (2 * d + 2.0 ** -17 + (len(pos) / 8 + 64) * U)
                    off_lse[n, x] = 2 * d + (len(pos) / 8 + 64) * U + 4 * U * abs(lse[n, x])
        weights.append((pos, w))
    return out, lse, weights, off, off_lse


def evict_positions(scores, length, budget, sinks, recent):
    """The kept tokens of one head by sorting (score, index) pairs."""
    if length <= budget:
        return list(range(length))
    lo = min(sinks, budget)
    tail = min(recent, budget - lo)
    middle = range(lo, length - tail)
    rank = sorted(middle, key=lambda i: (math.inf if math.isnan(scores[i]) else -scores[i], i))
    return list(range(lo)) + sorted(rank[:budget - lo - tail]) + list(range(length - tail, length))
