"""Decoding on a transferred prefix: the block transfer, then the cache operators on the pages that it filled.

A holder's pool has the KV pages of a prompt, every (layer, head) segment at its own address.  The prefix is
transferred into the receiver's pool (encode, plan, pack, seal) and the receiver decodes on it, with one Cache per layer
over the receiver's address table: new tokens are appended, each attends over the whole history, and when the history
is over its budget the tokens with the least attention weight are left behind.  There are no model weights here:
queries, keys and values are random, and the last step's attention is checked against a plain statement of it.

    python examples/decode_received_prefix.py
"""
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_kv_cache_kvx_gb300 import kvx, workloads as W  # noqa: E402


def main(layers=3, heads=4, group=4, dim=128, page=16, prompt_blocks=40, steps=24, budget=256, seed=0, verbose=True):
    dev, act = torch.device("cuda"), torch.bfloat16
    seg = page * dim * act.itemsize  # 4 KiB
    gen = torch.Generator(device=dev).manual_seed(seed)

    # ---- the holder: a bump-allocated prefix, its segments filled with keys and values
    wl = W.bump("prompt", prompt_blocks, layers * heads, seg, seed=seed)
    holder = torch.randn(wl.pool_bytes // 2, generator=gen, device=dev).to(act).view(torch.uint8)

    # ---- the receiver's pages: the prompt's, some for new tokens, some for what an eviction keeps
    more, kept_pages = -(-steps // page), -(-budget // page)
    blocks = prompt_blocks + more + kept_pages
    place = np.random.default_rng(seed).permutation(blocks).astype(np.int64)
    addr = torch.from_numpy(place[:, None] * (wl.lanes * seg) + np.arange(wl.lanes) * seg).to(dev)
    pool = torch.zeros(blocks * wl.lanes * seg, dtype=torch.uint8, device=dev)

    # ---- the transfer
    tr = kvx.Transfer(wl.blocks, wl.seg_len, wl.numa, wl.pool_bytes, device=dev)
    tr.set_addr(wl.addr)
    slab = torch.empty(tr.slab_bytes, dtype=torch.uint8, device=dev)
    tr.encode()
    tr.plan()
    tr.pack(holder, slab)
    tr.seal(slab, addr, pool)
    assert tr.read_status() == 0

    # ---- decoding: one cache per layer, all over the same pool and table
    caches = [kvx.Cache(pool, addr, heads, dim, act, page, first_lane=2 * heads * i) for i in range(layers)]
    q_heads, length = heads * group, prompt_blocks * page
    table = torch.arange(prompt_blocks + more, dtype=torch.int32, device=dev)[None]
    lens = torch.tensor([length], dtype=torch.int32, device=dev)
    scores = torch.zeros(layers, 1, heads, table.shape[1] * page, device=dev)
    angle = torch.arange(length + steps, dtype=torch.float64, device=dev)[:, None] * 10000.0 ** (
        -torch.arange(0, dim, 2, dtype=torch.float64, device=dev) / dim)
    cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    weight = torch.ones(2, dim, dtype=act, device=dev)
    out = torch.empty(layers, 1, q_heads, dim, dtype=act, device=dev)
    ws = caches[0].attend_workspace(1, q_heads, table.shape[1], scores=True)
    for step in range(steps):
        position = torch.tensor([length + step], dtype=torch.int32, device=dev)
        slot = torch.tensor([int(table[0, (length + step) // page]) * page + (length + step) % page], device=dev)
        lens += 1
        for i, cache in enumerate(caches):
            qkv = torch.randn(1, (q_heads + 2 * heads) * dim, generator=gen, device=dev).to(act)
            q, k, v = (x.unflatten(1, (-1, dim)) for x in qkv.split([q_heads * dim, heads * dim, heads * dim], dim=1))
            cache.append(q, k, v, position, slot, q, q_weight=weight[0], k_weight=weight[1], cos_sin=cos_sin)
            cache.attend(q, table, lens, out[i], ws, scores=scores[i])

    # ---- eviction: every head of every layer keeps what it has attended to
    dst = torch.arange(prompt_blocks + more, blocks, dtype=torch.int32, device=dev)[None]
    kept = torch.empty(layers, 1, heads, budget, dtype=torch.int32, device=dev)
    weights = torch.empty(layers, 1, heads, budget, device=dev)
    new_lens = torch.empty(1, dtype=torch.int32, device=dev)
    for i, cache in enumerate(caches):
        cache.evict(table, lens, scores[i], dst, kept[i], weights[i], new_lens,
                    cache.evict_workspace(1, table.shape[1], budget), sinks=4, recent=32)
        cache.attend(q, dst, new_lens, out[i], ws)
    torch.cuda.synchronize()
    assert all(cache.read_status() == 0 for cache in caches)

    # ---- the last attention, plainly, over the tokens that the last layer's heads kept
    rows = pool.view(act).view(-1, dim)
    at = kept[-1, 0].long()  # [heads, budget] tokens of the old pages
    lane = 2 * heads * (layers - 1) + 2 * torch.arange(heads, device=dev)[:, None]
    block = table[0].long()[at // page]
    k, v = (rows[addr[block, lane + kv] // (2 * dim) + at % page].double() for kv in (0, 1))
    p = (q.double().view(heads, group, dim) @ k.transpose(1, 2) / math.sqrt(dim)).softmax(-1)
    error = float((out[-1].double().view(heads, group, dim) - p @ v).abs().max())
    if verbose:
        print("%d blocks transferred, %d steps x %d layers, %d -> %d tokens a head, largest error %.4f" % (
            prompt_blocks, steps, layers, int(lens), int(new_lens), error))
    return error


if __name__ == "__main__":
    main()
