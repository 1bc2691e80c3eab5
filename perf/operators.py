"""Cases that time the cache operators of libkvx: appending tokens to a paged cache, attending over it with one new
token per sequence, and evicting tokens by accumulated attention weight.

The cache is the one that the block transfer fills: pages ("blocks") whose K and V segments of every head lie wherever
the address table ``addr[block, 2 * head + kv]`` says, in bytes from the pool's start.  ``own`` selects the library's
kernels; otherwise every operator is computed in its plain form, elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}
STORE = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _append(name, tokens, q_heads, heads, dim, page, act="bf16", store="bf16", rot=None, pairs="halves", norm=True,
            layout="head"):
    c = {"op": "append", "tokens": tokens, "q_heads": q_heads, "heads": heads, "dim": dim, "page": page, "act": act,
         "store": store, "rot": dim if rot is None else rot, "pairs": pairs, "norm": norm, "layout": layout}
    return {"name": name, **c} if name else c


def _attend(name, seqs, short, long, q_heads, heads, dim, page, act="bf16", store="bf16", window=0, sinks=0, empty=0,
            scores=False, layout="head"):
    c = {"op": "attend", "seqs": seqs, "short": short, "long": long, "empty": empty, "q_heads": q_heads, "heads": heads,
         "dim": dim, "page": page, "act": act, "store": store, "window": window, "sinks": sinks, "scores": scores,
         "layout": layout}
    return {"name": name, **c} if name else c


def _evict(name, seqs, short, long, budget, sinks, recent, heads, dim, page, store="bf16", layout="head"):
    c = {"op": "evict", "seqs": seqs, "short": short, "long": long, "budget": budget, "sinks": sinks, "recent": recent,
         "heads": heads, "dim": dim, "page": page, "store": store, "layout": layout}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One sequence decodes: the new token of one layer goes into a 4 KiB segment (16 tokens x 128 x 2 bytes).
        _append("append one token", 1, 32, 8, 128, 16),
        # A serving batch decodes into an 8-bit cache, each token into a page of another sequence.
        _append("append a batch, 8-bit cache", 200, 64, 8, 128, 64, store="e4m3"),
        # A prompt of the default transfer's 1000 blocks of 16 tokens.
        _append("append a prompt", 16000, 32, 8, 128, 16),
        # A ragged chunk of a prompt: heads of 96, a part of each rotated in neighbouring pairs, token-major pages.
        _append("append a ragged chunk", 4999, 24, 6, 96, 24, act="fp16", store="fp16", rot=64, pairs="neighbours",
                layout="token"),
        # A chat's first answer tokens: latency counts.
        _attend("attend, one short", 1, 77, 77, 32, 8, 128, 16),
        # One long document: all of the card for one sequence.
        _attend("attend, one long", 1, 131071, 131071, 32, 8, 128, 16),
        # Eight sequences of the default transfer's 16,000 tokens.
        _attend("attend, transferred prefixes", 8, 16000, 16000, 32, 8, 128, 16),
        # A ragged serving batch with an 8-bit cache, some of its places not in use.
        _attend("attend, ragged batch, 8-bit", 96, 30, 8192, 64, 8, 128, 64, store="e4m3", empty=5),
        # Streaming: long histories of which the last 4096 tokens and four first ones stay visible.
        _attend("attend, window and sinks", 48, 100, 40000, 64, 8, 64, 32, act="fp16", store="fp16", window=4096, sinks=4),
        # The step before an eviction: attention weights are added up per head and token.
        _attend("attend, weights added up", 32, 1000, 6001, 40, 8, 128, 16, scores=True),
        # One sequence over its budget.
        _evict("evict one", 1, 1500, 1500, 512, 4, 128, 8, 128, 16),
        # A batch of long sequences cut to 4096 tokens a head; the short ones stay whole.
        _evict("evict a batch", 24, 2000, 40000, 4096, 4, 512, 8, 128, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    act = rng.choice(["bf16", "bf16", "fp16"])
    store = rng.choice([act, act, "e4m3"])
    dim = rng.choice([64, 96, 128, 128, 128, 256])
    heads = rng.choice([1, 2, 4, 6, 8, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([2, 16, 16, 24, 32, 64, 256])
    layout = rng.choice(["head", "head", "token"])
    op = rng.choice(["append", "attend", "attend", "evict"])
    if op == "append":
        most = max(2, int(16000 * 48 * 128 / ((group + 2) * heads * dim)))
        return _append(None, _log(rng, 1, min(16000, most)), group * heads, heads, dim, page, act, store,
                       rng.choice([dim, dim, 32]), rng.choice(["halves", "neighbours"]), rng.random() < 0.8, layout)
    # at most about the cached values of the largest listed cases
    values = _log(rng, 1000, 120_000_000)
    tokens = max(2, values // (heads * dim))
    seqs = min(tokens, _log(rng, 1, 128))
    long = max(2, min(131071, tokens // seqs))
    short = max(1, int(long * rng.choice([1.0, 0.5, 0.03])))
    if op == "attend":
        window = rng.choice([0, 0, 1, _log(rng, 1, 8192)])
        return _attend(None, seqs, short, long, group * heads, heads, dim, page, act, store, window,
                       rng.choice([0, 1, 4, 64]) if window else 0, rng.choice([0, 0, 1]) if seqs > 1 else 0,
                       rng.random() < 0.3, layout)
    budget = max(1, int(long * rng.choice([0.05, 0.2, 0.5])))
    return _evict(None, seqs, short, long, budget, min(budget // 8, 4), budget // rng.choice([2, 4, 8]), heads, dim,
                  page, store, layout)


def _lens(case):
    """The sequences' lengths in no particular order: spread between the shortest and the longest, the empty ones first."""
    n, empty = case["seqs"], case.get("empty", 0)
    m = n - empty
    ratio = case["long"] / case["short"]
    lens = [int(round(case["short"] * ratio ** ((i + 1) / m))) for i in range(m)]
    return [0] * empty + lens


def _visible(length, window, sinks):
    return length if not window else min(length, min(sinks, length) + window)


def work(case):
    h, d, es = case["heads"], case["dim"], SIZE[case["store"]]
    if case["op"] == "append":
        t, hq = case["tokens"], case["q_heads"]
        rows_in, rot = hq + 2 * h, case["rot"]
        return {"bytes": t * d * (2 * rows_in + 2 * hq + 2 * h * es) + t * (4 * rot + 12),
                "flops": t * (hq + h) * (4 * d * case["norm"] + 3 * rot)}
    lens = _lens(case)
    if case["op"] == "attend":
        hq = case["q_heads"]
        keys = sum(_visible(n, case["window"], case["sinks"]) for n in lens)
        table = sum(-(-_visible(n, case["window"], case["sinks"]) // case["page"]) for n in lens) * (4 + 16 * h)
        return {"bytes": keys * h * (2 * d * es + 8 * case["scores"]) + len(lens) * hq * (4 * d + 4) + table,
                "flops": 4 * keys * hq * d}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": sum(lens) * h * 4 + kept * h * (4 * d * es + 8), "flops": sum(lens) * h}


# ------------------------------------------------------------------ inputs

def _fill(values, dtype, gen):
    """Normal values of the given type, made a part at a time."""
    pool = torch.empty(values, dtype=dtype, device="cuda")
    step = 1 << 26
    for a in range(0, values, step):
        n = min(step, values - a)
        pool[a:a + n] = torch.randn(n, generator=gen, device="cuda").to(dtype)
    return pool


def _cache(case, blocks, gen):
    """A pool of `blocks` pages in shuffled places, and its address table [blocks, 2 * heads] in bytes."""
    h, page, row = case["heads"], case["page"], case["dim"] * SIZE[case["store"]]
    pool = _fill(blocks * 2 * h * page * case["dim"], STORE[case["store"]], gen).view(torch.uint8)
    at = torch.randperm(blocks, generator=gen, device="cuda")[:, None] * (2 * h * page * row)
    lane = torch.arange(2 * h, device="cuda")[None, :]
    if case["layout"] == "head":  # a head's tokens together
        return pool, at + lane * (page * row), row
    head, kv = lane // 2, lane % 2  # a token's heads together
    return pool, at + kv * (h * page * row) + head * row, h * row


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h, d, page = case["heads"], case["dim"], case["page"]
    s = {"case": case}
    # k_scale and v_scale stand for an 8-bit cache's calibrated scales
    s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if case["store"] == "e4m3" else (1.0, 1.0)
    if case["op"] == "append":
        t, hq, act = case["tokens"], case["q_heads"], ACT[case["act"]]
        blocks = -(-t // page) + 3
        s["pool"], s["addr"], s["stride"] = _cache(case, blocks, gen)
        # q, k and v are parts of one projection's output
        qkv = torch.randn(t, (hq + 2 * h) * d, generator=gen, device="cuda").to(act)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, h * d, h * d], dim=1))
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (1 + 0.1 * torch.randn(2, d, generator=gen, device="cuda")).to(act)
        most = 32768
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        first = random.Random(seed).randrange(most - t)
        s["positions"] = torch.arange(first, first + t, dtype=torch.int32, device="cuda")
        s["slots"] = torch.randperm(blocks, generator=gen, device="cuda")[:, None] * page + torch.arange(page, device="cuda")
        s["slots"] = s["slots"].reshape(-1)[:t].contiguous()
        if t >= 100:  # a batch is padded now and then
            s["slots"][t // 2] = -1
        s["q_out"] = torch.empty(t, hq, d, dtype=act, device="cuda")
    else:
        lens = _lens(case)
        random.Random(seed).shuffle(lens)
        per = max(1, -(-max(lens) // page))
        need = [-(-n // page) for n in lens]
        extra = -(-case["budget"] // page) * len(lens) if case["op"] == "evict" else 0
        s["pool"], s["addr"], s["stride"] = _cache(case, sum(need) + extra, gen)
        ids = torch.randperm(sum(need) + extra, generator=gen, device="cuda").to(torch.int32)
        starts = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
        col = torch.arange(per, device="cuda")
        used = col[None, :] < torch.tensor(need, device="cuda")[:, None]
        s["blocks"] = torch.where(used, ids[(starts[:, None] + col).clamp(max=len(ids) - 1)], 0).to(torch.int32)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        n, s["most"] = len(lens), per * page
        if case["op"] == "attend":
            hq, act = case["q_heads"], ACT[case["act"]]
            spread = 2.0 / s["k_scale"]  # logits spread as after a norm of queries and keys
            s["q"] = (spread * torch.randn(n, hq, d, generator=gen, device="cuda")).to(act)
            s["out"] = torch.empty(n, hq, d, dtype=act, device="cuda")
            s["lse"] = torch.empty(n, hq, device="cuda")
            s["scores"] = torch.rand(n, h, s["most"], generator=gen, device="cuda") if case["scores"] else None
        else:
            budget = case["budget"]
            s["dst_blocks"] = ids[sum(need):].view(n, -1).contiguous()
            # a few tokens gather most of the weight
            s["scores"] = torch.randn(n, h, s["most"], generator=gen, device="cuda").mul_(2).exp_()
            s["kept"] = torch.empty(n, h, budget, dtype=torch.int32, device="cuda")
            s["kept_scores"] = torch.empty(n, h, budget, device="cuda")
            s["new_lens"] = torch.empty(n, dtype=torch.int32, device="cuda")
    if own:
        from paged_kv_cache_kvx_gb300 import kvx
        s["cache"] = kvx.Cache(s["pool"], s["addr"], heads=h, dim=d, dtype=STORE[case["store"]], page_tokens=page,
                               token_stride=s["stride"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if case["op"] == "attend":
            s["ws"] = s["cache"].attend_workspace(n, hq, per, window=case["window"], sinks=case["sinks"],
                                                  scores=case["scores"])
        elif case["op"] == "evict":
            s["ws"] = s["cache"].evict_workspace(n, per, case["budget"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_append(s):
    c = s["case"]
    s["cache"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], q_weight=s["q_weight"],
                      k_weight=s["k_weight"], eps=1e-6, cos_sin=s["cos_sin"], interleaved=c["pairs"] == "neighbours")
    return s["q_out"], s["pool"].view(STORE[c["store"]])


def _own_attend(s):
    c = s["case"]
    s["cache"].attend(s["q"], s["blocks"], s["lens"], s["out"], s["ws"], window=c["window"], sinks=c["sinks"],
                      lse=s["lse"], scores=s["scores"])
    return s["out"], s["lse"], s["scores"]


def _own_evict(s):
    c = s["case"]
    s["cache"].evict(s["blocks"], s["lens"], s["scores"], s["dst_blocks"], s["kept"], s["kept_scores"], s["new_lens"],
                     s["ws"], sinks=c["sinks"], recent=c["recent"])
    return s["kept"], s["kept_scores"], s["new_lens"], s["pool"].view(STORE[c["store"]])


_own = {"append": _own_append, "attend": _own_attend, "evict": _own_evict}


def _rows(s):
    """The cache as rows of one head's token, in the bytes' own type."""
    c = s["case"]
    return s["pool"].view(torch.uint8 if c["store"] == "e4m3" else STORE[c["store"]]).view(-1, c["dim"])


def _row_of(s, block, offset):
    """Row numbers [..., 2 * heads] of tokens at an offset of a block."""
    row = s["case"]["dim"] * SIZE[s["case"]["store"]]
    return (s["addr"][block] + (offset * s["stride"])[..., None]) // row


def _stored(s, x, scale):
    """Values as the cache holds them, in the type of _rows."""
    if s["case"]["store"] != "e4m3":
        return x.to(STORE[s["case"]["store"]])
    return (x / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _loaded(s, rows, scale):
    if s["case"]["store"] == "e4m3":
        rows = rows.view(torch.float8_e4m3fn)
    return rows.float() * scale


def _normed(x, weight, eps=1e-6):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()


def _rotated(x, cos, sin, pairs):
    """Rotates the first 2 * cos.shape[-1] values of each head."""
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "halves":
        a, b, rest = x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)
    a, b, rest = x[..., :rot:2], x[..., 1:rot:2], x[..., rot:]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), rest], dim=-1)


def _plain_append(s):
    c = s["case"]
    cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, dim=1)
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["pairs"]))
    k = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c["pairs"])
    slots = s["slots"]
    spare = slots.amax()  # a token without a place writes what the last place gets
    put = torch.where(slots < 0, spare, slots)
    take = torch.where(slots < 0, slots.argmax(), torch.arange(len(slots), device=slots.device))
    at = _row_of(s, put // c["page"], put % c["page"])
    rows = _rows(s)
    rows[at[:, 0::2]] = _stored(s, k[take], s["k_scale"])
    rows[at[:, 1::2]] = _stored(s, s["v"][take].float(), s["v_scale"])
    return s["q_out"], s["pool"].view(STORE[c["store"]])


def _plain_attend(s):
    c = s["case"]
    n, h, d = c["seqs"], c["heads"], c["dim"]
    lens, at = s["lens"].long()[:, None], torch.arange(s["most"], device="cuda")[None, :]
    seen = at < lens
    if c["window"]:
        seen = seen & ((at >= lens - c["window"]) | (at < c["sinks"]))
    block = s["blocks"].long()[:, torch.arange(s["most"], device="cuda") // c["page"]]
    rows, row = _rows(s), _row_of(s, block, (at % c["page"]).expand(n, -1))
    k = _loaded(s, rows[row[..., 0::2]], s["k_scale"]).permute(0, 2, 3, 1)  # [n, h, d, most]
    q = s["q"].float().view(n, h, -1, d)
    logits = (q @ k) * d ** -0.5
    del k
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = (logits - top).exp()
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    v = _loaded(s, rows[row[..., 1::2]], s["v_scale"])
    v = torch.where(seen[:, :, None, None], v, torch.zeros_like(v)).permute(0, 2, 1, 3)  # [n, h, most, d]
    s["out"].copy_((p @ v).view(n, -1, d))
    s["lse"].copy_((top + total.log()).view(n, -1))
    if s["scores"] is not None:
        s["scores"] += p.sum(2)
    return s["out"], s["lse"], s["scores"]


def _plain_evict(s):
    c = s["case"]
    n, h, budget, most = c["seqs"], c["heads"], c["budget"], s["most"]
    lens, at = s["lens"].long()[:, None], torch.arange(most, device="cuda")[None, :]
    sinks = min(c["sinks"], budget)
    recent = min(c["recent"], budget - sinks)
    # first the tokens that stay in any case, then by weight, ties to the lowest index
    stays = (at < sinks) | (at >= lens - recent)
    rank = torch.where(stays[:, None], math.inf, s["scores"])
    rank = torch.where((at < lens)[:, None], rank, -math.inf)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    width = best.shape[-1]
    new = lens.clamp(max=budget)
    used = torch.arange(budget, device="cuda")[None, :] < new
    kept = torch.where(used[:, None, :width], best, most).sort(dim=-1).values
    kept = torch.nn.functional.pad(kept, (0, budget - width), value=most)
    safe = torch.where(used[:, None], kept, 0)
    s["kept"].copy_(torch.where(used[:, None], kept, -1))
    s["kept_scores"].copy_(torch.where(used[:, None], s["scores"].gather(2, safe), 0))
    s["new_lens"].copy_(new[:, 0])
    lane = torch.arange(h, device="cuda")[None, :, None] * 2
    block = s["blocks"].long()[torch.arange(n, device="cuda")[:, None, None], safe // c["page"]]
    row = c["dim"] * SIZE[c["store"]]
    src = (s["addr"][block, lane] + safe % c["page"] * s["stride"]) // row
    src_v = (s["addr"][block, lane + 1] + safe % c["page"] * s["stride"]) // row
    to = torch.arange(budget, device="cuda")[None, None, :].expand(n, h, -1)
    block = s["dst_blocks"].long()[torch.arange(n, device="cuda")[:, None, None], to // c["page"]]
    dst = (s["addr"][block, lane] + to % c["page"] * s["stride"]) // row
    dst_v = (s["addr"][block, lane + 1] + to % c["page"] * s["stride"]) // row
    rows, here = _rows(s), used[:, None].expand(-1, h, -1)
    rows[torch.cat([dst[here], dst_v[here]])] = rows[torch.cat([src[here], src_v[here]])]
    return s["kept"], s["kept_scores"], s["new_lens"], s["pool"].view(STORE[c["store"]])


_plain = {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](prepare(case, seed))


def _places(s, block_ids, lane, offsets):
    """First element of each token's row in the pool, counted in values."""
    return (s["addr"][block_ids.long(), lane] + offsets * s["stride"]) // SIZE[s["case"]["store"]]


def _exact_append(s):
    c = s["case"]
    d, half, t = c["dim"], c["rot"] // 2, c["tokens"]
    # element i of a rotated head mixes with element partner[i], which enters with the given sign
    i = torch.arange(d, device="cuda")
    if c["pairs"] == "halves":
        partner, angle = torch.where(i < half, i + half, i - half), i % half
        sign = torch.where(i < half, -1.0, 1.0).double()
    else:
        partner, angle = i ^ 1, i // 2
        sign = torch.where(i % 2 == 0, -1.0, 1.0).double()
    turned = i < c["rot"]
    partner, angle = torch.where(turned, partner, i), torch.where(turned, angle, 0)
    table = s["cos_sin"].double()[s["positions"].long()]
    cos = torch.where(turned, table[:, angle], 1.0)
    sin = torch.where(turned, table[:, half + angle] * sign, 0.0)

    def head(x, weight):
        x = x.double()
        if weight is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * weight.double()
        return x * cos[:, None] + x[..., partner] * sin[:, None]

    pool = s["pool"].view(STORE[c["store"]]).double()
    has = s["slots"] >= 0
    slot = s["slots"][has]
    k, v = head(s["k"], s["k_weight"])[has] / s["k_scale"], s["v"].double()[has] / s["v_scale"]
    if c["store"] == "e4m3":
        k, v = k.clamp(-E4M3_MAX, E4M3_MAX), v.clamp(-E4M3_MAX, E4M3_MAX)
    for j in range(c["heads"]):
        for kv, x in ((0, k), (1, v)):
            at = _places(s, slot // c["page"], 2 * j + kv, slot % c["page"])
            pool[at[:, None] + i] = x[:, j]
    return head(s["q"], s["q_weight"]), pool


def _exact_attend(s):
    c = s["case"]
    g, d = c["q_heads"] // c["heads"], c["dim"]
    pool = s["pool"].view(STORE[c["store"]])
    out = torch.zeros(c["seqs"], c["q_heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if s["scores"] is not None else None
    elements = torch.arange(d, device="cuda")
    for n, length in enumerate(s["lens"].tolist()):
        pos = torch.arange(length, device="cuda")
        if c["window"]:
            pos = torch.cat([pos[:c["sinks"]], pos[max(min(c["sinks"], length), length - c["window"]):]])
        if not len(pos):
            continue
        for j in range(c["heads"]):
            block = s["blocks"][n][pos // c["page"]]
            k, v = (pool[_places(s, block, 2 * j + kv, pos % c["page"])[:, None] + elements] if c["store"] != "e4m3" else
                    s["pool"][_places(s, block, 2 * j + kv, pos % c["page"])[:, None] + elements].view(torch.float8_e4m3fn)
                    for kv in (0, 1))
            heads = slice(j * g, (j + 1) * g)
            x = (s["q"][n, heads].double() @ k.double().T) * (s["k_scale"] / math.sqrt(d))
            lse[n, heads] = torch.logsumexp(x, dim=1)
            p = (x - lse[n, heads, None]).exp()
            out[n, heads] = (p @ v.double()) * s["v_scale"]
            if scores is not None:
                scores[n, j, pos] += p.sum(0)
    return out, lse, scores


def _exact_evict(s):
    c = s["case"]
    n, h, budget = c["seqs"], c["heads"], c["budget"]
    sinks = min(c["sinks"], budget)
    recent = min(c["recent"], budget - sinks)
    kept = torch.full((n, h, budget), -1, dtype=torch.int32, device="cuda")
    kept_scores = torch.zeros(n, h, budget, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    pool = s["pool"].view(torch.uint8 if c["store"] == "e4m3" else STORE[c["store"]])
    after, elements = pool.clone(), torch.arange(c["dim"], device="cuda")
    for i in range(n):
        m = min(lens[i], budget)
        to = torch.arange(m, device="cuda")
        for j in range(h):
            weight = s["scores"][i, j, :lens[i]]
            if lens[i] > budget:
                middle = weight[sinks:lens[i] - recent].double()
                take = budget - sinks - recent
                cut = torch.sort(middle, descending=True).values[take - 1] if take else math.inf
                over = middle > cut
                ties = (middle == cut).nonzero()[:, 0][:take - int(over.sum())]
                chosen = torch.cat([over.nonzero()[:, 0], ties]).sort().values + sinks
                tail = torch.arange(lens[i] - recent, lens[i], device="cuda")
                pos = torch.cat([torch.arange(sinks, device="cuda"), chosen, tail])
            else:
                pos = to
            kept[i, j, :m] = pos.int()
            kept_scores[i, j, :m] = weight[pos].double()
            for kv in (0, 1):
                src = _places(s, s["blocks"][i][pos // c["page"]], 2 * j + kv, pos % c["page"])
                dst = _places(s, s["dst_blocks"][i][to // c["page"]], 2 * j + kv, to % c["page"])
                after[dst[:, None] + elements] = pool[src[:, None] + elements]
    return kept, kept_scores, s["lens"].clamp(max=budget), after.view(STORE[c["store"]]).double()
