"""Cases that time further cache operators of libkvx: appending tokens to a cache of 8-bit rows that carry a scale each,
reading tokens of a paged cache back into dense 16-bit tensors, and attending with a batch whose sequences share
prefixes.

The cache is the one that the block transfer fills: the K and V segments of every head of a page ("block") lie wherever
the address table ``addr[block, 2 * head + kv]`` says, in bytes from the pool's start.  Types: bf16, fp16, "e4m3" with
one scale for all keys and one for all values, and "rows": e4m3 with a power of two for each row (one token of one
head), whose exponents lie behind the rows of their segment and so travel with it.  ``own`` selects the library's
kernels; otherwise every operator is computed in its plain form, elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}
STORE = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "rows": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1, "rows": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _append(name, tokens, q_heads, heads, dim, page, act="bf16", rot=None, pairs="halves", norm=True, layout="head"):
    c = {"op": "append", "tokens": tokens, "q_heads": q_heads, "heads": heads, "dim": dim, "page": page, "act": act,
         "store": "rows", "rot": dim if rot is None else rot, "pairs": pairs, "norm": norm, "layout": layout}
    return {"name": name, **c} if name else c


def _read(name, seqs, short, long, skip, heads, dim, page, act="bf16", store="bf16", layout="head"):
    c = {"op": "read", "seqs": seqs, "short": short, "long": long, "skip": skip, "heads": heads, "dim": dim, "page": page,
         "act": act, "store": store, "layout": layout}
    return {"name": name, **c} if name else c


def _shared(name, seqs, groups, alone, prefix_short, prefix_long, short, long, q_heads, heads, dim, page, act="bf16",
            store="bf16", empty=0, layout="head"):
    c = {"op": "shared", "seqs": seqs, "groups": groups, "alone": alone, "prefix_short": prefix_short,
         "prefix_long": prefix_long, "short": short, "long": long, "empty": empty, "q_heads": q_heads, "heads": heads,
         "dim": dim, "page": page, "act": act, "store": store, "layout": layout}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One sequence decodes into a quantised cache: latency counts.
        _append("write one token", 1, 32, 8, 128, 16),
        # A serving batch decodes, each token into a page of another sequence.
        _append("write a batch", 200, 64, 8, 128, 64),
        # A prompt of the default transfer's 1000 blocks of 16 tokens.
        _append("write a prompt", 16000, 32, 8, 128, 16),
        # A ragged chunk of a prompt: heads of 96, a part of each rotated in neighbouring pairs, token-major pages.
        _append("write a ragged chunk", 4999, 24, 6, 96, 24, act="fp16", rot=64, pairs="neighbours", layout="token"),
        # A short prompt is read back for the next chunk's attention.
        _read("read one short", 1, 77, 77, 0, 8, 128, 16, store="rows"),
        # Eight transferred prefixes of 16,000 tokens, quantised, read back whole.
        _read("read transferred prefixes", 8, 16000, 16000, 0, 8, 128, 16, store="rows"),
        # A ragged batch of 16-bit histories, each read from some token on; token-major pages of 24, heads of 96.
        _read("read a ragged batch", 37, 100, 8000, 50, 6, 96, 24, act="fp16", store="fp16", layout="token"),
        # A few chats behind one short system prompt: latency counts.
        _shared("attend, short prefix", 4, 1, 0, 500, 500, 20, 60, 32, 8, 128, 16),
        # A serving batch behind one transferred prefix.
        _shared("attend, transferred prefix", 64, 1, 0, 16000, 16000, 16, 1000, 32, 8, 128, 16),
        # Many questions about one long document: the queries of a KV head fill the tensor cores.
        _shared("attend, one long document", 128, 1, 0, 100000, 100000, 30, 300, 64, 8, 128, 16),
        # Several system prompts of different lengths in a quantised cache; some sequences have none, some are padding.
        _shared("attend, several prefixes", 96, 6, 7, 1500, 16000, 30, 2000, 64, 8, 128, 64, store="rows", empty=3),
        # Plain decoding over a quantised cache, no two sequences alike; fp16, heads of 64, pages of 32.
        _shared("attend, nothing shared", 48, 0, 48, 0, 0, 100, 8000, 64, 8, 64, 32, act="fp16", store="rows"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    act = rng.choice(["bf16", "bf16", "fp16"])
    store = rng.choice([act, "rows", "rows", "e4m3"])
    dim = rng.choice([64, 96, 128, 128, 128, 256])
    heads = rng.choice([1, 2, 4, 6, 8, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    page = rng.choice([2, 16, 16, 24, 32, 64])
    layout = rng.choice(["head", "head", "token"])
    op = rng.choice(["append", "read", "shared", "shared"])
    if op == "append":
        most = max(2, int(16000 * 48 * 128 / ((group + 2) * heads * dim)))
        return _append(None, _log(rng, 1, min(16000, most)), group * heads, heads, dim, page, act,
                       rng.choice([dim, dim, 32]), rng.choice(["halves", "neighbours"]), rng.random() < 0.8, layout)
    if op == "read":
        values = _log(rng, 1000, 120_000_000)
        tokens = max(2, values // (heads * dim))
        seqs = min(tokens, _log(rng, 1, 128))
        long = max(2, min(131071, tokens // seqs))
        short = max(1, int(long * rng.choice([1.0, 0.5, 0.03])))
        return _read(None, seqs, short, long, rng.choice([0, 0, short // 2]), heads, dim, page, act, store, layout)
    seqs = _log(rng, 1, 256)
    groups = min(seqs, rng.choice([0, 1, 1, 1, 2, 5, 12]))
    # at most the multiplications and the cached values of the largest listed cases
    prefix = min(_log(rng, 100, 131071), max(1, int(128 * 64 * 100_000 * 128 // (seqs * group * heads * dim))),
                 max(1, 100_000_000 // (max(1, groups) * heads * dim)))
    long = max(1, min(_log(rng, 1, 8000), 120_000_000 // (seqs * heads * dim)))
    short = max(1, int(long * rng.choice([1.0, 0.3, 0.03])))
    alone = seqs if not groups else rng.choice([0, 0, (seqs - groups) // 4])
    return _shared(None, seqs, groups, alone, max(1, int(prefix * rng.choice([1.0, 0.2]))) if groups else 0,
                   prefix if groups else 0, short, long, group * heads, heads, dim, page, act, store,
                   rng.choice([0, 0, 1]) if seqs > 1 else 0, layout)


def _spread(n, short, long):
    """n lengths between the shortest and the longest."""
    return [int(round(short * (long / short) ** ((i + 1) / n))) for i in range(n)]


def _lens(case):
    """The sequences' own lengths in no particular order, the empty ones first."""
    empty = case.get("empty", 0)
    return [0] * empty + _spread(case["seqs"] - empty, case["short"], case["long"])


def _prefixes(case):
    return _spread(case["groups"], case["prefix_short"], case["prefix_long"]) if case["groups"] else []


def _sizes(case):
    """Sequences of each group: equal shares with a ragged end."""
    n, g = case["seqs"] - case["alone"], case["groups"]
    return [n * (i + 1) // g - n * i // g for i in range(g)]


def work(case):
    h, d, es = case["heads"], case["dim"], SIZE[case["store"]]
    row = d * es + (case["store"] == "rows")  # bytes of a token's key or value in one head
    if case["op"] == "append":
        t, hq, rot = case["tokens"], case["q_heads"], case["rot"]
        return {"bytes": t * d * (2 * (hq + 2 * h) + 2 * hq) + t * 2 * h * row + t * (4 * rot + 12),
                "flops": t * (hq + h) * (4 * d * case["norm"] + 3 * rot) + t * 2 * h * d * 3}
    if case["op"] == "read":
        tokens = sum(n - case["skip"] for n in _lens(case))
        pages = sum(-(-n // case["page"]) - case["skip"] // case["page"] for n in _lens(case))
        return {"bytes": tokens * 2 * h * (row + 2 * d) + pages * (4 + 16 * h), "flops": tokens * 2 * h * d * (es == 1)}
    hq, lens, prefixes = case["q_heads"], _lens(case), _prefixes(case)
    keys = sum(lens) + sum(prefixes)
    pages = sum(-(-n // case["page"]) for n in lens + prefixes)
    products = sum(lens) + sum(n * p for n, p in zip(_sizes(case), prefixes))
    return {"bytes": keys * h * 2 * row + pages * (4 + 16 * h) + len(lens) * hq * (4 * d + 4), "flops": 4 * products * hq * d}


# ------------------------------------------------------------------ inputs

def _layout(case):
    """Bytes of a page's K and V segments together, of a token's distance to the next, and of its scale's place in a
    segment (0 for none), and the segments' offsets [2 * heads] within the page."""
    h, page, row = case["heads"], case["page"], case["dim"] * SIZE[case["store"]]
    rows = case["store"] == "rows"
    lane = torch.arange(2 * h, device="cuda")
    if case["layout"] == "head" or page > case["dim"]:  # a head's tokens together, their scales behind them
        seg = page * row + (-(-page // 16) * 16 if rows else 0)
        return 2 * h * seg, row, page * row if rows else 0, lane * seg
    # a token's heads together; the scales take the place of one more token
    tokens = page + rows
    head, kv = lane // 2, lane % 2
    return 2 * h * tokens * row, h * row, page * h * row if rows else 0, kv * (h * tokens * row) + head * row


def _cache(s, case, blocks, gen):
    """A pool of `blocks` pages in shuffled places, and its address table [blocks, 2 * heads] in bytes."""
    size, stride, scales, lanes = _layout(case)
    h, d, page, es = case["heads"], case["dim"], case["page"], SIZE[case["store"]]
    at = torch.randperm(blocks, generator=gen, device="cuda")[:, None] * size
    pool = torch.empty(blocks * size, dtype=torch.uint8, device="cuda")
    step = 1 << 26
    for a in range(0, len(pool) // es, step):  # normal values, made a part at a time
        n = min(step, len(pool) // es - a)
        pool.view(STORE[case["store"]])[a:a + n] = torch.randn(n, generator=gen, device="cuda").mul_(
            64 if scales else 1).to(STORE[case["store"]])
    s["pool"], s["addr"], s["stride"], s["scale_offset"] = pool, (at + lanes).contiguous(), stride, scales
    # k_scale and v_scale stand for an 8-bit cache's calibrated scales
    s["k_scale"], s["v_scale"] = (0.0625, 0.03125) if case["store"] == "e4m3" else (1.0, 1.0)
    if scales:  # about unit values; now and then a row is larger or smaller
        exps = torch.randn(blocks, 2 * h, page, generator=gen, device="cuda").mul_(0.7).round_().add_(127 - 6)
        pool[(s["addr"][:, :, None] + scales + torch.arange(page, device="cuda"))] = exps.to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    h, d, page, act = case["heads"], case["dim"], case["page"], ACT[case["act"]]
    s = {"case": case}
    if case["op"] == "append":
        t, hq = case["tokens"], case["q_heads"]
        blocks = -(-t // page) + 3
        _cache(s, case, blocks, gen)
        # q, k and v are parts of one projection's output; some tokens' values are larger than others'
        qkv = torch.randn(t, (hq + 2 * h) * d, generator=gen, device="cuda")
        qkv = (qkv * torch.randn(t, 1, generator=gen, device="cuda").exp()).to(act)
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
        # the cache as a reader sees it: rows and their scales, by block and lane
        size, at = _layout(case)[0], _layout(case)[3]
        whole = s["pool"].view(blocks, size)
        if case["layout"] == "head" or page > d:
            segs = whole.view(blocks, 2 * h, -1)
            s["rows"], s["scales"] = segs[:, :, :page * d].unflatten(2, (page, d)), segs[:, :, page * d:page * d + page]
        else:
            segs = whole.view(blocks, 2, page + 1, h, d)
            s["rows"], s["scales"] = segs[:, :, :page], segs[:, :, page, :, :page]
        s["rows"], s["scales"] = s["rows"].view(torch.float8_e4m3fn), s["scales"].view(torch.float8_e8m0fnu)
    else:
        lens = _lens(case)
        random.Random(seed).shuffle(lens)
        n, per = len(lens), max(1, -(-max(lens) // page))
        prefixes = _prefixes(case) if case["op"] == "shared" else []
        need = [-(-x // page) for x in lens + prefixes]
        _cache(s, case, max(1, sum(need)), gen)
        ids = torch.randperm(max(1, sum(need)), generator=gen, device="cuda").to(torch.int32)

        def table(rows, first, width):
            starts = torch.tensor([sum(need[:first + i]) for i in range(rows)], dtype=torch.int64, device="cuda")
            used = torch.tensor(need[first:first + rows], dtype=torch.int64, device="cuda")
            col = torch.arange(width, device="cuda")
            got = torch.where(col < used[:, None], ids[(starts[:, None] + col).clamp(max=len(ids) - 1)], 0)
            return got.to(torch.int32)

        s["blocks"], s["most"] = table(n, 0, per), per * page
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if case["op"] == "read":
            starts = [0]
            for x in lens:
                starts.append(starts[-1] + x - case["skip"])
            s["first"] = torch.full((n,), case["skip"], dtype=torch.int32, device="cuda") if case["skip"] else None
            s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
            rows = starts[-1] + (-starts[-1]) % 64  # a captured batch is padded
            s["k_out"], s["v_out"] = torch.randn(2, rows, h, d, generator=gen, device="cuda").to(act)
        else:
            hq, groups = case["q_heads"], case["groups"]
            spread = 2.0 / s["k_scale"]  # logits spread as after a norm of queries and keys
            s["q"] = (spread * torch.randn(n, hq, d, generator=gen, device="cuda")).to(act)
            s["out"] = torch.empty(n, hq, d, dtype=act, device="cuda")
            s["lse"] = torch.empty(n, hq, device="cuda")
            s["prefix_blocks"] = table(groups, n, max([1] + need[n:]))
            s["prefix_lens"] = torch.tensor(prefixes, dtype=torch.int32, device="cuda")
            firsts = [0]
            for x in _sizes(case) if groups else []:
                firsts.append(firsts[-1] + x)
            s["group_first"] = torch.tensor(firsts, dtype=torch.int32, device="cuda")
            s["members"], s["prefix_most"] = max(_sizes(case), default=0) if groups else 0, s["prefix_blocks"].shape[1] * page
    if own:
        from paged_kv_cache_kvx_gb300 import kvx
        s["cache"] = kvx.Cache(s["pool"], s["addr"], heads=h, dim=d, dtype=STORE[case["store"]], page_tokens=page,
                               token_stride=s["stride"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                               scale_offset=s["scale_offset"])
        if case["op"] == "shared":
            s["ws"] = s["cache"].attend_shared_workspace(n, hq, per, groups, s["prefix_blocks"].shape[1])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_append(s):
    c = s["case"]
    s["cache"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"], q_weight=s["q_weight"],
                      k_weight=s["k_weight"], eps=1e-6, cos_sin=s["cos_sin"], interleaved=c["pairs"] == "neighbours")
    return s["q_out"], s["rows"], s["scales"]


def _own_read(s):
    s["cache"].read(s["blocks"], s["starts"], s["k_out"], s["v_out"], first=s["first"])
    return s["k_out"], s["v_out"]


def _own_shared(s):
    s["cache"].attend_shared(s["q"], s["prefix_blocks"], s["prefix_lens"], s["group_first"], s["blocks"], s["lens"],
                             s["out"], s["ws"], lse=s["lse"])
    return s["out"], s["lse"]


_own = {"append": _own_append, "read": _own_read, "shared": _own_shared}


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


def _power(e):
    """2 to whole numbers from -126 to 127, exactly."""
    return (e + 127 << 23).to(torch.int32).view(torch.float32)


def _quantised(x):
    """Rows as e4m3 (their bytes) and the exponent, biased by 127, of the smallest power of two that they fit over."""
    top = x.abs().amax(-1, keepdim=True)
    mantissa, exponent = torch.frexp(top)  # in [0.5, 1)
    e = (exponent - 9 + (mantissa > 0.875)).clamp(min=-126)
    e = torch.where(top > 0, e, -126)
    stored = (x * _power(-e)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return stored.view(torch.uint8), (e[..., 0] + 127).to(torch.uint8)


def _pieces(s, at):
    """Numbers of the 16-byte pieces of rows that start at bytes of the pool."""
    row = s["case"]["dim"] * SIZE[s["case"]["store"]]
    return at[..., None] // 16 + torch.arange(row // 16, device="cuda")


def _plain_append(s):
    c = s["case"]
    page = c["page"]
    cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, dim=1)
    s["q_out"].copy_(_rotated(_normed(s["q"], s["q_weight"]), cos, sin, c["pairs"]))
    k = _rotated(_normed(s["k"], s["k_weight"]), cos, sin, c["pairs"])
    slots = s["slots"]
    spare = slots.amax()  # a token without a place writes what the last place gets
    put = torch.where(slots < 0, spare, slots)
    take = torch.where(slots < 0, slots.argmax(), torch.arange(len(slots), device=slots.device))
    rows, exps = _quantised(torch.stack([k, s["v"].float()], dim=2)[take].flatten(1, 2))  # by lane
    seg, place = s["addr"][put // page], (put % page)[:, None]
    s["pool"].view(torch.int32).view(-1, 4)[_pieces(s, seg + place * s["stride"])] = rows.view(torch.int32).unflatten(-1, (-1, 4))
    s["pool"][seg + s["scale_offset"] + place] = exps
    return s["q_out"], s["rows"], s["scales"]


def _loaded(s, block, place):
    """The keys and values [..., heads, dim] of tokens at a place in a block."""
    c = s["case"]
    seg = s["addr"][block]
    at = _pieces(s, seg + (place * s["stride"])[..., None])
    x = s["pool"].view(torch.int32).view(-1, 4)[at].flatten(-2).view(STORE[c["store"]]).float()
    if c["store"] == "rows":
        e = s["pool"][seg + s["scale_offset"] + place[..., None]]
        x = x * _power(e.int()[..., None] - 127)
    return x[..., 0::2, :] * s["k_scale"], x[..., 1::2, :] * s["v_scale"]


def _plain_read(s):
    page = s["case"]["page"]
    row = torch.arange(len(s["k_out"]), device="cuda")
    seq = torch.bucketize(row, s["starts"].long(), right=True) - 1
    there = seq < len(s["lens"])
    seq = seq.clamp(max=len(s["lens"]) - 1)
    pos = row - s["starts"][seq]
    if s["first"] is not None:
        pos = pos + s["first"][seq]
    pos = torch.where(there, pos, 0)
    k, v = _loaded(s, s["blocks"].long()[seq, pos // page], pos % page)
    there = there[:, None, None]
    s["k_out"].copy_(torch.where(there, k.to(s["k_out"].dtype), s["k_out"]))
    s["v_out"].copy_(torch.where(there, v.to(s["v_out"].dtype), s["v_out"]))
    return s["k_out"], s["v_out"]


def _softmax_part(s, q, blocks, lens, most):
    """Attention of q [n, heads, queries, dim] over tables' tokens: outputs not yet divided, their maximum and sum."""
    c = s["case"]
    at = torch.arange(most, device="cuda")
    k, v = _loaded(s, blocks.long()[:, at // c["page"]], (at % c["page"]).expand(len(blocks), -1))
    seen = at < lens.long()[:, None]
    logits = (q @ k.permute(0, 2, 3, 1)) * c["dim"] ** -0.5
    del k
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = (logits - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
    v = torch.where(seen[:, :, None, None], v, torch.zeros_like(v)).permute(0, 2, 1, 3)
    return p @ v, top, p.sum(-1, keepdim=True)


def _plain_shared(s):
    c = s["case"]
    n, h, d = c["seqs"], c["heads"], c["dim"]
    q = s["q"].float().view(n, h, -1, d)
    out, top, total = _softmax_part(s, q, s["blocks"], s["lens"], s["most"])
    if c["groups"]:
        first = s["group_first"].long()
        seq = torch.arange(n, device="cuda")
        group = torch.bucketize(seq, first, right=True) - 1
        member = group < c["groups"]
        group = group.clamp(max=c["groups"] - 1)
        # the queries of a group's sequences together
        of = (first[:-1, None] + torch.arange(s["members"], device="cuda")).clamp(max=n - 1)
        parts = _softmax_part(s, q[of].transpose(1, 2).flatten(2, 3), s["prefix_blocks"], s["prefix_lens"], s["prefix_most"])
        g = q.shape[2]
        place = torch.where(member, seq - first[group], 0)
        p_out, p_top, p_total = (x.unflatten(2, (-1, g))[group, :, place] for x in parts)
        p_top = torch.where(member[:, None, None, None], p_top, -math.inf)
        both = torch.maximum(top, p_top)
        base = torch.where(torch.isinf(both), torch.zeros_like(both), both)
        a, b = (top - base).exp(), (p_top - base).exp()
        out, total, top = out * a + p_out * b, total * a + p_total * b, both
    s["out"].copy_(torch.where(total > 0, out / total, 0).view(n, -1, d))
    s["lse"].copy_((top + total.log()).view(n, -1))
    return s["out"], s["lse"]


_plain = {"append": _plain_append, "read": _plain_read, "shared": _plain_shared}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    return {"append": _exact_append, "read": _exact_read, "shared": _exact_shared}[case["op"]](prepare(case, seed))


def _exact_append(s):
    c = s["case"]
    d, half, h = c["dim"], c["rot"] // 2, c["heads"]
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

    rows, scales = s["rows"].double(), s["scales"].double()
    has = s["slots"] >= 0
    block, place = s["slots"][has] // c["page"], s["slots"][has] % c["page"]
    # a block's bytes, whichever way its address table leads to it
    size = len(s["pool"]) // len(s["addr"])
    block = s["addr"][block, 0] // size
    for kv, x in ((0, head(s["k"], s["k_weight"])[has]), (1, s["v"].double()[has])):
        top = x.abs().amax(-1)
        e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-126.0) + 127
        power = lambda b: b.clamp(1, 254).to(torch.uint8).view(torch.float8_e8m0fnu).double()  # noqa: E731
        e = torch.where(top > power(e) * E4M3_MAX, e + 1, torch.where(top <= power(e - 1) * E4M3_MAX, e - 1, e))
        scale = power(e)
        for j in range(h):
            if rows.dim() == 4:  # [blocks, lanes, tokens, dim]
                rows[block, 2 * j + kv, place] = x[:, j] / scale[:, j, None]
                scales[block, 2 * j + kv, place] = scale[:, j]
            else:  # [blocks, kv, tokens, heads, dim]
                rows[block, kv, place, j] = x[:, j] / scale[:, j, None]
                scales[block, kv, j, place] = scale[:, j]
    return head(s["q"], s["q_weight"]), rows, scales


def _head64(s, block, place, head, kv):
    """One head's keys or values [tokens, dim] in 64 bits."""
    c = s["case"]
    seg = s["addr"][block.long(), 2 * head + kv]
    size, row = SIZE[c["store"]], c["dim"] * SIZE[c["store"]]
    raw = s["pool"][(seg + place * s["stride"])[:, None] + torch.arange(row, device="cuda")]
    x = raw.view(STORE[c["store"]] if size == 2 else torch.float8_e4m3fn).double()
    if c["store"] == "rows":
        return x * s["pool"][seg + s["scale_offset"] + place].view(torch.float8_e8m0fnu).double()[:, None]
    return x * (s["v_scale"] if kv else s["k_scale"])


def _exact_read(s):
    c = s["case"]
    outs = [s["k_out"].double(), s["v_out"].double()]
    starts = s["starts"].tolist()
    for n in range(c["seqs"]):
        pos = torch.arange(starts[n + 1] - starts[n], device="cuda") + c["skip"]
        block = s["blocks"][n][pos // c["page"]]
        for j in range(c["heads"]):
            for kv in (0, 1):
                outs[kv][starts[n]:starts[n + 1], j] = _head64(s, block, pos % c["page"], j, kv)
    return tuple(outs)


def _exact_shared(s):
    c = s["case"]
    g, d, n = c["q_heads"] // max(1, c["heads"]), c["dim"], c["seqs"]
    out = torch.zeros(n, c["q_heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    firsts, lens, prefixes = s["group_first"].tolist(), s["lens"].tolist(), s["prefix_lens"].tolist()
    groups = [(list(range(firsts[i], firsts[i + 1])), prefixes[i]) for i in range(c["groups"])]
    groups.append((list(range(firsts[-1], n)), 0))
    for i, (members, prefix) in enumerate(groups):
        at = torch.arange(prefix, device="cuda")
        for j in range(c["heads"]):
            heads = slice(j * g, (j + 1) * g)
            if prefix:
                block = s["prefix_blocks"][i][at // c["page"]]
                pk, pv = (_head64(s, block, at % c["page"], j, kv) for kv in (0, 1))
            for m in members:
                pos = torch.arange(lens[m], device="cuda")
                block = s["blocks"][m][pos // c["page"]]
                k, v = (_head64(s, block, pos % c["page"], j, kv) for kv in (0, 1))
                if not len(k) and not prefix:
                    continue
                q = s["q"][m, heads].double() / math.sqrt(d)
                x = torch.cat([q @ pk.T, q @ k.T], dim=1) if prefix else q @ k.T
                lse[m, heads] = torch.logsumexp(x, dim=1)
                p = (x - lse[m, heads, None]).exp()
                out[m, heads] = p[:, :prefix] @ pv + p[:, prefix:] @ v if prefix else p @ v
    return out, lse
