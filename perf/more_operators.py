"""Workloads of the operators between projections and attention: norm and rotation of queries and keys (forward
and backward, and into the FP8 cache), and sparse attention over blocks (pages) of the FP8 cache.

``run`` makes ONE pass: with ``own`` the library's calls, without it the same operator from elementary torch
operations in 32 bits (sums that make 8-bit codes in 64), rounded once at the end.  ``exact`` is the definition in
64 bits, written apart from both.

Norm and rotation: y = w * x / sqrt(mean(x^2) + eps) of each head's row, then the pairs of its first R values turn by
the token's angles; cos_sin holds a position's R / 2 cosines, then its R / 2 sines.  Pair i is (i, i + R / 2),
or (2 i, 2 i + 1) where interleaved.  A token whose position is negative gives zeros, and is not written to the cache.

Blocks: a page's block key is the mean of its keys, for each head as signed 8-bit codes and one power of two, the
smallest with |mean| <= 127 of it.  A query of a sequence at place x has own block x // page; it attends to the first
`first` blocks, the last `last` (its own among them), and of those between the ones with the highest scores,
`top` blocks in all, equal scores by lower index.  A block's score is the largest, over the query heads that share the key head, of the
integer product of the query's 8-bit codes (made alike) and the block key's, times both scales.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", 0)
else:
    DEV = torch.device("cpu")

EPS = 1e-6
POSITIONS = 131072  # rows of the table of angles


# ---------------------------------------------------------------- cases
def _rope(name, op, tokens, heads, kv_heads, dim, rot, dtype, interleaved=False, skip=0, page=64):
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "dtype": dtype, "interleaved": interleaved, "skip": skip, "page": page}


def _keys(name, pages, kv_heads, dim, page, skip):
    return {"name": name, "op": "block_keys", "pages": pages, "kv_heads": kv_heads, "dim": dim, "page": page, "skip": skip}


def _sparse(name, batch, new, past, heads, kv_heads, dim, page, top, first=1, last=2, empty=0):
    return {"name": name, "op": "sparse", "batch": batch, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0],
            "past_hi": past[1], "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "top": top, "first": first,
            "last": last, "empty": empty}


def listed():
    return [
        # a training step's packed batch, forward and backward: bound by memory
        _rope("train_8192", "train", 8192, 32, 8, 128, 128, "bf16"),
        # FP32, odd counts, interleaved pairs, half of the values turned, a few padding tokens
        _rope("train_fp32_odd", "train", 1021, 9, 3, 64, 32, "fp32", True, 37),
        # one decode step of a padded batch: a call of a few kilobytes, all latency
        _rope("write_step", "write", 24, 32, 8, 128, 128, "bf16", False, 3),
        # a whole prompt's queries, keys and values
        _rope("write_prompt", "write", 8192, 32, 8, 128, 128, "bf16"),
        # wide heads, a quarter of the values turned, interleaved, an odd number of tokens on small pages
        _rope("write_wide_heads", "write", 1531, 16, 2, 256, 64, "bf16", True, 11, 16),
        # a decode step of 64 sequences, in which two fill their page
        _keys("block_keys_step", 64, 8, 128, 64, 62),
        # the pages of a long prompt
        _keys("block_keys_prompt", 2047, 8, 128, 64, 0),
        # one sequence, one new token: the shortest answer time
        _sparse("decode_one", 1, (1, 1), (16000, 16000), 32, 8, 128, 64, 16),
        # a full decode batch with contexts of every length, two of its places unused
        _sparse("decode_batch", 64, (1, 1), (0, 32767), 64, 8, 128, 64, 32, empty=2),
        # few sequences with a very long context
        _sparse("decode_long", 2, (1, 1), (100003, 131071), 32, 4, 128, 64, 64),
        # a chunk of a long prompt
        _sparse("chunk_2048", 1, (2048, 2048), (30720, 30720), 32, 8, 128, 64, 16),
        # chunks of several requests, groups of seven heads, half-size heads, small pages
        _sparse("chunk_ragged", 5, (1, 537), (0, 9001), 28, 4, 64, 16, 48, 2, 4),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the listed ranges."""
    while True:
        op = rng.choice(["train", "write", "block_keys", "sparse", "sparse", "sparse"])
        dim = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 64, 48, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8, 16])
        if op == "block_keys":
            pages = _log_between(rng, 1, 8192)
            c = {"op": op, "pages": pages, "kv_heads": kv_heads, "dim": dim, "page": page, "skip": rng.randint(0, (pages - 1) // 2)}
            if work(c)["bytes"] <= 137e6:
                return c
            continue
        if op != "sparse":
            tokens = _log_between(rng, 1, 8192)
            c = {"op": op, "tokens": tokens, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
                 "rot": rng.choice([dim, dim, dim // 2, dim // 4, 48]), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                 "interleaved": rng.random() < 0.4, "skip": rng.randint(0, (tokens - 1) // 4), "page": page}
            if work(c)["bytes"] <= 345e6:
                return c
            continue
        c = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "first": rng.randint(0, 2),
             "last": rng.randint(1, 4), "empty": 0}
        c["top"] = max(c["first"] + c["last"], _log_between(rng, 256, 4096) // page)
        if rng.random() < 0.6:  # single tokens, or a few speculated ones
            c["batch"] = _log_between(rng, 1, 128)
            c["new_lo"] = rng.choice([1, 1, 1, 2])
            c["new_hi"] = c["new_lo"] + rng.choice([0, 0, 0, 1, 4])
            c["past_hi"] = _log_between(rng, 16, 131071)
            c["empty"] = rng.randint(0, (c["batch"] - 1) // 16)
        else:  # chunks of prompts
            c["batch"] = rng.randint(1, 5)
            c["new_hi"] = _log_between(rng, 16, 2048)
            c["new_lo"] = rng.choice([c["new_hi"], rng.randint(1, c["new_hi"])])
            c["past_hi"] = rng.choice([0, _log_between(rng, 16, 32767)])
        c["past_lo"] = rng.randint(0, c["past_hi"])
        b, n, ctx = c["batch"], c["new_hi"], c["new_hi"] + c["past_hi"]
        if (b * n * kv_heads * c["top"] * page * dim <= 2048 * 8 * 1024 * 128 and b * ctx * kv_heads * dim <= 64 * 32768 * 8 * 128
                and b * n * c["heads"] * (ctx // page) <= 2048 * 32 * 512):
            return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(new tokens, context with them) of each sequence; the last `empty` ones have no context at all."""
    b = case["batch"]
    new = _spread(case["new_lo"], case["new_hi"], b)
    past = _spread(case["past_lo"], case["past_hi"], b)
    past = past[b // 2:] + past[: b // 2]  # (short chunks meet long contexts too)
    return [(n, 0 if i >= b - case["empty"] else n + p) for i, (n, p) in enumerate(zip(new, past))]


def work(case):
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] == "block_keys":
        rows = (case["pages"] - case["skip"]) * hk
        return {"bytes": rows * (case["page"] * (d + 1) + d + 4) + 4 * case["pages"], "flops": rows * case["page"] * d}
    if case["op"] != "sparse":
        t, n = case["tokens"] - case["skip"], case["heads"] + hk
        size = 2 if case["dtype"] == "bf16" else 4
        table = t * case["rot"] * 4 + case["tokens"] * 8
        if case["op"] == "train":  # (rows and their gradients, in and out)
            return {"bytes": 4 * t * n * d * size + table, "flops": 30 * t * n * d}
        return {"bytes": t * (n + hk) * d * size + t * case["heads"] * d * size + 2 * t * hk * (d + 1) + table + 8 * t,
                "flops": 12 * t * n * d}
    page, top = case["page"], case["top"]
    size = flops = 0
    for n, ctx in _lengths(case):
        if not ctx:
            continue
        blocks = -(-ctx // page)
        between = max(0, blocks - case["first"] - case["last"]) if blocks > top else 0  # blocks that are scored
        seen = min(top, blocks)
        size += between * hk * (d + 4) + 2 * hk * (d + 1) * min(ctx, n * top * page) + 4 * blocks
        size += n * case["heads"] * (2 * 2 * d + 4) + 4 * n * hk * top
        flops += n * case["heads"] * (2 * d * between + 4 * d * min(ctx, seen * page))
    return {"bytes": size + 8 * case["batch"], "flops": flops}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _encode(x):
    """E4M3 codes and UE8M0 scale codes of rows x [..., D] (FP32): the scale is the row's largest magnitude
    over 448, raised to a power of two; a row of zeros has scale 1."""
    t = x.abs().amax(-1) / 448.0
    bits = t.view(torch.int32)
    sf = ((bits >> 23) + ((bits & 0x7FFFFF) != 0)).clamp(min=1)
    sf = torch.where(t == 0, torch.full_like(sf, 127), sf)
    q = (x / (sf << 23).view(torch.float32).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), sf.to(torch.uint8)


def _decode(codes, sf):
    return codes.view(torch.float8_e4m3fn).float() * (sf.to(torch.int32) << 23).view(torch.float32).unsqueeze(-1)


def _rows(g, tokens, heads, dim):
    """Projections' outputs: normal, tokens of different size, a few large channels."""
    x = _normal(g, tokens, heads, dim)
    x *= torch.exp(0.5 * _normal(g, tokens, heads, 1))
    x *= 1.0 + 3.0 * (torch.rand((1, heads, dim), generator=g, device=DEV) < 0.03)
    return x


def _cache(g, pages, heads, page, dim, topics=None):
    """(codes, scale codes) of a cache whose every place holds a token; the keys of a page share a topic."""
    x = _rows(g, pages * page, heads, dim).view(pages, page, heads, dim)
    if topics is not None:
        x += topics.unsqueeze(1)
    q, sf = _encode(x)
    return q.transpose(1, 2).contiguous(), sf.transpose(1, 2).contiguous()


def _angles(rot):
    """[POSITIONS, rot]: cosines, then sines, of base 500000."""
    turn = torch.arange(POSITIONS, device=DEV, dtype=torch.float64)[:, None] * 500000.0 ** (
        -torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    return torch.cat([turn.cos(), turn.sin()], -1).float()


def prepare(case, seed):
    g = _generator(seed)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "block_keys":
        n = case["pages"]
        k_cache = _cache(g, n + 2, hk, page, d)
        pages = torch.randperm(n + 2, generator=g, device=DEV)[:n].to(torch.int32)
        pages[torch.randperm(n, generator=g, device=DEV)[: case["skip"]]] = -1
        return {"op": "block_keys", "k_cache": k_cache, "pages": pages,
                "block_keys": (torch.zeros((n + 2, hk, d), dtype=torch.int8, device=DEV),
                               torch.ones((n + 2, hk), dtype=torch.float32, device=DEV))}
    if case["op"] != "sparse":
        t, h, dtype = case["tokens"], case["heads"], _dtype(case)
        # queries, keys and values are slices of one projection's output
        qkv = _rows(g, t, h + 2 * hk, d).to(dtype)
        q, k, v = qkv.split((h, hk, hk), 1)
        # sequences one after the other, the first of them far into its context
        lens = max(1, t // 4)
        i = torch.arange(t, device=DEV)
        positions = i % lens + torch.where(i < lens, POSITIONS - lens, 0)
        dead = torch.randperm(t, generator=g, device=DEV)[: case["skip"]]
        positions[dead] = -1
        st = {"op": case["op"], "q": q, "k": k, "v": v, "positions": positions, "cos_sin": _angles(case["rot"]),
              "interleaved": case["interleaved"], "q_weight": (1 + 0.2 * _normal(g, d)).to(dtype),
              "k_weight": (1 + 0.2 * _normal(g, d)).to(dtype), "page": page}
        if case["op"] == "train":
            st["dq"], st["dk"] = _normal(g, t, h, d).to(dtype), _normal(g, t, hk, d).to(dtype)
            return st
        pages = -(-t // page) + 2
        order = torch.randperm(pages, generator=g, device=DEV)
        st["slots"] = order[i // page] * page + i % page
        st["slots"][dead] = -1
        st["k_cache"], st["v_cache"] = _cache(g, pages, hk, page, d), _cache(g, pages, hk, page, d)
        return st
    lens = _lengths(case)
    lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device=DEV).tolist()]
    new, ctx = [n for n, _ in lens], [c for _, c in lens]
    per = max(1, -(-max(ctx) // page))  # block-table columns
    used = [-(-c // page) for c in ctx]
    pages = sum(used) + 1
    table = torch.zeros((len(lens), per), dtype=torch.int32)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at: at + n]
        at += n
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(new, dtype=torch.int32).cumsum(0)
    total = sum(new)
    st = {"op": "sparse", "page": page, "top": case["top"], "first": case["first"], "last": case["last"],
          "table": table.to(DEV), "seq_lens": torch.tensor(ctx, dtype=torch.int32, device=DEV), "cu": cu.to(DEV),
          "max_new": max(new), "same_new": min(new) == max(new)}
    topics = 0.7 * _normal(g, pages, hk, d)
    st["k_cache"] = _cache(g, pages, hk, page, d, topics)
    st["v_cache"] = _cache(g, pages, hk, page, d)
    st["block_keys"] = _block_keys(*st["k_cache"])
    # runs of eight tokens ask for the topics of six pages of their context, weighted alike for a head's group
    t = torch.arange(total, device=DEV)
    seq = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    run_of = (t - st["cu"].long()[seq]) // 8 + seq * 1009
    pick = torch.rand((6, int(run_of.max()) + 1), generator=g, device=DEV)[:, run_of]
    blocks = torch.tensor(used, device=DEV)[seq].clamp(min=1)
    asked = st["table"][seq, (pick * blocks).long().clamp(max=per - 1)].long()
    q = _normal(g, total, hk, case["heads"] // hk, d) + 0.5 * topics[asked].sum(0).unsqueeze(2)
    st["q"] = q.view(total, case["heads"], d).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- one pass, plainly
def _cache_values(st):
    """The cache as the values it stands for."""
    return [t for codes, sf in (st["k_cache"], st["v_cache"])
            for t in (codes.view(torch.float8_e4m3fn), sf.view(torch.float8_e8m0fnu))]


def _cos_sin(st):
    """Cosines and sines [tokens, 1, R / 2], and which tokens count."""
    live = st["positions"] >= 0
    c, s = st["cos_sin"][st["positions"].clamp(min=0)].unsqueeze(1).chunk(2, -1)
    return c, s, live[:, None, None]


def _pairs(x, rot, interleaved):
    x = x[..., :rot]
    return (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)


def _join(a, b, rest, interleaved):
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), rest], -1)


def _norm_rope(x, weight, st):
    """FP32 rows."""
    c, s, live = _cos_sin(st)
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    rot = 2 * c.shape[-1]
    a, b = _pairs(y, rot, st["interleaved"])
    y = _join(a * c - b * s, a * s + b * c, y[..., rot:], st["interleaved"])
    return torch.where(live, y, 0.0)


def _norm_rope_backward(dout, x, weight, st):
    c, s, live = _cos_sin(st)
    x = x.float()
    dy = torch.where(live, dout.float(), 0.0)
    rot = 2 * c.shape[-1]
    a, b = _pairs(dy, rot, st["interleaved"])
    dy = _join(a * c + b * s, b * c - a * s, dy[..., rot:], st["interleaved"])
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    g = dy * weight.float()
    return r * (g - xh * (g * xh).mean(-1, keepdim=True)), (dy * xh).sum((0, 1))


def _plain_train(st):
    dtype = st["q"].dtype
    q, k = (_norm_rope(st[x], st[x + "_weight"], st).to(dtype) for x in "qk")
    dq, dwq = _norm_rope_backward(st["dq"], st["q"], st["q_weight"], st)
    dk, dwk = _norm_rope_backward(st["dk"], st["k"], st["k_weight"], st)
    return [q, k, dq.to(dtype), dk.to(dtype), dwq, dwk]


def _plain_write(st):
    q = _norm_rope(st["q"], st["q_weight"], st).to(st["q"].dtype)
    valid = st["slots"] >= 0
    i = torch.arange(valid.numel(), device=DEV)
    i = torch.where(valid, i, valid.to(torch.int32).argmax())  # a skipped token repeats the first one's write
    slots = st["slots"][i]
    at, place = slots // st["page"], slots % st["page"]
    kq, ks = _encode(_norm_rope(st["k"], st["k_weight"], st)[i])
    vq, vs = _encode(st["v"][i].float())
    st["k_cache"][0][at, :, place], st["k_cache"][1][at, :, place] = kq, ks
    st["v_cache"][0][at, :, place], st["v_cache"][1][at, :, place] = vq, vs
    return [q, *_cache_values(st)]


def _power_below(top):
    """The exponent e of the smallest power of two with top <= 127 * 2^e, at least -126; 0 for zeros (64 bits)."""
    frac, e = torch.frexp(top)  # frac in [1/2, 1); 127 = (127 / 128) * 2^7
    e = (e - 7 + (frac > 127.0 / 128.0).to(e.dtype)).clamp(-126, 127)
    return torch.where(top == 0, torch.zeros_like(e), e)


def _power(e):
    """2^e in FP32, by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _block_keys(codes, sf):
    """Codes [pages, heads, page, D] -> signed 8-bit codes [pages, heads, D] of the means and scales [pages, heads]."""
    mean = torch.nan_to_num(_decode(codes, sf)).double().sum(2) / codes.shape[2]
    scale = _power(_power_below(mean.abs().amax(-1)))
    return torch.round(mean / scale.double().unsqueeze(-1)).clamp(-127, 127).to(torch.int8), scale


def _plain_block_keys(st):
    valid = st["pages"] >= 0
    i = torch.arange(valid.numel(), device=DEV)
    pages = st["pages"][torch.where(valid, i, valid.to(torch.int32).argmax())].long()
    codes, scale = _block_keys(st["k_cache"][0][pages], st["k_cache"][1][pages])
    st["block_keys"][0][pages] = codes
    st["block_keys"][1][pages] = scale
    return [_block_key_values(st)]


def _block_key_values(st):
    return st["block_keys"][0] * st["block_keys"][1].unsqueeze(-1)


def _places(st):
    """Of each packed token: its sequence, its number among the sequence's new ones, its place."""
    cu, total = st["cu"].long(), st["q"].shape[0]
    t = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[seq]
    return seq, i, st["seq_lens"].long()[seq] - (cu[1:] - cu[:-1])[seq] + i


def _plain_select(st, seq, i, place):
    """int32 [tokens, key heads, top], ascending, then -1."""
    q, table, cu, n, top = st["q"], st["table"].long(), st["cu"].long(), st["max_new"], st["top"]
    total, heads, d = q.shape
    hk = st["block_keys"][0].shape[1]
    b, cols = table.shape
    # queries as 8-bit codes (exact in FP32, as are their products' sums: at most 2^22)
    x = q.float()
    sq = _power(_power_below(x.abs().amax(-1)))
    x = torch.round(x / sq.unsqueeze(-1))
    src = (cu[:-1, None] + torch.arange(n, device=DEV)).clamp(max=total - 1)
    x = x[src].view(b, n, hk, heads // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    keys = st["block_keys"][0][table].float().permute(0, 2, 3, 1)  # [b, hk, d, cols]
    s = torch.matmul(x, keys.contiguous()) * st["block_keys"][1][table].transpose(1, 2).unsqueeze(2)
    s = s.view(b, hk, n, heads // hk, cols)[seq, :, i] * sq.view(total, hk, heads // hk, 1)
    s = s.amax(2)  # [tokens, hk, cols]
    own_block = torch.div(place, st["page"], rounding_mode="floor")[:, None, None]
    j = torch.arange(cols, device=DEV)
    s = s.masked_fill_((j < st["first"]) | (j > own_block - st["last"]), math.inf).masked_fill_(j > own_block, -math.inf)
    best = torch.argsort(s, dim=-1, descending=True, stable=True)[..., :top]
    best = torch.nn.functional.pad(best, (0, top - best.shape[-1]), value=cols)
    best = torch.where(best > own_block, cols, best).sort(-1).values
    return torch.where(best >= cols, -1, best).to(torch.int32)


def _plain_sparse(st):
    seq, i, place = _places(st)
    blocks = _plain_select(st, seq, i, place)
    q, page = st["q"], st["page"]
    total, heads, d = q.shape
    hk = blocks.shape[1]
    pages = st["table"].long()[seq[:, None, None], blocks.long().clamp(min=0)]  # [tokens, hk, top]
    head = torch.arange(hk, device=DEV)[:, None]

    def rows(cache):  # [tokens, hk, top * page, d]
        return _decode(cache[0][pages, head], cache[1][pages, head]).flatten(2, 3)

    s = torch.matmul(q.float().view(total, hk, -1, d), rows(st["k_cache"]).transpose(2, 3)) * (1.0 / math.sqrt(d))
    j = blocks.long().unsqueeze(-1) * page + torch.arange(page, device=DEV)
    seen = ((blocks.unsqueeze(-1) >= 0) & (j <= place[:, None, None, None])).flatten(2).unsqueeze(2)
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows(st["v_cache"])) / torch.where(z == 0, torch.ones_like(z), z)
    return [blocks, o.view(total, heads, d).to(torch.bfloat16), (top + z.log()).view(total, heads)]


def run(state):
    st = state
    if own:
        import block_scaled_fp8_amd as dg
        if st["op"] == "block_keys":
            dg.fp8_kv_block_keys_update(st["k_cache"], st["block_keys"], st["pages"])
            return [_block_key_values(st)]
        if st["op"] == "sparse":
            cu = None if st["same_new"] else st["cu"]
            blocks = dg.fp8_kv_select_blocks(st["q"], st["block_keys"], st["table"], st["seq_lens"], st["page"], st["top"],
                                             first=st["first"], last=st["last"], cu_seqlens_q=cu, max_seqlen_q=st["max_new"])
            out, lse = dg.fp8_block_sparse_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq_lens"], blocks,
                                                     cu_seqlens_q=cu, max_seqlen_q=st["max_new"], return_lse=True)
            return [blocks, out, lse]
        weights = (st["q_weight"], st["k_weight"], st["cos_sin"], st["positions"])
        if st["op"] == "train":
            q, k = dg.qk_norm_rope(st["q"], st["k"], *weights, eps=EPS, interleaved=st["interleaved"])
            return [q, k, *dg.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], *weights, eps=EPS,
                                                    interleaved=st["interleaved"])]
        q = dg.qk_norm_rope_fp8_kv_cache_write(st["q"], st["k"], st["v"], *weights, st["k_cache"], st["v_cache"], st["slots"],
                                               eps=EPS, interleaved=st["interleaved"])
        return [q, *_cache_values(st)]
    return {"train": _plain_train, "write": _plain_write, "block_keys": _plain_block_keys, "sparse": _plain_sparse}[st["op"]](st)


# ---------------------------------------------------------------- the definition in 64 bits
def _e4m3_values():
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v.append(math.nan if (c & 127) == 127 else -mag if c & 128 else mag)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _power64(e):
    """2^e in 64 bits, by its bits: a computed power may be off in the last place, and ties would fall wrong."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values64(cache):
    codes, sf = cache
    return _e4m3_values()[codes.long()], _power64(sf.long() - 127)


def _least_power(top, most):
    """The smallest power of two p with top <= most * p; 1 for zeros."""
    frac, e = torch.frexp(top / most)  # (exact enough: a quotient equal to a power of two comes out as one)
    return _power64(torch.where(top == 0, torch.zeros_like(e), torch.where(frac == 0.5, e - 1, e)).clamp(min=-126))


def _turn64(x, st, sign):
    """Rows x turned forward (sign 1) or back (-1) by their tokens' angles, as complex numbers."""
    rot = st["cos_sin"].shape[1]
    angles = st["cos_sin"].double()[st["positions"].clamp(min=0)]
    z = torch.complex(angles[:, : rot // 2], sign * angles[:, rot // 2:])[:, None]
    even = torch.arange(0, rot, 2, device=DEV) if st["interleaved"] else torch.arange(rot // 2, device=DEV)
    odd = even + (1 if st["interleaved"] else rot // 2)
    turned = torch.complex(x[..., even], x[..., odd]) * z
    y = x.clone()
    y[..., even], y[..., odd] = turned.real, turned.imag
    return y


def _exact_rope(case, st):
    live = (st["positions"] >= 0)[:, None, None]
    out, grads, sums = [], [], []
    for x in "qk":
        v, w = st[x].double(), st[x + "_weight"].double()
        size = (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()
        unit = v / size
        out.append(torch.where(live, _turn64(unit * w, st, 1), 0.0))
        if case["op"] == "train":
            back = torch.where(live, _turn64(st["d" + x].double(), st, -1), 0.0)
            sums.append(torch.einsum("thd,thd->d", back, unit))
            along = torch.einsum("thd,thd->th", back * w, unit).unsqueeze(-1) / v.shape[-1]
            grads.append((back * w - unit * along) / size)
    if case["op"] == "train":
        return out + grads + sums
    page, res = st["page"], [out[0]]
    at = torch.nonzero(st["slots"] >= 0).flatten()
    slots = st["slots"][at]
    for x, cache in ((out[1][at], st["k_cache"]), (st["v"].double()[at], st["v_cache"])):
        val, scale = _values64(cache)
        s = _least_power(x.abs().amax(-1), 448.0)
        y = x / s.unsqueeze(-1)
        step = _power64(torch.frexp(y.abs())[1].clamp(min=-5) - 4)  # spacing of E4M3 at |y|
        val[slots // page, :, slots % page] = (torch.round(y / step) * step).clamp(-448, 448)
        scale[slots // page, :, slots % page] = s
        res += [val, scale]
    return res


def _exact_sparse(case, st):
    q, table, page, group = st["q"].double(), st["table"].long(), st["page"], case["heads"] // case["kv_heads"]
    total, heads, d = q.shape
    hk = case["kv_heads"]
    sq = _least_power(q.abs().amax(-1), 127.0)
    q8 = torch.round(q / sq.unsqueeze(-1))
    k8, sk = st["block_keys"][0].double(), st["block_keys"][1].double()
    o = torch.zeros((total, heads, d), dtype=torch.float64, device=DEV)
    lse = torch.full((total, heads), -math.inf, dtype=torch.float64, device=DEV)
    chosen = torch.full((total, hk, case["top"]), -1, dtype=torch.int32, device=DEV)
    cu, lens = st["cu"].tolist(), st["seq_lens"].tolist()
    for b, ctx in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if not ctx or lo == hi:
            continue
        blocks = -(-ctx // page)
        pages = table[b, :blocks]
        place = torch.arange(ctx - (hi - lo), ctx, device=DEV)
        mine = (place // page)[:, None]
        j = torch.arange(blocks, device=DEV)[None]
        key = torch.arange(ctx, device=DEV)[None]
        k, v = ((val * scale.unsqueeze(-1)).transpose(0, 1).flatten(1, 2)[:, :ctx]
                for val, scale in (_values64((c[pages], s[pages])) for c, s in (st["k_cache"], st["v_cache"])))
        for h in range(hk):
            hs = range(h * group, (h + 1) * group)
            score = torch.stack([(q8[lo:hi, x] @ k8[pages, h].T) * sk[pages, h] * sq[lo:hi, x, None] for x in hs]).amax(0)
            score[((j < case["first"]) | (j > mine - case["last"])).expand_as(score)] = math.inf
            score[(j > mine).expand_as(score)] = -math.inf
            order = torch.sort(-score, dim=-1, stable=True).indices
            rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order).contiguous())
            take = (rank < case["top"]) & (j <= mine)
            at = take.cumsum(-1) - 1
            t, c = torch.nonzero(take, as_tuple=True)
            chosen[lo + t, h, at[t, c]] = c.int()
            hidden = ~take[:, key[0] // page] | (key > place[:, None])
            for x in hs:
                s = q[lo:hi, x] @ k[h].T / math.sqrt(d)
                s[hidden] = -math.inf
                lse[lo:hi, x] = torch.logsumexp(s, -1)
                o[lo:hi, x] = torch.softmax(s, -1) @ v[h]
    return [chosen, o, lse]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "sparse":
        return _exact_sparse(case, st)
    if case["op"] != "block_keys":
        return _exact_rope(case, st)
    val = st["block_keys"][0].double() * st["block_keys"][1].double().unsqueeze(-1)
    pages = st["pages"][st["pages"] >= 0].long()
    codes, scale = _values64((st["k_cache"][0][pages], st["k_cache"][1][pages]))
    mean = (codes * scale.unsqueeze(-1)).mean(2)
    s = _least_power(mean.abs().amax(-1), 127.0).unsqueeze(-1)
    val[pages] = torch.round(mean / s) * s
    return [val]
