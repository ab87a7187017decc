"""The attention operators' workloads: an FP8 key/value cache in pages, written, read back and attended.

``run`` makes ONE pass: with ``own`` the library's calls, without it the same operator from
elementary torch operations in 32 bits, rounded once at the end.  ``exact`` is the definition
in 64 bits, written apart from both.

The cache holds E4M3 codes [pages, kv heads, page size, head dim] and one power-of-two scale per
(token, kv head) row as a UE8M0 code [pages, kv heads, page size]: value = code * 2^(sf - 127).
A token's slot is page * page_size + place in the page; a negative slot is skipped.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda", 0)
else:
    DEV = torch.device("cpu")


# ---------------------------------------------------------------- cases
def _write(name, tokens, heads, dim, page, dtype, skip):
    return {"name": name, "op": "write", "tokens": tokens, "kv_heads": heads, "dim": dim, "page": page, "dtype": dtype,
            "skip": skip}


def _read(name, tokens, heads, dim, page, dtype, skip):
    return {"name": name, "op": "read", "tokens": tokens, "kv_heads": heads, "dim": dim, "page": page, "dtype": dtype,
            "skip": skip}


def _attend(name, batch, new, past, heads, kv_heads, dim, page, window=0, sinks=0, lse=False, empty=0):
    return {"name": name, "op": "attend", "batch": batch, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0],
            "past_hi": past[1], "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "sinks": sinks, "lse": lse, "empty": empty}


def listed():
    return [
        # one decode step's keys and values of a padded batch: a call of a few kilobytes, all latency
        _write("write_step", 24, 8, 128, 64, "bf16", 3),
        # a whole prompt's keys and values: bound by memory
        _write("write_prompt", 8192, 8, 128, 64, "bf16", 0),
        # FP32 keys and values with half-size heads, an odd token count and pages of 16, padding rows among them
        _write("write_fp32_odd", 1021, 5, 64, 16, "fp32", 37),
        # a long shared prefix read back for a consumer that takes BF16
        _read("read_prefix", 16384, 8, 128, 64, "bf16", 0),
        # one sequence, one new token: the shortest answer time
        _attend("decode_one", 1, (1, 1), (1000, 1000), 32, 8, 128, 64),
        # a full decode batch with contexts of every length, two of its places unused
        _attend("decode_batch", 64, (1, 1), (0, 8191), 64, 8, 128, 64, empty=2),
        # few sequences with a very long context: the work has to be split along the keys
        _attend("decode_long", 2, (1, 1), (100003, 131071), 32, 8, 128, 64),
        # some speculated tokens each, groups of seven heads, half-size heads, small pages, sums returned
        _attend("decode_draft_tokens", 16, (3, 5), (17, 4099), 28, 4, 64, 16, lse=True),
        # old tokens out of sight except the first four
        _attend("decode_window", 128, (1, 1), (100, 16000), 32, 4, 128, 64, window=1024, sinks=4, empty=3),
        # a chunk of a long prompt
        _attend("chunk_2048", 1, (2048, 2048), (6144, 6144), 32, 8, 128, 64),
        # chunks of several requests in one call, pages that no tile's end falls on, sums returned
        _attend("chunk_ragged", 5, (1, 1537), (0, 4001), 32, 8, 128, 48, lse=True),
        # the same with a sliding window and the first tokens kept, half-size heads
        _attend("chunk_window", 2, (2048, 2048), (3001, 6144), 32, 4, 64, 64, window=1024, sinks=4),
    ]


def _log_between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the listed ranges."""
    while True:
        kind = rng.choice(["write", "read", "decode", "decode", "decode", "chunk", "chunk", "chunk"])
        dim = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 64, 48, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
        if kind in ("write", "read"):
            tokens = _log_between(rng, 1, 8192 if kind == "write" else 16384)
            c = {"op": kind, "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "page": page,
                 "dtype": rng.choice(["bf16", "bf16", "fp32"]), "skip": rng.randint(0, (tokens - 1) // 4)}
            if work(c)["bytes"] <= 101e6:
                return c
            continue
        window = rng.choice([0, 0, _log_between(rng, 64, 4096)])
        c = {"op": "attend", "heads": kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16]), "kv_heads": kv_heads, "dim": dim,
             "page": page, "window": window, "sinks": rng.randint(0, 8) if window else 0, "lse": rng.random() < 0.3,
             "empty": 0}
        if kind == "decode":
            c["batch"] = _log_between(rng, 1, 128)
            c["new_lo"] = rng.choice([1, 1, 1, 2])
            c["new_hi"] = c["new_lo"] + rng.choice([0, 0, 0, 1, 4])
            c["past_hi"] = _log_between(rng, 16, 131071)
            c["past_lo"] = rng.randint(0, c["past_hi"])
            c["empty"] = rng.randint(0, (c["batch"] - 1) // 16)
        else:
            c["batch"] = rng.randint(1, 5)
            c["new_hi"] = _log_between(rng, 16, 2048)
            c["new_lo"] = rng.choice([c["new_hi"], rng.randint(1, c["new_hi"])])
            c["past_hi"] = rng.choice([0, _log_between(rng, 16, 8192)])
            c["past_lo"] = rng.randint(0, c["past_hi"])
        keys = c["new_hi"] + c["past_hi"]
        w = work(c)
        if (c["batch"] * c["heads"] * c["new_hi"] * keys <= 2048 * 8192 * 32 and w["flops"] <= 2.4e11
                and c["batch"] * keys * c["kv_heads"] * dim <= 64 * 8192 * 8 * 128):
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


def _pairs_and_keys(case):
    """How many (query, key) pairs the masks leave, and how many keys some query of their sequence sees."""
    pairs = keys = 0
    w, s = case["window"], case["sinks"]
    for n, ctx in _lengths(case):
        if not ctx:
            continue
        seen = torch.arange(ctx - n + 1, ctx + 1, dtype=torch.int64)  # keys up to each query
        if w:
            near = seen.clamp(max=w)
            seen = near + (seen - near).clamp(max=s)
            first = max(0, ctx - n + 1 - w)
            keys += ctx - first + min(first, s)
        else:
            keys += ctx
        pairs += int(seen.sum())
    return pairs, keys


def work(case):
    d, hk = case["dim"], case["kv_heads"]
    if case["op"] != "attend":
        rows = 2 * (case["tokens"] - case["skip"]) * hk  # rows of keys and of values
        size = 2 if case["dtype"] == "bf16" else 4
        out = 2 * case["skip"] * hk * d * size if case["op"] == "read" else 0  # (skipped places read as zero)
        return {"bytes": rows * (d * (size + 1) + 1) + 8 * case["tokens"] + out, "flops": rows * d * 2}
    pairs, keys = _pairs_and_keys(case)
    new = sum(n for n, _ in _lengths(case))
    size = 2 * keys * hk * (d + 1) + new * case["heads"] * (2 * d * 2 + (4 if case["lse"] else 0))
    return {"bytes": size + 4 * (-(-keys // case["page"])) + 8 * case["batch"], "flops": 4 * d * case["heads"] * pairs}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _encode(x):
    """E4M3 codes and UE8M0 scale codes of rows x [..., D] (FP32): the scale is the row's largest magnitude
    over 448, raised to a power of two; a row of zeros has scale 1."""
    t = x.abs().amax(-1) / 448.0
    bits = t.view(torch.int32)
    sf = ((bits >> 23) + ((bits & 0x7FFFFF) != 0)).clamp(min=1)
    sf = torch.where(t == 0, torch.full_like(sf, 127), sf)
    q = (x / (sf << 23).view(torch.float32).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8), sf.to(torch.uint8)


def _rows(g, tokens, heads, dim):
    """Keys or values of `tokens` tokens: normal, tokens of different size, a few large channels."""
    x = _normal(g, tokens, heads, dim)
    x *= torch.exp(0.5 * _normal(g, tokens, heads, 1))
    x *= 1.0 + 3.0 * (torch.rand((1, heads, dim), generator=g, device=DEV) < 0.03)
    return x


def _filled_cache(g, pages, heads, page, dim):
    """(codes, scale codes) of a cache whose every place holds a token."""
    q, sf = _encode(_rows(g, pages * page, heads, dim))
    codes = q.view(pages, page, heads, dim).transpose(1, 2).contiguous()
    return codes, sf.view(pages, page, heads).transpose(1, 2).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] != "attend":
        t = case["tokens"]
        pages = -(-t // page) + 2
        st = {"op": case["op"], "page": page, "dtype": torch.bfloat16 if case["dtype"] == "bf16" else torch.float32}
        # whole pages in any order, as an allocator hands them out; the tokens of a page in a row
        order = torch.randperm(pages, generator=g, device=DEV)
        i = torch.arange(t, device=DEV)
        slots = order[i // page] * page + i % page
        slots[torch.randperm(t, generator=g, device=DEV)[: case["skip"]]] = -1
        st["slots"] = slots
        st["k_cache"] = _filled_cache(g, pages, hk, page, d)
        st["v_cache"] = _filled_cache(g, pages, hk, page, d)
        if case["op"] == "write":
            st["k"] = _rows(g, t, hk, d).to(st["dtype"])
            st["v"] = _rows(g, t, hk, d).to(st["dtype"])
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
    st = {"op": "attend", "page": page, "window": case["window"], "sinks": case["sinks"], "lse": case["lse"],
          "table": table.to(DEV), "seq_lens": torch.tensor(ctx, dtype=torch.int32, device=DEV), "cu": cu.to(DEV),
          "max_new": max(new), "max_ctx": max(ctx), "same_new": min(new) == max(new)}
    st["k_cache"] = _filled_cache(g, pages, hk, page, d)
    st["v_cache"] = _filled_cache(g, pages, hk, page, d)
    q = _normal(g, sum(new), case["heads"], d)
    st["q"] = q.to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- one pass
def _cache_values(st):
    """The cache as the values it stands for."""
    return [t for codes, sf in (st["k_cache"], st["v_cache"])
            for t in (codes.view(torch.float8_e4m3fn), sf.view(torch.float8_e8m0fnu))]


def _decode(codes, sf):
    return codes.view(torch.float8_e4m3fn).float() * (sf.to(torch.int32) << 23).view(torch.float32).unsqueeze(-1)


def _plain_write(st):
    valid = st["slots"] >= 0
    i = torch.arange(valid.numel(), device=DEV)
    i = torch.where(valid, i, valid.to(torch.int32).argmax())  # a skipped token repeats the first one's write
    slots = st["slots"][i]
    at, place = slots // st["page"], slots % st["page"]
    for x, (codes, sf) in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
        q, s = _encode(x[i].float())
        codes[at, :, place] = q
        sf[at, :, place] = s


def _plain_read(st):
    valid = st["slots"] >= 0
    slots = st["slots"].clamp(min=0)
    at, place = slots // st["page"], slots % st["page"]
    return [torch.where(valid[:, None, None], _decode(codes[at, :, place], sf[at, :, place]), 0.0).to(st["dtype"])
            for codes, sf in (st["k_cache"], st["v_cache"])]


def _plain_attend(st):
    q, table, cu, ctx = st["q"], st["table"].long(), st["cu"].long(), st["seq_lens"].long()
    total, heads, d = q.shape
    b, n = table.shape[0], st["max_new"]
    hk = st["k_cache"][0].shape[1]
    # queries padded to [b, hk, group * n, d]; row i of a sequence is its query i % n
    new = cu[1:] - cu[:-1]
    row = torch.arange(n, device=DEV)
    src = (cu[:-1, None] + row).clamp(max=total - 1)
    x = q[src].float().view(b, n, hk, heads // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)

    def keys(cache):  # [b, hk, columns * page, d]
        return _decode(*cache)[table].transpose(1, 2).reshape(b, hk, -1, d)

    s = torch.matmul(x, keys(st["k_cache"]).transpose(2, 3)) * (1.0 / math.sqrt(d))
    at = ctx[:, None, None] - new[:, None, None] + row[None, :, None]  # a query's place in its sequence
    j = torch.arange(s.shape[-1], device=DEV)[None, None, :]
    seen = j <= at
    if st["window"]:
        seen = seen & ((j > at - st["window"]) | (j < st["sinks"]))
    seen = seen[:, None, None]
    s = s.view(b, hk, heads // hk, n, -1).masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, hk, -1, p.shape[-1]), keys(st["v_cache"])).view(b, hk, heads // hk, n, d)
    o = o / torch.where(z == 0, torch.ones_like(z), z)
    # back to the packed rows
    t = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    place = t - cu[seq]
    out = [o.permute(0, 3, 1, 2, 4).reshape(b, n, heads, d)[seq, place].to(torch.bfloat16)]
    if st["lse"]:
        out.append((top + z.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(b, n, heads)[seq, place])
    return out


def run(state):
    st = state
    if own:
        import block_scaled_fp8_amd as dg
        if st["op"] == "write":
            dg.fp8_kv_cache_write(st["k"], st["v"], st["k_cache"], st["v_cache"], st["slots"])
            return _cache_values(st)
        if st["op"] == "read":
            return dg.fp8_kv_cache_read(st["k_cache"], st["v_cache"], st["slots"], out_dtype=st["dtype"])
        r = dg.fp8_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seq_lens"],
                                   cu_seqlens_q=None if st["same_new"] else st["cu"], max_seqlen_q=st["max_new"],
                                   max_seqlen_k=st["max_ctx"], window=st["window"], sinks=st["sinks"],
                                   return_lse=st["lse"])
        return r if st["lse"] else [r]
    if st["op"] == "write":
        _plain_write(st)
        return _cache_values(st)
    return _plain_read(st) if st["op"] == "read" else _plain_attend(st)


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


def exact(case, seed):
    st = prepare(case, seed)
    page = st["page"]
    if case["op"] == "write":
        out = []
        live = torch.nonzero(st["slots"] >= 0).flatten()
        slots = st["slots"][live]
        for x, cache in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
            val, scale = _values64(cache)
            x = x[live].double()
            top = x.abs().amax(-1)
            frac, e = torch.frexp(top / 448.0)  # frac in [1/2, 1): the next power of two is 2^e, or 2^(e-1) itself
            e = torch.where(top == 0, torch.zeros_like(e), torch.where(frac == 0.5, e - 1, e))
            y = x / _power64(e).unsqueeze(-1)
            step = _power64(torch.frexp(y.abs())[1].clamp(min=-5) - 4)  # spacing of E4M3 at |y|
            val[slots // page, :, slots % page] = torch.round(y / step) * step
            scale[slots // page, :, slots % page] = _power64(e)
            out += [val, scale]
        return out
    if case["op"] == "read":
        out = []
        for cache in (st["k_cache"], st["v_cache"]):
            val, scale = _values64(cache)
            x = (val * scale.unsqueeze(-1)).transpose(1, 2).flatten(0, 1)[st["slots"].clamp(min=0)]
            x[st["slots"] < 0] = 0.0
            out.append(x)
        return out
    total, heads, d = st["q"].shape
    hk = case["kv_heads"]
    group = heads // hk
    o = torch.zeros((total, heads, d), dtype=torch.float64, device=DEV)
    lse = torch.full((total, heads), -math.inf, dtype=torch.float64, device=DEV)
    cu, lens = st["cu"].tolist(), st["seq_lens"].tolist()
    for b, ctx in enumerate(lens):
        first, n = cu[b], cu[b + 1] - cu[b]
        if not ctx:
            continue
        pages = st["table"][b, : -(-ctx // page)].long()
        kv = []
        for codes, sf in (st["k_cache"], st["v_cache"]):
            val, scale = _values64((codes[pages], sf[pages]))
            kv.append((val * scale.unsqueeze(-1)).transpose(0, 1).flatten(1, 2)[:, :ctx])
        place = torch.arange(ctx - n, ctx, device=DEV)[:, None]
        j = torch.arange(ctx, device=DEV)[None, :]
        hidden = j > place
        if case["window"]:
            hidden |= (j <= place - case["window"]) & (j >= case["sinks"])
        for h in range(heads):
            s = st["q"][first: first + n, h].double() @ kv[0][h // group].T / math.sqrt(d)
            s[hidden] = -math.inf
            lse[first: first + n, h] = torch.logsumexp(s, -1)
            o[first: first + n, h] = torch.softmax(s, -1) @ kv[1][h // group]
    return [o, lse] if case["lse"] else [o]
