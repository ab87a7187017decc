"""GPU parity of the FP8 key/value cache (write, read back) and of the attention that reads it, through
the binding, against the float64 oracle."""
import contextlib

import numpy as np
import pytest
import torch

import block_scaled_fp8_amd as dg
import oracle
from tests import kv_gen

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print(*a, flush=True)


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def same(a, b):
    """Arrays equal, NaN for NaN (says where not, not what)."""
    a, b = np.asarray(a), np.asarray(b)
    ok = (a == b) | ((a != a) & (b != b))
    if not ok.all():
        at = np.argwhere(~ok)
        say("differ at", len(at), "places, first", at[:4].tolist(), a[~ok][:4], b[~ok][:4])
    return bool(ok.all())


@contextlib.contextmanager
def num_sms(n):
    """Plan for n compute units: more of them split the keys into more parts."""
    dg.set_num_sms(n)
    try:
        yield
    finally:
        dg.set_num_sms(0)


# ---------------------------------------------------------------- write
def rand_cache(rng, pages, heads, page, dim):
    return (rng.integers(0, 0x7F, (pages, heads, page, dim)).astype(np.uint8), rng.integers(100, 140, (pages, heads, page)).astype(np.uint8))


def tricky_rows(rng, tokens, heads, dim):
    """Rows whose scale or rounding sits on an edge: zeros, amax at and beside 448 * 2^e, halfway values,
    FP32 subnormals, the largest numbers."""
    x = kv_gen.rows(rng, tokens, heads, dim, wide=True)
    f = x.reshape(-1, dim)
    f[0] = 0.0
    f[1] = -0.0
    for i, e in enumerate((-130, -126, -100, -3, 0, 5, 100)):
        top = np.float32(448.0) * np.float32(2.0 ** e) if e > -127 else np.float32(2.0 ** -125)
        for j, t in enumerate((np.nextafter(top, np.float32(0)), top, np.nextafter(top, np.float32(np.inf)))):
            r = 2 + 3 * i + j
            f[r] = rng.uniform(-1, 1, dim).astype(np.float32) * t
            f[r, r % dim] = t * (-1 if j == 1 else 1)
    f[23] = np.float32(2.0 ** -149)
    f[24] = np.finfo(np.float32).max
    f[25] = (rng.integers(8, 16, dim) + 0.5).astype(np.float32) * 2.0 ** rng.integers(-6, 5, dim)  # ties
    f[25, 0] = 448.0
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,heads,page,order", [(64, 5, 16, "hpt"), (128, 8, 64, "hpt"), (128, 3, 48, "thd"), (256, 2, 7, "thd"),
                                                  (64, 1, 1, "hpt")])
def test_write_is_bitwise(dtype, dim, heads, page, order):
    rng = np.random.default_rng(dim + heads + page)
    tokens = 61
    x = [tricky_rows(rng, tokens, heads, dim) for _ in range(2)]
    if dtype == torch.bfloat16:
        x = [oracle.bf16_bits_to_f64(oracle.bf16_rne(np.clip(v, -3e38, 3e38))).astype(np.float32) for v in x]
    pages = -(-tokens // page) + 3
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[[3, 17]] = [-1, -(2 ** 40)]
    slots[[5, 20]] = [pages * page, 2 ** 40]
    before = [rand_cache(rng, pages, heads, page, dim) for _ in range(2)]
    say("kv write", dtype, dim, heads, page, order)
    # new tokens' keys and values as slices of one projection's output
    qkv = torch.empty((tokens, 3 * heads, dim), dtype=dtype, device=DEV)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    k.copy_(cuda(x[0]))
    v.copy_(cuda(x[1]))
    if order == "hpt":
        caches = [(cuda(c), cuda(s)) for c, s in before]
    else:  # tokens outermost within a page
        caches = [(cuda(c.swapaxes(1, 2)).transpose(1, 2), cuda(s.swapaxes(1, 2)).transpose(1, 2)) for c, s in before]
    dg.fp8_kv_cache_write(k, v, caches[0], caches[1], cuda(slots))
    torch.cuda.synchronize()
    for i in range(2):
        codes, sf = oracle.kv_write(before[i], x[i], slots)
        assert same(caches[i][1].cpu().numpy(), sf), i
        assert same(caches[i][0].cpu().numpy(), codes), i


def test_write_infinities_and_nans():
    """An infinity saturates and does not count for the scale; a NaN becomes the NaN code; neighbours are not touched."""
    rng = np.random.default_rng(0)
    x = kv_gen.rows(rng, 3, 2, 64)
    want = [oracle.kv_encode(x), None]
    y = x.copy()
    at = np.abs(y).argmin(axis=-1)  # (an element that does not set the scale)
    y[0, 0, at[0, 0]], y[0, 1, at[0, 1]] = np.inf, -np.inf
    y[1, 0, at[1, 0]] = np.nan
    k_cache, v_cache = dg.fp8_kv_cache_empty(1, 2, 4, 64, device=DEV)
    say("kv write, non-finite values")
    dg.fp8_kv_cache_write(cuda(y), cuda(x), k_cache, v_cache, torch.arange(3, device=DEV))
    torch.cuda.synchronize()
    codes, sf = want[0][0].copy(), want[0][1]
    codes[0, 0, at[0, 0]], codes[0, 1, at[0, 1]] = 0x7E, 0xFE
    got = k_cache[0][0].cpu().numpy().swapaxes(0, 1)[:3]
    assert got[1, 0, at[1, 0]] & 0x7F == 0x7F
    codes[1, 0, at[1, 0]] = got[1, 0, at[1, 0]]
    assert same(got, codes) and same(k_cache[1][0].cpu().numpy().T[:3], sf)
    assert same(v_cache[0][0].cpu().numpy().swapaxes(0, 1)[:3], want[0][0])
    allinf = torch.full((1, 2, 64), float("inf"), device=DEV)
    dg.fp8_kv_cache_write(allinf, allinf, k_cache, v_cache, torch.tensor([3], device=DEV))
    torch.cuda.synchronize()
    assert (k_cache[0][0, :, 3].cpu() == 0x7E).all() and (k_cache[1][0, :, 3].cpu() == 127).all()


def test_write_and_read_of_nothing():
    k_cache, v_cache = dg.fp8_kv_cache_empty(2, 2, 4, 64, device=DEV)
    x = torch.empty((0, 2, 64), device=DEV)
    slots = torch.empty((0,), dtype=torch.int64, device=DEV)
    dg.fp8_kv_cache_write(x, x, k_cache, v_cache, slots)
    k, v = dg.fp8_kv_cache_read(k_cache, v_cache, slots)
    assert k.shape == (0, 2, 64) and v.dtype == torch.bfloat16


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 8, 64), (256, 1, 5)])
def test_read_is_exact(dtype, dim, heads, page):
    rng = np.random.default_rng(dim)
    pages = 6
    cache = [(rng.integers(0, 256, (pages, heads, page, dim)).astype(np.uint8), rng.integers(20, 230, (pages, heads, page)).astype(np.uint8))
             for _ in range(2)]
    slots = rng.integers(-2, pages * page + 2, 77).astype(np.int64)
    say("kv read", dtype, dim, heads, page)
    out = tuple(torch.full((77, heads + 1, dim), 5.0, dtype=dtype, device=DEV)[:, :heads] for _ in range(2))
    got = dg.fp8_kv_cache_read(*[(cuda(c).view(torch.float8_e4m3fn), cuda(s).view(torch.float8_e8m0fnu)) for c, s in cache], cuda(slots),
                               out_dtype=dtype, out=out)
    torch.cuda.synchronize()
    for i in range(2):
        assert same(got[i].double().cpu().numpy(), oracle.kv_read(cache[i], slots))


# ---------------------------------------------------------------- attention
def run(p, window=0, sinks=0, lse=True, scale=None, **kw):
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    r = dg.fp8_paged_attention(q, caches[0], caches[1], cuda(p["table"]), cuda(p["lens"]), cu_seqlens_q=cuda(p["cu"]),
                               max_seqlen_q=max(p["news"]), sm_scale=scale, window=window, sinks=sinks, return_lse=lse, **kw)
    torch.cuda.synchronize()
    return r


def check(p, got, window=0, sinks=0, scale=None):
    o = oracle.paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"],
                               scale if scale is not None else p["dim"] ** -0.5, window, sinks)
    tol, tol_lse = kv_gen.bounds(o, p["dim"])
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    err = np.abs(out - o["out"])
    say("largest error / bound", float((err / tol).max()) if err.size else 0.0)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(~(err <= tol))[:5])
    blind = np.isneginf(o["lse"])
    assert same(np.isneginf(lse), blind) and (out[blind] == 0).all()
    with np.errstate(invalid="ignore"):
        assert (np.abs(lse - o["lse"])[~blind] <= tol_lse[~blind]).all()


# lengths (tokens in the cache) and new tokens; heads, key heads, head dim, page size
CASES = {
    "one_token": ([1], [1], 4, 1, 128, 16),
    "single_tokens": ([0, 1, 31, 32, 33, 64, 65, 127, 300], [1] * 9, 16, 2, 128, 16),
    "single_tokens_64": ([5, 0, 700], [1] * 3, 5, 5, 64, 1),
    "single_tokens_256": ([130, 63, 1], [1] * 3, 8, 2, 256, 32),
    "groups_of_seven": ([100, 37, 64], [3, 5, 4], 14, 2, 64, 16),
    "forty_heads_one_key_head": ([90, 17], [1, 2], 40, 1, 128, 100),
    "more_new_than_held": ([3, 0, 40], [5, 2, 41], 4, 2, 128, 16),
    "chunks": ([200, 129, 64, 1], [130, 129, 1, 1], 4, 2, 128, 48),
    "chunks_64": ([300, 100, 65], [64, 100, 33], 12, 4, 64, 7),
    "chunks_256": ([190, 70], [140, 70], 2, 1, 256, 64),
    "long": ([1500, 1027], [70, 2], 8, 2, 128, 64),
}


@pytest.mark.parametrize("mask", [(0, 0), (1, 0), (40, 0), (70, 4), (33, 100), (5, 1)])
@pytest.mark.parametrize("name", sorted(CASES))
def test_attention(name, mask):
    lens, news, *shape = CASES[name]
    p = kv_gen.problem(lens, news, *shape, seed=len(name))
    say("attention", name, mask)
    check(p, run(p, *mask), *mask)


@pytest.mark.parametrize("mask", [(0, 0), (300, 5)])
@pytest.mark.parametrize("name", ["chunks", "long", "single_tokens", "more_new_than_held", "single_tokens_256"])
def test_attention_in_parts(name, mask):
    """As many parts of the keys as the planner ever makes, some of them without a key for a row."""
    lens, news, *shape = CASES[name]
    p = kv_gen.problem(lens, news, *shape, seed=3)
    say("attention in parts", name, mask)
    with num_sms(1 << 14):
        # (a host bound far above the lengths asks for parts that have no tile)
        got = run(p, *mask, max_seqlen_k=1 << 16)
    check(p, got, *mask)


@pytest.mark.parametrize("hint", [0, 1, 40, 1 << 20])
@pytest.mark.parametrize("name", ["single_tokens", "long"])
def test_attention_with_a_wrong_bound_of_the_lengths(name, hint):
    """max_seqlen_k guides the split and nothing else, whatever it says."""
    lens, news, *shape = CASES[name]
    p = kv_gen.problem(lens, news, *shape, seed=12)
    say("attention, bound", name, hint)
    for sms in (0, 3, 1 << 14):
        with num_sms(sms):
            got = run(p, max_seqlen_k=hint)
        check(p, got)


@pytest.mark.parametrize("new", [1, 3, 40])
def test_attention_of_many_sequences(new):
    """More items than the lanes that look them up, empty sequences among them, whole and in parts."""
    rng = np.random.default_rng(new)
    lens = [int(x) for x in rng.integers(0, 400, 75)]
    lens[0] = lens[64] = lens[74] = 0
    p = kv_gen.problem(lens, [new if i % 7 else 0 for i in range(75)], 8, 2, 64, 16, seed=new)
    say("attention, many sequences", new)
    for sms in (0, 1 << 12):
        with num_sms(sms):
            check(p, run(p))
            check(p, run(p, 50, 3), 50, 3)


@pytest.mark.parametrize("sms", [24, 40, 150])
@pytest.mark.parametrize("dim,new", [(64, 1), (64, 11), (128, 2), (128, 30), (256, 1), (256, 9)])
def test_attention_few_rows_in_few_parts(dim, new, sms):
    """Ragged batches of few rows whose items are cut into two or three parts, or stay whole."""
    rng = np.random.default_rng(dim + new)
    lens = [int(x) for x in rng.integers(0, 900, 30)]
    lens[3], lens[17] = 0, 1
    news = [int(x) for x in rng.integers(0, new + 1, 30)]
    news[29] = new
    p = kv_gen.problem(lens, news, 8, 2, dim, 32, seed=dim + new)
    say("attention, few parts", dim, new, sms)
    with num_sms(sms):
        check(p, run(p, max_seqlen_k=1 << 14))
        check(p, run(p, 100, 3, max_seqlen_k=1 << 14), 100, 3)


@pytest.mark.parametrize("seqs,sms", [(1, 1), (2, 2), (5, 5), (5, 12), (128, 100), (130, 100)])
@pytest.mark.parametrize("dim,group,mask", [(64, 4, (0, 0)), (128, 8, (200, 3)), (256, 4, (0, 0))])
def test_attention_pieces_by_size(dim, group, mask, seqs, sms):
    """Many rows of unequal sequences: whole and cut items of all sizes in one call, up to as many as are sorted
    and more; two rows of a lane group in the join (5 compute units for 5 sequences, say)."""
    rng = np.random.default_rng(seqs)
    small = seqs > 8
    lens = [int(x) for x in rng.integers(0, 120 if small else 1500, seqs)]
    lens[-1] = 130 if small else 2600
    news = [int(x) for x in rng.integers(0, 4 if small else 90, seqs)]
    news[seqs // 2] = 256 // group + 3 if dim == 128 else 128 // group + 3
    p = kv_gen.problem(lens, news, 2 * group, 2, dim, 16, seed=seqs)
    say("attention, pieces by size", dim, mask, seqs, sms)
    for most in (None, 1 << 14):
        with num_sms(sms):
            got = run(p, *mask) if most is None else run(p, *mask, max_seqlen_k=most)
        check(p, got, *mask)


def test_attention_scale_and_large_scores():
    """Scores of hundreds: the running maximum moves far, weights underflow."""
    p = kv_gen.problem([200, 77], [70, 1], 4, 2, 128, 16, seed=9)
    say("attention, large scores")
    for scale in (1e-3, 3.0):
        check(p, run(p, scale=scale), scale=scale)


def test_attention_strides_and_rows_of_no_sequence():
    """q and out as slices, cache with tokens outermost in a page; rows outside the sequences stay as they were."""
    p = kv_gen.problem([70, 33], [40, 1], 6, 3, 64, 16, seed=4)
    caches = [(cuda(p[x][0].swapaxes(1, 2)).transpose(1, 2), cuda(p[x][1].swapaxes(1, 2)).transpose(1, 2)) for x in "kv"]
    big = torch.full((45, 12, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    big[2:43, 3:9] = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    table = torch.full((2, p["table"].shape[1] + 3), -7, dtype=torch.int32, device=DEV)
    table[:, :-3] = cuda(p["table"])
    for sms in (0, 4096):
        out = torch.full((45, 9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        say("attention, strided", sms)
        with num_sms(sms):
            got, lse = dg.fp8_paged_attention(big[:, 3:9], *caches, table[:, :-3], cuda(p["lens"]), cu_seqlens_q=cuda(p["cu"] + 2),
                                              max_seqlen_q=40, max_seqlen_k=1 << 16 if sms else 70, out=out[:, 1:7], return_lse=True)
        torch.cuda.synchronize()
        check(p, (got[2:43], lse[2:43]))
        keep = torch.ones(45, 9, dtype=torch.bool, device=DEV)
        keep[2:43, 1:7] = False
        assert (out[keep] == 7.0).all()


def test_attention_equal_lengths_without_cu():
    p = kv_gen.problem([50, 51, 100], [2, 2, 2], 8, 2, 128, 16, seed=5)
    a = run(p)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    b = dg.fp8_paged_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), return_lse=True)
    torch.cuda.synchronize()
    check(p, b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_is_deterministic_on_another_stream_and_in_a_graph():
    p = kv_gen.problem([900, 33, 0, 500], [1, 1, 1, 1], 8, 2, 128, 16, seed=6)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    table, lens = cuda(p["table"]), cuda(p["lens"])
    out = torch.empty_like(q)

    def call():
        return dg.fp8_paged_attention(q, *caches, table, lens, max_seqlen_k=900, out=out)

    say("attention, stream and graph")
    first = call().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        again = call().clone()
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for step in range(3):  # (lengths change between replays, as in a decode loop)
        lens.copy_(cuda(np.maximum(p["lens"] - step, 0)))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(4.0)
        assert torch.equal(call(), got), step
        torch.cuda.synchronize()


def test_cache_past_4_gib():
    """Pages whose byte offsets pass 32 bits: written, attended, read back."""
    heads, page, dim, pages = 2, 16, 128, 9
    stride = (1 << 29) + 16  # 8 * stride > 2^32
    buf = torch.empty((8 * stride + 2 * heads * page * dim,), dtype=torch.uint8, device=DEV)
    shape, st = (pages, heads, page, dim), (stride, page * dim, dim, 1)
    say("cache past 4 GiB")
    k_codes, v_codes = buf.as_strided(shape, st), buf[heads * page * dim:].as_strided(shape, st)
    sf = torch.full((2, pages, heads, page), 127, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(1)
    n = 50
    x = [kv_gen.rows(rng, n, heads, dim) for _ in range(2)]
    table = np.array([[8, 0, 7, 5]], np.int32)
    slots = table[0][np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
    caches = (k_codes, sf[0]), (v_codes, sf[1])
    dg.fp8_kv_cache_write(cuda(x[0]), cuda(x[1]), *caches, cuda(slots))
    back = dg.fp8_kv_cache_read(*caches, cuda(slots), out_dtype=torch.float32)
    torch.cuda.synchronize()
    for i in range(2):
        assert same(back[i].double().cpu().numpy(), oracle.kv_decode(*oracle.kv_encode(x[i])))
    p = {"dim": dim, "page": page, "table": table, "lens": np.array([n], np.int32)}
    host = [(np.zeros(shape, np.uint8), np.full(shape[:3], 127, np.uint8)) for _ in range(2)]
    p["k"], p["v"] = (oracle.kv_write(host[i], x[i], slots) for i in range(2))
    for new in (1, 50):
        q = rng.standard_normal((new, 4, dim))
        p["q_bits"] = oracle.bf16_rne(q)
        p["q"], p["cu"], p["news"] = oracle.bf16_bits_to_f64(p["q_bits"]), np.array([0, new], np.int32), [new]
        got = dg.fp8_paged_attention(cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16), *caches, cuda(table), cuda(p["lens"]),
                                     return_lse=True)
        torch.cuda.synchronize()
        check(p, got)


def test_write_then_attend_matches_unquantised_attention():
    """End to end through the library's own cache: within E4M3's step of attention over the keys and values themselves."""
    rng = np.random.default_rng(8)
    n, heads, dim, page = 90, 2, 128, 16
    x = [rng.standard_normal((n, heads, dim)).astype(np.float32) for _ in range(2)]
    k_cache, v_cache = dg.fp8_kv_cache_empty(8, heads, page, dim, device=DEV)
    table = torch.tensor([[7, 2, 5, 0, 1, 3]], dtype=torch.int32, device=DEV)
    i = torch.arange(n, device=DEV)
    slots = table[0, i // page].long() * page + i % page
    dg.fp8_kv_cache_write(cuda(x[0]), cuda(x[1]), k_cache, v_cache, slots)
    q = torch.randn((3, 4, dim), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).bfloat16()
    out = dg.fp8_paged_attention(q, k_cache, v_cache, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    k, v = (torch.from_numpy(a).double().repeat_interleave(2, 1) for a in x)
    s = torch.einsum("qhd,khd->hqk", q.double().cpu(), k) / dim ** 0.5
    s = s.masked_fill(torch.arange(n)[None, None] > torch.arange(n - 3, n)[None, :, None], float("-inf"))
    want = torch.einsum("hqk,khd->qhd", s.softmax(-1), v)
    rel = float((out.double().cpu() - want).norm() / want.norm())
    # E4M3 rounds values by up to 2^-4; errors of different keys average out
    assert rel < 2.0 ** -4, rel


@pytest.mark.parametrize("mask", [(0, 0), (50, 4)])
def test_attention_layer_example(mask):
    """The library's parts together as a serving layer uses them.  Chunks and single tokens differ from one chunk by
    the rounding of the attention's output to BF16 (2^-8) and of that to E4M3 (2^-4), where a last bit may flip."""
    from examples import attention_layer
    say("attention layer", mask)
    off, moved = attention_layer.main(*mask)
    assert moved and off < 2.0 ** -6


def test_quantised_values_survive_being_written_again():
    """Reading back and writing again gives the same values, whatever the scales: E4M3 values times a power of two.
    (The row of FP32's largest number is rounded up to 2^128, which FP32 does not have: it reads as infinity.)"""
    rng = np.random.default_rng(3)
    x = tricky_rows(rng, 30, 2, 128)
    k_cache, v_cache = dg.fp8_kv_cache_empty(4, 2, 16, 128, device=DEV)
    slots = torch.arange(30, device=DEV)
    dg.fp8_kv_cache_write(cuda(x), cuda(x[::-1]), k_cache, v_cache, slots)
    first = dg.fp8_kv_cache_read(k_cache, v_cache, slots, out_dtype=torch.float32)
    dg.fp8_kv_cache_write(*first, k_cache, v_cache, slots + 30)
    again = dg.fp8_kv_cache_read(k_cache, v_cache, slots + 30, out_dtype=torch.float32)
    torch.cuda.synchronize()
    for a, b in zip(first, again):
        fine = torch.isfinite(a).all(-1)
        assert int((~fine).sum()) == 1
        assert same(a[fine].cpu().numpy(), b[fine].cpu().numpy())


# ---------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("sms", [0, 24, 1 << 14])
@pytest.mark.parametrize("name", ["single_tokens", "single_tokens_256", "groups_of_seven", "chunks", "chunks_64", "chunks_256", "long"])
def test_a_query_that_is_not_a_number_gives_no_number(name, sms):
    """A NaN or infinite query shows in its own output and log-sum, whole and however its keys are cut, and in no
    other's; one that sees no key gives zeros and -infinity like every other."""
    lens, news, *shape = CASES[name]
    p = kv_gen.problem(lens, news, *shape, seed=21)
    heads, dim = shape[0], shape[2]
    keys = np.concatenate([np.arange(n) + length - n + 1 for length, n in zip(lens, news)])  # that a row sees
    seen = keys > 0
    rng = np.random.default_rng(5)
    rows = np.unique(np.concatenate([np.flatnonzero(seen)[::3], np.flatnonzero(~seen)[:2], np.flatnonzero(seen)[-1:]]))
    bad = np.zeros((len(seen), heads), bool)
    q = p["q_bits"].copy()
    for i, t in enumerate(rows):
        h = int(rng.integers(heads))
        bad[t, h] = True
        if i % 3 == 0:
            q[t, h, int(rng.integers(dim))] = 0x7FC0   # one NaN
        elif i % 3 == 1 or keys[t] < 40:
            q[t, h] = 0x7F80                           # all infinite: products of both signs for every key
        else:
            q[t, h, int(rng.integers(dim))] = 0x7F80   # one infinity: scores of both signs
    say("attention, queries that are not numbers", name, sms)
    with num_sms(sms):
        got = run({**p, "q_bits": q}, max_seqlen_k=1 << 16 if sms else None)
    nan_out, nan_lse = got[0].isnan().cpu().numpy(), got[1].isnan().cpu().numpy()
    want = bad & seen[:, None]
    assert same(nan_lse, want) and same(nan_out.all(-1), want) and same(nan_out.any(-1), want)
    # (the others as the oracle has them without; their last bits may move, since rows of a wave raise their running
    # maxima together)
    o = oracle.paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], dim ** -0.5)
    tol, tol_lse = kv_gen.bounds(o, dim)
    assert (np.abs(got[0].double().cpu().numpy() - o["out"]) <= tol)[~want].all()
    lse = got[1].double().cpu().numpy()
    blind = np.isneginf(o["lse"])
    assert same(np.isneginf(lse)[~want], blind[~want])
    assert (np.abs(lse - np.where(blind, 0.0, o["lse"])) <= tol_lse)[~want & ~blind].all()


def test_one_row_of_the_block_table_for_all_sequences():
    """A shared prompt with several samples: an expanded table, whole and cut, gives what its copy gives."""
    p = kv_gen.problem([300], [1], 8, 2, 128, 16, seed=31)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    table = cuda(p["table"]).expand(5, -1)
    assert table.stride(0) == 0
    lens = torch.tensor([300, 17, 0, 299, 160], dtype=torch.int32, device=DEV)
    for new in (1, 40):
        q = torch.randn((5 * new, 8, 128), generator=torch.Generator(DEV).manual_seed(new), device=DEV).bfloat16()
        for sms in (0, 1 << 12):
            say("attention, expanded table", new, sms)
            with num_sms(sms):
                got, want = (dg.fp8_paged_attention(q, *caches, t, lens, return_lse=True) for t in (table, table.contiguous()))
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_tokens_than_a_launch_holds():
    """2^28 rows of 128 values take 16 lanes each, 2^32 threads; every token but six has no slot, and all share one row."""
    n = (1 << 28) + 9
    k_cache, v_cache = dg.fp8_kv_cache_empty(1, 1, 16, 128, device=DEV)
    row = torch.from_numpy(kv_gen.rows(np.random.default_rng(2), 1, 1, 128)).to(DEV)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    for i, t in enumerate((0, (1 << 26) + 1, (1 << 28) - 1, 1 << 28, n - 2, n - 1)):
        slots[t] = i
    say("kv write, 2^28 tokens")
    x = row.expand(n, -1, -1)
    dg.fp8_kv_cache_write(x, x, k_cache, v_cache, slots)
    torch.cuda.synchronize()
    codes, sf = oracle.kv_encode(row.cpu().numpy())
    for c, s in (k_cache, v_cache):
        assert same(c[0, 0, :6].cpu().numpy(), np.repeat(codes[:, 0], 6, 0)) and same(s[0, 0, :6].cpu().numpy(), np.repeat(sf[:, 0], 6))
        assert (c[0, 0, 6:] == 0).all()


@pytest.mark.parametrize("max_q", [2, 30, 200])
def test_a_call_whose_sequences_have_no_rows(max_q):
    """cu_seqlens_q of one number, with rows present and keys enough to be cut: nothing is written."""
    p = kv_gen.problem([900, 500, 0], [0, 0, 0], 8, 2, 128, 16, seed=41)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    q = torch.randn((200, 8, 128), device=DEV).bfloat16()
    for first in (0, 7, 200):
        cu = torch.full((4,), first, dtype=torch.int32, device=DEV)
        for sms in (0, 1 << 12):
            out = torch.full_like(q, 3.0)
            say("attention, no rows", max_q, first, sms)
            with num_sms(sms):
                dg.fp8_paged_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), cu_seqlens_q=cu, max_seqlen_q=max_q, max_seqlen_k=900,
                                       out=out, return_lse=True)
            torch.cuda.synchronize()
            assert (out == 3.0).all()


@pytest.mark.parametrize("batch,max_q", [(0, 5), (2, 0)])
def test_rows_of_a_call_without_sequences_or_new_tokens(batch, max_q):
    """Rows that can belong to no sequence see nothing: zeros and -infinity; a given out stays as it was."""
    k_cache, v_cache = dg.fp8_kv_cache_empty(2, 2, 16, 64, device=DEV)
    q = torch.randn((6, 4, 64), device=DEV).bfloat16()
    table, lens = torch.zeros((batch, 2), dtype=torch.int32, device=DEV), torch.full((batch,), 20, dtype=torch.int32, device=DEV)
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
    say("attention, no sequences", batch, max_q)
    left = torch.full_like(q, 7.0), torch.full((6, 4), 7.0, device=DEV)  # (memory that the call's results are likely to get)
    del left
    out, lse = dg.fp8_paged_attention(q, k_cache, v_cache, table, lens, cu_seqlens_q=cu, max_seqlen_q=max_q, return_lse=True)
    mine = torch.full_like(q, 3.0)
    dg.fp8_paged_attention(q, k_cache, v_cache, table, lens, cu_seqlens_q=cu, max_seqlen_q=max_q, out=mine)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all() and (mine == 3.0).all()


@pytest.mark.parametrize("sms", [0, 24, 1 << 14])
@pytest.mark.parametrize("mask", [(0, 0), (33, 0), (20, 9), (40, 70)])
@pytest.mark.parametrize("name", ["single_tokens", "groups_of_seven", "more_new_than_held", "forty_heads_one_key_head", "chunks", "chunks_64",
                                  "chunks_256", "long"])
def test_a_value_that_is_not_a_number_reaches_the_queries_that_see_it(name, mask, sms):
    """NaN among values and keys: exactly the queries that see their token, and of values exactly their places of the head,
    give no number; all others give what the cache without them gives."""
    lens, news, *shape = CASES[name]
    p = kv_gen.problem(lens, news, *shape, seed=51)
    heads, hk, dim, page = shape
    rng = np.random.default_rng(len(name) + sum(mask))
    first = np.concatenate([[0], np.cumsum(news)])
    want_out, want_lse = np.zeros((first[-1], heads, dim), bool), np.zeros((first[-1], heads), bool)
    k, v = (tuple(a.copy() for a in p[x]) for x in "kv")
    for b, (length, n) in enumerate(zip(lens, news)):
        seen = oracle.visible(length, n, *mask)
        # new tokens that only some queries see, and old ones at the window's end
        at = set(rng.choice(length, min(length, 2), replace=False).tolist()) | {j for j in (length - 1, length - n // 2 - 1, length - n - mask[0] + 1) if 0 <= j < length}
        for i, j in enumerate(sorted(at)):
            h, d = int(rng.integers(hk)), int(rng.integers(dim))
            rows, heads_of = first[b] + np.flatnonzero(seen[:, j]), slice(h * (heads // hk), (h + 1) * (heads // hk))
            page_at = p["table"][b, j // page], h, j % page
            if i % 3 != 2:
                v[0][page_at + (d,)] = 0x7F if i % 2 else 0xFF
                want_out[rows, heads_of, d] = True
            else:
                k[0][page_at + (d,)] = 0x7F
                want_out[rows, heads_of], want_lse[rows, heads_of] = True, True
    say("attention, cache with NaN", name, mask, sms)
    with num_sms(sms):
        got = run({**p, "k": k, "v": v}, *mask, max_seqlen_k=1 << 16 if sms else None)
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    assert same(np.isnan(lse), want_lse)
    assert same(np.isnan(out), want_out)
    o = oracle.paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], dim ** -0.5, *mask)
    tol, tol_lse = kv_gen.bounds(o, dim)
    blind = np.isneginf(o["lse"])
    assert (np.abs(out - o["out"]) <= tol)[~want_out].all()
    assert same(np.isneginf(lse), blind)
    assert (np.abs(lse - np.where(blind, 0.0, o["lse"])) <= tol_lse)[~want_lse & ~blind].all()


@pytest.mark.parametrize("name", ["groups_of_seven", "chunks", "chunks_64", "chunks_256"])
def test_a_value_past_bf16_reaches_the_queries_that_see_it(name):
    """Codes whose value BF16 does not hold (FP32 rows near its largest number, or scales of another writer): queries that see the token
    give no finite number at these places of the head, all others what they give without it."""
    lens, news, *shape = CASES[name]
    p = kv_gen.problem(lens, news, *shape, seed=61)
    heads, hk, dim, page = shape
    first = np.concatenate([[0], np.cumsum(news)])
    want, big = np.zeros((first[-1], heads, dim), bool), []
    v = tuple(a.copy() for a in p["v"])
    for b, (length, n) in enumerate(zip(lens, news)):
        j = length - 1 - n // 3
        at = p["table"][b, j // page], hk - 1, j % page
        v[0][at] = 0x30              # (1/2)
        v[0][at + (5,)], v[0][at + (dim - 3,)] = 0x7E, 0xFE
        v[1][at] = 250               # 448 * 2^123
        rows = first[b] + np.flatnonzero(oracle.visible(length, n)[:, j])
        for d in (5, dim - 3):
            want[rows, heads - heads // hk:, d] = True
        big.append(rows)             # (their other places hold 2^122 times a weight: not compared)
    say("attention, values past BF16", name)
    for sms in (0, 1 << 14):
        with num_sms(sms):
            out = run({**p, "v": v}, max_seqlen_k=1 << 16 if sms else None)[0].double().cpu().numpy()
        finite = np.isfinite(out)
        assert same(~finite, want)
        o = oracle.paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], dim ** -0.5)
        tol, _ = kv_gen.bounds(o, dim)
        plain = np.ones((first[-1], heads), bool)
        plain[np.concatenate(big), heads - heads // hk:] = False
        assert (np.abs(out - o["out"]) <= tol)[plain].all()


@pytest.mark.parametrize("page", [1, 3, 8, 15])
@pytest.mark.parametrize("dim,new", [(64, 1), (128, 1), (128, 6), (256, 2), (64, 50), (128, 50), (256, 40)])
def test_attention_small_pages_in_parts(dim, new, page):
    """Pages that hold no row of 16 keys together, cut into many parts and few; pages that end anywhere in a tile."""
    p = kv_gen.problem([700, 0, 333, 64], [new, 1, max(1, new - 1), new], 8, 2, dim, page, seed=page + dim)
    say("attention, small pages", dim, new, page)
    for sms in (0, 24, 1 << 14):
        for mask in ((0, 0), (90, 2)):
            with num_sms(sms):
                check(p, run(p, *mask, max_seqlen_k=1 << 14), *mask)


@pytest.mark.parametrize("batch,new", [(1024, 1), (1025, 1), (1500, 2), (520, 33)])
def test_attention_of_more_items_than_are_cut(batch, new):
    """Around the number of items up to which they may be cut, which more compute units than there are ask for."""
    rng = np.random.default_rng(batch)
    lens = [int(x) for x in rng.integers(0, 70, batch)]
    lens[-1] = 600
    news = [min(new, int(x)) for x in rng.integers(0, new + 2, batch)]
    news[-1] = new
    p = kv_gen.problem(lens, news, 4, 1, 64, 16, seed=batch)
    say("attention, many items", batch, new)
    for sms in (0, 1 << 12):
        with num_sms(sms):
            check(p, run(p, max_seqlen_k=1 << 13))
