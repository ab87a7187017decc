"""GPU parity of block keys, the choice of blocks and attention over chosen blocks, through the binding, against the float64 oracle."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_amd as dg
import oracle
from tests import kv_gen
from tests.test_gpu_kv import cuda, num_sms, same, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# ---------------------------------------------------------------- block keys
@pytest.mark.parametrize("dim,heads,page,order", [(64, 5, 16, "hpt"), (128, 8, 64, "hpt"), (128, 3, 48, "thd"), (256, 2, 7, "thd"), (64, 1, 1, "hpt"),
                                                  (256, 1, 100, "hpt"), (128, 2, 129, "hpt")])
def test_block_keys_are_exact(dim, heads, page, order):
    say("block keys", dim, heads, page, order)
    rng = np.random.default_rng(dim + page)
    pages = 9
    codes = rng.integers(0, 256, (pages, heads, page, dim)).astype(np.uint8)
    if page > 1:  # (some NaN codes stay, which count as zeros)
        codes = np.where((codes & 0x7F) == 0x7F, np.where(rng.random(codes.shape) < 0.9, 0x30, codes), codes)
    sf = rng.integers(110, 130, (pages, heads, page)).astype(np.uint8)
    codes[1], codes[2, 0] = 0, 0x80  # zeros: scale 1
    sf[3], sf[4] = 1, 240            # the smallest scales, and large ones
    codes[5, :, :, :] = 0x7E         # all 448: |mean| = 127 s has to hold exactly
    sf[5] = 127
    x = (cuda(codes), cuda(sf)) if order == "hpt" else (cuda(codes.swapaxes(1, 2)).transpose(1, 2), cuda(sf.swapaxes(1, 2)).transpose(1, 2))
    keys = dg.fp8_kv_block_keys_empty(pages, heads, dim, device=DEV)
    keys[0].fill_(55)
    entries = torch.tensor([5, 0, -1, 8, 4, 3, pages, 2 ** 31 - 1, 2, 1, 5, 5, -2 ** 31], dtype=torch.int32, device=DEV)
    dg.fp8_kv_block_keys_update(x, keys, entries)
    torch.cuda.synchronize()
    want, scale = oracle.block_keys((codes, sf))
    want[[6, 7]], scale[[6, 7]] = 55, 1.0
    assert same(keys[1].double().cpu().numpy(), scale)
    assert same(keys[0].cpu().numpy(), want)
    dg.fp8_kv_block_keys_update(x, keys, entries[:0])


def test_block_keys_of_more_entries_than_one_launch_holds():
    n = 2 ** 25 + 3
    cache = dg.fp8_kv_cache_empty(3, 1, 1, 64, device=DEV)[0]
    cache[0].copy_(torch.arange(0x20, 0x23, device=DEV, dtype=torch.uint8)[:, None, None, None].expand(3, 1, 1, 64))
    keys = dg.fp8_kv_block_keys_empty(3, 1, 64, device=DEV)
    entries = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    entries[0], entries[2 ** 25 - 1], entries[-1] = 0, 1, 2
    dg.fp8_kv_block_keys_update(cache, keys, entries)
    torch.cuda.synchronize()
    want, scale = oracle.block_keys(tuple(x.cpu().numpy() for x in cache))
    assert same(keys[0].cpu().numpy(), want) and same(keys[1].double().cpu().numpy(), scale)


# ---------------------------------------------------------------- choosing
def select_problem(lens, news, heads, kv_heads, dim, page, seed, ties=False, cols=None):
    rng = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    pages = max(sum(used), 1) + 1
    order = rng.permutation(pages)
    cols = cols or max(1, max(used)) + 1
    # unused entries name pages that do not exist
    table = np.where(rng.random((len(lens), cols)) < 0.5, -1, 2 ** 31 - 1).astype(np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at: at + n]
        at += n
    if ties:
        codes, scales = rng.integers(-1, 2, (pages, kv_heads, dim)), 2.0 ** rng.integers(0, 2, (pages, kv_heads))
    else:
        codes, scales = rng.integers(-127, 128, (pages, kv_heads, dim)), 2.0 ** rng.integers(-9, 3, (pages, kv_heads))
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), heads, dim)) * np.exp(2.0 * rng.standard_normal((int(cu[-1]), heads, 1)))
    if ties:
        q = np.sign(q) * (rng.random(q.shape) < 0.1)
    qb = oracle.bf16_rne(q)
    return {"keys": (codes.astype(np.int8), scales), "table": table, "lens": np.array(lens, np.int32), "cu": cu, "news": news, "q_bits": qb,
            "q": oracle.bf16_bits_to_f64(qb), "page": page}


def select(p, top, first, last, **kw):
    keys = cuda(p["keys"][0]), cuda(p["keys"][1].astype(np.float32))
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    r = dg.fp8_kv_select_blocks(q, keys, cuda(p["table"]), cuda(p["lens"]), p["page"], top, first, last, cu_seqlens_q=cuda(p["cu"]),
                                max_seqlen_q=max(p["news"]), **kw)
    torch.cuda.synchronize()
    return r.cpu().numpy()


# lengths, new tokens; heads, key heads, head dim, page
CHOICES = {
    "one": ([700], [1], 4, 1, 128, 16),
    "single_tokens": ([0, 1, 15, 16, 17, 400, 1000, 33], [1] * 8, 16, 2, 64, 16),
    "groups_of_seven": ([300, 37, 964], [3, 5, 4], 14, 2, 64, 16),
    "forty_heads_one_key_head": ([900, 17], [5, 2], 40, 1, 128, 10),
    "groups_of_three": ([500, 100], [70, 100], 9, 3, 256, 7),
    "no_groups": ([333, 258], [33, 1], 5, 5, 128, 2),
    "two_a_group": ([900], [100], 4, 2, 64, 5),
    "groups_of_sixteen": ([640, 640], [9, 9], 32, 2, 256, 16),
    "more_new_than_held": ([30, 0, 40], [50, 2, 41], 4, 2, 128, 1),
    "long": ([9000], [6], 8, 1, 64, 1),
    "long_ragged": ([5000, 700, 2500, 0], [2, 1, 5, 1], 4, 2, 128, 1),
}


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("top,first,last", [(8, 1, 2), (1, 0, 1), (5, 2, 3), (16, 0, 1), (70, 3, 1), (300, 1, 1), (200, 0, 2)])
@pytest.mark.parametrize("name", sorted(CHOICES))
def test_choice_is_exact(name, top, first, last, ties):
    say("choice", name, top, first, last, ties)
    p = select_problem(*CHOICES[name], seed=top, ties=ties)
    want = oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], p["page"], top, first, last)
    assert same(select(p, top, first, last), want)
    for sms in (1, 4000):  # (larger tiles of tokens; more workgroups for the blocks of a tile)
        with num_sms(sms):
            assert same(select(p, top, first, last), want)


def test_choice_from_a_wide_table():
    p = select_problem([32768 * 2, 20000], [3, 2], 4, 2, 64, 2, 0, cols=32768)
    assert same(select(p, 40, 1, 1), oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], 2, 40, 1, 1))


# lengths, new tokens; heads, key heads, head dim, page
FEW_LONG = {
    "wide_heads": ([1300], [1], 4, 1, 256, 1),
    "wide_heads_two": ([1300, 2900], [2, 1], 14, 2, 256, 2),
    "forty_heads_one_key_head": ([1500], [2], 40, 1, 128, 1),
    "forty_heads_one_key_head_64": ([1700, 900], [1, 1], 40, 1, 64, 1),
    "forty_heads_one_key_head_256": ([1250], [1], 40, 1, 256, 1),
}


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("top,first,last", [(8, 1, 2), (70, 3, 1), (600, 0, 2)])
@pytest.mark.parametrize("name", sorted(FEW_LONG))
def test_choice_in_parts(name, top, first, last, ties):
    """Few tokens over more than 512 blocks: the scores by several workgroups, in several rounds where a key head has more than 16 heads."""
    say("choice in parts", name, top, first, last, ties)
    heads, kv_heads, dim, page = FEW_LONG[name][2:]
    p = select_problem(*FEW_LONG[name], seed=top, ties=ties)
    assert dg.lib().dg_fp8_kv_select_blocks_workspace(len(p["lens"]), int(p["cu"][-1]), heads, kv_heads, dim, 0, max(p["news"]), p["table"].shape[1], top,
                                                      first, last) > 0
    want = oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], page, top, first, last)
    assert same(select(p, top, first, last), want)
    with num_sms(1):
        assert same(select(p, top, first, last), want)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_choice_from_a_wide_table_in_one_kernel(dim):
    """All of a token's 32768 scores in one workgroup's LDS."""
    say("wide table in one kernel", dim)
    p = select_problem([32768 * 2, 20000], [3, 2], 4, 2, dim, 2, 1, cols=32768)
    with num_sms(1):
        assert same(select(p, 40, 1, 1), oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], 2, 40, 1, 1))


@pytest.mark.parametrize("cols", [1000, 1900])
@pytest.mark.parametrize("heads,dim", [(8, 128), (2, 64)])
def test_choice_of_a_chunk_over_many_blocks(heads, dim, cols):
    """Tiles of fewer tokens than LDS has room for, so that two workgroups share a compute unit."""
    p = select_problem([cols - 1], [135], heads, 2, dim, 1, 2, cols=cols)
    want = oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], 1, 20, 1, 2)
    for sms in (256, 1):
        with num_sms(sms):
            assert same(select(p, 20, 1, 2), want)


def test_choice_with_queries_that_are_no_numbers():
    """They count as zeros: the choice of the other heads of the group, and of other tokens, stays."""
    p = select_problem([500], [20], 8, 2, 128, 8, 3)
    q = p["q"].copy()
    q[3, 1, 7], q[4, 5, 100], q[5, 2, 0] = np.nan, np.inf, -np.inf
    q[6, :4] = np.nan
    p["q_bits"] = oracle.bf16_rne(np.where(np.isnan(q), 0, q))
    p["q_bits"][np.isnan(q)] = 0x7FC0
    assert same(select(p, 9, 1, 1), oracle.select_blocks(q, p["keys"], p["table"], p["lens"], p["cu"], 8, 9, 1, 1))


def test_choice_leaves_rows_behind_the_last_sequence():
    p = select_problem([200, 90], [3, 2], 4, 2, 64, 16, 4)
    keys = cuda(p["keys"][0]), cuda(p["keys"][1].astype(np.float32))
    q = torch.cat([cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)] * 2)
    out = torch.full((10, 2, 6), 77, dtype=torch.int32, device=DEV)
    dg.fp8_kv_select_blocks(q, keys, cuda(p["table"]), cuda(p["lens"]), 16, 6, cu_seqlens_q=cuda(p["cu"]), max_seqlen_q=2, out=out)
    want = oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], 16, 6, 1, 1)
    assert (out[5:] == 77).all()
    got = out[:5].cpu().numpy()
    assert same(got[[0, 1, 3, 4]], want[[0, 1, 3, 4]]) and (got[2] == 77).all()  # (past the bound of two new tokens)
    none = dg.fp8_kv_select_blocks(q, keys, cuda(p["table"]), cuda(p["lens"]), 16, 6, cu_seqlens_q=cuda(p["cu"]), max_seqlen_q=0)
    assert (none == -1).all()


def test_choice_of_strided_queries_and_an_expanded_table():
    p = select_problem([300] * 3, [4] * 3, 8, 2, 128, 8, 5)
    p["table"][1:] = p["table"][0]
    wide = torch.zeros((12, 11, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10] = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    keys = cuda(p["keys"][0]), cuda(p["keys"][1].astype(np.float32))
    got = dg.fp8_kv_select_blocks(wide[:, 2:10], keys, cuda(p["table"])[:1].expand(3, -1), cuda(p["lens"]), 8, 7)
    assert same(got.cpu().numpy(), oracle.select_blocks(p["q"], p["keys"], p["table"], p["lens"], p["cu"], 8, 7, 1, 1))


# ---------------------------------------------------------------- attention
def lists(p, kv_heads, top, seed, near=False):
    """Random ascending lists of the blocks up to a token's own, some empty, some past the token's place.  near: neighbours' are alike."""
    rng = np.random.default_rng(seed)
    seq, place = oracle.blocks.places(p["lens"], p["cu"])
    out = np.full((len(seq), kv_heads, top), -1, dtype=np.int32)
    for t in range(len(seq)):
        for h in range(kv_heads):
            n = max(place[t] // p["page"] + 1, 0) + (1 if rng.random() < 0.2 else 0)  # (one more than it has)
            n = min(n, p["table"].shape[1])
            k = min(top, n) if rng.random() < 0.7 else rng.integers(0, min(top, n) + 1)
            if near and t and seq[t] == seq[t - 1] and rng.random() < 0.8:
                out[t, h] = out[t - 1, h]
            else:
                out[t, h, :k] = np.sort(rng.choice(n, k, replace=False))
    return out


def run(p, blocks, lse=True, scale=None, **kw):
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    r = dg.fp8_block_sparse_attention(q, caches[0], caches[1], cuda(p["table"]), cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]),
                                      max_seqlen_q=max(p["news"]), sm_scale=scale, return_lse=lse, **kw)
    torch.cuda.synchronize()
    return r


def check(p, got, blocks, scale=None):
    o = oracle.block_sparse_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], blocks, scale if scale is not None else p["dim"] ** -0.5)
    tol, tol_lse = kv_gen.bounds(o, p["dim"])
    out, lse = got[0].double().cpu().numpy(), got[1].double().cpu().numpy()
    err = np.abs(out - o["out"])
    say("largest error / bound", float((err / tol).max()) if err.size else 0.0)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(~(err <= tol))[:5])
    blind = np.isneginf(o["lse"])
    assert same(np.isneginf(lse), blind) and (out[blind] == 0).all()
    with np.errstate(invalid="ignore"):
        assert (np.abs(lse - o["lse"])[~blind] <= tol_lse[~blind]).all()


# lengths, new tokens; heads, key heads, head dim, page
CASES = {
    "one_token": ([1], [1], 4, 1, 128, 16),
    "single_tokens": ([0, 1, 31, 32, 33, 64, 65, 127, 300], [1] * 9, 16, 2, 128, 16),
    "single_tokens_64": ([5, 0, 300], [1] * 3, 5, 5, 64, 1),
    "single_tokens_256": ([130, 63, 1], [1] * 3, 8, 2, 256, 32),
    "groups_of_seven": ([100, 37, 64], [3, 5, 4], 14, 2, 64, 16),
    "forty_heads_one_key_head": ([90, 17], [1, 2], 40, 1, 128, 100),
    "more_new_than_held": ([3, 0, 40], [5, 2, 41], 4, 2, 128, 16),
    "chunks": ([200, 129, 64, 1], [130, 129, 1, 1], 4, 1, 128, 48),
    "chunks_64": ([300, 100, 65], [64, 100, 33], 12, 4, 64, 7),
    "chunks_256": ([190, 70], [40, 70], 2, 1, 256, 64),
    "no_groups": ([150], [90], 3, 3, 64, 16),
    "large_pages": ([700, 300], [9, 1], 8, 2, 128, 300),
    "long": ([1500, 1027], [20, 2], 8, 2, 128, 64),
}


@pytest.mark.parametrize("sms", [256, 1, 4000])
@pytest.mark.parametrize("top,near", [(4, True), (1, False), (9, False)])
@pytest.mark.parametrize("name", sorted(CASES))
def test_attention(name, top, near, sms):
    say("attention over blocks", name, top, near, sms)
    p = kv_gen.problem(*CASES[name], seed=top)
    blocks = lists(p, CASES[name][3], top, top, near)
    with num_sms(sms):  # (more compute units: tiles shared by more workgroups)
        check(p, run(p, blocks), blocks)


def test_many_blocks():
    """Lists of more than the 64 entries that a wave takes at a time, all blocks, and equal new tokens without first rows."""
    p = kv_gen.problem([600, 600], [4, 4], 8, 2, 64, 4, 11)
    blocks = np.full((8, 2, 200), -1, dtype=np.int32)
    seq, place = oracle.blocks.places(p["lens"], p["cu"])
    for t in range(8):
        n = place[t] // 4 + 1
        blocks[t, :, :n] = np.arange(n)
    for sms in (1, 256, 4000):
        with num_sms(sms):
            check(p, run(p, blocks), blocks)
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    check(p, dg.fp8_block_sparse_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), cuda(blocks), return_lse=True), blocks)
    whole = dg.fp8_paged_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), return_lse=True)
    check(p, whole, blocks)


def test_many_short_sequences_without_a_bound():
    """No max_seqlen_q: a launch has a tile for every token of every sequence, of which few have rows."""
    say("many short sequences")
    news = [1 + (b % 97 == 5) for b in range(1024)]
    p = kv_gen.problem([1 + 7 * b % 60 for b in range(1024)], news, 16, 1, 64, 16, 14)
    blocks = lists(p, 1, 3, 4)
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    check(p, dg.fp8_block_sparse_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]), return_lse=True), blocks)


def test_lists_past_32_bits():
    """A token's lists of 4097 key heads and 2^19 entries: the last head's begins 2^31 entries behind the first one's."""
    heads, top = 4097, 2 ** 19
    say("lists past 32 bits")
    p = kv_gen.problem([40], [1], heads, heads, 64, 16, 15)
    few = lists(p, heads, 2, 6)
    few[0, [0, heads - 1]] = [[0, 2], [1, 2]]
    blocks = torch.full((1, heads, top), -1, dtype=torch.int32, device=DEV)
    blocks[:, :, :2] = cuda(few)
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    check(p, dg.fp8_block_sparse_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), blocks, return_lse=True), few)


@pytest.mark.parametrize("sms", [256, 1, 4000])
@pytest.mark.parametrize("heads,top", [(8, 1500), (4, 1300), (8, 5000), (2, 300)])
def test_lists_that_fill_a_tiles_room(heads, top, sms):
    """Long lists of several new tokens: tiles of two tokens, of three, of one, and of 13 (4096 entries of LDS)."""
    say("long lists", heads, top, sms)
    p = kv_gen.problem([5200, 4100], [5, 14], heads, 2, 64, 1, 16)
    blocks = lists(p, 2, top, top, near=True)
    with num_sms(sms):
        check(p, run(p, blocks), blocks)


def test_scale_and_strides():
    p = kv_gen.problem([90, 70, 33], [5, 2, 9], 6, 2, 128, 16, 12)
    blocks = lists(p, 2, 3, 0)
    caches = [(cuda(p[x][0].swapaxes(1, 2)).transpose(1, 2), cuda(p[x][1].swapaxes(1, 2)).transpose(1, 2)) for x in "kv"]  # tokens outermost
    wide = torch.zeros((16, 9, 128), dtype=torch.bfloat16, device=DEV)
    wide[:, 1:7] = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    out = torch.full((20, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    table = torch.full((3, p["table"].shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    table[:, 2:-3] = cuda(p["table"])
    got = dg.fp8_block_sparse_attention(wide[:, 1:7], *caches, table[:, 2:-3], cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]),
                                        max_seqlen_q=9, sm_scale=0.3, out=out[:16, 2:], return_lse=True)
    check(p, got, blocks, 0.3)
    assert (out[16:] == 3).all() and (out[:, :2] == 3).all()


def test_rows_of_no_sequence():
    p = kv_gen.problem([90, 70], [5, 2], 4, 2, 64, 16, 13)
    blocks = np.concatenate([lists(p, 2, 3, 0)] * 2)
    q = torch.cat([cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)] * 2)
    caches = [(cuda(p[x][0]), cuda(p[x][1])) for x in "kv"]
    for sms in (1, 4000):
        with num_sms(sms):
            out = torch.full((14, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
            got = dg.fp8_block_sparse_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]), max_seqlen_q=5,
                                                out=out, return_lse=True)
            assert (out[7:] == 3).all()
            check(p, (got[0][:7], got[1][:7]), blocks[:7])
            out, lse = dg.fp8_block_sparse_attention(q, *caches, cuda(p["table"]), cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]),
                                                     max_seqlen_q=0, return_lse=True)
            assert (out == 0).all() and lse.isneginf().all()


@pytest.mark.parametrize("sms", [1, 4000])
@pytest.mark.parametrize("name", ["chunks", "groups_of_seven", "chunks_64", "chunks_256", "single_tokens"])
def test_lists_that_break_the_rules_read_nothing_else(name, sms):
    """Unordered, repeated, negative in between, far past the table: any result, but of finite values, and it ends."""
    p = kv_gen.problem(*CASES[name], seed=1, garbage=False)
    rng = np.random.default_rng(5)
    total = int(p["cu"][-1])
    blocks = rng.integers(-3, p["table"].shape[1] + 3, (total, CASES[name][3], 11)).astype(np.int32)
    blocks[rng.random(blocks.shape) < 0.1] = 2 ** 31 - 1
    blocks[rng.random(blocks.shape) < 0.1] = -2 ** 31
    with num_sms(sms):
        out, lse = run(p, blocks)
    assert out.isfinite().all() and not lse.isnan().any()


@pytest.mark.parametrize("sms", [1, 4000])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 7)])
def test_values_that_are_no_numbers_reach_who_sees_them(dim, page, sms):
    p = kv_gen.problem([200], [12], 4, 2, dim, page, 21)
    blocks = lists(p, 2, 5, 3, near=True)
    with num_sms(sms):
        clean = run(p, blocks)
    seen = lambda t, h, j: (blocks[t, h] == j // page).any() and j <= 188 + t  # noqa: E731
    for kind, code, sf in (("nan", 0x7F, None), ("inf", 0x7E, 250), ("key", 0x7F, None)):
        for j in (int(blocks[5, 0][blocks[5, 0] >= 0][0]) * page, 190, 199):
            r = {x: (p[x][0].copy(), p[x][1].copy()) for x in "kv"}
            c, s = r["k" if kind == "key" else "v"]
            pg, at = p["table"][0, j // page], j % page
            c[pg, 0, at, 5] = code
            if sf:
                s[pg, 0, at] = sf
            with num_sms(sms):
                got = run({**p, **r}, blocks)
            for t in range(12):
                for h in range(4):
                    row = got[0][t, h].float().cpu().numpy()
                    if h < 2 and seen(t, 0, j):
                        # (a value of 2^132 counts by its weight)
                        assert not (np.abs(row if kind == "key" else row[5]) < 1e30).any(), (kind, j, t, h)
                    else:
                        # (a NaN score raises no maximum, and the rows of a tile raise theirs together: last bits may change)
                        was = clean[0][t, h].float().cpu().numpy()
                        assert np.allclose(row, was, rtol=2 ** -6, atol=1e-2) if kind == "key" else same(row, was), (kind, j, t, h)


def test_queries_that_are_no_numbers():
    p = kv_gen.problem([100, 50], [6, 1], 8, 2, 128, 16, 22)
    blocks = lists(p, 2, 4, 1)
    blocks[:, :, 0] = np.where(blocks[:, :, 0] < 0, 0, blocks[:, :, 0])
    p["q_bits"][2, 3, 9] = 0x7FC0
    for sms in (1, 4000):
        with num_sms(sms):
            out, lse = run(p, blocks)
        assert out[2, 3].isnan().all() and lse[2, 3].isnan()
        rest = torch.ones((7, 8), dtype=torch.bool, device=DEV)
        rest[2, 3] = False
        assert out[rest].isfinite().all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
def test_beside_queries_that_are_no_numbers(dim, bad):
    """A NaN or infinite query's row sends its tile over the keys again with care: the other rows are within their bounds as ever."""
    p = kv_gen.problem([100, 50], [6, 1], 8, 2, dim, 16, 24)
    blocks = lists(p, 2, 4, 1, near=True)
    blocks[:, :, 0] = np.where(blocks[:, :, 0] < 0, 0, blocks[:, :, 0])
    clean = oracle.block_sparse_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], blocks, dim ** -0.5)
    p["q_bits"][2, 3, 9] = bad
    for sms in (1, 4000):
        with num_sms(sms):
            out, lse = run(p, blocks)
        assert out[2, 3].isnan().all() and not lse[2, 3].isfinite()
        out[2, 3] = torch.from_numpy(clean["out"][2, 3])
        lse[2, 3] = float(clean["lse"][2, 3])
        check(p, (out, lse), blocks)


@pytest.mark.parametrize("dim,news", [(128, [3, 1]), (64, [1, 1]), (256, [2, 9])])
def test_a_cache_between_2_and_4_gib(dim, news):
    """Offsets past 2^31 in the form of 32-bit offsets: on the last pages below 4 GiB."""
    heads, page = 8, 64
    pages = 2 ** 32 // (heads * page * dim) - 1
    k_cache, v_cache = dg.fp8_kv_cache_empty(pages, heads, page, dim, device=DEV)
    p = kv_gen.problem([500, 300], news, 16, heads, dim, page, 25)
    blocks = lists(p, heads, 4, 2)
    used = p["table"][p["table"] >= 0]
    used = np.unique(used[used < len(p["k"][0])])
    high = {int(pg): pages - 1 - 7 * i if i % 3 else pages // 2 - 1 + i for i, pg in enumerate(used)}
    for x, c in (("k", k_cache), ("v", v_cache)):
        for pg, to in high.items():
            c[0][to], c[1][to] = cuda(p[x][0][pg]), cuda(p[x][1][pg])
    table = np.vectorize(lambda x: high.get(int(x), -1))(p["table"]).astype(np.int32)
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    for sms in (1, 256, 4000):
        say("2 to 4 GiB", dim, sms)
        with num_sms(sms):
            got = dg.fp8_block_sparse_attention(q, k_cache, v_cache, cuda(table), cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]),
                                                max_seqlen_q=max(news), return_lse=True)
        check(p, got, blocks)


@pytest.mark.parametrize("dim,news", [(128, [3, 1]), (64, [5, 2]), (256, [2, 9]), (64, [1, 1]), (128, [1, 1]), (256, [1, 1])])
def test_a_cache_past_4_gib(dim, news):
    heads, page = 8, 64
    pages = 2 ** 32 // (heads * page * dim) + 3000
    k_cache, v_cache = dg.fp8_kv_cache_empty(pages, heads, page, dim, device=DEV)
    p = kv_gen.problem([500, 300], news, 16, heads, dim, page, 23)
    blocks = lists(p, heads, 4, 2)
    used = p["table"][p["table"] >= 0]
    used = np.unique(used[used < len(p["k"][0])])
    far = {int(pg): pages - 1 - 7 * i for i, pg in enumerate(used)}
    for x, c in (("k", k_cache), ("v", v_cache)):
        for pg, to in far.items():
            c[0][to], c[1][to] = cuda(p[x][0][pg]), cuda(p[x][1][pg])
    table = np.vectorize(lambda x: far.get(int(x), -1))(p["table"]).astype(np.int32)
    q = cuda(p["q_bits"].view(np.int16)).view(torch.bfloat16)
    for sms in (1, 256, 4000):
        with num_sms(sms):
            got = dg.fp8_block_sparse_attention(q, k_cache, v_cache, cuda(table), cuda(p["lens"]), cuda(blocks), cu_seqlens_q=cuda(p["cu"]),
                                                max_seqlen_q=max(news), return_lse=True)
        check(p, got, blocks)
    keys = dg.fp8_kv_block_keys_empty(pages, heads, dim, device=DEV)
    to = torch.tensor(sorted(far.values()), dtype=torch.int32, device=DEV)
    dg.fp8_kv_block_keys_update(k_cache, keys, to)
    want, scale = oracle.block_keys(tuple(x[to.long()].cpu().numpy() for x in k_cache))
    assert same(keys[0][to.long()].cpu().numpy(), want) and same(keys[1][to.long()].double().cpu().numpy(), scale)


# ---------------------------------------------------------------- as they are used
def test_a_sequence_grows():
    """Prompt in chunks, then token by token: keys normed, turned and written, block keys as pages fill up, blocks chosen, attended; on a
    side stream, and captured and replayed for the single tokens."""
    heads, kv_heads, dim, page, top = 8, 2, 128, 16, 6
    g = torch.Generator(DEV).manual_seed(0)
    n = 400
    qkv = torch.randn((n, heads + 2 * kv_heads, dim), generator=g, device=DEV).bfloat16()
    w, pos = torch.ones(dim, device=DEV), torch.arange(n, device=DEV)
    turn = pos[:, None].double() * 10000.0 ** (-torch.arange(0, dim, 2, device=DEV).double() / dim)
    cs = torch.cat([turn.cos(), turn.sin()], 1).float()
    pages = n // page
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[None].contiguous()
    slots = table[0, pos // page].long() * page + pos % page
    k_cache, v_cache = dg.fp8_kv_cache_empty(pages, kv_heads, page, dim, device=DEV)
    keys = dg.fp8_kv_block_keys_empty(pages, kv_heads, dim, device=DEV)

    def feed(x, at, slot, full, length):
        q, k, v = x.split((heads, kv_heads, kv_heads), 1)
        q = dg.qk_norm_rope_fp8_kv_cache_write(q, k, v, w, w, cs, at, k_cache, v_cache, slot)
        dg.fp8_kv_block_keys_update(k_cache, keys, full)
        blocks = dg.fp8_kv_select_blocks(q, keys, table, length, page, top, first=1, last=2)
        return q, blocks, *dg.fp8_block_sparse_attention(q, k_cache, v_cache, table, length, blocks, return_lse=True)

    def inputs(a, b):
        full = table[0, a // page: b // page]
        return qkv[a:b], pos[a:b], slots[a:b], full, torch.tensor([b], dtype=torch.int32, device=DEV)

    def verify(a, b, r):
        lens, cu = np.array([b]), np.array([0, b - a])
        qf = r[0].double().cpu().numpy()
        kc, vc = (tuple(x.cpu().numpy() for x in c) for c in (k_cache, v_cache))
        t = table.cpu().numpy()
        want, scale = oracle.block_keys(tuple(x[t[0, :b // page]] for x in kc))
        assert same(keys[0].cpu().numpy()[t[0, :b // page]], want)
        blocks = oracle.select_blocks(qf, (keys[0].cpu().numpy(), keys[1].double().cpu().numpy()), t, lens, cu, page, top, 1, 2)
        assert same(r[1].cpu().numpy(), blocks)
        p = {"q": qf, "k": kc, "v": vc, "table": t, "lens": lens, "cu": cu, "dim": dim}
        check(p, (r[2], r[3]), blocks)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in [(0, 150), (150, 151), (151, 300), (300, 303), (303, 390)]:
            r = feed(*inputs(a, b))
            side.synchronize()
            verify(a, b, r)
        static = [x.clone() for x in inputs(390, 391)]
        static[3] = torch.full((1,), -1, dtype=torch.int32, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r = feed(*static)
        for a in range(390, 400):
            now = list(inputs(a, a + 1))
            now[3] = now[3] if now[3].numel() else torch.full((1,), -1, dtype=torch.int32, device=DEV)
            for x, y in zip(static, now):
                x.copy_(y)
            graph.replay()
            side.synchronize()
            verify(a, a + 1, r)
            eager = feed(*now)  # (writes the same values again)
            side.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(r, eager))
