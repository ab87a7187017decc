"""CPU tests of block keys, the choice of blocks and attention over them: argument validation (before any HIP call), the binding's
refusals, and pins of the oracle against something other than itself."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_scaled_fp8_amd as dg
import oracle
from oracle.blocks import int8_scale
from tests import kv_gen
from tests.test_kv_host import CACHE_FAULTS, OnGpu, cache, fake_cache, recorder  # noqa: F401

DG_OK, NULL, DTYPE, SHAPE, LAYOUT, UNSUPPORTED, HIP = 0, -1, -2, -3, -4, -5, -6
P, P_MIS, P_ODD = 4096, 4104, 4097   # fake addresses: never dereferenced


def keys(**kw):
    f = dict(codes=P, scales=P, num_pages=10, num_heads=4, head_dim=128)
    f.update(kw)
    return dg._BlockKeys(*f.values())


KEY_FAULTS = [(dict(head_dim=96), UNSUPPORTED), (dict(num_heads=0), SHAPE), (dict(num_heads=65536), SHAPE), (dict(num_pages=-1), SHAPE),
              (dict(num_pages=0), SHAPE), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(codes=P_MIS), LAYOUT), (dict(scales=P_ODD), LAYOUT)]


def update(c=None, b=None, n=3, pages=P):
    return dg.lib().dg_fp8_kv_block_keys_update(ctypes.byref(cache() if c is None else c), ctypes.byref(keys() if b is None else b), n, pages, None)


def select(b=None, **kw):
    a = dict(page=16, batch=2, total_q=4, hq=8, q=P, qts=1024, qhs=128, cu=P, max_q=2, table=P, ts=5, cols=5, lens=P, top=4, first=1, last=1,
             blocks=P, work=None, work_bytes=0, stream=None)
    a.update(kw)
    return dg.lib().dg_fp8_kv_select_blocks(ctypes.byref(keys() if b is None else b), *a.values())


def attend(c=None, **kw):
    a = dict(batch=2, total_q=4, hq=8, q=P, qts=1024, qhs=128, cu=P, max_q=2, table=P, ts=5, cols=5, lens=P, blocks=P, top=4, scale=0.1,
             out=P, ots=1024, ohs=128, lse=None, work=None, work_bytes=0, stream=None)
    a.update(kw)
    return dg.lib().dg_fp8_block_sparse_attention(ctypes.byref(cache() if c is None else c), *a.values())


SHARED_FAULTS = [(dict(batch=-1), SHAPE), (dict(total_q=-4), SHAPE), (dict(hq=6), SHAPE), (dict(hq=0), SHAPE), (dict(hq=-4), SHAPE),
                 (dict(total_q=1 << 29), SHAPE), (dict(max_q=-1), SHAPE), (dict(cu=None, total_q=5), SHAPE), (dict(cols=-1), LAYOUT), (dict(ts=4), LAYOUT),
                 (dict(cols=1 << 27, ts=1 << 27), SHAPE), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(q=None), NULL), (dict(blocks=None), NULL),
                 (dict(q=P_MIS), LAYOUT), (dict(qts=1028), LAYOUT), (dict(qhs=-128), LAYOUT), (dict(lens=P_ODD), LAYOUT), (dict(cu=P_ODD), LAYOUT),
                 (dict(table=P_ODD), LAYOUT), (dict(blocks=P_ODD), LAYOUT), (dict(top=0), SHAPE), (dict(top=(1 << 20) + 1), SHAPE)]


def test_block_keys_refuse():
    for kw, code in CACHE_FAULTS:
        if "v" not in kw and "v_sf" not in kw:
            assert update(cache(**kw)) == code, kw
    assert update(cache(v=None, v_sf=None), n=0) == DG_OK  # (values are not read)
    for kw, code in KEY_FAULTS:
        assert update(b=keys(**kw)) == code, kw
        assert dg.lib().dg_get_last_error()
    for b in (keys(num_pages=9), keys(num_heads=5), keys(head_dim=64)):
        assert update(b=b) == SHAPE
    assert update(n=-1) == SHAPE and update(pages=None) == NULL and update(pages=P_ODD) == LAYOUT
    assert dg.lib().dg_fp8_kv_block_keys_update(None, ctypes.byref(keys()), 1, P, None) == NULL
    assert dg.lib().dg_fp8_kv_block_keys_update(ctypes.byref(cache()), None, 1, P, None) == NULL
    assert update(cache(k=None, k_sf=None), keys(codes=None, scales=None), n=0, pages=None) == DG_OK


def test_select_refuses():
    for kw, code in KEY_FAULTS:
        assert select(keys(**kw)) == code, kw
    for kw, code in SHARED_FAULTS + [(dict(page=0), SHAPE), (dict(page=-16), SHAPE), (dict(first=-1), SHAPE), (dict(last=0), SHAPE), (dict(first=4), SHAPE),
                                     (dict(first=2, last=3), SHAPE), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), SHAPE),
                                     (dict(cols=32769, ts=32769), UNSUPPORTED)]:
        assert select(**kw) == code, kw
    for kw in (dict(batch=0), dict(total_q=0), dict(max_q=0)):
        assert select(keys(codes=None), q=None, table=None, lens=None, blocks=None, **kw) == DG_OK, kw
    assert dg.lib().dg_fp8_kv_select_blocks(None, *[0] * 4, None, 0, 0, None, 0, None, 0, 0, None, 1, 0, 1, None, None, 0, None) == NULL


def test_attention_refuses():
    for kw, code in CACHE_FAULTS:
        assert attend(cache(**kw)) == code, kw
    for kw, code in SHARED_FAULTS + [(dict(scale=0.0), SHAPE), (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE), (dict(out=None), NULL),
                                     (dict(out=P_MIS), LAYOUT), (dict(ohs=132), LAYOUT), (dict(lse=P_ODD), LAYOUT)]:
        assert attend(**kw) == code, kw
    for kw in (dict(batch=0), dict(total_q=0), dict(max_q=0)):
        assert attend(cache(k=None), q=None, out=None, table=None, lens=None, blocks=None, **kw) == DG_OK, kw


def test_more_tiles_than_a_launch_holds_are_refused():
    dg.set_num_sms(256)
    try:
        many = dict(batch=1 << 20, total_q=1 << 20, hq=4, max_q=1 << 20)
        assert select(**many) == SHAPE and b"max_seqlen_q" in dg.lib().dg_get_last_error()
        assert attend(**many) == SHAPE and b"max_seqlen_q" in dg.lib().dg_get_last_error()
    finally:
        dg.set_num_sms(0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch kernels on fake addresses")
def test_ordinary_calls_of_many_tiles_reach_the_launch():
    """Without a device they end in a launch error: no check of sizes refuses them, here or in the choice of blocks."""
    heads = cache(num_heads=8, page_size=64, page_stride=65536, head_stride=8192, sf_page_stride=512, sf_head_stride=64)
    dg.set_num_sms(256)
    try:
        for kw in (dict(batch=32, total_q=8192, hq=64, max_q=8192), dict(batch=128, total_q=8192, hq=32, max_q=8192),
                   dict(batch=1, total_q=131072, hq=128, max_q=131072), dict(batch=1, total_q=131072, hq=128, cu=None, max_q=0)):
            d = dict(kw, qts=kw["hq"] * 128, top=16)
            assert attend(heads, ots=kw["hq"] * 128, **d) == HIP, kw
            assert select(keys(num_heads=8), page=64, **d) == HIP, kw
        # the most that a launch of four waves holds, and one tile more
        for batch, code in ((32, HIP), (33, SHAPE)):
            assert attend(heads, batch=batch, total_q=1 << 17, hq=64, max_q=(1 << 17) - 2, qts=8192, ots=8192, top=16) == code, batch
    finally:
        dg.set_num_sms(0)


def test_a_workspace_that_is_missing_or_small_is_refused():
    dg.set_num_sms(256)
    try:
        size = dg.lib().dg_fp8_kv_select_blocks_workspace
        need = size(1, 1, 32, 4, 128, 1, 0, 2000, 20, 1, 1)
        assert need > 0
        a = dict(batch=1, total_q=1, hq=32, cu=None, cols=2000, ts=2000, top=20)
        assert select(**a) == NULL and select(work=P, work_bytes=need - 1, **a) == SHAPE and select(work=P_MIS, work_bytes=need, **a) == LAYOUT
        assert size(64, 64, 32, 4, 128, 1, 0, 2000, 20, 1, 1) == 0 and size(1, 1, 32, 4, 128, 1, 0, 100, 20, 1, 1) == 0
        assert size(0, 0, 32, 4, 128, 1, 0, 2000, 20, 1, 1) == 0 and size(1, 1, 32, 4, 128, 1, 0, 20, 20, 1, 1) == 0
        for bad, code in [((1, 1, 32, 4, 96, 1, 0, 100, 20, 1, 1), UNSUPPORTED), ((1, 1, 30, 4, 128, 1, 0, 100, 20, 1, 1), SHAPE),
                          ((1, 1, 32, 4, 128, 1, 0, 100, 20, 10, 11), SHAPE), ((1, 1, 32, 4, 128, 1, 0, -1, 20, 1, 1), LAYOUT),
                          ((1, 1, 32, 4, 128, 1, 0, 40000, 20, 1, 1), UNSUPPORTED)]:
            assert size(*bad) == code, bad
        size = dg.lib().dg_fp8_block_sparse_attention_workspace
        need = size(1, 1, 32, 8, 128, 1, 0, 64, 64)
        assert need > 0
        a = dict(batch=1, total_q=1, hq=32, cu=None, top=64)
        c = lambda: cache(num_heads=8, page_size=64, page_stride=65536, head_stride=8192, sf_page_stride=512, sf_head_stride=64)  # noqa: E731
        assert attend(c(), **a) == NULL
        assert attend(c(), work=P, work_bytes=need - 1, **a) == SHAPE
        assert attend(c(), work=P_MIS, work_bytes=need, **a) == LAYOUT
        assert size(4096, 4096, 32, 8, 128, 1, 0, 64, 64) == 0  # (enough work for whole tiles)
        assert size(0, 0, 32, 8, 128, 1, 0, 64, 64) == 0
        assert size(1, 1, 32, 8, 96, 1, 0, 64, 64) == UNSUPPORTED and size(1, 1, 30, 8, 128, 1, 0, 64, 64) == SHAPE and size(1, 1, 32, 8, 128, 1, 0, 0, 64) == SHAPE
    finally:
        dg.set_num_sms(0)


def test_a_tiles_segments_stay_within_32_bits():
    """The largest pages that a cache may have, 2^19 segments of 64 keys each: 16 tokens of 256 blocks would be 2^31 segments, so a tile has eight."""
    dg.set_num_sms(256)
    try:
        size = dg.lib().dg_fp8_block_sparse_attention_workspace
        tiles = lambda page, top: size(1, 16, 1, 1, 64, 1, 0, page, top) // (64 * 16 * (64 + 2) * 4)  # noqa: E731  (of 64 parts each)
        assert tiles((1 << 25) - 1, 256) == 2 and tiles((1 << 25) - 1, 128) == 1 and tiles(1 << 24, 256) == 1 and tiles(1 << 24, 128) == 1
    finally:
        dg.set_num_sms(0)


def test_the_binding_refuses():
    codes, scales = dg.fp8_kv_block_keys_empty(4, 2, 64, device="cpu")
    assert codes.dtype == torch.int8 and (scales == 1).all()
    q, table, lens = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in [(codes, scales), (codes.int(), scales), (codes[:, :, ::2], scales), (codes, scales[:3]), (codes, scales.double()), (codes[0], scales)]:
        with pytest.raises(ValueError):  # (the first: not on a GPU)
            dg.fp8_kv_select_blocks(q, bad, table, lens, 16, 4)
    cache_ = (torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 16), dtype=torch.uint8))
    with pytest.raises(ValueError):
        dg.fp8_kv_block_keys_update(cache_, (codes, scales), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        dg.fp8_block_sparse_attention(q, cache_, cache_, table, lens, torch.zeros((3, 2, 4), dtype=torch.int32))


def test_numbers_past_32_bits_are_refused(recorder):  # noqa: F811
    """None reaches the library cut to its low 32 bits, large or negative; what 32 bits hold does, for the library to refuse."""
    keys_ = tuple(OnGpu(x) for x in dg.fp8_kv_block_keys_empty(6, 2, 64, device="cpu"))
    q, table = OnGpu(torch.zeros((3, 4, 64), dtype=torch.bfloat16)), OnGpu(torch.zeros((3, 5), dtype=torch.int32))
    lens, out = OnGpu(torch.zeros(3, dtype=torch.int32)), OnGpu(torch.zeros((3, 2, 4), dtype=torch.int32))
    good = dict(page_size=16, top=4, first=1, last=2)

    def call(**kw):
        dg.fp8_kv_select_blocks(q, keys_, table, lens, out=out, **{**good, **kw})

    for name, x in good.items():
        for cut in (2 ** 32, -2 ** 32, 2 ** 64, -2 ** 70):
            with pytest.raises(ValueError, match="32 bits"):
                call(**{name: x + cut})
        with pytest.raises(TypeError):
            call(**{name: "4" if name != "top" else None})
    with pytest.raises(ValueError, match="32 bits"):
        call(first=2 ** 31)
    assert not recorder.calls
    call(first=-2 ** 31, last=np.int64(2), page_size=np.int32(16), top=np.int64(4))
    args = recorder.calls["dg_fp8_kv_select_blocks"][-1]
    assert args[1] == 16 and args[14:17] == (4, -2 ** 31, 2) and all(type(args[i]) is int for i in (1, 14, 15, 16))
    assert recorder.calls["dg_fp8_kv_select_blocks_workspace"][-1][8:] == (4, -2 ** 31, 2)
    # attention's bound saturates, as full attention's does
    cu = OnGpu(torch.zeros(4, dtype=torch.int32))
    attn_out = OnGpu(torch.zeros((3, 4, 64), dtype=torch.bfloat16))
    for given, passed in ((2 ** 32 + 5, 2 ** 31 - 1), (-2 ** 32, -1)):
        dg.fp8_block_sparse_attention(q, *fake_cache(), table, lens, out, cu_seqlens_q=cu, max_seqlen_q=given, out=attn_out)
        assert recorder.calls["dg_fp8_block_sparse_attention"][-1][8] == passed


# ---------------------------------------------------------------- pins of the oracle
def test_oracle_scale_is_the_smallest():
    rng = np.random.default_rng(0)
    tops = np.concatenate([np.exp(rng.uniform(-60, 60, 200)), 127.0 * 2.0 ** np.arange(-20, 20), np.nextafter(127.0 * 2.0 ** np.arange(-20, 20), np.inf),
                           2.0 ** np.arange(-20.0, 20.0), [2.0 ** -140]])
    for t, s in zip(tops, int8_scale(tops)):
        assert Fraction(t) <= 127 * Fraction(s) and math.frexp(s)[0] == 0.5
        assert s == 2.0 ** -126 or Fraction(t) > 127 * Fraction(s) / 2
    assert int8_scale(0.0) == 1.0


def test_oracle_block_keys_by_fractions():
    rng = np.random.default_rng(1)
    c, s = oracle.kv_encode(kv_gen.rows(rng, 2, 3, 5, 64))
    codes, scale = oracle.block_keys((c, s))
    val = oracle.kv_decode(c, s)
    for p in range(2):
        for h in range(3):
            mean = [sum(Fraction(v) for v in val[p, h, :, d]) / 5 for d in range(64)]
            k = Fraction(float(scale[p, h]))
            assert k / 2 * 127 < max(abs(m) for m in mean) <= 127 * k
            assert [round(m / k) for m in mean] == codes[p, h].tolist()  # (Python rounds ties to even)


def test_oracle_choice_by_brute_force():
    rng = np.random.default_rng(2)
    page, top, first, last = 4, 5, 1, 2
    keys = (rng.integers(-2, 3, (12, 2, 64)).astype(np.int8), 2.0 ** rng.integers(-1, 2, (12, 2)))  # (many ties)
    q = np.sign(rng.standard_normal((6, 4, 64)))
    lens, cu = np.array([41, 9]), np.array([0, 4, 6])
    table = np.array([rng.permutation(12), rng.permutation(12)])
    got = oracle.select_blocks(q, keys, table, lens, cu, page, top, first, last)
    for t, (b, place) in enumerate([(0, 37), (0, 38), (0, 39), (0, 40), (1, 7), (1, 8)]):
        n = place // page + 1
        for h in range(2):
            # (a query of ones has codes of 64 under 2^-6)
            score = [max(int(np.sign(q[t, x]) @ keys[0][table[b, j], h].astype(int)) * keys[1][table[b, j], h] for x in (2 * h, 2 * h + 1)) for j in range(n)]
            take = {j for j in range(n) if j < first or j >= n - last}
            while len(take) < min(top, n):
                take.add(max((j for j in range(n) if j not in take), key=lambda j: (score[j], -j)))
            assert got[t, h].tolist() == sorted(take) + [-1] * (top - len(take))


def test_oracle_attention_over_all_blocks_is_attention():
    p = kv_gen.problem([37, 5], [4, 2], 4, 2, 64, 16, 0, garbage=False)
    blocks = np.broadcast_to(np.arange(3, dtype=np.int32), (6, 2, 3))
    a = oracle.block_sparse_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], blocks, 0.1)
    b = oracle.paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], 0.1)
    for x in a:
        assert np.allclose(a[x], b[x], rtol=1e-13, atol=1e-13), x
    # and a window of whole blocks is attention over the last ones
    one = np.full((6, 2, 1), -1, dtype=np.int32)
    one[:4] = 2
    c = oracle.block_sparse_attention(p["q"][:4], p["k"], p["v"], p["table"], p["lens"], np.array([0, 4, 4]), one[:4], 0.1)
    d = oracle.paged_attention(p["q"][3:4], p["k"], p["v"], p["table"], p["lens"][:1], np.array([0, 1]), 0.1, window=5)
    assert np.allclose(c["out"][3], d["out"][0], rtol=1e-13, atol=1e-13)
