"""CPU tests of the FP8 key/value cache: argument validation (before any HIP call), the binding's
refusals, the workspace's size, and pins of the oracle against something other than itself."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_scaled_fp8_amd as dg
import oracle
from tests import kv_gen

DG_OK, NULL, DTYPE, SHAPE, LAYOUT, UNSUPPORTED, HIP = 0, -1, -2, -3, -4, -5, -6
P, P_MIS, P_ODD = 4096, 4104, 4097   # fake addresses: never dereferenced


def cache(**kw):
    f = dict(k=P, v=P, k_sf=P, v_sf=P, num_pages=10, num_heads=4, page_size=16, head_dim=128, page_stride=8192,
             head_stride=2048, token_stride=128, sf_page_stride=64, sf_head_stride=16, sf_token_stride=1)
    f.update(kw)
    return dg._KvCache(*f.values())


CACHE_FAULTS = [
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED),
    (dict(num_heads=0), SHAPE), (dict(num_heads=65536), SHAPE), (dict(page_size=0), SHAPE), (dict(num_pages=-1), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 20, page_size=1 << 11), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k_sf=None), NULL), (dict(v_sf=None), NULL),
    (dict(k=P_MIS), LAYOUT), (dict(v=P_MIS), LAYOUT), (dict(page_stride=8200), LAYOUT), (dict(head_stride=2056), LAYOUT),
    (dict(token_stride=136), LAYOUT), (dict(token_stride=64), LAYOUT), (dict(page_stride=-8192), LAYOUT), (dict(sf_head_stride=-1), LAYOUT),
    (dict(token_stride=1 << 24), LAYOUT), (dict(sf_token_stride=1 << 24), LAYOUT),
]


def move(fn, c=None, **kw):
    a = dict(n=3, k=P, kts=512, khs=128, v=P, vts=512, vhs=128, dtype=1, slots=P, stream=None)
    a.update(kw)
    return getattr(dg.lib(), fn)(ctypes.byref(cache() if c is None else c), *a.values())


@pytest.mark.parametrize("fn", ["dg_fp8_kv_cache_write", "dg_fp8_kv_cache_read"])
def test_write_and_read_refuse(fn):
    for kw, code in CACHE_FAULTS:
        assert move(fn, cache(**kw)) == code, kw
        assert dg.lib().dg_get_last_error()
    for kw, code in [(dict(dtype=0), DTYPE), (dict(n=-1), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL),
                     (dict(k=P_MIS), LAYOUT), (dict(v=P_MIS), LAYOUT), (dict(kts=516), LAYOUT), (dict(vhs=132), LAYOUT),
                     (dict(kts=514, dtype=2), LAYOUT), (dict(khs=-128), LAYOUT), (dict(slots=P_ODD), LAYOUT)]:
        assert move(fn, **kw) == code, kw
    assert getattr(dg.lib(), fn)(None, 0, None, 0, 0, None, 0, 0, 1, None, None) == NULL
    # no tokens: nothing is read or written, so pointers may be NULL
    assert move(fn, cache(k=None, v=None, k_sf=None, v_sf=None, num_pages=0), n=0, k=None, v=None, slots=None) == DG_OK


def attend(c=None, **kw):
    a = dict(batch=2, total_q=4, hq=8, q=P, qts=1024, qhs=128, cu=P, max_q=2, table=P, ts=5, cols=5, lens=P, max_k=80, scale=0.1,
             window=0, sinks=0, out=P, ots=1024, ohs=128, lse=None, work=None, work_bytes=0, stream=None)
    a.update(kw)
    return dg.lib().dg_fp8_paged_attention(ctypes.byref(cache() if c is None else c), *a.values())


def test_attention_refuses():
    for kw, code in CACHE_FAULTS:
        assert attend(cache(**kw)) == code, kw
    for kw, code in [(dict(batch=-1), SHAPE), (dict(total_q=-4), SHAPE), (dict(hq=6), SHAPE), (dict(hq=0), SHAPE), (dict(hq=-4), SHAPE),
                     (dict(total_q=1 << 29), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(max_q=-1), SHAPE),
                     (dict(max_k=-1), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=math.inf), SHAPE),
                     (dict(scale=math.nan), SHAPE), (dict(cu=None, total_q=5), SHAPE), (dict(cols=-1), LAYOUT), (dict(ts=4), LAYOUT),
                     (dict(cols=1 << 27, ts=1 << 27), SHAPE), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(q=None), NULL),
                     (dict(out=None), NULL), (dict(q=P_MIS), LAYOUT), (dict(out=P_MIS), LAYOUT), (dict(qts=1028), LAYOUT),
                     (dict(ohs=132), LAYOUT), (dict(lse=P_ODD), LAYOUT), (dict(lens=P_ODD), LAYOUT), (dict(cu=P_ODD), LAYOUT),
                     (dict(table=P_ODD), LAYOUT)]:
        assert attend(**kw) == code, kw
    for kw in (dict(batch=0), dict(total_q=0), dict(max_q=0)):
        assert attend(cache(k=None), q=None, out=None, table=None, lens=None, **kw) == DG_OK, kw


def test_a_workspace_that_is_missing_or_small_is_refused():
    lib = dg.lib()
    assert lib.dg_set_num_sms(256) == DG_OK
    try:
        args = (2, 4, 8, 4, 128, 0, 2, 1 << 16, 0, 0)
        need = lib.dg_fp8_paged_attention_workspace(*args)
        assert need > 0
        assert attend(max_k=1 << 16) == NULL
        assert attend(max_k=1 << 16, work=P, work_bytes=need - 1) == SHAPE
        assert attend(max_k=1 << 16, work=P_MIS, work_bytes=need) == LAYOUT
        # a window bounds the keys, and with them the parts
        assert lib.dg_fp8_paged_attention_workspace(*args[:-2], 20, 4) == 0
        assert lib.dg_fp8_paged_attention_workspace(0, 0, 8, 4, 128, 0, 2, 1 << 16, 0, 0) == 0
        assert lib.dg_fp8_paged_attention_workspace(2, 4, 8, 3, 128, 0, 2, 1 << 16, 0, 0) == SHAPE
        assert lib.dg_fp8_paged_attention_workspace(2, 4, 8, 4, 80, 0, 2, 1 << 16, 0, 0) == UNSUPPORTED
    finally:
        lib.dg_set_num_sms(0)


def test_binding_refuses():
    k, v = dg.fp8_kv_cache_empty(4, 2, 16, 64, device="cpu")
    x, slots = torch.zeros((3, 2, 64)), torch.arange(3)
    with pytest.raises(ValueError, match="GPU"):
        dg.fp8_kv_cache_write(x, x, k, v, slots)
    with pytest.raises(TypeError, match="codes"):
        dg.fp8_kv_cache_read((k[0].float(), k[1]), v, slots)
    with pytest.raises(TypeError, match="scales"):
        dg.fp8_kv_cache_read((k[0], k[1].int()), v, slots)
    with pytest.raises(ValueError, match="same shape"):
        dg.fp8_kv_cache_read(k, (v[0][:3], v[1]), slots)
    with pytest.raises(ValueError, match="scales"):
        dg.fp8_kv_cache_read(k, (v[0], v[1].transpose(1, 2)), slots)
    with pytest.raises(ValueError, match="GPU"):
        dg.fp8_paged_attention(torch.zeros((1, 2, 64), dtype=torch.bfloat16), k, v, torch.zeros((1, 1), dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32))


# ---------------------------------------------------------------- the oracle's pins
def test_encode_against_torch_and_hand_values():
    rng = np.random.default_rng(0)
    x = kv_gen.rows(rng, 200, 3, 64, wide=True)
    codes, sf = oracle.kv_encode(x)
    s = np.ldexp(1.0, sf.astype(int) - 127)
    amax = np.abs(x).max(-1).astype(np.float64)
    assert (amax <= 448 * s).all() and (amax > 224 * s).all()   # the smallest power of two that holds the row
    q = torch.from_numpy((x / s[..., None]).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q, codes)
    y = np.zeros((3, 64), np.float32)
    y[1, 5], y[2, 7] = 448.0, -449.0
    codes, sf = oracle.kv_encode(y)
    assert sf.tolist() == [127, 127, 128] and codes[1, 5] == 0x7E and codes[2, 7] == 0xF6   # -449 / 2 -> -224
    # the cast's power-of-two recipe on one 128-long group gives the same
    z = kv_gen.rows(rng, 50, 128, wide=True)
    q, s = oracle.per_token_group_cast(z, ue8m0=True)
    codes, sf = oracle.kv_encode(z)
    assert np.array_equal(q, codes) and np.array_equal(s[:, 0].astype(np.float64), oracle.ue8m0_decode(sf))


def test_write_then_read_goes_by_slots():
    rng = np.random.default_rng(1)
    x = kv_gen.rows(rng, 6, 2, 64)
    empty = np.zeros((3, 2, 4, 64), np.uint8), np.full((3, 2, 4), 127, np.uint8)
    slots = [11, 0, -1, 5, 12, 6]
    c = oracle.kv_write(empty, x, slots)
    back = oracle.kv_read(c, slots)
    assert (back[2] == 0).all() and (back[4] == 0).all()
    for t in (0, 1, 3, 5):
        assert (np.abs(back[t] - x[t]) <= np.abs(x[t]) / 16 + 1e-3 * np.abs(x[t]).max()).all()
    assert (oracle.kv_read(c, [1, 2, 3, 4, 7, 8, 9, 10]) == 0).all()
    assert np.array_equal(c[0][1, :, 1], oracle.kv_encode(x[3])[0])   # slot 5 of pages of 4: page 1, place 1


def test_attention_against_exact_sums():
    """Scores whose exponentials are rational: s = log 2 times a whole number, so weights are powers of two."""
    D, page = 64, 2
    k = np.zeros((5, 1, D), np.float32)
    k[:, 0, 0] = [1, 2, 0, 3, 1]
    v = np.zeros((5, 1, D), np.float32)
    v[:, 0, 0] = [1, -2, 4, 8, 16]
    codes = np.zeros((4, 1, page, D), np.uint8), np.full((4, 1, page), 127, np.uint8)
    table = [[2, 0, 3]]
    slots = [table[0][j // page] * page + j % page for j in range(5)]
    kc, vc = oracle.kv_write(codes, k, slots), oracle.kv_write(codes, v, slots)
    q = np.zeros((3, 2, D))
    q[:, 0, 0], q[:, 1, 0] = 1.0, 2.0
    for window, sinks in ((0, 0), (2, 0), (2, 1), (1, 0)):
        r = oracle.paged_attention(q, kc, vc, np.array(table), [5], [0, 3], math.log(2.0), window, sinks)
        for t in range(3):
            x = 2 + t
            for h in range(2):
                num = den = Fraction(0)
                for j in range(5):
                    if j <= x and (not window or x - j < window or j < sinks):
                        w = Fraction(2) ** int((h + 1) * k[j, 0, 0])
                        num, den = num + w * int(v[j, 0, 0]), den + w
                assert abs(r["out"][t, h, 0] - float(num / den)) < 1e-12
                assert abs(r["lse"][t, h] - math.log(den)) < 1e-12


def test_attention_of_rows_that_see_nothing():
    p = kv_gen.problem([2, 0], [4, 1], 2, 1, 64, 4, seed=1)
    r = oracle.paged_attention(p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"], 0.1)
    assert np.isneginf(r["lse"][[0, 1, 4]]).all() and (r["out"][[0, 1, 4]] == 0).all() and np.isfinite(r["lse"][[2, 3]]).all()
    assert r["seen"].tolist() == [0, 0, 1, 2, 0]


def test_visible_by_brute_force():
    for length, n, w, s in ((7, 3, 0, 0), (7, 7, 2, 1), (5, 8, 3, 2), (0, 2, 0, 0), (9, 1, 100, 3)):
        got = oracle.visible(length, n, w, s)
        for i in range(n):
            for j in range(length):
                x = length - n + i
                assert got[i, j] == (j <= x and (w == 0 or j > x - w or j < s))


def test_bounds_pass_a_correct_result_and_catch_mistakes():
    """The bounds hold for the oracle rounded to BF16, and not for results with one key left out, one key too
    many, a neighbour's scale, or weights that are not normalised."""
    p = kv_gen.problem([40], [5], 2, 1, 64, 16, seed=2)
    args = (p["q"], p["k"], p["v"], p["table"], p["lens"], p["cu"])
    r = oracle.paged_attention(*args, 0.125)
    tol, tol_lse = kv_gen.bounds(r, 64)
    rounded = oracle.bf16_bits_to_f64(oracle.bf16_rne(r["out"]))
    assert (np.abs(rounded - r["out"]) <= tol).all()
    fewer = oracle.paged_attention(*args, 0.125, window=36)["out"]
    more = oracle.paged_attention(*args[:4], p["lens"] - 1, p["cu"], 0.125)["out"]
    sf = p["k"][1].copy()
    sf[p["table"][0][0]] += 1
    scaled = oracle.paged_attention(p["q"], (p["k"][0], sf), *args[2:], 0.125)["out"]
    for wrong in (fewer, more, scaled, r["out"] * (1 + 2.0 ** -5)):
        assert not (np.abs(wrong - r["out"]) <= tol).all()


# ---------------------------------------------------------------- what the binding hands to the library
class OnGpu:
    """A CPU tensor that says it is on a GPU, for calls whose library side is replaced."""

    def __init__(self, t, index=0):
        self.t, self.device = t, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)


class Recorder:
    """Stands in for the library: keeps the arguments by function and says that all went well."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            self.calls.setdefault(name, []).append(args)
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(dg, "lib", lambda: r)
    monkeypatch.setattr(dg, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(dg, "_current_device", lambda: 0, raising=False)
    return r


def fake_cache(index=0):
    return [tuple(OnGpu(t, index) for t in x) for x in dg.fp8_kv_cache_empty(6, 2, 16, 64, device="cpu")]


def fake_attention(table, batch, index=0, **kw):
    q = OnGpu(torch.zeros((batch, 4, 64), dtype=torch.bfloat16), index)
    lens = OnGpu(torch.zeros(batch, dtype=torch.int32), index)
    return dg.fp8_paged_attention(q, *fake_cache(index), OnGpu(table, index), lens, out=q, **kw)


TABLE_STRIDE, TABLE_COLS = 10, 11  # their places among dg_fp8_paged_attention's arguments


def test_the_block_table_goes_by_its_own_stride(recorder):
    """Every row that the kernels may read lies in the table's storage: an expanded table has one row for all."""
    one = torch.zeros((1, 5), dtype=torch.int32)
    big = torch.zeros((7, 9), dtype=torch.int32)
    for table, batch in [(one, 1), (one.expand(4, -1), 4), (big, 7), (big[:, :5], 7), (big[::2, 2:6], 4), (big[:1, :3], 1), (big[:, :1], 7),
                         (one[:, :1].expand(3, 1), 3), (big[:, :0], 7), (torch.zeros(5, dtype=torch.int32).as_strided((1, 5), (2, 1)), 1)]:
        fake_attention(table, batch)
        args = recorder.calls["dg_fp8_paged_attention"][-1]
        stride, cols = args[TABLE_STRIDE], args[TABLE_COLS]
        assert cols == table.shape[1] and (stride >= cols or stride == 0)
        if batch > 1:
            assert stride == table.stride(0)
        assert table.storage_offset() + (batch - 1) * stride + cols <= table.untyped_storage().nbytes() // 4


def test_a_table_with_one_row_for_all_is_taken():
    """A row stride of zero passes the checks of the arguments (the next fault is found), one below the columns does not."""
    assert attend(ts=0, lens=None) == NULL
    assert attend(ts=3) == LAYOUT and attend(ts=-5) == LAYOUT


def test_more_tiles_than_a_launch_holds_are_refused():
    """batch * tiles of max_seqlen_q past 32 bits, with the binding's default bound (all rows) for example.  (The tables and
    queries are fake: none of these calls may reach a launch.)"""
    lib = dg.lib()
    assert lib.dg_set_num_sms(256) == DG_OK
    try:
        for batch, total, hq, hk in [(65537, 1 << 20, 16, 1), (8193, 1 << 20, 128, 1), ((1 << 31) - 1, 1 << 20, 16, 1), (1 << 20, 1 << 20, 16, 4)]:
            assert lib.dg_fp8_paged_attention_workspace(batch, total, hq, hk, 128, 0, total, 80, 0, 0) == SHAPE, batch
            assert attend(cache(num_heads=hk), batch=batch, total_q=total, hq=hq, max_q=total) == SHAPE, batch
            assert b"max_seqlen_q" in lib.dg_get_last_error()
        # a bound of the new tokens is what such calls lack
        assert lib.dg_fp8_paged_attention_workspace(65537, 1 << 20, 16, 1, 128, 0, 16, 80, 0, 0) >= 0
        # 1024 tiles of 256 rows a sequence, 512 threads each: 2^32 threads with 8192 sequences
        assert lib.dg_fp8_paged_attention_workspace(8191, 1 << 14, 16, 1, 128, 0, 1 << 14, 80, 0, 0) >= 0
        assert lib.dg_fp8_paged_attention_workspace(8192, 1 << 14, 16, 1, 128, 0, 1 << 14, 80, 0, 0) == SHAPE
    finally:
        lib.dg_set_num_sms(0)


WINDOW, SINKS, MAX_Q, MAX_K = 15, 16, 8, 13


def test_numbers_past_32_bits_are_not_cut(recorder):
    """A window or bound past what the library's 32-bit numbers hold means the same as the largest of them."""
    table = torch.zeros((2, 3), dtype=torch.int32)
    cu = OnGpu(torch.tensor([0, 1, 2], dtype=torch.int32))
    top = 2 ** 31 - 1
    for big in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 70):
        fake_attention(table, 2, window=big, sinks=big, cu_seqlens_q=cu, max_seqlen_q=big, max_seqlen_k=big)
        args = recorder.calls["dg_fp8_paged_attention"][-1]
        assert [args[i] for i in (WINDOW, SINKS, MAX_Q, MAX_K)] == [top] * 4
        assert recorder.calls["dg_fp8_paged_attention_workspace"][-1][6:] == (top,) * 4
    fake_attention(table, 2, window=-2 ** 32, sinks=-2 ** 40, cu_seqlens_q=cu, max_seqlen_q=-2 ** 32, max_seqlen_k=-2 ** 32)
    args = recorder.calls["dg_fp8_paged_attention"][-1]
    assert all(-2 ** 31 <= args[i] < 0 for i in (WINDOW, SINKS, MAX_Q, MAX_K))   # refused by the library
    fake_attention(table, 2, window=np.int64(7), sinks=np.int32(2))
    args = recorder.calls["dg_fp8_paged_attention"][-1]
    assert (args[WINDOW], args[SINKS]) == (7, 2) and type(args[WINDOW]) is int


def test_shapes_past_32_bits_are_refused(recorder):
    """No dimension reaches the library cut to its low 32 bits."""
    (kc, ks), (vc, vs) = fake_cache()
    many = 2 ** 32 + 6
    x = OnGpu(torch.zeros((1, 2, 64)).expand(many, -1, -1))

    class Slots(OnGpu):
        shape = (many,)

        def dim(self):
            return 1

        def is_contiguous(self):
            return True

    with pytest.raises(ValueError, match="32 bits"):
        dg.fp8_kv_cache_write(x, x, (kc, ks), (vc, vs), Slots(torch.zeros(1, dtype=torch.int64)))
    big = [OnGpu(t.t[:1].expand(many, *t.shape[1:])) for t in (kc, ks)]
    with pytest.raises(ValueError, match="32 bits"):
        dg.fp8_kv_cache_read(big, big, OnGpu(torch.zeros(1, dtype=torch.int64)), out=(x, x))
    with pytest.raises(ValueError, match="32 bits"):
        q = OnGpu(torch.zeros((1, 4, 64), dtype=torch.bfloat16).expand(many, -1, -1))
        dg.fp8_paged_attention(q, *fake_cache(), OnGpu(torch.zeros((1, 3), dtype=torch.int32)), OnGpu(torch.zeros(1, dtype=torch.int32)), out=q)
    assert not recorder.calls


def test_the_tensors_gpu_is_the_current_one_during_a_call(recorder, monkeypatch):
    """The default stream's handle names no GPU, and a launch goes to the current one."""
    now, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.index = torch.device(dev).index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *a):
            now[0] = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(dg, "_current_device", lambda: now[0])
    monkeypatch.setattr(dg, "_current_stream", lambda dev: seen.append((dev.index, now[0])) or 0)
    x, slots = (torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int64))
    for index in (0, 2, 0):
        k, v = fake_cache(index)
        dg.fp8_kv_cache_write(OnGpu(x, index), OnGpu(x, index), k, v, OnGpu(slots, index))
        dg.fp8_kv_cache_read(k, v, OnGpu(slots, index), out=(OnGpu(x, index), OnGpu(x, index)))
        fake_attention(torch.zeros((2, 3), dtype=torch.int32), 2, index)
        assert now == [0]
    assert len(seen) == 9 and all(a == b for a, b in seen)
