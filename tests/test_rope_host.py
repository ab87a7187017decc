"""CPU tests of norm and rotation of queries and keys: argument validation (before any HIP call), the binding's
refusals, and pins of the oracle against something other than itself."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_amd as dg
import oracle
from tests import rope_gen
from tests.test_kv_host import CACHE_FAULTS, cache

DG_OK, NULL, DTYPE, SHAPE, LAYOUT, UNSUPPORTED, HIP = 0, -1, -2, -3, -4, -5, -6
P, P_MIS, P_ODD = 4096, 4104, 4097   # fake addresses: never dereferenced


def call(**kw):
    a = dict(num_tokens=3, num_q_heads=8, num_kv_heads=4, head_dim=128, dtype=1, weight_dtype=1, q_weight=P, k_weight=P, cos_sin=P,
             cos_sin_stride=128, num_positions=10, positions=P, rot_dim=128, interleaved=0, eps=1e-6)
    a.update({k: v for k, v in kw.items() if k in a})
    return dg._NormRope(*a.values())


def rows(name, kw):
    return kw.get(name, (P, 1024, 128))


def forward(**kw):
    return dg.lib().dg_qk_norm_rope(call(**kw), *sum((rows(x, kw) for x in ("q", "k", "q_out", "k_out")), ()), None)


def backward(**kw):
    return dg.lib().dg_qk_norm_rope_backward(call(**kw), *sum((rows(x, kw) for x in ("dq_out", "dk_out", "q", "k", "dq", "dk")), ()),
                                             kw.get("dqw", P), kw.get("dkw", P), kw.get("work"), kw.get("work_bytes", 0), None)


def write(c=None, **kw):
    return dg.lib().dg_qk_norm_rope_fp8_kv_cache_write(call(**kw), *sum((rows(x, kw) for x in ("q", "k", "v", "q_out")), ()),
                                                       ctypes.byref(cache() if c is None else c), kw.get("slots", P), None)


FAULTS = [
    (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), UNSUPPORTED), (dict(num_tokens=-1), SHAPE), (dict(num_tokens=(1 << 30) + 1), SHAPE),
    (dict(num_q_heads=0), SHAPE), (dict(num_kv_heads=0), SHAPE), (dict(num_q_heads=65536), SHAPE), (dict(dtype=0), DTYPE), (dict(weight_dtype=3), DTYPE),
    (dict(rot_dim=0), SHAPE), (dict(rot_dim=24), SHAPE), (dict(rot_dim=144), SHAPE), (dict(rot_dim=-16), SHAPE), (dict(eps=-1e-6), SHAPE),
    (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE), (dict(num_positions=-1), SHAPE), (dict(cos_sin_stride=127), LAYOUT),
    (dict(cos_sin_stride=130), LAYOUT), (dict(cos_sin=P_MIS), LAYOUT), (dict(cos_sin=None), NULL), (dict(positions=None), NULL),
    (dict(positions=P_ODD), LAYOUT), (dict(q_weight=None), NULL), (dict(k_weight=None), NULL), (dict(k_weight=P_MIS), LAYOUT),
    (dict(q=(None, 1024, 128)), NULL), (dict(k=(P_MIS, 1024, 128)), LAYOUT), (dict(q=(P, 1028, 128)), LAYOUT), (dict(k=(P, 1024, 132)), LAYOUT),
    (dict(q=(P, 1024, -128)), LAYOUT), (dict(q=(P, 1026, 128), dtype=2), LAYOUT),
]


@pytest.mark.parametrize("fn", [forward, backward, write])
def test_refusals(fn):
    for kw, code in FAULTS:
        assert fn(**kw) == code, kw
        assert dg.lib().dg_get_last_error()


def test_refusals_of_each():
    for name in ("q_out", "k_out"):
        assert forward(**{name: (None, 1024, 128)}) == NULL
        assert forward(**{name: (P, 1028, 128)}) == LAYOUT
    for name in ("dq_out", "dk_out", "dq", "dk"):
        assert backward(**{name: (None, 1024, 128)}) == NULL
        assert backward(**{name: (P_MIS, 1024, 128)}) == LAYOUT
    assert backward(dqw=None) == NULL and backward(dkw=None) == NULL and backward(dkw=P_ODD) == LAYOUT
    assert backward(num_tokens=0, q_weight=None) == NULL  # (a kernel runs, and writes zeros)
    for kw, code in CACHE_FAULTS:
        assert write(cache(**kw), **({"head_dim": kw["head_dim"]} if kw.get("head_dim") == 0 else {})) in (code, UNSUPPORTED), kw
    assert write(cache(num_heads=5, page_stride=16384)) == SHAPE and write(cache(head_dim=64)) == SHAPE
    assert write(slots=None) == NULL and write(slots=P_ODD) == LAYOUT and write(v=(None, 1024, 128)) == NULL
    assert dg.lib().dg_qk_norm_rope(None, *[P, 1024, 128] * 4, None) == NULL
    # no tokens: nothing is read or written, so pointers may be NULL
    none = dict(num_tokens=0, q_weight=None, k_weight=None, cos_sin=None, positions=None)
    assert forward(**none, q=(None, 0, 0), q_out=(None, 0, 0)) == DG_OK
    assert write(cache(k=None, v=None, k_sf=None, v_sf=None), **none, q=(None, 0, 0), slots=None) == DG_OK


def test_workspace_is_checked():
    dg.set_num_sms(256)
    try:
        f = dg.lib().dg_qk_norm_rope_backward_workspace
        need = f(5000, 8, 4, 128)
        assert need == 1024 * 2 * 128 * 4
        assert f(1, 8, 4, 128) == 0 and f(0, 8, 4, 128) == 0
        assert f(5, 8, 4, 96) == UNSUPPORTED and f(-1, 8, 4, 128) == SHAPE
        assert backward(num_tokens=5000, work=None, work_bytes=need) == NULL
        assert backward(num_tokens=5000, work=P, work_bytes=need - 1) == SHAPE
        assert backward(num_tokens=5000, work=P_MIS, work_bytes=need) == LAYOUT
    finally:
        dg.set_num_sms(0)


def test_the_binding_refuses():
    q, k, w = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64), torch.ones(64)
    cs, pos = torch.zeros(9, 64), torch.zeros(4, dtype=torch.int64)
    for bad in [(q.half(), k.half(), w, w, cs, pos), (q, k.bfloat16(), w, w, cs, pos)]:
        with pytest.raises(TypeError):
            dg.qk_norm_rope(*bad)
    with pytest.raises(TypeError):
        dg.qk_norm_rope(q, k, w.half(), w.half(), cs, pos)
    for bad in [(q, k[:3], w, w, cs, pos), (q, k, w[:32], w, cs, pos), (q[0], k, w, w, cs, pos), (q, k, w, w, cs.double(), pos),
                (q, k, w, w, cs.T, pos), (q, k, w, w, cs, pos.int()), (q, k, w, w, cs, pos[:3]), (q, k, w, w, cs, pos),
                (q, k, torch.ones(64, 2)[:, 0], w, cs, pos)]:
        with pytest.raises(ValueError):  # (the last but one: not on a GPU)
            dg.qk_norm_rope(*bad)


# ---------------------------------------------------------------- pins of the oracle
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 48, 64])
def test_oracle_turns_as_complex_numbers_do(rot, interleaved):
    p = rope_gen.problem(7, 3, 1, 64, rot, False, rot)
    y, _ = oracle.norm_rope(p["q"], p["qw"], p["cs"], p["pos"], 1e-6, interleaved)
    for t in range(7):
        for h in range(3):
            x = p["q"][t, h]
            if not 0 <= p["pos"][t] < 500:
                assert (y[t, h] == 0).all()
                continue
            n = p["qw"] * x / math.sqrt(math.fsum(x * x) / 64 + 1e-6)
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                c = complex(p["cs"][p["pos"][t], i], p["cs"][p["pos"][t], rot // 2 + i]) * complex(n[a], n[b])
                assert abs(y[t, h, a] - c.real) < 1e-12 and abs(y[t, h, b] - c.imag) < 1e-12
            assert np.allclose(y[t, h, rot:], n[rot:], rtol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradients_are_those_of_differences(interleaved):
    p = rope_gen.problem(6, 2, 1, 64, 32, False, 3)
    x, w, rng = p["q"], p["qw"], np.random.default_rng(0)
    f = lambda x, w: (oracle.norm_rope(x, w, p["cs"], p["pos"], 1e-6, interleaved)[0] * p["dq"]).sum()  # noqa: E731
    dx, dw = oracle.norm_rope_backward(p["dq"], x, w, p["cs"], p["pos"], 1e-6, interleaved)[:2]
    for _ in range(20):
        # central differences: the error is h^2 / 6 of the third derivative and rounding / h
        v = rng.standard_normal(x.shape) * np.abs(x).max(-1, keepdims=True)
        h = 1e-5
        got = (f(x + h * v, w) - f(x - h * v, w)) / (2 * h)
        assert abs(got - (dx * v).sum()) < 1e-6 * np.abs(dx * v).sum()
        v = rng.standard_normal(w.shape)
        got = (f(x, w + h * v) - f(x, w - h * v)) / (2 * h)
        assert abs(got - (dw * v).sum()) < 1e-6 * np.abs(dw * v).sum()
