"""GPU parity of norm and rotation of queries and keys, forward, backward and into the FP8 cache, through the
binding, against the float64 oracle."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_amd as dg
import oracle
from tests import rope_gen
from tests.test_gpu_kv import num_sms, same, say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5


def cuda(x, bf16):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(torch.bfloat16 if bf16 else torch.float32)


def operands(p):
    """q, k, v as slices of one projection's output, and the shared arguments."""
    x = torch.cat([cuda(p[n], p["bf16"]) for n in "qkv"], 1)
    q, k, v = x.split([p[n].shape[1] for n in "qkv"], 1)
    return q, k, v, (cuda(p["qw"], p["weights_bf16"]), cuda(p["kw"], p["weights_bf16"]), torch.from_numpy(p["cs"]).to(DEV),
                     torch.from_numpy(p["pos"]).to(DEV))


def inside(got, ref, tol, what):
    got = got.double().cpu().numpy()
    err = np.abs(got - ref)
    say(what, "largest error / bound", float((err / tol).max()) if err.size else 0.0)
    assert (err <= tol).all(), (what, float((err / tol).max()), np.argwhere(~(err <= tol))[:5])


def check_forward(p, got, interleaved, names="qk"):
    for n, y in zip(names, got):
        ref, size = oracle.norm_rope(p[n], p[n + "w"], p["cs"], p["pos"], EPS, interleaved)
        inside(y, ref, rope_gen.rounded(rope_gen.forward32(size), ref, p["bf16"]), n)


def check_backward(p, got, interleaved, in_turn=1):
    for i, n in enumerate("qk"):
        dx, dw, big, along, total = oracle.norm_rope_backward(p["d" + n], p[n], p[n + "w"], p["cs"], p["pos"], EPS, interleaved)
        inside(got[i], dx, rope_gen.rounded(rope_gen.backward32(big, along), dx, p["bf16"]), "d" + n)
        inside(got[2 + i], dw, rope_gen.weights32(total, in_turn), "d" + n + "_weight")


# tokens, heads, key heads, head dim, rotated dim
CASES = [(1, 32, 8, 128, 128), (37, 9, 3, 64, 32), (50, 5, 5, 64, 64), (130, 8, 1, 128, 48), (24, 7, 2, 128, 64), (65, 4, 2, 256, 256),
         (33, 3, 1, 256, 16), (9, 33, 17, 64, 16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, bf16, interleaved):
    say("norm and rotation", case, bf16, interleaved)
    p = rope_gen.problem(*case, bf16, sum(case), weights_bf16=bf16 != (case[0] == 130))
    q, k, _, args = operands(p)
    check_forward(p, dg.qk_norm_rope(q, k, *args, eps=EPS, interleaved=interleaved), interleaved)
    got = dg.qk_norm_rope_backward(cuda(p["dq"], bf16), cuda(p["dk"], bf16), q, k, *args, eps=EPS, interleaved=interleaved)
    check_backward(p, got, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 32), (128, 128), (256, 48)])
def test_gradients_are_those_of_differences(dim, rot, interleaved):
    """Along random directions, the library's FP32 gradients against central differences of the forward in 64 bits (off by h^2 / 6 of
    the third derivative, and rounding / h: 1e-6 of the magnitudes as the oracle's own), within the bounds of their arithmetic."""
    p = rope_gen.problem(9, 3, 2, dim, rot, False, 15)
    q, k, _, args = operands(p)
    got = dg.qk_norm_rope_backward(cuda(p["dq"], False), cuda(p["dk"], False), q, k, *args, eps=EPS, interleaved=interleaved)
    rng, h = np.random.default_rng(1), 1e-5
    for i, n in enumerate("qk"):
        x, w, g = p[n], p[n + "w"], p["d" + n]
        dx, dw = (got[j].double().cpu().numpy() for j in (i, 2 + i))
        _, _, big, along, total = oracle.norm_rope_backward(g, x, w, p["cs"], p["pos"], EPS, interleaved)
        tol, tol_w = rope_gen.rounded(rope_gen.backward32(big, along), dx, False), rope_gen.weights32(total, 1)
        f = lambda x, w: (oracle.norm_rope(x, w, p["cs"], p["pos"], EPS, interleaved)[0] * g).sum()  # noqa: E731
        for _ in range(10):
            v = rng.standard_normal(x.shape) * np.abs(x).max(-1, keepdims=True)
            want = (f(x + h * v, w) - f(x - h * v, w)) / (2 * h)
            assert abs((dx * v).sum() - want) <= (tol * np.abs(v)).sum() + 1e-6 * np.abs(dx * v).sum()
            v = rng.standard_normal(w.shape)
            want = (f(x, w + h * v) - f(x, w - h * v)) / (2 * h)
            assert abs((dw * v).sum() - want) <= (tol_w * np.abs(v)).sum() + 1e-6 * np.abs(dw * v).sum()


@pytest.mark.parametrize("sms", [1, 3])
def test_backward_with_many_rows_a_wave(sms):
    p = rope_gen.problem(301, 12, 3, 128, 128, True, 5)
    q, k, _, args = operands(p)
    with num_sms(sms):  # 4 sms workgroups of 4 waves
        got = dg.qk_norm_rope_backward(cuda(p["dq"], True), cuda(p["dk"], True), q, k, *args, eps=EPS)
        check_backward(p, got, False, -(-301 * 2 // (16 * sms)))
        again = dg.qk_norm_rope_backward(cuda(p["dq"], True), cuda(p["dk"], True), q, k, *args, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("bf16", [True, False])
def test_in_place(bf16):
    p = rope_gen.problem(40, 6, 2, 128, 64, bf16, 1)
    q, k, _, args = operands(p)
    want = dg.qk_norm_rope(q, k, *args)
    grads = cuda(p["dq"], bf16), cuda(p["dk"], bf16)
    back = dg.qk_norm_rope_backward(*grads, q, k, *args)
    again = dg.qk_norm_rope_backward(*grads, q, k, *args, out=grads)
    assert again[0] is grads[0] and all(torch.equal(a, b) for a, b in zip(back, again))
    got = dg.qk_norm_rope(q, k, *args, out=(q, k))
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("offset,gap", [(8, 0), (0, 8), (32, 0), (0, 32)])
def test_results_at_any_address(dim, offset, gap):
    """Rows that begin 16 or 64 bytes into a line, and rows with gaps between them: the same values, and nothing beside them."""
    p = rope_gen.problem(21, 9, 2, dim, dim, True, 11)
    q, k, _, args = operands(p)
    grads = cuda(p["dq"], True), cuda(p["dk"], True)
    want, back = dg.qk_norm_rope(q, k, *args), dg.qk_norm_rope_backward(*grads, q, k, *args)
    wide = [torch.full((21 * h * (dim + gap) + offset,), 77, dtype=torch.bfloat16, device=DEV) for h in (9, 2)]
    out = [x[offset:].view(21, -1, dim + gap)[..., :dim] for x in wide]
    for call, ref in ((lambda: dg.qk_norm_rope(q, k, *args, out=tuple(out)), want),
                      (lambda: dg.qk_norm_rope_backward(*grads, q, k, *args, out=tuple(out)), back)):
        assert all(torch.equal(x, y) for x, y in zip(call(), ref))
        assert all((x[:offset] == 77).all() and (x[offset:].view(-1, dim + gap)[:, dim:] == 77).all() for x in wide)


def test_a_table_without_positions():
    p = rope_gen.problem(5, 3, 1, 64, 64, True, 12)
    q, k, _, (qw, kw, cs, pos) = operands(p)
    args = qw, kw, cs[:0], pos
    assert all((x == 0).all() for x in dg.qk_norm_rope(q, k, *args))
    assert all((x == 0).all() for x in dg.qk_norm_rope_backward(cuda(p["dq"], True), cuda(p["dk"], True), q, k, *args))


def test_no_tokens():
    w, cs = torch.ones(128, device=DEV), torch.zeros((4, 128), device=DEV)
    q, k = torch.zeros((0, 4, 128), device=DEV), torch.zeros((0, 2, 128), device=DEV)
    pos = torch.zeros((0,), dtype=torch.int64, device=DEV)
    assert dg.qk_norm_rope(q, k, w, w, cs, pos)[0].shape == (0, 4, 128)
    dq, dk, dqw, dkw = dg.qk_norm_rope_backward(q, k, q, k, w, w, cs, pos)
    assert (dqw == 0).all() and (dkw == 0).all() and dk.shape == (0, 2, 128)
    k_cache, v_cache = dg.fp8_kv_cache_empty(2, 2, 16, 128, device=DEV)
    assert dg.qk_norm_rope_fp8_kv_cache_write(q, k, k, w, w, cs, pos, k_cache, v_cache, pos).shape == (0, 4, 128)


def test_numbers_that_are_none_stay_in_their_row():
    p = rope_gen.problem(20, 4, 2, 64, 64, False, 2)
    q, k, _, args = operands(p)
    want = dg.qk_norm_rope(q, k, *args)
    q[7, 2, 5] = float("nan")
    k[9, 1, 3] = float("inf")
    got = dg.qk_norm_rope(q, k, *args)
    assert got[0][7, 2].isnan().all() and got[1][9, 1].isnan().any()
    got[0][7, 2], got[1][9, 1] = want[0][7, 2], want[1][9, 1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a padding token's rows and gradients are not read for what they are
    q[0] = float("nan")
    q[7, 2, 5] = 1.0
    assert args[3][0] == -1 and (dg.qk_norm_rope(q, k, *args)[0][0] == 0).all()
    back = dg.qk_norm_rope_backward(q, k[:, :1].expand_as(k).contiguous(), q, k, *args)
    assert (back[0][0] == 0).all() and back[2].isfinite().all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 48), (256, 256)])
def test_rows_of_large_numbers(dim, rot, bf16, interleaved):
    """Up to 2^59 they are like any other; those whose squares pass FP32's range are zeros, up to the largest numbers and under weights above 1."""
    p = rope_gen.problem(24, 4, 2, dim, rot, bf16, 13)
    for n in "qk":
        p[n] /= np.abs(p[n]).max(-1, keepdims=True)  # (by the largest, which becomes 1)
        p[n] = rope_gen.to_type(p[n], bf16) * 2.0 ** 59
        p[n + "w"] = rope_gen.to_type(1.3 + 0.1 * np.abs(p[n + "w"]), bf16)
    q, k, v, args = operands(p)
    grads = cuda(p["dq"], bf16), cuda(p["dk"], bf16)
    want, back = dg.qk_norm_rope(q, k, *args, eps=EPS, interleaved=interleaved), dg.qk_norm_rope_backward(*grads, q, k, *args, eps=EPS, interleaved=interleaved)
    check_forward(p, want, interleaved)
    # (gradients come out under 2^-59, still well above the smallest numbers)
    check_backward(p, back, interleaved)
    huge = {5: 2.0 ** 66, 6: 2.0 ** 100, 7: 3.3e38, 8: -3.3e38}
    for t, x in huge.items():
        q[t, 1], k[t, 0] = x, x
        q[t, 1, ::3] *= -1
    k[9, 1], k[9, 1, dim - 1] = 1.0, 2.0 ** 127  # (one such value)
    caches = dg.fp8_kv_cache_empty(2, 2, 16, dim, device=DEV)
    for call in (lambda: dg.qk_norm_rope(q, k, *args, eps=EPS, interleaved=interleaved),
                 lambda: (dg.qk_norm_rope_fp8_kv_cache_write(q, k, v, *args, *caches, torch.arange(24, device=DEV), eps=EPS, interleaved=interleaved),)):
        for y, was, rows in zip(call(), want, ([(t, 1) for t in huge], [(t, 0) for t in huge] + [(9, 1)])):
            for t, h in rows:
                assert (y[t, h] == 0).all(), (t, h, y[t, h])
                y[t, h] = was[t, h]
            assert torch.equal(y, was)
    codes, sf = (x.transpose(1, 2).flatten(0, 1)[:24] for x in caches[0])
    assert all(not (codes[t, h] & 0x7F).any() and sf[t, h] == 127 for t, h in [(t, 0) for t in huge] + [(9, 1)])
    got = dg.qk_norm_rope_backward(*grads, q, k, *args, eps=EPS, interleaved=interleaved)
    assert all((got[0][t, 1] == 0).all() and (got[1][t, 0] == 0).all() for t in huge) and got[2].isfinite().all() and got[3].isfinite().all()


def test_infinities_among_large_numbers_stay():
    p = rope_gen.problem(8, 2, 1, 64, 32, False, 14)
    q, k, _, args = operands(p)
    q[5, 0] = 3e38
    q[5, 0, 40], q[6, 1, 50], q[7, 0, 3] = float("inf"), float("nan"), float("-inf")
    got = dg.qk_norm_rope(q, k, *args)[0]
    # what does not turn and is infinite is NaN, the rest of the row zero; a pair that turns has it in both places; a NaN is in all sums
    assert got[5, 0, 40].isnan() and got[5, 0].isnan().sum() == 1 and (got[5, 0, :40] == 0).all()
    assert got[6, 1].isnan().all() and got[7, 0].isnan().nonzero().flatten().tolist() == [3, 19]


@pytest.mark.parametrize("order", ["hpt", "thd"])
@pytest.mark.parametrize("bf16,interleaved", [(True, False), (True, True), (False, False)])
@pytest.mark.parametrize("case,page", [((61, 8, 2, 128, 128), 16), ((40, 9, 3, 64, 32), 7), ((23, 4, 2, 256, 64), 64), ((1, 32, 8, 128, 128), 64)])
def test_into_the_cache(case, page, bf16, interleaved, order):
    say("into the cache", case, page, bf16, interleaved, order)
    p = rope_gen.problem(*case, bf16, 7)
    tokens, heads, kv_heads, dim, _ = case
    q, k, v, args = operands(p)
    pages = -(-tokens // page) + 2
    rng = np.random.default_rng(1)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 10:
        slots[[5, 6, 7]] = [-1, pages * page, 2 ** 40]
    slots = torch.from_numpy(slots).to(DEV)

    def new_cache():
        c = dg.fp8_kv_cache_empty(pages, kv_heads, page, dim, device=DEV)
        for codes, sf in c:
            codes.fill_(0x33)
            sf.fill_(77)
        if order == "thd":
            c = tuple((codes.transpose(1, 2).contiguous().transpose(1, 2), sf.transpose(1, 2).contiguous().transpose(1, 2)) for codes, sf in c)
        return c

    caches, want = new_cache(), new_cache()
    got = dg.qk_norm_rope_fp8_kv_cache_write(q, k, v, *args, *caches, slots, eps=EPS, interleaved=interleaved)
    check_forward(p, [got], interleaved)
    # the same as the steps one by one, the keys between them in FP32
    keys = dg.qk_norm_rope(q.float(), k.float(), *args, eps=EPS, interleaved=interleaved)[1]
    live = (args[3] >= 0) & (args[3] < len(p["cs"]))
    dg.fp8_kv_cache_write(keys, v.float(), *want, torch.where(live, slots, -1))
    for a, b in zip(caches, want):
        assert same(a[0].cpu().numpy(), b[0].cpu().numpy()) and same(a[1].cpu().numpy(), b[1].cpu().numpy())
    # and near the oracle's keys: half a step of E4M3 (2^-4 of the value, 2^-10 of the scale) from what FP32 may give
    ref, size = oracle.norm_rope(p["k"], p["kw"], p["cs"], p["pos"], EPS, interleaved)
    tol = rope_gen.forward32(size)
    s = slots.cpu().numpy()
    codes, sf = caches[0][0].cpu().numpy(), caches[0][1].cpu().numpy()
    for t in range(tokens):
        if not live[t] or not 0 <= s[t] < pages * page:
            continue
        scale = 2.0 ** (sf[s[t] // page, :, s[t] % page].astype(np.float64) - 127)
        top = np.abs(ref[t]).max(-1)
        slack = tol[t].max(-1) * 1.01
        assert (top - slack <= 448 * scale).all() and (top + slack > 224 * scale).all()
        val = oracle.kv_decode(codes[s[t] // page, :, s[t] % page], sf[s[t] // page, :, s[t] % page])
        assert (np.abs(val - ref[t]) <= np.maximum(np.abs(ref[t]) * 2.0 ** -4, scale[:, None] * 2.0 ** -10) + 2 * tol[t]).all()


def test_other_streams_and_graphs():
    p = rope_gen.problem(64, 8, 2, 128, 128, True, 9)
    q, k, v, args = operands(p)
    dq, dk = cuda(p["dq"], True), cuda(p["dk"], True)
    caches = dg.fp8_kv_cache_empty(5, 2, 16, 128, device=DEV)
    slots = torch.arange(64, device=DEV)

    def step():
        a = dg.qk_norm_rope(q, k, *args)
        b = dg.qk_norm_rope_backward(dq, dk, q, k, *args)
        return [*a, *b, dg.qk_norm_rope_fp8_kv_cache_write(q, k, v, *args, *caches, slots)]

    want = [t.clone() for t in step()] + [c.clone() for x in caches for c in x]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(3):
        q.copy_(q.flip(0)), k.copy_(k.flip(0)), v.copy_(v.flip(0)), dq.copy_(dq.flip(0)), dk.copy_(dk.flip(0)), args[3].copy_(args[3].flip(0))
        eager = [t.clone() for t in step()] + [c.clone() for x in caches for c in x]
        for codes, sf in caches:
            codes.zero_(), sf.fill_(1)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out + [c for x in caches for c in x]
        # (padding tokens' slots keep what they held: zeros now, older tokens before)
        live = torch.zeros(80, dtype=torch.bool, device=DEV)
        live[:64] = (args[3] >= 0) & (args[3] < 500)
        for i, (a, b) in enumerate(zip(got, eager)):
            if i < 7:
                assert torch.equal(a, b), (turn, i)
            else:
                a, b = (x.transpose(1, 2).flatten(0, 1)[live] for x in (a, b))
                assert torch.equal(a, b), (turn, i)
    assert len(want) == 11


def test_more_tokens_than_one_launch_holds():
    """2^25 + 77 tokens: two launches, offsets past 32 bits; the last tokens against the same tokens alone."""
    n, tail = 2 ** 25 + 77, 100
    q = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(DEV).manual_seed(0)
    q[-tail:] = torch.randn((tail, 1, 64), generator=g, device=DEV)
    k[-tail:] = torch.randn((tail, 1, 64), generator=g, device=DEV)
    w, cs = torch.rand(64, generator=g, device=DEV), torch.from_numpy(rope_gen.table(300, 64)).to(DEV)
    pos = torch.arange(n, device=DEV) % 300
    say("many tokens")
    got = dg.qk_norm_rope(q, k, w, w, cs, pos, out=(q.clone().fill_(5), k.clone().fill_(5)))
    want = dg.qk_norm_rope(q[-tail:], k[-tail:], w, w, cs, pos[-tail:])
    assert torch.equal(got[0][-tail:], want[0]) and torch.equal(got[1][-tail:], want[1])
    assert not got[0][:-tail].any() and not got[1][:-tail].any()
    del got
    back = dg.qk_norm_rope_backward(q, k, q, k, w, w, cs, pos, out=(q, k))
    assert back[0] is q and not q[:-tail].any() and back[2].isfinite().all() and back[2].any()
