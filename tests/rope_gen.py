"""Seeded inputs for the tests of norm and rotation, and the error bounds of their FP32 arithmetic."""
import numpy as np

import oracle

E = 2.0 ** -24  # half a step of FP32, relative


def to_type(x, bf16):
    """float64 rows rounded to BF16 (as values) or FP32."""
    return oracle.bf16_bits_to_f64(oracle.bf16_rne(x)) if bf16 else x.astype(np.float32).astype(np.float64)


def table(positions, rot, base=10000.0):
    turn = np.arange(positions)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(turn), np.sin(turn)], -1).astype(np.float32)


def problem(tokens, heads, kv_heads, dim, rot, bf16, seed, weights_bf16=None, positions=500):
    rng = np.random.default_rng(seed)
    size = np.exp(2.0 * rng.standard_normal((tokens, 1, 1)))

    def rows(h):
        return to_type(rng.standard_normal((tokens, h, dim)) * size, bf16)

    weights_bf16 = bf16 if weights_bf16 is None else weights_bf16
    pos = rng.integers(0, positions, tokens).astype(np.int64)
    if tokens > 4:  # padding tokens, and the table's ends
        pos[[0, 1, 2, 3]] = [-1, positions, positions - 1, 0]
        pos[tokens // 2] = -2 ** 40
    return {"q": rows(heads), "k": rows(kv_heads), "v": rows(kv_heads), "dq": rows(heads), "dk": rows(kv_heads),
            "qw": to_type(1.0 + 0.3 * rng.standard_normal(dim), weights_bf16),
            "kw": to_type(1.0 + 0.3 * rng.standard_normal(dim), weights_bf16),
            "cs": table(positions, rot), "pos": pos, "bf16": bf16, "weights_bf16": weights_bf16}


def half(bf16):
    return 2.0 ** -8 if bf16 else E


def forward32(size):
    """Largest error of a result before its last rounding.  The sum of D <= 256 squares is 16 of a lane and at most 4 joins
    (20 roundings), its mean plus eps one more, the square root halves what came before and adds one, the quotient
    another: 13 E; times x and w, two more; the turn's products and sum, two: 17 E of the magnitudes added."""
    return 17 * E * size


def rounded(tol, ref, bf16):
    """With the result's own rounding (and FP32's smallest numbers)."""
    return tol + (np.abs(ref) + tol) * half(bf16) + 1e-37


def backward32(big, along):
    """A turned gradient has 3 roundings and w one: g is off by 4 E; u = x r by 14 E; their products by 19 E, the mean over D adds 21: 40 E;
    times u 15 more, the difference 1, times r 14: 19 E on g's side, 70 E on the other."""
    return 19 * E * big + 70 * E * along


def weights32(total, rows_in_turn):
    """Each term is off by 3 + 14 + 1 roundings; a lane adds `rows_in_turn` of them, its wave at most 4 more, the
    workgroup 4, the sums of workgroups 32 + at most 32."""
    return (18 + rows_in_turn + 72) * E * total + 1e-37
