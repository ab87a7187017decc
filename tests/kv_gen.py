"""Seeded inputs for the FP8 key/value cache tests, and the error bounds of the attention tests."""
import numpy as np

import oracle


def rows(rng, *shape, wide=False):
    """Keys or values: normal, rows of different size, some large channels."""
    x = rng.standard_normal(shape) * np.exp((3.0 if wide else 0.5) * rng.standard_normal(shape[:-1] + (1,)))
    x *= 1.0 + 7.0 * (rng.random(shape[-1]) < 0.05)
    return x.astype(np.float32)


def problem(lens, news, heads, kv_heads, dim, page, seed, garbage=True):
    """A cache holding every sequence on pages in random order.  With ``garbage``, every place that belongs to no
    token holds a NaN code under a large scale, and unused table entries name pages that do not exist."""
    rng = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 2
    order = rng.permutation(pages)
    cols = max(1, max(used)) + 1
    table = np.where(rng.random((len(lens), cols)) < 0.5, -1, 2 ** 31 - 1).astype(np.int32) if garbage else np.zeros((len(lens), cols), np.int32)
    codes = [np.full((pages, kv_heads, page, dim), 0x7F if garbage else 0, np.uint8) for _ in range(2)]
    sfs = [np.full((pages, kv_heads, page), 200 if garbage else 127, np.uint8) for _ in range(2)]
    at = 0
    for b, n in enumerate(lens):
        table[b, :used[b]] = order[at: at + used[b]]
        for x in range(2):
            c, s = oracle.kv_encode(rows(rng, n, kv_heads, dim)) if n else (None, None)
            for j in range(n):
                pg = order[at + j // page]
                codes[x][pg, :, j % page], sfs[x][pg, :, j % page] = c[j], s[j]
        at += used[b]
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = rng.standard_normal((int(cu[-1]), heads, dim)).astype(np.float32)
    qb = oracle.bf16_rne(q.astype(np.float64))  # BF16 bits
    return {"k": (codes[0], sfs[0]), "v": (codes[1], sfs[1]), "table": table, "lens": np.array(lens, np.int32),
            "cu": cu, "news": news, "q_bits": qb, "q": oracle.bf16_bits_to_f64(qb), "dim": dim, "page": page}


def bounds(r, dim):
    """Largest error of out (BF16) and lse (FP32) that the arithmetic allows, from the oracle's sums:
      * a score is D exact products summed in FP32: off by at most D 2^-23 of the sum of their
        magnitudes, with one more rounding for scale and maximum and the hardware exponential
        (2^-20 in all): weights are off by a relative e = size * (D + 4) 2^-23 + 2^-20, which the
        quotient of two sums doubles;
      * a weight is rounded to BF16 (8 significant bits: 2^-8 of it at most) before it multiplies its value, and not in the sum of weights;
      * the sums over n keys add n 2^-23;
      * the result is rounded to BF16, 2^-8 of it."""
    n = r["seen"][:, None].astype(np.float64)
    e = r["size"] * (dim + 4) * 2.0 ** -23 + 2.0 ** -20
    tol = (2.0 ** -8 + 2 * e + 2 * n * 2.0 ** -23)[..., None] * r["abs"]
    tol = tol + (np.abs(r["out"]) + tol) * 2.0 ** -8 + 1e-30
    lse = np.where(np.isfinite(r["lse"]), r["lse"], 0.0)
    return tol, e + n * 2.0 ** -23 + (np.abs(lse) + 16) * 2.0 ** -22
