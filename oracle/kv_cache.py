"""The FP8 key/value cache and the attention that reads it, in float64.

Test infrastructure only (see the package docstring).

A row (one token and head, D values) is held as E4M3 codes and one power-of-two scale kept as a
UE8M0 code: the scale is max|x| / 448 raised to the next power of two, 1 for a row of zeros, at
least 2^-126 (the cast's UE8M0 recipe with the row as its group).  A token's slot is
page * page_size + place.

Attention: query i of a sequence's n new tokens stands at place x = len - n + i and sees keys
j <= x; with a window W only those with j > x - W or j < sinks.
"""
import numpy as np

from .codecs import e4m3_decode, ue8m0_decode, ue8m0_encode
from .quant import E4M3_MAX, e4m3_encode_rne, pow2_ceil


def kv_encode(x):
    """x [..., D] float32, finite -> (codes uint8 [..., D], scale codes uint8 [...])."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(axis=-1)
    s = pow2_ceil((amax / np.float32(E4M3_MAX)).astype(np.float32))
    q = np.clip(x.astype(np.float64) / s.astype(np.float64)[..., None], -E4M3_MAX, E4M3_MAX)
    return e4m3_encode_rne(q), ue8m0_encode(s)


def kv_decode(codes, sf):
    """Codes [..., D] and scale codes [...] -> float64 values."""
    return e4m3_decode(codes) * ue8m0_decode(sf)[..., None]


def kv_write(cache, x, slots):
    """The cache (codes [P, H, page, D], sf [P, H, page]) with rows x [T, H, D] written to their slots."""
    codes, sf = cache[0].copy(), cache[1].copy()
    page, total = codes.shape[2], codes.shape[0] * codes.shape[2]
    for t, slot in enumerate(slots):
        if 0 <= slot < total:
            codes[slot // page, :, slot % page], sf[slot // page, :, slot % page] = kv_encode(x[t])
    return codes, sf


def kv_read(cache, slots):
    codes, sf = cache
    page, total = codes.shape[2], codes.shape[0] * codes.shape[2]
    out = np.zeros((len(slots), codes.shape[1], codes.shape[3]))
    for t, slot in enumerate(slots):
        if 0 <= slot < total:
            out[t] = kv_decode(codes[slot // page, :, slot % page], sf[slot // page, :, slot % page])
    return out


def visible(length, n, window=0, sinks=0):
    """Boolean [n, length]: which keys each of the n newest queries sees."""
    x = (length - n + np.arange(n))[:, None]
    j = np.arange(max(length, 0))[None, :]
    seen = j <= x
    if window:
        seen &= (j > x - window) | (j < sinks)
    return seen


def paged_attention(q, k_cache, v_cache, table, lens, cu, scale, window=0, sinks=0):
    """q [T, Hq, D] float64.  Returns a dict of float64 arrays: out [T, Hq, D], lse [T, Hq], and for
    error bounds abs [T, Hq, D] = sum softmax |v|, size [T, Hq] = max over visible keys of
    scale * sum |q_d k_d|, and seen [T] (visible keys)."""
    T, Hq, D = q.shape
    H, page = k_cache[0].shape[1:3]
    group = Hq // H
    r = {"out": np.zeros((T, Hq, D)), "lse": np.full((T, Hq), -np.inf), "abs": np.zeros((T, Hq, D)),
         "size": np.zeros((T, Hq)), "seen": np.zeros(T, dtype=np.int64)}
    for b, length in enumerate(lens):
        first, n = int(cu[b]), int(cu[b + 1] - cu[b])
        if length <= 0 or n <= 0:
            continue
        pages = table[b][: -(-length // page)]
        k, v = (np.moveaxis(kv_decode(c[0][pages], c[1][pages]), 1, 0).reshape(H, -1, D)[:, :length]
                for c in (k_cache, v_cache))
        seen = visible(length, n, window, sinks)
        r["seen"][first:first + n] = seen.sum(1)
        for h in range(Hq):
            qq, kk, vv = q[first:first + n, h], k[h // group], v[h // group]
            s = np.where(seen, scale * (qq @ kk.T), -np.inf)
            top = s.max(1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            p = np.exp(s - top)
            z = p.sum(1, keepdims=True)
            safe = np.where(z > 0, z, 1.0)
            r["out"][first:first + n, h] = p @ vv / safe
            r["abs"][first:first + n, h] = p @ np.abs(vv) / safe
            with np.errstate(divide="ignore"):
                r["lse"][first:first + n, h] = (top + np.log(z))[:, 0]
            r["size"][first:first + n, h] = np.where(seen, scale * (np.abs(qq) @ np.abs(kk).T), 0.0).max(1)
    return r
