"""Block keys, the choice of blocks by them, and attention over chosen blocks, in float64.

Test infrastructure only (see the package docstring).

A block is a page.  Its block key is, for each head, the mean of its keys as codes -127..127 under a power of two s, the smallest
with |mean| <= 127 s.  A query at place x has the own block x // page; it gets the first `first` blocks, the last `last`, and of those
between the ones of the highest score, `top` in all, equal scores by lower index.  A block's score is the largest, over the
query heads of the key head, of (codes . codes) * block scale * query scale.
"""
import numpy as np

from .kv_cache import kv_decode


def int8_scale(top):
    """The smallest power of two s >= 2^-126 with top <= 127 s; 1 for zeros."""
    top = np.asarray(top, dtype=np.float64)
    _, e = np.frexp(top)  # top = f 2^e, f in [1/2, 1): 2^(e - 7) is the only candidate but the next
    s = np.ldexp(1.0, np.maximum(e - 7, -126))
    s = np.where(top > 127.0 * s, 2.0 * s, s)
    return np.where(top == 0, 1.0, s)


def int8_rows(x):
    """Rows x [..., D] -> (codes as float64, scales [...]); what is no number counts as zero."""
    x = np.where(np.isfinite(x), x, 0.0)
    s = int8_scale(np.abs(x).max(-1))
    return np.rint(x / s[..., None]), s


def block_keys(k_cache):
    """(codes [pages, heads, page, D], scale codes) -> (codes int8 [pages, heads, D], scales [pages, heads])."""
    val = kv_decode(*k_cache)
    codes, s = int8_rows(np.where(np.isnan(val), 0.0, val).sum(2) / val.shape[2])
    return codes.astype(np.int8), s


def places(lens, cu):
    """For each packed token its sequence and place."""
    seq = np.concatenate([np.full(int(cu[b + 1] - cu[b]), b) for b in range(len(lens))] + [np.zeros(0)]).astype(np.int64)
    i = np.arange(len(seq)) - cu[seq]
    return seq, lens[seq] - (cu[seq + 1] - cu[seq]) + i


def select_blocks(q, keys, table, lens, cu, page, top, first, last):
    """q [T, Hq, D] float64 -> int32 [T, H, top]."""
    codes, scales = keys[0].astype(np.float64), keys[1]
    T, Hq, _ = q.shape
    H = codes.shape[1]
    out = np.full((T, H, top), -1, dtype=np.int32)
    qc, qs = int8_rows(q)
    seq, place = places(lens, cu)
    for t in range(T):
        own = place[t] // page
        n = own + 1
        if n <= top:
            out[t, :, :max(n, 0)] = np.arange(max(n, 0))
            continue
        pages = table[seq[t]][:n]
        pages = np.where((pages >= 0) & (pages < len(codes)), pages, 0)
        for h in range(H):
            hs = slice(h * (Hq // H), (h + 1) * (Hq // H))
            score = ((codes[pages, h] @ qc[t, hs].T) * scales[pages, h][:, None] * qs[t, hs]).max(1)
            between = np.arange(first, n - last)
            best = between[np.argsort(-score[between], kind="stable")][:top - first - last]
            out[t, h] = np.sort(np.concatenate([np.arange(first), best, np.arange(n - last, n)]))
    return out


def block_sparse_attention(q, k_cache, v_cache, table, lens, cu, blocks, scale):
    """As kv_cache.paged_attention, over the keys of `blocks` [T, H, top] (negative: none)."""
    T, Hq, D = q.shape
    H, page = k_cache[0].shape[1:3]
    r = {"out": np.zeros((T, Hq, D)), "lse": np.full((T, Hq), -np.inf), "abs": np.zeros((T, Hq, D)),
         "size": np.zeros((T, Hq)), "seen": np.zeros(T, dtype=np.int64)}
    seq, place = places(lens, cu)
    for t in range(T):
        for h in range(H):
            b = blocks[t, h][blocks[t, h] >= 0].astype(np.int64)
            j = (b[:, None] * page + np.arange(page)).ravel()
            j = j[j <= place[t]]
            if not len(j):
                continue
            pg = table[seq[t]][j // page]
            k, v = (kv_decode(c[0][pg, h, j % page], c[1][pg, h, j % page]) for c in (k_cache, v_cache))
            hs = slice(h * (Hq // H), (h + 1) * (Hq // H))
            s = scale * (q[t, hs] @ k.T)
            p = np.exp(s - s.max(1, keepdims=True))
            z = p.sum(1, keepdims=True)
            r["out"][t, hs] = p @ v / z
            r["abs"][t, hs] = p @ np.abs(v) / z
            r["lse"][t, hs] = (s.max(1, keepdims=True) + np.log(z))[:, 0]
            r["size"][t, hs] = scale * (np.abs(q[t, hs]) @ np.abs(k).T).max(1)
            r["seen"][t] = max(r["seen"][t], len(j))
    return r
