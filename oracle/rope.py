"""Norm and rotation of queries and keys in float64, and its gradients.

Test infrastructure only (see the package docstring).

y = w x / sqrt(mean(x^2) + eps) of a row, whose first R values turn in pairs (i, i + R/2), or (2i, 2i + 1)
interleaved, by the angles of the token's position; cos_sin [positions, R] holds R/2 cosines, then R/2 sines.  A
token whose position is not a row of the table gives zeros.
"""
import numpy as np


def _pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(y, cos_sin, positions, interleaved, back):
    """(turned rows, the sums of magnitudes that each value was made of)."""
    rot = cos_sin.shape[1]
    a, b = _pairs(rot, interleaved)
    at = np.clip(positions, 0, len(cos_sin) - 1)
    c = cos_sin[at, None, :rot // 2].astype(np.float64)
    s = cos_sin[at, None, rot // 2:].astype(np.float64) * (-1.0 if back else 1.0)
    out, size = y.copy(), np.abs(y)
    out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    size[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
    size[..., b] = np.abs(y[..., a] * s) + np.abs(y[..., b] * c)
    return out, size


def live_tokens(cos_sin, positions):
    return (positions >= 0) & (positions < len(cos_sin))


def norm_rope(x, w, cos_sin, positions, eps, interleaved=False):
    """x [T, H, D] -> (y, size): the result, and for error bounds the magnitudes that were added up to it."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y, size = _turn(x * r * w, cos_sin, positions, interleaved, False)
    dead = ~live_tokens(cos_sin, positions)
    y[dead] = 0.0
    size[dead] = 0.0
    return y, size


def norm_rope_backward(dout, x, w, cos_sin, positions, eps, interleaved=False):
    """Returns dx [T, H, D], dw [D], and for error bounds what their sums' magnitudes are: (|g|, |u| mean |g u|) times r,
    and sum |t u|."""
    dead = ~live_tokens(cos_sin, positions)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    t, size = _turn(dout, cos_sin, positions, interleaved, True)
    t[dead], size[dead] = 0.0, 0.0
    u, g = x * r, t * w
    dx = r * (g - u * (g * u).mean(-1, keepdims=True))
    big = size * np.abs(w)
    return (dx, (t * u).sum((0, 1)), r * big, r * np.abs(u) * (big * np.abs(u)).mean(-1, keepdims=True),
            (size * np.abs(u)).sum((0, 1)))
