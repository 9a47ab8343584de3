"""Plain CPU oracle of the norm and rotary operators.

TEST INFRASTRUCTURE ONLY, as ``msa_oracle``: only ``tests/`` imports it, and it
shares no code with the CUDA library.  fp64 throughout; the rotation is a
product of complex numbers.
"""
from __future__ import annotations

import numpy as np

from oracle.cache_oracle import E2M1, E4M3

D = 128


def turns(positions, inv_freq, axes):
    """Complex numbers of length 1, [tokens, pairs]: positions [tokens, columns] times radians per position."""
    pos = np.asarray(positions, np.float64)
    pos = pos[:, None] if pos.ndim == 1 else pos
    return np.exp(1j * pos[:, np.asarray(axes, int)] * np.asarray(inv_freq, np.float64))


def _pairs(x, n, adjacent):
    """The first 2 n dims as complex numbers [..., n]."""
    r = x[..., :2 * n]
    return r[..., 0::2] + 1j * r[..., 1::2] if adjacent else r[..., :n] + 1j * r[..., n:]


def _dims(x, z, adjacent):
    out, n = x.copy(), z.shape[-1]
    if adjacent:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = z.real, z.imag
    else:
        out[..., :n], out[..., n:2 * n] = z.real, z.imag
    return out


def rotate(x, turn, adjacent):
    """x fp64 [tokens, heads, 128]; turn [tokens, pairs]."""
    return _dims(x, _pairs(x, turn.shape[1], adjacent) * turn[:, None], adjacent)


def norm_rope(x, w, turn, adjacent, eps, scale=1.0):
    """x fp64 [tokens, heads, 128]; w fp64 weights (offset added) that broadcast over it, or None: no norm; turn None:
    no rotation.  scale multiplies the rotated dims."""
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return n if turn is None else rotate(n, turn * scale, adjacent)


def norm_rope_grad(x, w, dy, turn, adjacent, eps, scale=1.0):
    """Gradients of sum(dy * norm_rope(x)): to x, and to w for every row and head ([tokens, heads, 128]; None without
    a norm)."""
    g = dy if turn is None else rotate(dy, turn.conj() * scale, adjacent)
    if w is None:
        return g, None
    n = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return g * w / n - x * (g * w * x).sum(-1, keepdims=True) / (D * n ** 3), g * x / n


def round_values(x, exp):
    """Codes uint8 [..., 128] and e4m3 patterns uint8 [..., 8] of fp64 rows by the cache's rule."""
    g = (x * 2.0 ** -exp).reshape(*x.shape[:-1], 8, 16)
    finite = np.isfinite(g).all(-1)
    g = np.where(finite[..., None], g, 0.0)
    mids = (E4M3[:-1] + E4M3[1:]) / 2 * 6
    amax = np.abs(g).max(-1)
    idx = np.searchsorted(mids, amax, side="left")
    tie = mids[np.minimum(idx, len(mids) - 1)] == amax
    idx = np.where(tie & (idx % 2 == 1), idx + 1, idx)
    s = E4M3[idx][..., None]
    code = np.zeros(g.shape, np.int64)
    for i in range(1, 8):
        mid = (E2M1[i - 1] + E2M1[i]) / 2 * s
        code = np.where((np.abs(g) > mid) if i % 2 else (np.abs(g) >= mid), i, code)
    code = np.where(s > 0, code + 8 * ((g < 0) & (code > 0)), 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(finite, idx, 0x7F).astype(np.uint8)
