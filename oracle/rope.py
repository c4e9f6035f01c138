"""Rotary positions and the latent cache (oracle side), in float64.

Test infrastructure only (see :mod:`oracle`). The runner page takes queries and
keys that are already rotated; the rotation before it is defined here:

* frequency ``i`` of a token turns one pair of channels by
  ``position[axis(i)] * inv_freq[i]``; pairs are ``(i, i + n)`` or
  ``(2i, 2i + 1)`` of the first ``2n`` channels, the others pass;
* a latent row is 512 latent codes and 64 codes of the rotated key part, e4m3,
  each part with its own scale;
* absorbed latent attention: every head's key is the whole row, its value the
  first 512 channels.

The angle is reduced with integers: ``inv_freq / 2 pi`` as a fraction of 2^96
times the position, modulo a turn, so that positions near 2^40 keep their
angles.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

# pi to 60 decimals
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def angles(positions, inv_freq, freq_axis=None):
    """float64 [T, n]: position times frequency, reduced to [0, 2 pi).
    ``positions``: integers [T] or [axes, T]."""
    pos = np.asarray(positions, dtype=np.int64)
    pos = pos[None] if pos.ndim == 1 else pos
    n = len(inv_freq)
    axis = [0] * n if freq_axis is None else [min(int(a), pos.shape[0] - 1) for a in freq_axis]
    one = 1 << 96
    out = np.empty((pos.shape[1], n))
    for i in range(n):
        turn = round(Fraction(float(inv_freq[i])) / (2 * PI) * one)
        out[:, i] = [float((int(p) * turn) % one) / one for p in pos[axis[i]]]
    return out * (2 * np.pi)


def rotate(x, ang, interleaved, scale=1.0):
    """x float64 [T, heads, d]; the first 2n channels rotated by ang [T, n]."""
    x = np.array(x, dtype=np.float64)
    n = ang.shape[1]
    c, s = np.cos(ang)[:, None] * scale, np.sin(ang)[:, None] * scale
    a = x[..., 0:2 * n:2].copy() if interleaved else x[..., :n].copy()
    b = x[..., 1:2 * n:2].copy() if interleaved else x[..., n:2 * n].copy()
    lo, hi = a * c - b * s, b * c + a * s
    if interleaved:
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = lo, hi
    else:
        x[..., :n], x[..., n:2 * n] = lo, hi
    return x


def latent_attention(q, rows, softmax_scale, seq_len, causal):
    """One request: q float64 [q_len, h, 576], rows float64 [L, 576] (codes
    times their scales). Returns (out [q_len, h, 512], lse [q_len, h]); a row
    that sees no key is 0 with LSE -inf."""
    q_len, h, _ = q.shape
    out, lse = np.zeros((q_len, h, 512)), np.full((q_len, h), -np.inf)
    for t in range(q_len):
        n = seq_len if not causal else min(seq_len, seq_len - q_len + t + 1)
        if n <= 0:
            continue
        logit = q[t] @ rows[:n].T * softmax_scale
        top = logit.max(axis=1, keepdims=True)
        w = np.exp(logit - top)
        total = w.sum(axis=1, keepdims=True)
        out[t] = (w / total) @ rows[:n, :512]
        lse[t] = (top + np.log(total))[:, 0]
    return out, lse
