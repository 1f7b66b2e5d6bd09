"""Plain float64 definitions of the norm of q and k with the position rotation and of its gradients
(numpy; angles from whole-number arithmetic).  They share nothing with the library."""
from __future__ import annotations

import functools
from fractions import Fraction

import numpy as np

BITS = 240


@functools.lru_cache(maxsize=None)
def two_pi() -> int:
    """floor(2 pi 2^BITS), by Machin's formula: pi / 4 = 4 arctan(1/5) - arctan(1/239)."""
    one = 1 << (BITS + 32)

    def arctan_inverse(n):
        total, term, k, sign = 0, one // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return total

    return (8 * (4 * arctan_inverse(5) - arctan_inverse(239))) >> 32


def angles(positions, inv_freq) -> np.ndarray:
    """positions [..] x inv_freq [n] (float32) modulo 2 pi, each product exact, [.., n] float64."""
    pos = np.asarray(positions)
    out = np.empty(pos.shape + (len(inv_freq),))
    full = two_pi()
    steps = [int(Fraction(float(f)) * (1 << BITS)) for f in np.asarray(inv_freq, np.float32)]
    for at in np.ndindex(pos.shape):
        for i, f in enumerate(steps):
            out[at + (i,)] = (int(pos[at]) * f % full) / (1 << BITS)
    return out


def rotate(x, angle, interleaved, sign=1.0):
    """x [B, S, H, d], its first 2 n channels by angle [B, S, n]."""
    n = angle.shape[-1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    c, s = np.cos(angle)[:, :, None], sign * np.sin(angle)[:, :, None]
    y = np.array(x, np.float64)
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, b * c + a * s
    else:
        y[..., :n], y[..., n:2 * n] = a * c - b * s, b * c + a * s
    return y


def forward(x, angle, w=None, eps=None, interleaved=False):
    """eps None: no norm."""
    x = np.asarray(x, np.float64)
    if eps is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    return rotate(x, angle, interleaved)


def backward(x, dy, angle, w=None, eps=None, interleaved=False):
    """(dx, dw, what the sum of dw adds up in magnitudes); the last two None without a norm."""
    g = rotate(np.asarray(dy, np.float64), angle, interleaved, -1.0)
    if eps is None:
        return g, None, None
    x = np.asarray(x, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    e = g * (1.0 if w is None else w)
    return r * (e - xh * (e * xh).mean(-1, keepdims=True)), (g * xh).sum((0, 1, 2)), np.abs(g * xh).sum((0, 1, 2))
