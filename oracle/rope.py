"""Rotary positions and the norms of queries and keys in fp64 (numpy), with the norms' gradients.

x [..., S, D], positions integers that broadcast to [..., S].  Pairs (a, b) of the first
rotary_dim values turn by t = position * inv_freq: gain * (a cos t - b sin t, b cos t + a sin t).
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def rotate(x, positions, inv_freq, interleaved=False, gain=1.0, inverse=False):
    x = np.asarray(x, np.float64)
    inv_freq = np.asarray(inv_freq, np.float64)
    n = inv_freq.size
    # whole turns leave first, in rational numbers: an angle of 2^31 radians keeps 2^-22 in fp64
    per = np.array([Fraction(float(f)) / (2 * _PI) for f in inv_freq], object)
    turns = np.asarray(positions).astype(object)[..., None] * per
    t = np.array([float(u % 1) for u in turns.reshape(-1)]).reshape(turns.shape) * (2 * np.pi)
    c, s = gain * np.cos(t), gain * np.sin(t) * (-1.0 if inverse else 1.0)
    y = x.copy()
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


_PI = Fraction("3.14159265358979323846264338327950288419716939937510")


def norm_rope(x, weight, eps, positions=None, inv_freq=(), interleaved=False, gain=1.0):
    x = np.asarray(x, np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = n * (1.0 if weight is None else np.asarray(weight, np.float64))
    return rotate(z, positions, inv_freq, interleaved, gain) if len(inv_freq) else z


def norm_rope_backward(dy, x, weight, eps, positions=None, inv_freq=(), interleaved=False, gain=1.0):
    """(dx, dweight) from the gradient of norm_rope's output."""
    x = np.asarray(x, np.float64)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    dz = rotate(dy, positions, inv_freq, interleaved, gain, inverse=True) if len(inv_freq) else np.asarray(dy, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dx = r * (w * dz - n * (w * dz * n).mean(-1, keepdims=True))
    return dx, (dz * n).reshape(-1, x.shape[-1]).sum(0)
