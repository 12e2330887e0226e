"""RMS norm of query and key heads and the rotation of their positions, in float64.

Test infrastructure only (see the package docstring).  Angles are formed in long
double, whose 64 bits or more hold p * w to 2^-33 radians for any int32 p.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_max_position=0,
                low=None, high=None):
    """(radians a position for each pair, magnitude)."""
    half = rotary_dim // 2
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    out, magnitude = [], 1.0
    for i in range(half):
        w = base ** (-2 * i / rotary_dim)
        if scaling == "linear":
            w = w / factor
        elif scaling == "yarn":
            lo, hi = (1 if low is None else low), (32 if high is None else high)

            def pair(turns):
                return half * math.log(original_max_position / (turns * 2 * math.pi)) / \
                    math.log(base)
            first = max(math.floor(pair(hi)), 0)
            last = min(math.ceil(pair(lo)), rotary_dim - 1)
            t = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            w = w * (1 - t) + w / factor * t
            magnitude = 0.1 * math.log(factor) + 1
        elif scaling == "bands":
            lo, hi = (1 if low is None else low), (4 if high is None else high)
            t = (original_max_position * w / (2 * math.pi) - lo) / (hi - lo)
            t = min(max(t, 0.0), 1.0)
            w = w * t + w / factor * (1 - t)
        out.append(w)
    return out, magnitude


def angles(positions, freq):
    """p * w modulo a turn, [tokens, pairs]."""
    p = np.asarray(positions).astype(np.longdouble)[:, None]
    two_pi = 8 * np.arctan(np.longdouble(1))
    return np.fmod(p * np.asarray(freq, dtype=np.float64).astype(np.longdouble)[None, :],
                   two_pi).astype(np.float64)


def norm_rope(x, weight, eps, positions, freq, interleaved=False, magnitude=1.0):
    """x [tokens, heads, D] -> the same, normed (weight None: not) and with its first
    2 len(freq) entries rotated."""
    y = np.asarray(x, dtype=np.float64).copy()
    if weight is not None:
        mean = (y * y).mean(-1, keepdims=True)
        y = y / np.sqrt(mean + eps) * np.asarray(weight, dtype=np.float64)
    r = 2 * len(freq)
    if r == 0:
        return y
    t = angles(positions, freq)[:, None, :]
    c, s = magnitude * np.cos(t), magnitude * np.sin(t)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                 slice(r // 2, r))
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y
