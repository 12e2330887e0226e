"""The 8-bit KV cache, restated on the CPU in float64.

Test infrastructure only (see the package docstring).

e4m3: 1 sign, 4 exponent (bias 7), 3 fraction bits; no infinities, one NaN
pattern a sign (0x7f, 0xff), largest value 448, subnormals below 2^-6.  A cache
holds codes (num_blocks, block_size, Hkv, D) uint8 and scales
(num_blocks, Hkv); an entry's value is its code's value times the scale of its
block and head.
"""
from __future__ import annotations

import math

import numpy as np

MAX = 448.0
EXP_LO, EXP_HI = -64, 119


def _values() -> np.ndarray:
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if c & 127 == 127 else (-mag if c & 128 else mag)
    return out


VALUES = _values()
_MAGS = VALUES[:127]                            # 0 .. 448, increasing


def encode(y) -> np.ndarray:
    """Codes of the e4m3 values nearest to y: of two equally near ones the even
    code, magnitudes above 448 become 448, NaN 0x7f."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    hi = np.clip(np.searchsorted(_MAGS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):         # infinities: hi is the last code anyway
        up, down = np.abs(_MAGS[hi] - a), np.abs(a - _MAGS[lo])
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= MAX, 126, code)
    code = np.where(np.signbit(y), code | 128, code)
    return np.where(np.isnan(y), 127, code).astype(np.uint8)


def scale_for(amax: float) -> float:
    """2^e for the least e with amax <= 448 * 2^e, clamped to [-64, 119]."""
    e = EXP_LO
    while e < EXP_HI and amax > MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def usable(scale: float) -> bool:
    return bool(2.0 ** -96 <= scale <= np.finfo(np.float32).max)


def kv_store(k, v, k_codes, v_codes, k_scale, v_scale, slot_mapping):
    """Stores rows k, v (N, Hkv, D) float64 into copies of the caches, block by
    block; returns (k_codes, v_codes, k_scale, v_scale, bad slots, bad scales)."""
    k_codes, v_codes = k_codes.copy(), v_codes.copy()
    k_scale, v_scale = np.array(k_scale, np.float64), np.array(v_scale, np.float64)
    num_blocks, block_size, heads, _ = k_codes.shape
    rows: dict[int, dict[int, int]] = {}
    bad_slots, bad_scales = [], 0
    for t, s in enumerate(np.asarray(slot_mapping).tolist()):
        if s < 0:
            continue
        if s >= num_blocks * block_size:
            bad_slots.append(s)
            continue
        rows.setdefault(s // block_size, {})[s % block_size] = t      # the last one stays
    for x, codes, scale in ((k, k_codes, k_scale), (v, v_codes, v_scale)):
        for blk, at in rows.items():
            for h in range(heads):
                old = scale[blk, h] if 0 not in at else 0.0
                if old != 0.0 and not usable(old):
                    bad_scales += 1
                    old = 0.0
                new = np.stack([x[t, h] for t in at.values()])
                finite = np.abs(new[np.isfinite(new)])
                c = max(old, scale_for(float(finite.max()) if finite.size else 0.0))
                if old > 0.0 and c > old:
                    others = [o for o in range(block_size) if o not in at]
                    # the ratio and the product are fp32 in the kernel; both are
                    # exact for powers of two
                    ratio = np.float64(np.float32(old / c))
                    codes[blk, others, h] = encode(
                        (VALUES[codes[blk, others, h]] * ratio).astype(np.float32))
                for o, t in at.items():
                    codes[blk, o, h] = encode((x[t, h] / c).astype(np.float32))
                scale[blk, h] = c
    return k_codes, v_codes, k_scale, v_scale, bad_slots, bad_scales


def decode_values(codes, scale) -> np.ndarray:
    """The cache's values, (num_blocks, block_size, Hkv, D) float64."""
    return VALUES[codes] * np.asarray(scale, np.float64)[:, None, :, None]
