"""Helpers of the 8-bit cache's GPU tests: inputs, and error bounds.

Bounds, from the kernels' roundings (a value rounded to t is off by at most
finfo(t).eps / 2 relative: bf16 2^-8, f16 2^-11, fp32 2^-24):
  * q . K: operands are exact (q times a power of two in f16, codes in f16);
    fp32 sums of at most 128 products, each partial sum off by at most 2^-23 of
    the magnitudes summed (a tensor core may cut instead of round), so the
    exponent x is off by at most dx = 128 * 2^-23 * X with X = scale * max_j
    sum |q K_j|, and by 4 * 2^-24 * X from the fp32 steps behind it;
  * p is rounded to f16 (decode) or bf16 (prefill) for the product with V, and
    to bf16 the result; exp2 is good to 2^-22.
With A = max |V| over the row's keys, an error d in every log weight moves the
output by at most 2 d A (a weighted mean of values within A), and the rounding
of p by its half step times A.  So
    |out - ref| <= 2^-8 |ref| + A (rp + 2 (dx + 2^-21 X + 2^-21)),
rp = 2^-11 or 2^-8.  The bound is taken against the largest sums of the case."""
from __future__ import annotations

import numpy as np
import torch

from oracle import fp8_cache as ofp

RP_DECODE, RP_PREFILL = 2.0 ** -11, 2.0 ** -8


def bound(ref, q, k_values, v_values, scale, rp):
    """Elementwise error bound for outputs `ref` [.., D] of queries q [.., D]
    over the finite entries of the given key and value rows [.., D]."""
    kmax = np.abs(np.where(np.isfinite(k_values), k_values, 0.0)).reshape(-1, q.shape[-1]).max(0)
    big_x = abs(scale) * (np.abs(q) * kmax).sum(-1).max()
    a = np.abs(np.where(np.isfinite(v_values), v_values, 0.0)).max()
    d = (128 * 2.0 ** -23 + 2.0 ** -21) * big_x + 2.0 ** -21
    return 2.0 ** -8 * np.abs(ref) + a * (rp + 2 * d)


class Pool:
    """A random e4m3 cache of sequences of the given lengths: codes of about
    N(0, 1) rows, power-of-two (or arbitrary) scales, NaN codes in every slot
    that holds no token."""

    def __init__(self, lens, bs, hkv, d, seed, spread=2, arbitrary=False, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.bs = list(lens), bs
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + spare
        perm = rng.permutation(nb)
        width = max(1, max(need))
        self.bt = np.full((len(lens), width), -1, np.int32)
        used = np.zeros((nb, bs), bool)
        at = 0
        for i, n in enumerate(lens):
            blocks = perm[at:at + need[i]]
            at += need[i]
            self.bt[i, :need[i]] = blocks
            for j, blk in enumerate(blocks):
                used[blk, :min(bs, n - j * bs)] = True
        self.codes, self.scale = {}, {}
        for name in "kv":
            c = ofp.encode(rng.normal(size=(nb, bs, hkv, d)) * 80)
            c[~used] = 0x7F
            s = 2.0 ** rng.integers(-7 - spread, -6, (nb, hkv))
            if arbitrary:
                s = s * rng.uniform(1, 2, s.shape)
            self.codes[name], self.scale[name] = c, s.astype(np.float32)

    def values(self, name):
        return ofp.decode_values(self.codes[name], self.scale[name])

    def on(self, dev):
        """(k_cache, v_cache, k_scale, v_scale, block_tables) on the GPU."""
        f8 = lambda c: torch.from_numpy(c).to(dev).view(torch.float8_e4m3fn)  # noqa: E731
        return (f8(self.codes["k"]), f8(self.codes["v"]),
                torch.from_numpy(self.scale["k"]).to(dev),
                torch.from_numpy(self.scale["v"]).to(dev), torch.from_numpy(self.bt).to(dev))


def bf16(rng, *shape, mag=1.0):
    return torch.from_numpy((rng.normal(size=shape) * mag).astype(np.float32)).to(torch.bfloat16)
