"""Helpers of the 8-bit cache's GPU tests: inputs, and error bounds.

Bounds, from the kernels' roundings (a value rounded to t is off by at most
finfo(t).eps / 2 relative: bf16 2^-8, f16 2^-11, fp32 2^-24):
  * q . K: codes are exact.  The decode takes a q row, scaled so that its largest
    entry lies in [2^7, 2^8), as two e4m3 parts of 4 significant bits, the second
    16 times finer: exact for bf16's 8 bits down to the second part's smallest
    step, 2^-9 / 16, so off by 2^-14 < 2^-21 of the largest entry.  fp32 sums of at
    most 128 products, each partial sum off by at most 2^-23 of the magnitudes
    summed (a tensor core may cut instead of round).  With
    X = scale * max_j sum |q K_j| the exponent is off by at most
    dx = 128 * 2^-23 X + 2^-21 * scale * sum_d max|q| max_j |K_jd|,
    and by 4 * 2^-24 X from the fp32 steps behind it;
  * p is rounded for the product with V: in the prefill to bf16, 2^-8 of itself; in
    the decode to f16 and then to two parts as q is, 2^-11 + 2^-9 of itself (the
    first part leaves at most 2^-4 of [1, 2), the second rounds that to 4 bits)
    or 2^-14 / 2^8 of the row's largest p, whichever is more;
  * the result is rounded to bf16; exp2 is good to 2^-22.
With A = max |V| over the row's keys, an error d in every log weight moves the
output by at most 2 d A (a weighted mean of values within A), a rounding of
every p by r of itself by r A, and one of n weights by f of the largest by n f A.
    |out - ref| <= 2^-8 |ref| + A (r + n f + 2 (dx + 2^-21 X + 2^-21)).
The bound is taken against the largest sums of the case."""
from __future__ import annotations

import numpy as np
import torch

from oracle import fp8_cache as ofp

DECODE, PREFILL = (2.0 ** -9 + 2.0 ** -11, 2.0 ** -22), (2.0 ** -8, 0.0)      # r, f


def bound(ref, q, k_values, v_values, scale, rounding, n):
    """Elementwise error bound for outputs `ref` [.., D] of queries q [.., D]
    over at most n of the finite entries of the given key and value rows [.., D]."""
    r, f = rounding
    kmax = np.abs(np.where(np.isfinite(k_values), k_values, 0.0)).reshape(-1, q.shape[-1]).max(0)
    big_x = abs(scale) * (np.abs(q) * kmax).sum(-1).max()
    worst_q = abs(scale) * np.abs(q).max() * kmax.sum()
    a = np.abs(np.where(np.isfinite(v_values), v_values, 0.0)).max()
    d = (128 * 2.0 ** -23 + 2.0 ** -21) * big_x + 2.0 ** -21 * worst_q + 2.0 ** -21
    return 2.0 ** -8 * np.abs(ref) + a * (r + n * f + 2 * d)


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
