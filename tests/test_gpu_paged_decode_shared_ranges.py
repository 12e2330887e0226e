"""paged_decode_shared at the ends of its ranges: scores far from one."""
import numpy as np
import pytest
import torch

from gpu_util import f64, lib, status_word
from test_gpu_paged_decode_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs,d", [(16, 128), (256, 64), (24, 64), (20, 128)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(cuda, bs, d, sign):
    """A key's score is q0 K0 scale, K0 one of bf16's values in [1, 2): scores that differ do so by
    2^-7 of the largest, thousands here, so that the result is the value of the one key ahead,
    in the first tile or a later one, among the common keys or a sequence's own.  Its weight and
    its value's product are rounded to bf16: twice 2^-8."""
    pkv = lib()
    b = Batch([6, 3, 1], [400, 150, 0], [300, 1, 0, 77, 500, 20, 140, 5, 260, 33], 4, 2, d, bs,
              cuda, seed=bs)
    rng = np.random.default_rng(d)
    nb = b.tk.shape[0]
    k0 = torch.from_numpy(rng.integers(0, 127, nb * bs) / 128 + 1).to(torch.bfloat16).to(cuda)
    b.tk[torch.isfinite(b.tk)] = 0
    rows = lambda i, t: t.view(nb * bs, 2, d)[  # noqa: E731
        torch.from_numpy(b.bt[i, np.arange(b.ctx[i]) // bs].astype(np.int64) * bs +
                         np.arange(b.ctx[i]) % bs).to(cuda)]
    b.tk.view(-1, 2, d)[:, :, 0] = torch.where(b.tk.view(-1, 2, d)[:, :, 0].isnan(),
                                               b.tk.view(-1, 2, d)[:, :, 0], k0[:, None])
    for g, p in enumerate(b.prefix):               # the members' copies of a common row stay alike
        first, last = b.offsets[g], b.offsets[g + 1]
        if p % bs:
            head = b.tk[int(b.bt[first, p // bs]), :p % bs].clone()
            for i in range(first, last):
                b.tk[int(b.bt[i, p // bs]), :p % bs] = head
    # one key of each sequence ahead of its others: a common one of the first group, own ones of
    # the second and third
    ahead = [int(rng.integers(0, 400))] * 6 + [int(b.ctx[i]) - 1 for i in range(6, 10)]
    at = {}
    for i in range(10):
        j = ahead[i]
        at[i] = int(b.bt[i, j // bs]) * bs + j % bs
    lead = 1 + 127 / 128 if sign > 0 else 1 - 2.0 ** -7
    for i in range(10):
        b.tk.view(-1, 2, d)[at[i], :, 0] = lead
    # (its copies in blocks that are common only in part)
    p = int(b.prefix[0])
    if ahead[0] >= p // bs * bs:
        for i in range(6):
            b.tk[int(b.bt[i, p // bs]), ahead[0] % bs, :, 0] = lead
    want = torch.stack([rows(i, b.tv)[ahead[i]] for i in range(10)])       # [10, 2, d]
    want = f64(want)[:, [0, 0, 1, 1]]
    for top in (2.0 ** 20, 2.0 ** 24 + 2, 1.3 * 2.0 ** 26, 2.0 ** 27, 1.9 * 2.0 ** 28,
                1.1 * 2.0 ** 30, 1.7 * 2.0 ** 31, 1.3 * 2.0 ** 32, 1.9 * 2.0 ** 33,
                1.2 * 2.0 ** 40, 1.6 * 2.0 ** 63, 1.4 * 2.0 ** 100):
        for e in (0, 20):                          # the scale's part in a query's
            b.tq[:] = 0
            b.tq[:, :, 0] = sign * 2.0 ** e
            st = pkv.new_status(cuda)
            got = f64(pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, b.tctx, b.toff, b.tpre,
                                              top * 2.0 ** -e * 0.7, b.max_ctx, status=st))
            assert status_word(st) == 0
            assert np.isfinite(got).all(), (top, e)
            bound = np.abs(want) * (2.0 ** -7 + 2.0 ** -14)
            assert (np.abs(got - want) <= bound).all(), (top, e)


@pytest.mark.parametrize("bs,d", [(16, 64), (64, 128), (20, 64)])
@pytest.mark.parametrize("scale", [0.7, 2.0 ** -20 / 3, 1.0])
def test_scores_from_near_to_far(cuda, bs, d, scale):
    """Scores that cross every power of two from one tile to the next, rising, falling, of both
    signs, with equal maxima in several tiles.  They are K0's values, exact in 32 bits, so that
    the exponents are exact but for the product with the scale: weights within 2^-8 by their
    rounding, and by exponents of at most 126 times 2^-23."""
    pkv = lib()
    n = 12
    suffix = [900, 0, 130, 500, 1, 777, 640, 128, 300, 64, 1000, 250]
    b = Batch([4, 5, 1, 1, 1], [600, 300, 0, 0, 0], suffix, 2, 1, d, bs, cuda, seed=bs)
    rng = np.random.default_rng(d + bs)
    nb = b.tk.shape[0]
    b.tk[torch.isfinite(b.tk)] = 0
    flat = b.tk.view(nb * bs, d)
    logical = np.zeros((n, int(b.ctx.max())))
    for i in range(n):
        j = np.arange(b.ctx[i])
        slots = torch.from_numpy(b.bt[i, j // bs].astype(np.int64) * bs + j % bs).to(cuda)
        g = int(np.searchsorted(b.offsets, i, "right")) - 1
        first, p = int(b.offsets[g]), int(b.prefix[g])
        kind = i % 4
        e = (j // 16) if kind == 0 else (70 - j // 16) if kind == 1 else rng.integers(0, 80, len(j))
        v = 2.0 ** e.clip(0, 90) * (1 + rng.integers(0, 128, len(j)) / 128)
        if kind == 2:
            v = -v
        if kind == 3:                              # two maxima alike, of some sign
            v = np.where(rng.random(len(j)) < 0.5, -v, v)
            v[len(j) // 3] = v[-1] = 2.0 ** 85
        if i != first:
            v[:p] = logical[first, :p]
        logical[i, :len(j)] = v
        flat[slots, 0] = torch.from_numpy(v).to(cuda).to(torch.bfloat16)
    for sign in (1, -1):
        b.tq[:] = 0
        b.tq[:, 0, 0] = sign * 1.0
        b.tq[:, 1, 0] = sign * 2.0 ** -30
        st = pkv.new_status(cuda)
        got = f64(pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, b.tctx, b.toff, b.tpre, scale,
                                          b.max_ctx, status=st))
        assert status_word(st) == 0
        v = f64(b.tv).reshape(nb * bs, d)
        for i in range(n):
            j = np.arange(b.ctx[i])
            rows = v[b.bt[i, j // bs].astype(np.int64) * bs + j % bs]
            for h, f in enumerate((1.0, 2.0 ** -30)):
                x = scale * sign * f * logical[i, :len(j)]
                w = np.exp(x - x.max())
                w /= w.sum()
                ref, size = w @ rows, w @ np.abs(rows)
                bound = 2.0 ** -8 * (np.abs(ref) + size) + (2 * 126 * 2.0 ** -23 + 2.0 ** -14) * size
                err = np.abs(got[i, h] - ref)
                assert (err <= bound).all(), (i, h, sign, float((err / bound).max()))


@pytest.mark.parametrize("bs,d", [(16, 128), (20, 64)])
@pytest.mark.parametrize("e", [-126, -110, 100, 117, 120])
def test_values_of_any_size(cuda, bs, d, e):
    """Values of size 2^e, bf16's own range: with scores that rise from tile to tile by less than
    a new maximum is taken for, and without.  The sums pass neither end of 32 bits where the
    results are within bf16's.  Near its smallest each of n products adds 2^-149, the last
    place there, over a sum of weights of n 2^-18 or more (2^-16 for the first tile's maximum,
    whose other weights are within 2^-2 of it), and the result's half step is 2^-134."""
    pkv = lib()
    n = 100                                        # enough for runs of several tiles
    b = Batch([3, 2, n - 5], [500, 300, 0], [400, 1, 0, 130, 260] + [900 - i for i in range(n - 5)],
              4, 2, d, bs, cuda, seed=e + 200)
    keep = b.tv.isnan()
    b.tv = torch.where(keep, b.tv, (b.tv.clamp(-2, 2).float() * 2.0 ** e).to(torch.bfloat16))
    for slope in (0.0, 12 / 900):                  # base 2, over a context
        nb = b.tk.shape[0]
        b.tk[torch.isfinite(b.tk)] = 0
        b.tq[:], b.tq[:, :, 0] = 0, 1.0
        flat = b.tk.view(nb * bs, 2, d)
        logical = {}
        for i in range(n):
            j = np.arange(b.ctx[i])
            slots = torch.from_numpy(b.bt[i, j // bs].astype(np.int64) * bs + j % bs).to(cuda)
            logical[i] = slots
            flat[slots, :, 0] = torch.from_numpy(slope * j).to(cuda).to(torch.bfloat16)[:, None]
        st = pkv.new_status(cuda)
        got = f64(pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, b.tctx, b.toff, b.tpre,
                                          float(np.log(2)), b.max_ctx, status=st))
        assert status_word(st) == 0
        k, v = f64(flat[:, 0, 0]), f64(b.tv).reshape(nb * bs, 2, d)
        for i in range(n):
            at = logical[i].cpu().numpy()
            w = 2.0 ** k[at]
            w /= w.sum()
            for h in range(4):
                ref, size = w @ v[at, h // 2], w @ np.abs(v[at, h // 2])
                bound = 2.0 ** -8 * (np.abs(ref) + size) + 2.0 ** -12 * size + \
                    2.0 ** -131 + 2.0 ** -134
                err = np.abs(got[i, h] - ref)
                assert np.isfinite(got[i, h]).all(), (i, h, slope)
                assert (err <= bound).all(), (i, h, slope, float((err / bound).max()))


@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** 127, 3.4e38])
def test_scales_whose_scores_pass_32_bits(cuda, scale):
    """Scores of both signs around the ends of 32 bits, times log2 e as the kernel takes them: NaN
    where the largest passes them, zeros (no keys) where all are -infinite, else the value
    of the key ahead."""
    pkv = lib()
    for size in (0.25, 1.0, 16.0):
        b = Batch([3, 1, 1], [200, 0, 0], [40, 1, 90, 300, 100], 2, 1, 64, 16, cuda, seed=70)
        nb = b.tk.shape[0]
        rng = np.random.default_rng(1)
        k0 = torch.from_numpy(rng.integers(-127, 127, nb * 16) / 128 * size).to(torch.bfloat16)
        b.tk[torch.isfinite(b.tk)] = 0
        flat = b.tk.view(nb * 16, 64)
        flat[:, 0] = torch.where(flat[:, 0].isnan(), flat[:, 0], k0.to(cuda))
        b.tq[:], b.tq[:, :, 0] = 0, 1.0
        for i in range(3):                           # members' copies of a block common in part
            b.tk[int(b.bt[i, 12]), :8] = b.tk[int(b.bt[0, 12]), :8]
        got = f64(pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, b.tctx, b.toff, b.tpre, scale,
                                          b.max_ctx))
        k, v = f64(flat[:, 0]), f64(b.tv).reshape(nb * 16, 64)
        for i in range(5):
            j = np.arange(b.ctx[i])
            at = b.bt[i, j // 16].astype(np.int64) * 16 + j % 16
            top = k[at] == k[at].max()
            want = v[at][top].mean(0)
            size_of = np.abs(v[at][top]).mean(0)
            for h in range(2):
                with np.errstate(over="ignore"):
                    scale2 = float(np.float32(scale) * np.float32(1.4426950408889634))
                most = k[at].max() * scale2
                if not most <= 3.4028e38:
                    assert np.isnan(got[i, h]).all(), (size, i, h)
                elif most < -3.4028e38:
                    assert (got[i, h] == 0).all(), (size, i, h)
                else:
                    bound = 2.0 ** -7 * (size_of + np.abs(want))
                    assert (np.abs(got[i, h] - want) <= bound).all(), (size, i, h)
