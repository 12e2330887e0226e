"""paged_decode_shared row by row: each query row within a bound of its own, so that one key lost or
counted twice shows; block ids outside the pool; waits that run out in mid-item; pools beyond
2^31 elements.

Bound of a row of n keys, from the kernel's roundings (those of test_gpu_paged_decode_shared.py, with
the row's own sizes).  W = sum of weight |V| per entry, X = scale * sum_d |q_d| max_j |K_jd|.  A
weight is off by its exponent, (132 * 2^-23 X + 2^-21) of itself, in the product with V and in
the sum; for the product with V it is rounded to bf16 as well, 2^-8 of itself, and n products are
summed in fp32, 2^-23 of W each at most.  The result is rounded to bf16:
    |out - ref| <= 2^-8 |ref| + W (2^-8 + 2 (132 * 2^-23 X + 2^-21) + 2^-23 n), times 1 + 2^-7
for products of these terms.  One of n keys of equal weight moves a row by 1/n of |V - ref|, which
is beyond that for some entry of a row of up to 200 keys."""
import numpy as np
import pytest
import torch

from gpu_util import f64, lib, status_word
from test_gpu_paged_decode_shared import BF, PLANS, Batch

pytestmark = pytest.mark.gpu


def check_rows(b, got, skip=()):
    """Every row of `got` against the definition; keys in the blocks (sequence, place) of `skip`
    are left out."""
    q, k, v = f64(b.tq), f64(b.tk), f64(b.tv)
    bs, hkv = k.shape[1:3]
    g = b.hq // hkv
    worst = 0.0
    for i in range(len(b.ctx)):
        j = np.arange(b.ctx[i])
        j = j[~np.isin(j // bs, [at for s, at in skip if s == i])]
        if len(j) == 0:
            assert (got[i] == 0).all()
            continue
        blk = b.bt[i, j // bs]
        kk, vv = k[blk, j % bs], v[blk, j % bs]                    # [n, hkv, d]
        out = f64(got[i])
        for h in range(hkv):
            rows = q[i, h * g:(h + 1) * g]
            s = b.scale * rows @ kk[:, h].T
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            ref, size = w @ vv[:, h], w @ np.abs(vv[:, h])
            x = b.scale * np.abs(rows) @ np.abs(kk[:, h]).max(0)
            rel = 2.0 ** -8 + 2 * (132 * 2.0 ** -23 * x + 2.0 ** -21) + 2.0 ** -23 * len(j)
            bound = (2.0 ** -8 * np.abs(ref) + size * rel[:, None]) * (1 + 2.0 ** -7)
            err = np.abs(out[h * g:(h + 1) * g] - ref) / bound
            worst = max(worst, float(err.max()))
            assert worst <= 1, (i, h, worst)
    return worst


def test_the_bound_sees_one_key(cuda):
    """With one key left out of the reference, or counted as another, the check fails."""
    pkv = lib()
    b = Batch([3], [70], [60, 130, 5], 2, 1, 64, 16, cuda, seed=50)
    got = b.run(pkv)
    check_rows(b, got)
    for i, ctx in enumerate(b.ctx.copy()):
        b.ctx[i] = ctx - 1
        with pytest.raises(AssertionError):
            check_rows(b, got)
        b.ctx[i] = ctx


@pytest.mark.parametrize("name", PLANS)
def test_plans_row_by_row(cuda, name):
    pkv = lib()
    sizes, prefixes, suffixes, hq, hkv, d, bs = PLANS[name]
    if isinstance(suffixes, int):
        suffixes = np.random.default_rng(2).integers(0, suffixes + 1, sum(sizes)).tolist()
    b = Batch(sizes, prefixes, suffixes, hq, hkv, d, bs, cuda, seed=21)
    st = pkv.new_status(cuda)
    got = b.run(pkv, status=st)
    assert status_word(st) == 0
    check_rows(b, got)


SHAPES = [  # sizes, prefixes, suffixes' bound, hq, hkv, d, block size
    ([3, 1, 90, 40], [64, 63, 128, 129], 70, 8, 8, 64, 16),
    ([128], [129], 3, 4, 4, 128, 8),                    # no own keys, or one tile of few
    ([200, 100], [65, 190], 130, 14, 2, 64, 20),
    ([33, 34, 35], [120, 121, 240], 121, 5, 1, 128, 24),
    ([257], [100], 129, 2, 2, 64, 1),
    ([513, 2], [70, 80], 20, 1, 1, 128, 48),
    ([1025], [96], 40, 1, 1, 64, 32),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_shapes_row_by_row(cuda, case):
    pkv = lib()
    sizes, prefixes, most, hq, hkv, d, bs = SHAPES[case]
    suffixes = np.random.default_rng(case).integers(0, most + 1, sum(sizes)).tolist()
    b = Batch(sizes, prefixes, suffixes, hq, hkv, d, bs, cuda, seed=30 + case)
    st = pkv.new_status(cuda)
    got = b.run(pkv, status=st)
    assert status_word(st) == 0
    check_rows(b, got)


@pytest.mark.parametrize("bs,d", [(16, 128), (20, 64), (24, 128), (256, 64), (5, 64)])
@pytest.mark.parametrize("where", ["common", "own", "both"])
def test_blocks_outside_the_pool(cuda, bs, d, where):
    """Their keys are left out, of all members where they are common, and no others: behind the first
    such tile every tile of its CTA takes its mask from the producer, for a dozen more and
    several items."""
    pkv = lib()
    sizes, prefixes = [40, 24], [1280, 512]
    suffixes = np.random.default_rng(bs).integers(1, 1200, 64).tolist()
    b = Batch(sizes, prefixes, suffixes, 4, 4, d, bs, cuda, seed=40)
    good = b.run(pkv)
    bt, skip, touched = b.bt.copy(), [], set()
    outside = [-1, b.tk.shape[0], 2**31 - 1, -2**31]
    if where != "own":
        for at, bad in ((0, outside[1]), (7 if bs < 100 else 2, outside[0])):
            bt[:40, at] = bad                           # each member's table, or its first's
            skip += [(i, at) for i in range(40)]
        touched |= set(range(40))
    if where != "common":
        for i, bad in zip((3, 41, 63), outside[1:]):
            first = prefixes[i >= 40] // bs + (1 if prefixes[i >= 40] % bs else 0)
            at = first if first * bs < b.ctx[i] else None
            if at is not None:
                bt[i, at] = bad
                skip.append((i, at))
                touched.add(i)
    st = pkv.new_status(cuda)
    got = pkv.paged_decode_shared(b.tq, b.tk, b.tv, torch.from_numpy(bt).to(cuda), b.tctx, b.toff,
                                  b.tpre, b.scale, b.max_ctx, status=st)
    assert status_word(st) == pkv.STATUS["BAD_BLOCK_ID"]
    check_rows(b, got, skip)
    rest = [i for i in range(64) if i not in touched]
    assert torch.equal(got[rest], good[rest])


@pytest.mark.parametrize("d,bs", [(128, 16), (64, 20), (64, 256), (128, 24)])
def test_waits_that_run_out_in_mid_item(cuda, d, bs):
    """With a few polls some waits succeed and some give up: the call unwinds with copies and products
    in flight, reports nothing else, and the next one is right."""
    pkv = lib()
    b = Batch([90, 3], [1300, 200], [300] * 93, 8, 2, d, bs, cuda, seed=13)
    ref = b.run(pkv)
    ws = pkv.paged_decode_plan_shared(b.tctx, b.toff, b.tpre, 8, b.max_ctx, b.tbt.shape[1], b.tk)
    for polls in (1, 2, 3, 5):
        st = pkv.new_status(cuda)
        pkv.set_wait_poll_limit(polls)
        try:
            pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws,
                                        status=st)
        finally:
            pkv.set_wait_poll_limit()
        assert status_word(st) & ~pkv.STATUS["WAIT_TIMEOUT"] == 0
        got = pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws,
                                          status=st.zero_())
        assert torch.equal(got, ref) and status_word(st) == 0


@pytest.mark.parametrize("bs", [16, 20, 256])
def test_a_pool_beyond_32_bit_offsets(cuda, bs):
    """Blocks at the end of a pool of more than 2^31 elements: the bits of a small pool's."""
    pkv = lib()
    hkv, d = 8, 128
    b = Batch([5, 2], [300, 140], [200, 0, 33, 1, 700, 128, 90], 16, hkv, d, bs, cuda, seed=60)
    ref = b.run(pkv)
    nb = b.tk.shape[0]
    far = (1 << 31) // (bs * hkv * d) + 5               # the first block used there
    pools = []
    for small in (b.tk, b.tv):
        big = torch.empty((far + nb, bs, hkv, d), dtype=BF, device=cuda)
        assert big[far:].storage_offset() > 1 << 31
        big[far:] = small
        pools.append(big)
    bt = torch.where(b.tbt >= 0, b.tbt + far, b.tbt)
    st = pkv.new_status(cuda)
    got = pkv.paged_decode_shared(b.tq, *pools, bt, b.tctx, b.toff, b.tpre, b.scale, b.max_ctx,
                                  status=st)
    assert status_word(st) == 0 and torch.equal(got, ref)
