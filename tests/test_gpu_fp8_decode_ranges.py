"""paged_decode_fp8 at the ends of its stated ranges: scores, queries, key scales and value
scales far from one, each with and without a combine, in boxes and gathered."""
import math

import numpy as np
import pytest
import torch

import fp8_util as F
import gpu_util as U
from oracle import attention as oatt

pytestmark = pytest.mark.gpu


def _decode(pkv, cuda, q, pool, scale, max_context_len=None):
    st = pkv.new_status(cuda)
    ctx = torch.tensor(pool.lens, dtype=torch.int32, device=cuda)
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda), ctx, scale,
                               max_context_len or max(pool.lens), status=st)
    assert U.status_word(st) == 0
    return U.f64(out)


def _check(got, q, pool, scale):
    kv, vv = pool.values("k"), pool.values("v")
    ref = oatt.paged_decode(U.f64(q), kv, vv, pool.bt, pool.lens, scale)
    assert np.isfinite(got).all()
    tol = F.bound(ref, U.f64(q), kv, vv, scale, F.DECODE, max(pool.lens))
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 128), (256, 64), (24, 64)])
@pytest.mark.parametrize("n,most", [(300, 300), (700, 5000), (2500, 1 << 20)])
@pytest.mark.parametrize("group", [2, 8])
def test_scores_of_any_size(cuda, bs, d, n, most, group):
    """The largest score anywhere between 2^20 and 2^29 (base 2), of either sign, the others
    far below it: the output is that key's value, which e4m3 times a power of two
    holds exactly and bf16 too."""
    pkv = U.lib()
    rng = np.random.default_rng(bs + n)
    tops = [s * t for t in (2.0 ** 20, 2.0 ** 24 + 2.0, 2.0 ** 25, 2.0 ** 26, 1.3 * 2.0 ** 26,
                            1.9 * 2.0 ** 26, 2.0 ** 27, 2.0 ** 27 + 16, 1.3 * 2.0 ** 27,
                            1.9 * 2.0 ** 27, 2.0 ** 28, 1.7 * 2.0 ** 28, 2.0 ** 29)
            for s in (1, -1)]
    for top in tops:
        pool = F.Pool([n], bs, 1, d, seed=bs)
        at = int(rng.integers(0, n))
        # every key's first code is 448 below zero or 224 above it; the top one's is
        # 448, or -224 where all scores are negative
        best, rest = (0x7E, 0x76) if top > 0 else (0xF6, 0xFE)
        pool.codes["k"][:, :, 0, 0] = np.where(pool.codes["k"][:, :, 0, 0] == 0x7F, 0x7F, rest)
        pool.codes["k"][pool.bt[0, at // bs], at % bs, 0, 0] = best
        pool.scale["k"][:] = 1.0
        pool.scale["v"][:] = 2.0 ** -7
        q = torch.zeros((1, group, d), dtype=torch.bfloat16)
        q[:, :, 0] = 1.0
        scale = abs(top) / (448 if top > 0 else 224) * math.log(2)
        got = _decode(pkv, cuda, q, pool, scale, most)
        want = pool.values("v")[pool.bt[0, at // bs], at % bs, 0]
        np.testing.assert_array_equal(got, np.broadcast_to(want, got.shape), err_msg=str(top))


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 128), (40, 64)])
@pytest.mark.parametrize("q_mag", [6e37, 1e37, 1e36, 1e-31, 1e-33, 1e-35, 1e-37, 1e-39])
def test_queries_of_any_size(cuda, bs, d, q_mag):
    """Down to bf16's subnormals and up to its largest values, with key scales and a
    softmax scale that make the scores ordinary."""
    pkv = U.lib()
    rng = np.random.default_rng(11)
    hkv, group, lens = 2, 4, [200, 77]
    pool = F.Pool(lens, bs, hkv, d, seed=4)
    # the keys' scales take what they can of it (2^-96 .. 2^127), the softmax scale the rest
    exp = -round(math.log2(q_mag))
    k_exp = min(max(exp, -80), 120)
    pool.scale["k"] = np.ldexp(pool.scale["k"], k_exp).astype(np.float32)
    scale = math.ldexp(0.125, exp - k_exp)
    q = F.bf16(rng, 2, hkv * group, d, mag=q_mag)
    assert torch.isfinite(q).all() and (q != 0).float().mean() > 0.9
    q[0, 0, :5] = 0.0
    q[1, 3] = 0.0
    if q_mag > 1:
        q[1, 0, 7] = -torch.finfo(torch.bfloat16).max
    _check(_decode(pkv, cuda, q, pool, scale), q, pool, scale)


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 128), (24, 64)])
@pytest.mark.parametrize("q_exp", [20, 60])
def test_zero_keys_under_a_large_scale(cuda, bs, d, q_exp):
    """A block of zero K codes under a scale of 2^125 beside queries of 2^20 and more: the scores
    of its keys are zero, not zero times an overflow."""
    pkv = U.lib()
    rng = np.random.default_rng(bs + q_exp)
    lens = [4 * bs + 5, 3 * bs]
    pool = F.Pool(lens, bs, 1, d, seed=bs)
    pool.scale["k"] = np.ldexp(pool.scale["k"], -q_exp).astype(np.float32)
    for row in pool.bt:
        blk = int(row[1])
        pool.scale["k"][blk] = 2.0 ** 125
        pool.codes["k"][blk] = rng.choice(np.asarray([0, 0x80], np.uint8), pool.codes["k"][blk].shape)
    q = F.bf16(rng, 2, 8, d, mag=2.0 ** q_exp)
    q[:, ::3] = F.bf16(rng, 2, 3, d)             # heads of ordinary size in the same unit
    _check(_decode(pkv, cuda, q, pool, 0.125), q, pool, 0.125)


# the V scales' exponents by block
SPREADS = [(-64, 110), (110, -64), (-96, 112), (-75, 75), (100, -40), (0, 13), (13, 0), (-7, -20)]


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 128), (256, 64), (24, 64)])
# one unit of several stages, units of one stage, units of 2048 keys
@pytest.mark.parametrize("lens,most", [([500, 90], 500), ([3000, 1300], 3000),
                                       ([5000, 1300], 1 << 20)])
@pytest.mark.parametrize("halves", [False, True])    # small and large blocks in two halves, in turn
def test_value_scales_far_apart(cuda, bs, d, lens, most, halves):
    """Blocks whose V scales differ by up to 2^208: the small ones' keys carry their weight
    in the normaliser, whether they come before the large ones or behind them."""
    pkv = U.lib()
    rng = np.random.default_rng(bs)
    for lo, hi in SPREADS:
        pool = F.Pool(lens, bs, 1, d, seed=bs, spread=0)
        exps = np.full(pool.scale["v"].shape[0], hi)
        for row, n in zip(pool.bt, lens):
            used = row[:-(-n // bs)]
            exps[used[:len(used) // 2] if halves else used[::2]] = lo
        pool.scale["v"] = np.ldexp(np.ones_like(pool.scale["v"]), exps[:, None]).astype(np.float32)
        q = F.bf16(rng, len(lens), 8, d)
        _check(_decode(pkv, cuda, q, pool, 0.125, most), q, pool, 0.125)


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 128), (24, 64)])
@pytest.mark.parametrize("apart", [0, 6, 13])
@pytest.mark.parametrize("n,most", [(500, 500), (5000, 1 << 20)])
def test_small_values_beside_large_ones(cuda, bs, d, apart, n, most):
    """Every second block's V scale is 2^apart larger, but its codes are zero in half of the
    entries, where the output is made of the small blocks' values alone.  Entry by entry, with
    s_j = w_j vs_j the share of a key (its weight times its V scale) and C its codes:
    each share is kept to r of itself (2^-9 + 2^-11) or 2^-22 of the largest, and the
    log weights to d as in fp8_util, so
      |out - ref| <= 2^-8 |ref| + sum_j |C_j| (s_j (r + 2 d) + 2^-22 max s)."""
    pkv = U.lib()
    rng = np.random.default_rng(bs + apart)
    pool = F.Pool([n], bs, 1, d, seed=bs, spread=0)
    large = pool.bt[0, ::2]
    pool.scale["v"][large] *= np.float32(2.0 ** apart)
    zeros = pool.codes["v"][large][..., :d // 2]
    pool.codes["v"][np.ix_(large, range(bs), [0], range(d // 2))] = np.where(zeros == 0x7F, 0x7F, 0)
    q = F.bf16(rng, 1, 4, d)
    scale = 0.125
    got = _decode(pkv, cuda, q, pool, scale, most)
    rows = lambda x: x[pool.bt[0, np.arange(n) // bs], np.arange(n) % bs, 0]  # noqa: E731
    K, V = rows(pool.values("k")), rows(pool.values("v"))
    vs = pool.scale["v"].astype(np.float64)[pool.bt[0, np.arange(n) // bs], 0]
    C = np.abs(V) / vs[:, None]
    for h in range(4):
        qh = U.f64(q)[0, h]
        x = scale * (K @ qh)
        w = np.exp(x - x.max())
        s = w / w.sum() * vs
        ref = (w / w.sum()) @ V
        big_x = scale * (np.abs(K) @ np.abs(qh)).max()
        worst_q = scale * np.abs(qh).max() * np.abs(K).sum(1).max()
        dx = (128 * 2.0 ** -23 + 2.0 ** -21) * big_x + 2.0 ** -21 * worst_q + 2.0 ** -20
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -9 + 2.0 ** -11 + 2 * dx) * (s @ C) + \
            2.0 ** -22 * s.max() * C.sum(0)
        err = np.abs(got[0, h] - ref)
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 64)])
@pytest.mark.parametrize("scale", [-0.125, 0.0, -1e-20])
def test_softmax_scales_of_either_sign(cuda, bs, d, scale):
    pkv = U.lib()
    rng = np.random.default_rng(bs)
    pool = F.Pool([700, 33], bs, 2, d, seed=bs)
    q = F.bf16(rng, 2, 8, d)
    _check(_decode(pkv, cuda, q, pool, scale), q, pool, scale)
