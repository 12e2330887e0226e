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
