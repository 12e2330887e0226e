"""Pins of the CPU oracle's e4m3 cache and logit rules (no GPU)."""
import math

import numpy as np
import torch

from oracle import fp8_cache as ofp
from oracle import logit_rules as olr


def _torch_codes(y):
    return torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def test_code_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(codes, ofp.VALUES)


def test_encode_rounds_as_torch_does():
    mags = ofp.VALUES[:127]
    mids = (mags[1:] + mags[:-1]) / 2                    # ties
    near = np.concatenate([np.nextafter(mids.astype(np.float32), np.float32(np.inf)),
                           np.nextafter(mids.astype(np.float32), np.float32(-np.inf))])
    rng = np.random.default_rng(0)
    rnd = rng.normal(size=20000) * 2.0 ** rng.integers(-12, 8, 20000)
    y = np.concatenate([mags, mids, near, np.clip(rnd, -448, 448)]).astype(np.float32)
    y = np.concatenate([y, -y])
    np.testing.assert_array_equal(ofp.encode(y), _torch_codes(y))


def test_encode_saturates_and_keeps_nan():
    got = ofp.encode([449.0, 1e9, math.inf, -math.inf, -500.0, math.nan])
    assert got.tolist() == [126, 126, 126, 254, 254, 127]


def test_scales_are_the_least_power_of_two():
    for amax in (1e-30, 0.3, 1.0, 3.5, 3.5 + 1e-6, 447.9, 448.0, 448.1, 1e30):
        c = ofp.scale_for(amax)
        assert amax <= 448 * c and (amax > 448 * c / 2 or c == 2.0 ** -64)
    assert ofp.scale_for(0.0) == 2.0 ** -64
    assert ofp.scale_for(float(np.finfo(np.float32).max)) == 2.0 ** 119


def _empty(nb, bs, h, d):
    return np.zeros((nb, bs, h, d), np.uint8), np.zeros((nb, h))


def test_store_row_by_row_is_store_at_once():
    """Powers of two: growing a block's scale keeps its codes' significant bits,
    so the two agree except among the subnormals of the final scale."""
    rng = np.random.default_rng(1)
    n, bs, h, d = 14, 4, 2, 8
    x = rng.normal(size=(n, h, d)) * 2.0 ** rng.integers(-3, 4, (n, 1, 1))
    x = x.astype(np.float32).astype(np.float64)
    slots = np.concatenate([np.arange(8, 12), np.arange(0, 4), np.arange(16, 20), [4, 5]])
    kc, ks = _empty(6, bs, h, d)
    once = ofp.kv_store(x, x, kc, kc, ks, ks, slots)
    c, s = kc, ks
    for t in range(n):
        c, _, s, _, _, _ = ofp.kv_store(x[t:t + 1], x[t:t + 1], c, c, s, s, slots[t:t + 1])
    np.testing.assert_array_equal(s, once[2])
    a, b = ofp.decode_values(c, s), ofp.decode_values(once[0], once[2])
    step = (s * 2.0 ** -9)[:, None, :, None]            # the subnormals' step
    assert (np.abs(a - b) <= np.where(np.abs(b) < 2.0 ** -6 * s[:, None, :, None], step, 0)).all()
    # a stored entry is within half a step of the row's
    for t, slot in enumerate(slots):
        err = np.abs(b[slot // bs, slot % bs] - x[t])
        half = np.maximum(np.abs(x[t]) * 2.0 ** -4, s[slot // bs][:, None] * 2.0 ** -10)
        assert (err <= half).all()


def test_store_rules_of_a_block():
    h, d = 1, 4
    kc, ks = _empty(2, 4, h, d)
    one = lambda v: np.full((1, h, d), float(v))        # noqa: E731
    c, _, s, _, _, _ = ofp.kv_store(one(1.0), one(1.0), kc, kc, ks, ks, [0])
    assert s[0, 0] == 2.0 ** -8 and ofp.decode_values(c, s)[0, 0, 0, 0] == 1.0
    # the next row is larger: the block grows, the first row keeps its value
    c, _, s, _, _, _ = ofp.kv_store(one(7.0), one(7.0), c, c, s, s, [1])
    assert s[0, 0] == 2.0 ** -6
    assert ofp.decode_values(c, s)[0, :2, 0, 0].tolist() == [1.0, 7.0]
    # a smaller row leaves the scale
    c, _, s, _, _, _ = ofp.kv_store(one(0.5), one(0.5), c, c, s, s, [2])
    assert s[0, 0] == 2.0 ** -6
    # offset 0 begins the block anew: the other rows keep their codes
    before = c.copy()
    c, _, s, _, _, _ = ofp.kv_store(one(0.25), one(0.25), c, c, s, s, [0])
    assert s[0, 0] == 2.0 ** -10 and (c[0, 1:] == before[0, 1:]).all()
    # the last token of a slot is stored; -1 skipped; a slot past the pool listed
    x = np.stack([np.full((h, d), v) for v in (1.0, 2.0, 3.0, 4.0)])
    c, _, s, _, bad, _ = ofp.kv_store(x, x, c, c, s, s, [4, -1, 4, 8])
    assert bad == [8] and ofp.decode_values(c, s)[1, 0, 0, 0] == 3.0


def test_logit_rules_by_hand():
    x = np.array([[2.0, -2.0, 0.0, 1.0, 5.0]])
    ids = np.array([[0, 1, 1, 3, 3, 4]])
    out, spread = olr.apply(x, ids, np.array([2]), np.array([5]), np.array([2.0]),
                            np.array([0.25]), np.array([0.5]), np.array([0, 3]),
                            np.array([2, 4, 2]), np.array([9.0, 1.0, -3.0]),
                            np.array([[0b10111]]))
    # 0: prompt only, 2/2; 1: prompt and once generated, -2*2 - .5 - .25;
    # 2: unseen, its last bias; 3: twice generated but not allowed; 4: behind the
    # row's tokens, bias 1
    assert out.tolist() == [[1.0, -4.75, -3.0, -math.inf, 6.0]]
    assert spread[0, 1] == 4.75
