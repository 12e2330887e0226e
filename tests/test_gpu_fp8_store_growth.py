"""Blocks of the 8-bit cache whose scale grows so far that the ratio of the two
scales is small, subnormal or zero in fp32: the block's other rows are re-scaled all
the same, bit for bit as the oracle does (codes to signed zeros in the end)."""
import numpy as np
import pytest
import torch

import fp8_util as F
import gpu_util as U
from oracle import fp8_cache as ofp

pytestmark = pytest.mark.gpu

# (exponent of the scale before, magnitude of the new row): the scale becomes the least
# 2^e with magnitude <= 448 * 2^e, clamped to 2^119
GROWTHS = [(-64, 1e30), (-64, 3e38), (-96, 1e20), (-96, 3e38), (-64, 2.0 ** 93), (-64, 2.0 ** 70),
           (-20, 1e30), (-64, 1.0), (-7, 1.0)]


@pytest.mark.parametrize("n", [len(GROWTHS), 2100])     # both forms of the store
@pytest.mark.parametrize("bs,hkv,d", [(16, 2, 128), (24, 3, 64)])
def test_other_rows_follow_any_growth(cuda, n, bs, hkv, d):
    pkv = U.lib()
    rng = np.random.default_rng(n + bs)
    nb = n + 1
    codes = {c: rng.integers(0, 256, (nb, bs, hkv, d)).astype(np.uint8) for c in "kv"}
    scale = {c: np.empty((nb, hkv), np.float32) for c in "kv"}
    rows = {c: np.zeros((n, hkv, d)) for c in "kv"}
    for b in range(n):
        for c in "kv":
            for h in range(hkv):
                e, mag = GROWTHS[(b + h + (c == "v")) % len(GROWTHS)]
                scale[c][b, h] = 2.0 ** e
                rows[c][b, h] = rng.uniform(-1, 1, d) * mag
                rows[c][b, h, 0] = mag
    for c in "kv":
        scale[c][n] = 1.0
    # one new row in each block, never the first
    slots = np.asarray([b * bs + 1 + b % (bs - 1) for b in range(n)], np.int32)
    k, v = (torch.from_numpy(rows[c].astype(np.float32)).to(torch.bfloat16) for c in "kv")
    f8 = lambda c: torch.from_numpy(c.copy()).to(cuda).view(torch.float8_e4m3fn)  # noqa: E731
    kc, vc = f8(codes["k"]), f8(codes["v"])
    ks, vs = (torch.from_numpy(scale[c].copy()).to(cuda) for c in "kv")
    st = pkv.new_status(cuda)
    pkv.kv_store_fp8(k.to(cuda), v.to(cuda), kc, vc, ks, vs, torch.from_numpy(slots).to(cuda),
                     status=st)
    assert U.status_word(st) == 0
    ref = ofp.kv_store(U.f64(k), U.f64(v), codes["k"], codes["v"], scale["k"], scale["v"], slots)
    for got, want in ((ks, ref[2]), (vs, ref[3])):
        np.testing.assert_array_equal(U.f64(got), want)
    for got, want in ((kc, ref[0]), (vc, ref[1])):
        got = got.view(torch.uint8).cpu().numpy()
        # a NaN code that was re-scaled may come back with either sign
        assert ((got == want) | ((got & 127 == 127) & (want & 127 == 127))).all()


def test_a_tiny_row_stays_tiny(cuda):
    """What a later read of the cache sees: a row near 2^-60 stored first and one of 1e30
    behind it; the first row's value is next to nothing, not 1e28."""
    pkv = U.lib()
    bs, hkv, d = 16, 1, 64
    kc = torch.zeros((1, bs, hkv, d), dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
    vc = kc.clone()
    ks, vs = torch.zeros((1, hkv), device=cuda), torch.zeros((1, hkv), device=cuda)
    for slot, value in ((0, 2.0 ** -60), (1, 1e30)):
        x = torch.full((1, hkv, d), value, dtype=torch.bfloat16, device=cuda)
        pkv.kv_store_fp8(x, x, kc, vc, ks, vs, torch.tensor([slot], dtype=torch.int32, device=cuda))
    held = ofp.decode_values(kc.view(torch.uint8).cpu().numpy(), U.f64(ks))
    assert (held[0, 0] == 0).all()
    # one code step of a row whose largest entry is 1e30: 1e30 / 448 * 2^-9 at least
    assert np.abs(held[0, 1] - 1e30).max() <= 1e30 * (2.0 ** -4 + 2.0 ** -8)
