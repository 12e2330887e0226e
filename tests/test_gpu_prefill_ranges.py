"""paged_prefill_varlen and its form over the 8-bit cache: scores far from one.

A key's score is q0 K0 scale with K0 exact in 32 bits; one key, which every row sees, is ahead of the
others by 2^-8 of its score and more, thousands here, so that a row is that key's value.  Its
weight and the result are rounded to bf16: twice 2^-8."""
import numpy as np
import pytest
import torch

import fp8_util as F
import gpu_util as U
from test_gpu_prefill import _prefill, make_case

pytestmark = pytest.mark.gpu

TOPS = (2.0 ** 20, 2.0 ** 24 + 2, 1.3 * 2.0 ** 26, 1.9 * 2.0 ** 28, 1.1 * 2.0 ** 30, 1.7 * 2.0 ** 31,
        1.3 * 2.0 ** 32, 1.9 * 2.0 ** 33, 1.2 * 2.0 ** 40, 1.6 * 2.0 ** 63, 1.4 * 2.0 ** 100)


@pytest.mark.parametrize("d,bs", [(128, 256), (64, 16), (128, 48), (64, 64)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(cuda, d, bs, sign):
    pkv = U.lib()
    lens, cached = [200, 1, 129, 64, 300], [0, 48, 100, 300, 2 * bs]
    c = make_case(d + bs, lens, cached, 4, 2, d, bs)
    rng = np.random.default_rng(bs)
    k0 = lambda *shape: torch.from_numpy(  # noqa: E731
        rng.integers(0, 127, shape) / 128 + 1).to(torch.bfloat16)
    lead = 1 + 127 / 128 if sign > 0 else 1 - 2.0 ** -7
    c["k"][:], c["q"][:] = 0, 0
    c["k"][:, :, 0] = k0(c["k"].shape[0], 1)
    c["q"][:, :, 0] = sign
    kept = torch.isfinite(c["kc"])
    c["kc"][kept] = 0
    first = k0(*c["kc"].shape[:2], 1)
    c["kc"][..., 0] = torch.where(kept[..., 0], first, c["kc"][..., 0])
    want = []
    for b, n in enumerate(lens):
        if cached[b]:
            at = (int(c["bt"][b, 0]), 0)
            c["kc"][at][:, 0] = lead
            v = c["vc"][at]
        else:
            at = int(c["cu_q"][b])
            c["k"][at, :, 0] = lead
            v = c["v"][at]
        want += [U.f64(v)[[0, 0, 1, 1]]] * n
    want = np.stack(want)
    for top in TOPS:
        st = pkv.new_status(cuda)
        got = U.f64(_prefill(pkv, cuda, c["q"], c["k"], c["v"], c["kc"], c["vc"], c["cu_q"],
                             c["cu_k"], c["bt"], top * 0.7, c["max_sq"], c["max_sk"], status=st))
        assert U.status_word(st) == 0
        assert np.isfinite(got).all(), top
        assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -7 + 2.0 ** -14)).all(), top


@pytest.mark.parametrize("bs,d", [(16, 128), (64, 64)])
@pytest.mark.parametrize("place", [0, 2500, 5499])
def test_scores_of_any_size_in_splits(cuda, bs, d, place):
    """Few queries over many cached keys: splits' maxima, near and far, merged."""
    pkv = U.lib()
    lq, lp, hkv, group = [20, 130], [5500, 900], 1, 2
    pool = F.Pool(lp, bs, hkv, d, seed=4)
    rng = np.random.default_rng(place)
    codes = pool.codes["k"]
    codes[:, :, 0, 0] = np.where(codes[:, :, 0, 0] == 0x7F, 0x7F, 0x76)        # 224
    at = []
    for b, j in enumerate((place, place % 900)):
        at.append((pool.bt[b, j // bs], j % bs))
        codes[at[b]][0, 0] = 0x7E                                               # 448
    pool.scale["k"][:], pool.scale["v"][:] = 1.0, 2.0 ** -7
    q, k = (torch.zeros((150, h, d), dtype=torch.bfloat16) for h in (hkv * group, hkv))
    q[:, :, 0] = 1
    k[:, :, 0] = torch.from_numpy(rng.integers(-127, 127, (150, 1)).astype(np.float32)).bfloat16()
    v = F.bf16(rng, 150, hkv, d)
    cu = lambda x: torch.from_numpy(np.concatenate([[0], np.cumsum(x)]).astype(np.int32)).to(  # noqa: E731,E501
        cuda)
    *cache, bt = pool.on(cuda)
    want = np.concatenate([np.broadcast_to(pool.values("v")[at[b]][0], (lq[b], group, d))
                           for b in range(2)])
    for top in TOPS:
        st = pkv.new_status(cuda)
        got = U.f64(pkv.paged_prefill_varlen_fp8(q.to(cuda), k.to(cuda), v.to(cuda), *cache, cu(lq),
                                                 cu(np.add(lq, lp)), max(lq),
                                                 max(a + b for a, b in zip(lq, lp)), bt,
                                                 top / 448 * 0.7, status=st))
        assert U.status_word(st) == 0
        assert np.isfinite(got).all(), top
        assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -7 + 2.0 ** -14)).all(), top
