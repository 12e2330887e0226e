"""Prefill over the 8-bit cache with a tile's keys in splits: its bounded waits run out."""
import numpy as np
import pytest
import torch

import fp8_util as F
import gpu_util as U
from test_gpu_fp8_cache import _prefill

pytestmark = pytest.mark.gpu

CASES = [([20, 160], [5500, 900], 16, 1, 2, 128), ([1, 300], [4200, 6000], 64, 1, 2, 64)]


def _splits(lq, max_k, heads):
    """At least 32 key tiles of 128, and fewer than 304 items of (128-query tile, head): the
    sizes at which a call's keys are split over work items."""
    return max_k // 128 + 2 >= 32 and (sum(lq) // 128 + len(lq)) * heads < 304


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("polls", [0, 1, 2, 3, 5])
def test_gives_up_then_recovers(cuda, case, polls):
    """At a limit of 0 the time-out is reported; at a few polls it or nothing is, and where
    nothing is the rows are those of the default limit."""
    pkv = U.lib()
    lq, lp, bs, hkv, group, d = case
    max_k = max(a + b for a, b in zip(lq, lp))
    assert _splits(lq, max_k, hkv * group)
    rng = np.random.default_rng(4)
    pool = F.Pool(lp, bs, hkv, d, seed=4)
    q, k, v = (F.bf16(rng, sum(lq), h, d).to(cuda) for h in (hkv * group, hkv, hkv))
    cu = lambda x: torch.from_numpy(np.concatenate([[0], np.cumsum(x)]).astype(np.int32)).to(  # noqa: E731,E501
        cuda)
    *cache, bt = pool.on(cuda)
    cu_q, cu_k = cu(lq), cu(np.add(lq, lp))

    def call():
        st = pkv.new_status(cuda)
        out = pkv.paged_prefill_varlen_fp8(q, k, v, *cache, cu_q, cu_k, max(lq), max_k, bt, 0.1,
                                           status=st)
        return out, U.status_word(st)            # synchronises: the kernels returned
    want, word = call()
    assert word == 0
    pkv.set_wait_poll_limit(polls)
    try:
        out, word = call()
    finally:
        pkv.set_wait_poll_limit()
    assert word in (0, pkv.STATUS["WAIT_TIMEOUT"])
    if polls == 0:
        assert word == pkv.STATUS["WAIT_TIMEOUT"]
    if word == 0:
        assert torch.equal(out, want)
    out, word = call()
    assert word == 0 and torch.equal(out, want)
    _prefill(pkv, cuda, *case, seed=4)
