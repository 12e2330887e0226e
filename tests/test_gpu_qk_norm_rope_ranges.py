"""qk_norm_rope of rows whose squares 32 bits do not hold, within the bound of
test_gpu_qk_norm_rope.py (a power of two before the sum rounds nothing)."""
import numpy as np
import pytest
import torch

from gpu_util import lib, status_word
from oracle import head_rotation as ohr
from test_gpu_qk_norm_rope import BF, FP, HF, check

pytestmark = pytest.mark.gpu

SIZES = [2.0 ** -146, 2.0 ** -120, 2.0 ** -76, 2.0 ** -63, 2.0 ** -51, 2.0 ** -49, 2.0 ** -20, 1.0,
         2.0 ** 40, 2.0 ** 58, 2.0 ** 60, 2.0 ** 62, 2.0 ** 64, 2.0 ** 90, 2.0 ** 122]


def _rows(rng, n, heads, d, dtype, dev):
    """Heads of every size beside one another; some of zeros."""
    size = rng.choice(SIZES if dtype != HF else [2.0 ** -20, 2.0 ** -10, 1.0, 2.0 ** 11],
                      (n, heads, 1))
    if dtype == BF:
        size = np.maximum(size, 2.0 ** -120)
    x = torch.from_numpy(rng.normal(size=(n, heads, d)).clip(-4, 4) * size).to(dtype)
    return x.to(dev)


@pytest.mark.parametrize("n", [3, 300, 2300])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (80, 20, False), (72, 40, False),
                                         (64, 32, True), (256, 250, False), (96, 0, False)])
@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_rows_of_any_size(cuda, n, d, rot, inter, dtype):
    pkv = lib()
    rng = np.random.default_rng(n + d)
    q, k = _rows(rng, n, 5, d, dtype, cuda), _rows(rng, n, 2, d, dtype, cuda)
    qw, kw = (torch.from_numpy(1 + 0.5 * rng.normal(size=d)).to(FP).to(cuda) for _ in range(2))
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    freq, mag = ohr.frequencies(rot, 1e4) if rot else ([], 1.0)
    rope = pkv.rotary(rot, frequencies=freq, interleaved=inter) if rot else None
    dpos = torch.from_numpy(pos).to(cuda)
    for eps in (0.0, 1e-38, 1e-20, 1e-6, 3.0):
        qo, ko = pkv.qk_norm_rope(q, k, qw, kw, eps, dpos, rope)
        for at in (slice(0, 40), slice(max(n - 40, 0), n)):
            check(qo[at], q[at], qw, eps, pos[at], freq, inter, mag, ("q", eps))
            check(ko[at], k[at], kw, eps, pos[at], freq, inter, mag, ("k", eps))
        few = slice(n // 2, n // 2 + 3)              # the same bits in any batch
        qf, kf = pkv.qk_norm_rope(q[few], k[few], qw, kw, eps, dpos[few], rope)
        assert torch.equal(qo[few], qf) and torch.equal(ko[few], kf)


@pytest.mark.parametrize("n", [7, 2100])
def test_into_the_cache(cuda, n):
    pkv = lib()
    rng = np.random.default_rng(n)
    q, k, v = (_rows(rng, n, h, 128, BF, cuda) for h in (4, 2, 2))
    w = torch.from_numpy(1 + 0.5 * rng.normal(size=128)).to(BF).to(cuda)
    pos = torch.from_numpy(rng.integers(0, 9999, n).astype(np.int32)).to(cuda)
    rope = pkv.rotary(128)
    kc = torch.zeros(n // 16 + 1, 16, 2, 128, dtype=BF, device=cuda)
    vc, st = kc.clone(), pkv.new_status(cuda)
    slots = torch.from_numpy(rng.permutation(n).astype(np.int32)).to(cuda)
    ref = pkv.qk_norm_rope(q, k, w, w, 0.0, pos, rope)
    got = pkv.qk_norm_rope_kv_store(q, k, v, w, w, 0.0, pos, rope, kc, vc, slots, status=st)
    assert status_word(st) == 0 and torch.equal(got, ref[0])
    assert torch.equal(kc.view(-1, 2, 128)[slots.long()], ref[1])
    assert torch.equal(vc.view(-1, 2, 128)[slots.long()], v)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("n", [3, 2100])
def test_zeros_infinite_and_nan_entries(cuda, n, dtype):
    """As the formula has them: zeros over eps are zeros, an infinite entry is NaN beside zeros, a
    NaN makes its head NaN."""
    pkv = lib()
    q = torch.zeros(n, 3, 64, dtype=dtype, device=cuda)
    q[:, 1] = 2.0 ** 100
    q[1, 1, 5] = float("inf")
    q[2, 1, 6] = float("nan")
    k = torch.full((n, 1, 64), 2.0 ** -60, dtype=dtype, device=cuda)
    w = torch.ones(64, device=cuda)
    pos = torch.zeros(n, dtype=torch.int32, device=cuda)
    qo, ko = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, None)
    assert (qo[:, [0, 2]] == 0).all() and (qo[0, 1] == 1).all()
    rest = [i for i in range(64) if i != 5]
    assert qo[1, 1, 5].isnan() and (qo[1, 1, rest] == 0).all() and qo[2, 1].isnan().all()
    qo, ko = pkv.qk_norm_rope(q, k, w, w, 0.0, pos, None)
    assert qo[:, [0, 2]].isnan().all() and (ko == 1).all() and (qo[0, 1] == 1).all()
