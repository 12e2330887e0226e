"""qk_norm_rope and qk_norm_rope_kv_store against the float64 oracle.

Bound, from the kernel's roundings.  An entry is r * (A x + B x'), with A = w m cos,
B = +-w' m sin in fp32.  In units of 2^-24 relative: the residual angle 1 (of at most
pi / 4, so at most 1 of the cosine or sine), sincospi 4, magnitude and weight 1 each;
the product and the sum 2; r: the sum of at most 256 squares in 8 + 5 steps and a product
each 14, halved by the root, plus the mean's division and eps 2, halved, plus rsqrt 4; the
last product 1.  Together less than 22, taken as 24, of |r A x| + |r B x'|; then the
rounding to the rows' type, eps / 2 of the result or half its smallest step."""
import numpy as np
import pytest
import torch

from gpu_util import bits, f64, lib, status_word
from oracle import head_rotation as ohr

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def check(got, x, weight, eps, pos, freq, interleaved, magnitude, what):
    ref = ohr.norm_rope(f64(x), None if weight is None else f64(weight), eps, pos, freq,
                        interleaved, magnitude)
    # |r A x| + |r B x'| is at most the sum of the pair's normed sizes times the magnitude
    y = np.abs(ohr.norm_rope(f64(x), None if weight is None else f64(weight), eps, pos, []))
    r = 2 * len(freq)
    if r:
        i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                     slice(r // 2, r))
        both = (y[..., i] + y[..., j]) * abs(magnitude)
        y[..., i], y[..., j] = both, both
    info = torch.finfo(x.dtype)
    step = info.smallest_normal * info.eps
    bound = np.abs(ref) * info.eps / 2 + 24 * 2.0 ** -24 * y * (1 + info.eps) + step / 2
    assert got.shape == x.shape and got.dtype == x.dtype
    err = np.abs(f64(got) - ref)
    assert (err <= bound).all(), (what, float((err / bound).max()))


def rows(rng, n, heads, d, dtype, dev, packed, mag=1.0):
    x = torch.from_numpy(rng.normal(size=(n, sum(heads), d)) * mag).to(dtype).to(dev)
    parts = x.split(heads, dim=1)
    return parts if packed else tuple(p.contiguous() for p in parts)


CASES = [  # tokens, hq, hkv, d, rotary_dim, interleaved, dtype, weights' dtype, packed
    (1, 16, 8, 128, 128, False, BF, BF, True),
    (1, 1, 1, 8, 8, True, FP, FP, False),
    (3, 1, 1, 64, 64, False, HF, FP, True),
    (33, 7, 1, 128, 64, True, BF, FP, True),
    (5, 32, 8, 128, 32, False, HF, HF, True),
    (17, 3, 3, 80, 20, False, BF, BF, True),          # partners through memory
    (9, 5, 1, 80, 80, False, FP, BF, False),
    (2, 40, 40, 96, 96, True, BF, BF, True),
    (65, 4, 2, 192, 48, False, FP, FP, True),
    (4, 9, 3, 256, 256, False, BF, BF, True),
    (6, 2, 1, 256, 2, False, HF, HF, False),
    (7, 2, 1, 24, 10, True, BF, HF, True),
    (11, 64, 8, 128, 128, False, BF, BF, True),       # several passes over the heads
    (300, 6, 2, 64, 0, False, BF, BF, True),          # no rotation
    (300, 6, 2, 72, 40, False, FP, None, True),       # no norm
]


@pytest.mark.parametrize("case", CASES)
def test_against_oracle(cuda, case):
    pkv = lib()
    n, hq, hkv, d, rot, inter, dtype, wtype, packed = case
    rng = np.random.default_rng(n * 1000 + d)
    q, k = rows(rng, n, (hq, hkv), d, dtype, cuda, packed, 3.0)
    qw = kw = None
    if wtype is not None:
        qw, kw = (torch.from_numpy(1 + 0.5 * rng.normal(size=d)).to(wtype).to(cuda)
                  for _ in range(2))
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    freq, mag = ohr.frequencies(rot, 1e4, "yarn", 4, 4096) if rot > 2 else ([0.3] * (rot // 2),
                                                                            1.25)
    rope = pkv.rotary(rot, frequencies=freq, magnitude=mag, interleaved=inter) if rot else None
    qo, ko = pkv.qk_norm_rope(q, k, qw, kw, 1e-5, torch.from_numpy(pos).to(cuda), rope)
    assert qo.is_contiguous() and ko.is_contiguous()
    check(qo, q, qw, 1e-5, pos, freq, inter, mag, "q")
    check(ko, k, kw, 1e-5, pos, freq, inter, mag, "k")


def test_positions_of_the_whole_int32_range(cuda):
    pkv = lib()
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 2**31 - 1, -2**31, 2**31 - 2, 1 << 24, (1 << 24) + 1, 123456789],
                   np.int32)
    freq = [1.0, 0.9999999, 3.14159, 1e-9, 1e-5, 0.017, 1000.0, 65536.0]
    q, k = rows(rng, len(pos), (2, 1), 16, FP, cuda, False)
    rope = pkv.rotary(16, frequencies=freq)
    qo, ko = pkv.qk_norm_rope(q, k, None, None, 0.0, torch.from_numpy(pos).to(cuda), rope)
    check(qo, q, None, 0, pos, freq, False, 1.0, "q")
    check(ko, k, None, 0, pos, freq, False, 1.0, "k")


def test_one_norm_zero_rows_and_odd_values(cuda):
    pkv = lib()
    q = torch.zeros(2, 2, 64, device=cuda)
    q[0, 1, 3] = float("inf")
    q[1, 0, 5] = float("nan")
    q[1, 1] = 1e-3
    k = torch.ones(2, 1, 64, device=cuda) * 2
    w = torch.ones(64, device=cuda)
    rope = pkv.rotary(16)
    pos = torch.zeros(2, dtype=torch.int32, device=cuda)
    qo, ko = pkv.qk_norm_rope(q, k, w, None, 1e-6, pos, rope)
    assert torch.equal(ko, k)                          # no norm, position 0
    assert torch.equal(qo[0, 0], q[0, 0])              # zeros stay zeros
    assert qo[1, 0].isnan().all() and qo[0, 1, 3].isnan()
    assert torch.allclose(qo[1, 1], torch.full_like(qo[1, 1], 2 ** -0.5), rtol=1e-5)
    # without a norm, an infinite entry behind the rotated ones passes through alone
    q[1, 0, 5] = 0
    q[0, 1, 3], q[0, 1, 17] = 0, float("inf")
    for inter in (False, True):
        got, _ = pkv.qk_norm_rope(q, k, None, None, 0.0, pos, pkv.rotary(16, interleaved=inter))
        assert torch.equal(got, q)
        got, _ = pkv.qk_norm_rope(q, k, None, None, 0.0, pos, pkv.rotary(10, interleaved=inter))
        assert torch.equal(got, q)


@pytest.mark.parametrize("rot,inter", [(128, False), (20, False), (64, True)])
def test_in_place_packed_rows(cuda, rot, inter):
    """In place within packed rows: the columns between stay as they were."""
    pkv = lib()
    rng = np.random.default_rng(7)
    x = torch.from_numpy(rng.normal(size=(50, 9, 128))).to(BF).to(cuda)
    before = x.clone()
    q, k = x[:, 1:5], x[:, 6:8]
    w = torch.from_numpy(1 + 0.1 * rng.normal(size=128)).to(BF).to(cuda)
    pos = torch.arange(50, dtype=torch.int32, device=cuda)
    rope = pkv.rotary(rot, interleaved=inter)
    ref = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope)
    got = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope, q_out=q, k_out=k)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for at in (0, 5, 8):
        assert torch.equal(x[:, at], before[:, at])


def test_rows_beyond_32_bit_offsets(cuda):
    pkv = lib()
    stride = (1 << 31) + 8                              # elements between two tokens
    big = torch.empty(stride + 3 * 64, dtype=BF, device=cuda)
    view = big.as_strided((2, 3, 64), (stride, 64, 1))
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(size=(2, 3, 64))).to(BF).to(cuda)
    view.copy_(x)
    pos = torch.tensor([5, 9], dtype=torch.int32, device=cuda)
    rope = pkv.rotary(64)
    ref = pkv.qk_norm_rope(x[:, :2].contiguous(), x[:, 2:].contiguous(), None, None, 0, pos, rope)
    got = pkv.qk_norm_rope(view[:, :2], view[:, 2:], None, None, 0, pos, rope)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


STORES = [  # tokens, hq, hkv, d, rotary_dim, interleaved, block size, norm
    (1, 16, 8, 128, 128, False, 256, True), (40, 4, 1, 64, 64, False, 1, True),
    (77, 6, 2, 128, 64, True, 20, True), (130, 8, 8, 80, 20, False, 16, False),
    (600, 64, 8, 128, 128, False, 64, True)]


@pytest.mark.parametrize("case", STORES)
def test_store(cuda, case):
    pkv = lib()
    n, hq, hkv, d, rot, inter, bs, norm = case
    rng = np.random.default_rng(n)
    q, k, v = rows(rng, n, (hq, hkv, hkv), d, BF, cuda, True)
    w = torch.from_numpy(1 + 0.5 * rng.normal(size=d)).to(BF).to(cuda) if norm else None
    nb = -(-n // bs) + 3
    kc0 = torch.from_numpy(rng.normal(size=(nb, bs, hkv, d))).to(BF).to(cuda)
    vc0 = -kc0
    kc, vc = kc0.clone(), vc0.clone()
    slots = rng.permutation(nb * bs)[:n].astype(np.int32)
    slots[::7] = -1 - slots[::7]                       # padding
    pos = torch.from_numpy(rng.integers(0, 100000, n).astype(np.int32)).to(cuda)
    rope = pkv.rotary(rot, interleaved=inter, base=1e6)
    qr, kr = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope)
    ko = torch.empty_like(kr)
    st = pkv.new_status(cuda)
    got = pkv.qk_norm_rope_kv_store(q, k, v, w, w, 1e-6, pos, rope, kc, vc,
                                    torch.from_numpy(slots).to(cuda), k_out=ko, status=st)
    assert status_word(st) == 0
    assert torch.equal(got, qr) and torch.equal(ko, kr)
    real = torch.from_numpy(np.flatnonzero(slots >= 0)).to(cuda)
    to = torch.from_numpy(slots[slots >= 0].astype(np.int64)).to(cuda)
    kc0.view(-1, hkv, d)[to], vc0.view(-1, hkv, d)[to] = kr[real], v[real]
    assert np.array_equal(bits(kc), bits(kc0)) and np.array_equal(bits(vc), bits(vc0))


def test_store_reports_slots_outside_and_keeps_one_of_equal_slots(cuda):
    pkv = lib()
    rng = np.random.default_rng(3)
    q, k, v = rows(rng, 6, (2, 1, 1), 64, BF, cuda, True)
    kc = torch.zeros(2, 4, 1, 64, dtype=BF, device=cuda)
    vc = kc.clone()
    slots = torch.tensor([8, 0, 2**31 - 1, 3, 3, -2**31], dtype=torch.int32, device=cuda)
    pos = torch.zeros(6, dtype=torch.int32, device=cuda)
    st = pkv.new_status(cuda)
    rope = pkv.rotary(64)
    qo = pkv.qk_norm_rope_kv_store(q, k, v, None, None, 0.0, pos, rope, kc, vc, slots, status=st)
    assert status_word(st) == pkv.STATUS["SLOT_OUT_OF_RANGE"]
    assert torch.equal(qo, q)                          # position 0
    flat_k, flat_v = kc.view(8, 64), vc.view(8, 64)
    assert torch.equal(flat_k[0], k[1, 0]) and torch.equal(flat_v[0], v[1, 0])
    assert any(torch.equal(flat_k[3], k[i, 0]) for i in (3, 4))
    assert any(torch.equal(flat_v[3], v[i, 0]) for i in (3, 4))
    rest = [1, 2, 4, 5, 6, 7]
    assert (flat_k[rest] == 0).all() and (flat_v[rest] == 0).all()


def test_empty_other_stream_and_graph(cuda):
    pkv = lib()
    rng = np.random.default_rng(4)
    q, k, v = rows(rng, 12, (4, 2, 2), 128, BF, cuda, True)
    w = torch.ones(128, dtype=BF, device=cuda)
    rope = pkv.rotary(128)
    pos = torch.arange(12, dtype=torch.int32, device=cuda)
    e, f = pkv.qk_norm_rope(q[:0], k[:0], w, w, 1e-6, pos[:0], rope)
    assert e.shape == (0, 4, 128) and f.shape == (0, 2, 128)
    ref = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    kc = torch.zeros(4, 16, 2, 128, dtype=BF, device=cuda)
    vc = kc.clone()
    slots = torch.arange(12, dtype=torch.int32, device=cuda)
    qo = torch.empty_like(ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.qk_norm_rope_kv_store(q, k, v, w, w, 1e-6, pos, rope, kc, vc, slots, q_out=qo)
    pos += 3                                            # what a replay reads
    slots += 20
    graph.replay()
    ref = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope)
    assert torch.equal(qo, ref[0])
    assert torch.equal(kc.view(64, 2, 128)[20:32], ref[1])
    assert torch.equal(vc.view(64, 2, 128)[20:32], v)
    assert (kc.view(64, 2, 128)[:20] == 0).all()


MANY = [  # as CASES, of so many tokens that warps work through runs of them
    (2048, 1, 1, 8, 8, True, FP, FP, False),
    (2100, 9, 2, 256, 256, False, FP, BF, True),
    (2049, 3, 3, 80, 20, False, BF, BF, True),
    (2300, 5, 1, 72, 40, False, FP, None, False),
    (2077, 4, 2, 24, 10, False, HF, HF, True),
    (5000, 2, 1, 136, 34, True, HF, FP, True),
    (2050, 33, 1, 128, 64, False, BF, BF, True),
    (20000, 1, 1, 64, 64, False, BF, BF, False),
    (2500, 6, 2, 64, 0, False, BF, BF, True),
]


@pytest.mark.parametrize("case", MANY)
def test_many_tokens(cuda, case):
    """Against the oracle at both ends, and all of it against calls of fewer tokens:
    a token's bits do not depend on the batch."""
    pkv = lib()
    n, hq, hkv, d, rot, inter, dtype, wtype, packed = case
    rng = np.random.default_rng(n * 1000 + d)
    q, k = rows(rng, n, (hq, hkv), d, dtype, cuda, packed, 3.0)
    qw = kw = None
    if wtype is not None:
        qw, kw = (torch.from_numpy(1 + 0.5 * rng.normal(size=d)).to(wtype).to(cuda)
                  for _ in range(2))
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    dpos = torch.from_numpy(pos).to(cuda)
    freq, mag = ohr.frequencies(rot, 1e4, "yarn", 4, 4096) if rot else ([], 1.0)
    rope = pkv.rotary(rot, frequencies=freq, magnitude=mag, interleaved=inter) if rot else None
    qo, ko = pkv.qk_norm_rope(q, k, qw, kw, 1e-5, dpos, rope)
    for at in (slice(0, 20), slice(n - 20, n)):
        check(qo[at], q[at], qw, 1e-5, pos[at], freq, inter, mag, "q")
        check(ko[at], k[at], kw, 1e-5, pos[at], freq, inter, mag, "k")
    for at in range(0, n, 2000):
        few = slice(at, min(at + 2000, n))
        qf, kf = pkv.qk_norm_rope(q[few], k[few], qw, kw, 1e-5, dpos[few], rope)
        assert torch.equal(qo[few], qf) and torch.equal(ko[few], kf)
    # in place; the same weights for one of the two only
    ref = pkv.qk_norm_rope(q, k, qw, None, 1e-5, dpos, rope) if qw is not None else (qo, ko)
    got = pkv.qk_norm_rope(q, k, qw, None, 1e-5, dpos, rope, q_out=q, k_out=k)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter", [(2048, 4, 1, 64, 64, False),
                                                  (2300, 9, 3, 80, 20, False),
                                                  (3333, 32, 8, 128, 128, True)])
def test_many_tokens_into_the_cache(cuda, n, hq, hkv, d, rot, inter):
    pkv = lib()
    rng = np.random.default_rng(n)
    q, k, v = rows(rng, n, (hq, hkv, hkv), d, BF, cuda, True)
    w = torch.from_numpy(1 + 0.5 * rng.normal(size=d)).to(BF).to(cuda)
    nb = n // 16 + 3
    kc0 = torch.from_numpy(rng.normal(size=(nb, 16, hkv, d))).to(BF).to(cuda)
    vc0 = -kc0
    kc, vc = kc0.clone(), vc0.clone()
    slots = rng.permutation(nb * 16)[:n].astype(np.int32)
    slots[::7] = -1 - slots[::7]                       # padding
    slots[5] = nb * 16                                 # outside
    pos = torch.from_numpy(rng.integers(0, 100000, n).astype(np.int32)).to(cuda)
    rope = pkv.rotary(rot, interleaved=inter, base=1e6)
    qr, kr = pkv.qk_norm_rope(q, k, w, w, 1e-6, pos, rope)
    st, ko = pkv.new_status(cuda), torch.empty_like(kr)
    got = pkv.qk_norm_rope_kv_store(q, k, v, w, w, 1e-6, pos, rope, kc, vc,
                                    torch.from_numpy(slots).to(cuda), k_out=ko, status=st)
    assert status_word(st) == pkv.STATUS["SLOT_OUT_OF_RANGE"]
    assert torch.equal(got, qr) and torch.equal(ko, kr)
    slots[5] = -1
    real = torch.from_numpy(np.flatnonzero(slots >= 0)).to(cuda)
    to = torch.from_numpy(slots[slots >= 0].astype(np.int64)).to(cuda)
    kc0.view(-1, hkv, d)[to], vc0.view(-1, hkv, d)[to] = kr[real], v[real]
    assert np.array_equal(bits(kc), bits(kc0)) and np.array_equal(bits(vc), bits(vc0))


def test_odd_values_of_many_tokens(cuda):
    """Infinite and NaN entries stay in their rows, and in their entries without a norm."""
    pkv = lib()
    q = torch.ones(2200, 2, 64, device=cuda)
    k = torch.ones(2200, 1, 64, device=cuda) * 2
    q[7, 0, 3], q[8, 1, 5], q[9, 0, 17] = float("inf"), float("nan"), float("inf")
    pos = torch.zeros(2200, dtype=torch.int32, device=cuda)
    w = torch.ones(64, device=cuda)
    qo, ko = pkv.qk_norm_rope(q, k, w, w, 0.0, pos, pkv.rotary(64))
    odd = torch.zeros(2200, 2, dtype=torch.bool, device=cuda)
    odd[7, 0] = odd[8, 1] = odd[9, 0] = True
    assert torch.equal(qo.isnan().any(-1), odd) and (ko == 1).all() and (qo[~odd] == 1).all()
    q[7, 0, 3] = q[8, 1, 5] = 1
    for rot, inter in [(16, False), (16, True), (10, False), (10, True)]:
        got, _ = pkv.qk_norm_rope(q, k, None, None, 0.0, pos, pkv.rotary(rot, interleaved=inter))
        assert torch.equal(got, q)


@pytest.mark.parametrize("n,hq,hkv,d,slots", [(2, 2, 1, 64, 1), (300, 4, 2, 64, 40),
                                              (2047, 2, 1, 128, 900), (2048, 2, 1, 64, 3),
                                              (5001, 9, 3, 80, 4000), (20000, 4, 2, 64, 15000),
                                              (160001, 1, 1, 8, 120000)])
def test_the_last_of_equal_slots_is_stored(cuda, n, hq, hkv, d, slots):
    """Whatever runs first: of one launch, and of the several that very many tokens take."""
    pkv = lib()
    rng = np.random.default_rng(n)
    q, k, v = rows(rng, n, (hq, hkv, hkv), d, BF, cuda, True)
    nb = -(-slots // 16)
    kc0 = torch.from_numpy(rng.normal(size=(nb, 16, hkv, d))).to(BF).to(cuda)
    kc, vc = kc0.clone(), kc0.clone()
    to = rng.integers(0, slots, n).astype(np.int32)
    to[rng.random(n) < 0.1] = -5                       # padding
    pos = torch.from_numpy(rng.integers(0, 100000, n).astype(np.int32)).to(cuda)
    rope = pkv.rotary(d)
    qr, kr = pkv.qk_norm_rope(q, k, None, None, 0.0, pos, rope)
    st = pkv.new_status(cuda)
    got = pkv.qk_norm_rope_kv_store(q, k, v, None, None, 0.0, pos, rope, kc, vc,
                                    torch.from_numpy(to).to(cuda), status=st)
    assert status_word(st) == 0 and torch.equal(got, qr)
    last = np.full(nb * 16, -1)
    last[to[to >= 0]] = np.flatnonzero(to >= 0)        # assignments in order: the last stays
    have = torch.from_numpy(np.flatnonzero(last >= 0)).to(cuda)
    src = torch.from_numpy(last[last >= 0]).to(cuda)
    kw, vw = kc0.clone(), kc0.clone()
    kw.view(-1, hkv, d)[have], vw.view(-1, hkv, d)[have] = kr[src], v[src]
    assert np.array_equal(bits(kc), bits(kw)) and np.array_equal(bits(vc), bits(vw))
