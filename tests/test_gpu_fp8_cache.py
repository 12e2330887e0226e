"""The 8-bit KV cache on the GPU against the float64 oracle: the store bit for
bit, decode and prefill within the bounds of fp8_util."""
import math

import numpy as np
import pytest
import torch

import fp8_util as F
import gpu_util as U
from oracle import attention as oatt
from oracle import fp8_cache as ofp

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------
# store
# ----------------------------------------------------------------------------
def _store_case(rng, n, nb, bs, hkv, d, pattern):
    if pattern == "runs":                       # sequences in order, ragged
        slots = []
        perm = rng.permutation(nb)
        at = 0
        while len(slots) < n and at < nb:
            take = min(int(rng.integers(1, 3 * bs + 1)), n - len(slots))
            pos = int(rng.integers(0, bs))
            blocks = perm[at:at + -(-(pos + take) // bs)]
            at += len(blocks)
            for p in range(pos, pos + take):
                if p // bs < len(blocks):
                    slots.append(int(blocks[p // bs]) * bs + p % bs)
        slots += [-1] * (n - len(slots))
    elif pattern == "shuffled":                 # any order, padding, one slot often twice
        slots = rng.integers(-2, nb * bs, n).tolist()
    elif pattern == "same":                     # every token to one slot
        slots = [bs // 2] * n
    else:                                       # one token per block, as a decode step
        slots = (rng.permutation(nb)[:n] * bs + rng.integers(0, bs, n)).tolist()
    return np.asarray(slots, np.int32)


def _run_store(pkv, dev, k, v, pool, slots, expect=0, **kw):
    kc, vc, ks, vs, _ = pool.on(dev)
    st = pkv.new_status(dev)
    pkv.kv_store_fp8(k.to(dev), v.to(dev), kc, vc, ks, vs, torch.from_numpy(slots).to(dev),
                     status=st, **kw)
    assert U.status_word(st) == expect
    ref = ofp.kv_store(U.f64(k), U.f64(v), pool.codes["k"], pool.codes["v"], pool.scale["k"],
                       pool.scale["v"], slots)
    for got, want in ((ks, ref[2]), (vs, ref[3])):
        np.testing.assert_array_equal(U.f64(got), want)
    for got, want in ((kc, ref[0]), (vc, ref[1])):
        got = got.view(torch.uint8).cpu().numpy()
        same = got == want
        # a NaN code that was re-scaled may come back with either sign
        assert (same | ((got & 127 == 127) & (want & 127 == 127))).all()


@pytest.mark.parametrize("n,nb,bs,hkv,d,pattern", [
    (1, 2, 16, 1, 64, "step"), (37, 60, 256, 8, 128, "step"), (5, 9, 1, 2, 64, "step"),
    (300, 30, 16, 8, 128, "runs"), (513, 9, 256, 2, 128, "runs"), (100, 40, 7, 3, 64, "runs"),
    (700, 3, 1024, 1, 128, "runs"), (2048, 20, 128, 4, 64, "runs"),
    (200, 12, 24, 5, 128, "shuffled"), (2048, 6, 48, 2, 64, "shuffled"),
    (2049, 200, 16, 2, 128, "runs"), (3000, 40, 100, 3, 64, "shuffled"),
    (5000, 3, 512, 20, 64, "shuffled"), (2500, 2, 8, 1, 64, "same"), (90, 2, 8, 1, 128, "same"),
    (4097, 4500, 1, 1, 64, "step"),
])
def test_store_is_the_oracles(cuda, n, nb, bs, hkv, d, pattern):
    pkv = U.lib()
    rng = np.random.default_rng(n * 131 + bs)
    slots = _store_case(rng, n, nb, bs, hkv, d, pattern)
    pool = F.Pool([nb * bs - bs], bs, hkv, d, seed=n, spare=1)
    mag = 2.0 ** rng.integers(-5, 4, (n, hkv, 1))
    _run_store(pkv, cuda, F.bf16(rng, n, hkv, d, mag=mag), F.bf16(rng, n, hkv, d, mag=mag), pool,
               slots)


def _run_edges(rng, nb, bs):
    """Runs of 1 to bs rows around the 16 that a lane group keeps: in line, with two rows
    swapped, a slot left out or stored twice, padding inside, and two runs of one block
    with another block's rows between them."""
    slots, perm = [], rng.permutation(nb)
    for i in range(0, nb - 1, 2):
        b, c = int(perm[i]) * bs, int(perm[i + 1]) * bs
        rows = int(rng.choice([1, 2, 15, 16, 17, 18, 33, bs]))
        rows = min(rows, bs)
        pos = int(rng.integers(0, bs - rows + 1))
        run = list(range(b + pos, b + pos + rows))
        kind = int(rng.integers(0, 6))
        at = int(rng.integers(0, rows))
        if kind == 1 and rows > 2:
            run[at - 1], run[at - 2] = run[at - 2], run[at - 1]
        elif kind == 2 and rows > 1:
            del run[at]
        elif kind == 3:
            run.insert(at, run[-1])
        elif kind == 4:
            run.insert(at, -1)
        elif kind == 5 and rows > 6:            # slot after slot again sixteen tokens on
            run[2:5] = [c, c + bs // 2, c + bs - 1]
        slots += run
    return np.asarray(slots, np.int32)


@pytest.mark.parametrize("nb,bs,hkv,d", [(260, 48, 8, 128), (700, 20, 3, 64), (120, 256, 2, 128),
                                         (150, 200, 20, 64)])
def test_store_runs_of_few_and_many_rows(cuda, nb, bs, hkv, d):
    rng = np.random.default_rng(bs)
    slots = _run_edges(rng, nb, bs)
    n = len(slots)
    assert n > 2048
    pool = F.Pool([nb * bs - bs], bs, hkv, d, seed=n, spare=1)
    mag = 2.0 ** rng.integers(-5, 4, (n, hkv, 1))
    _run_store(U.lib(), cuda, F.bf16(rng, n, hkv, d, mag=mag), F.bf16(rng, n, hkv, d, mag=mag),
               pool, slots)


def test_store_one_row_each_of_many_sequences(cuda):
    rng = np.random.default_rng(4)
    n, nb, bs, hkv, d = 2500, 2600, 64, 2, 128
    slots = _store_case(rng, n, nb, bs, hkv, d, "step")
    pool = F.Pool([nb * bs - bs], bs, hkv, d, seed=n, spare=1)
    _run_store(U.lib(), cuda, F.bf16(rng, n, hkv, d), F.bf16(rng, n, hkv, d), pool, slots)


@pytest.mark.parametrize("n", [6, 2100])
def test_store_special_values_and_scales(cuda, n):
    """Infinities saturate and do not widen the scale, NaN stays; zero rows;
    values at a power of two's edge; a scale of 0, one that is no power of two,
    and one that cannot be used."""
    pkv = U.lib()
    rng = np.random.default_rng(3)
    bs, hkv, d = 16, 4, 64
    pool = F.Pool([16 * bs], bs, hkv, d, seed=5, arbitrary=True, spare=2200)
    k, v = F.bf16(rng, n, hkv, d), F.bf16(rng, n, hkv, d)
    k[0, 0, 3], k[0, 0, 4], k[1, 1, 0] = math.inf, -math.inf, math.nan
    k[2], v[2] = 0.0, 0.0
    v[3, 0] = 3.5                                # exactly 448 * 2^-7
    v[3, 1] = 3.515625                           # the next bf16
    v[3, 2, 0], v[3, 3] = 3.38e38, 1e-38
    k[4, 0] = math.inf                           # no finite entry at all
    slots = np.asarray([b * bs + 5 for b in range(n)], np.int32)
    pool.scale["k"][1, 2], pool.scale["v"][1, 3] = 0.0, 0.0
    _run_store(pkv, cuda, k, v, pool, slots)
    pool.scale["k"][0, 1], pool.scale["v"][2, 0] = -1.0, math.inf
    pool.scale["k"][3, 3] = math.nan
    _run_store(pkv, cuda, k, v, pool, slots, expect=pkv.STATUS["BAD_SCALE"])


def test_store_row_by_row_is_store_at_once(cuda):
    """Up to the subnormals of a block's final scale."""
    pkv = U.lib()
    rng = np.random.default_rng(8)
    n, bs, hkv, d = 40, 16, 2, 64
    k = F.bf16(rng, n, hkv, d, mag=2.0 ** rng.integers(-3, 4, (n, 1, 1))).to(cuda)
    slots = torch.arange(n, dtype=torch.int32, device=cuda) + 2 * bs
    caches = [[torch.zeros((6, bs, hkv, d), dtype=torch.uint8, device=cuda).view(torch.float8_e4m3fn)
               for _ in "kv"] + [torch.zeros((6, hkv), device=cuda) for _ in "kv"]
              for _ in range(2)]
    pkv.kv_store_fp8(k, k, *caches[0], slots)
    for t in range(n):
        pkv.kv_store_fp8(k[t:t + 1], k[t:t + 1], *caches[1], slots[t:t + 1])
    assert torch.equal(caches[0][2], caches[1][2])
    a, b = (c[0].double() * c[2].double()[:, None, :, None] for c in caches)
    s = caches[0][2].double()[:, None, :, None]
    assert ((a - b).abs() <= torch.where(a.abs() < s * 2.0 ** -6, s * 2.0 ** -9, 0.0)).all()


@pytest.mark.parametrize("n", [50, 3000])
def test_store_reports_slots_outside_the_pool(cuda, n):
    pkv = U.lib()
    rng = np.random.default_rng(1)
    bs, hkv, d = 16, 2, 64
    pool = F.Pool([300 * bs], bs, hkv, d, seed=2)
    slots = rng.integers(0, 302 * bs, n).astype(np.int32)
    slots[7], slots[20] = 302 * bs, 2 ** 31 - 1
    _run_store(pkv, cuda, F.bf16(rng, n, hkv, d), F.bf16(rng, n, hkv, d), pool, slots,
               expect=pkv.STATUS["SLOT_OUT_OF_RANGE"])


def test_empty_store_and_padding_only(cuda):
    pkv = U.lib()
    pool = F.Pool([32], 16, 1, 64, seed=1)
    none = torch.zeros((0, 1, 64), dtype=torch.bfloat16)
    _run_store(pkv, cuda, none, none, pool, np.zeros(0, np.int32))
    rows = torch.ones((9, 1, 64), dtype=torch.bfloat16)
    _run_store(pkv, cuda, rows, rows, pool, np.full(9, -1, np.int32))


# ----------------------------------------------------------------------------
# decode
# ----------------------------------------------------------------------------
def _check_decode(got, pool, q, scale):
    kv, vv = pool.values("k"), pool.values("v")
    ref = oatt.paged_decode(U.f64(q), kv, vv, pool.bt, pool.lens, scale)
    got = U.f64(got)
    assert np.isfinite(got).all()
    tol = F.bound(ref, U.f64(q), kv, vv, scale, F.DECODE, max(pool.lens))
    err = np.abs(got - ref)
    assert (err <= tol).all(), (err - tol).max()
    return ref


@pytest.mark.parametrize("lens,bs,hkv,group,d", [
    ([1], 16, 1, 1, 64), ([1], 256, 8, 2, 128), ([0], 64, 2, 2, 128), ([1000], 256, 8, 2, 128),
    ([0, 1, 15, 16, 17, 64, 65, 300], 16, 2, 4, 128), ([5, 700, 64, 0, 129], 64, 2, 8, 128),
    ([5, 700, 64, 0, 129], 64, 2, 8, 64), ([33, 100, 7], 24, 3, 7, 128), ([33, 100, 7], 1, 1, 3, 64),
    ([255, 256, 257, 1023, 1025], 256, 1, 16, 128), ([255, 256, 257, 1023], 256, 2, 9, 64),
    ([2000, 1], 1024, 1, 4, 128), ([190, 193, 600], 192, 4, 1, 64), ([500, 13], 100, 2, 5, 128),
    ([4100, 129, 3], 128, 1, 4, 128), ([40] * 70, 32, 2, 2, 64),
])
@pytest.mark.parametrize("arbitrary", [False, True])
def test_decode_is_the_oracles(cuda, lens, bs, hkv, group, d, arbitrary):
    pkv = U.lib()
    rng = np.random.default_rng(len(lens) * 7 + bs)
    pool = F.Pool(lens, bs, hkv, d, seed=bs + d, spread=4, arbitrary=arbitrary)
    q = F.bf16(rng, len(lens), hkv * group, d)
    st = pkv.new_status(cuda)
    scale = 1 / math.sqrt(d)
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda),
                               torch.tensor(lens, dtype=torch.int32, device=cuda), scale,
                               max(lens), status=st)
    assert U.status_word(st) == 0
    ref = _check_decode(out, pool, q, scale)
    assert (ref[[i for i, n in enumerate(lens) if n == 0]] == 0).all()


@pytest.mark.parametrize("lens", [[2047, 2049, 0, 1985, 6200], [4097] + [130] * 32 + [2048]])
@pytest.mark.parametrize("bs,d", [(16, 128), (64, 128), (256, 64), (24, 64)])
def test_decode_longest_units(cuda, lens, bs, d):
    """A stated maximum so large that units have 2048 keys, with and without a plan
    kernel."""
    pkv = U.lib()
    rng = np.random.default_rng(bs)
    pool = F.Pool(lens, bs, 2, d, seed=bs + d, spread=4)
    q = F.bf16(rng, len(lens), 16, d)
    st = pkv.new_status(cuda)
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda),
                               torch.tensor(lens, dtype=torch.int32, device=cuda), 0.09, 1 << 20,
                               status=st)
    assert U.status_word(st) == 0
    _check_decode(out, pool, q, 0.09)


@pytest.mark.parametrize("bs", [16, 64, 40])
@pytest.mark.parametrize("q_mag,vexp", [(1e25, -60), (1e-30, 100), (3e4, 0), (1.0, -86)])
def test_decode_ranges(cuda, bs, q_mag, vexp):
    """Queries and scales far outside f16's range: only the products count."""
    pkv = U.lib()
    rng = np.random.default_rng(11)
    hkv, group, d, lens = 2, 4, 128, [200, 77]
    pool = F.Pool(lens, bs, hkv, d, seed=4)
    kexp = -round(math.log2(q_mag))
    pool.scale["k"] = np.ldexp(pool.scale["k"], kexp).astype(np.float32)
    pool.scale["v"] = np.ldexp(pool.scale["v"], vexp).astype(np.float32)
    q = F.bf16(rng, 2, hkv * group, d, mag=q_mag)
    q[0, 0, :5] = 0.0
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda),
                               torch.tensor(lens, dtype=torch.int32, device=cuda), 0.125, 200)
    _check_decode(out, pool, q, 0.125)


@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [100, 5000])          # with and without a combine
def test_decode_infinities_and_nan(cuda, bs, d, most):
    """NaN or an infinity in a head's query: NaN for that head alone.  A NaN code in
    a key that counts: NaN for its kv head; in a value: for that entry."""
    pkv = U.lib()
    rng = np.random.default_rng(19)
    pool = F.Pool([most, 90], bs, 2, d, seed=4)
    blk = int(pool.bt[1, 0])
    pool.codes["k"][blk, 3, 0, 5] = 0x7F
    pool.codes["v"][blk, 3, 1, 7] = 0xFF
    q = F.bf16(rng, 2, 8, d)
    ctx = torch.tensor([most, 90], dtype=torch.int32, device=cuda)
    clean = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda), ctx, 0.125, most)
    q[0, 1, 0], q[0, 2, 9], q[0, 6, d - 1] = math.inf, math.nan, -math.inf
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda), ctx, 0.125, most)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, [1, 2, 6]] = True
    bad[1, :4] = True                            # kv head 0
    bad[1, 4:, 7] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("bs", [16, 64, 40])
def test_decode_values_of_very_different_scales(cuda, bs):
    """Blocks whose V scales differ by 2^80: the small ones' keys still carry
    their weight in the normaliser."""
    pkv = U.lib()
    rng = np.random.default_rng(12)
    hkv, group, d, lens = 1, 8, 64, [10 * bs]
    pool = F.Pool(lens, bs, hkv, d, seed=4)
    pool.scale["v"][::2] = np.ldexp(pool.scale["v"][::2], -80)
    q = F.bf16(rng, 1, hkv * group, d)
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda),
                               torch.tensor(lens, dtype=torch.int32, device=cuda), 0.125, lens[0])
    _check_decode(out, pool, q, 0.125)


@pytest.mark.parametrize("bs", [16, 64, 48, 256])
def test_decode_leaves_out_blocks_it_cannot_read(cuda, bs):
    """A block id outside the pool, and a block whose scale cannot be used: the
    status says so, the other keys are attended to."""
    pkv = U.lib()
    rng = np.random.default_rng(13)
    hkv, group, d = 2, 2, 128
    n = 4 * bs + 3
    for what in ("id", "k", "v"):
        pool = F.Pool([n, bs + 1], bs, hkv, d, seed=6)
        q = F.bf16(rng, 2, hkv * group, d)
        kept = [0, 2, 3, 4]                      # blocks of sequence 0 without its second
        bad_blk = int(pool.bt[0, 1])
        dense = np.concatenate([pool.bt[0, kept], [-1]])
        args = list(pool.on(cuda))
        if what == "id":
            args[4][0, 1] = pool.codes["k"].shape[0] if bs == 16 else -7
        else:
            args[2 if what == "k" else 3][bad_blk] = 0.0 if bs == 16 else math.nan
        st = pkv.new_status(cuda)
        out = pkv.paged_decode_fp8(q.to(cuda), *args,
                                   torch.tensor([n, bs + 1], dtype=torch.int32, device=cuda), 0.1,
                                   n, status=st)
        name = "BAD_BLOCK_ID" if what == "id" else "BAD_SCALE"
        assert U.status_word(st) == pkv.STATUS[name]
        pool.bt[0] = dense[:pool.bt.shape[1]]
        pool.lens[0] = n - bs
        _check_decode(out, pool, q, 0.1)


def test_decode_bad_context_lens(cuda):
    pkv = U.lib()
    rng = np.random.default_rng(14)
    pool = F.Pool([40, 40, 40, 40], 16, 1, 64, seed=6)
    q = F.bf16(rng, 4, 2, 64)
    st = pkv.new_status(cuda)
    ctx = torch.tensor([40, -1, 49, 40], dtype=torch.int32, device=cuda)
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda), ctx, 0.1, 48, status=st)
    assert U.status_word(st) == pkv.STATUS["BAD_CONTEXT_LEN"]
    pool.lens = [40, 0, 0, 40]
    _check_decode(out, pool, q, 0.1)


@pytest.mark.parametrize("B", [31, 32, 33, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("bs,most", [(16, 300), (64, 1500)])      # without and with a combine
def test_decode_batches_around_a_warps_lanes(cuda, B, bs, most):
    """With and without a plan kernel: many sequences, some without keys, some of a
    length that is out of range (reported, zero rows), some of several chunks."""
    pkv = U.lib()
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 40, B).tolist()
    for i in (0, 5, B // 2, B - 1):
        lens[i] = most
    pool = F.Pool(lens, bs, 1, 64, seed=B)
    q = F.bf16(rng, B, 3, 64)
    st = pkv.new_status(cuda)
    run = lambda ctx: pkv.paged_decode_fp8(  # noqa: E731
        q.to(cuda), *pool.on(cuda), torch.tensor(ctx, dtype=torch.int32, device=cuda), 0.1, most,
        status=st)
    out = run(lens)
    assert U.status_word(st) == 0
    _check_decode(out, pool, q, 0.1)
    bad = list(lens)
    bad[B - 2], bad[3] = -5, most + 1
    out = run(bad)
    assert U.status_word(st) == pkv.STATUS["BAD_CONTEXT_LEN"]
    pool.lens[B - 2] = pool.lens[3] = 0
    _check_decode(out, pool, q, 0.1)


def test_plan_and_runs_are_the_whole_call(cuda):
    pkv = U.lib()
    rng = np.random.default_rng(15)
    lens = [300, 5, 0, 1000]
    pool = F.Pool(lens, 64, 2, 128, seed=6)
    args = pool.on(cuda)
    ctx = torch.tensor(lens, dtype=torch.int32, device=cuda)
    ws = pkv.paged_decode_plan_fp8(ctx, 8, 1000, args[4].shape[1], args[0])
    assert ws.numel() >= pkv.paged_decode_fp8_workspace_bytes(4, 8, 1000, args[0])
    for i in range(3):
        q = F.bf16(rng, 4, 8, 128).to(cuda)
        whole = pkv.paged_decode_fp8(q, *args, ctx, 0.1, 1000)
        assert torch.equal(pkv.paged_decode_run_fp8(q, *args, ctx, 0.1, 1000, ws), whole)


@pytest.mark.parametrize("n,bs", [(4, 16), (4, 256), (2200, 16)])
def test_store_and_decode_in_one_call(cuda, n, bs):
    """A step's fused call is its two calls, bit for bit; n = 2200 tokens is a
    call of the store's list form (most of them padding for the decode)."""
    pkv = U.lib()
    rng = np.random.default_rng(16)
    lens = [1, bs, 3 * bs + 2, 2 * bs + 1]
    pool = F.Pool(lens, bs, 2, 128, seed=6, spare=150)
    q, k, v = F.bf16(rng, 4, 8, 128), F.bf16(rng, n, 2, 128), F.bf16(rng, n, 2, 128)
    free = sorted(set(range(pool.codes["k"].shape[0])) - set(pool.bt.reshape(-1).tolist()))
    slots = [int(pool.bt[i, (m - 1) // bs]) * bs + (m - 1) % bs for i, m in enumerate(lens)]
    slots += [free[i // bs] * bs + i % bs for i in range(n - 4)]
    slots = torch.tensor(slots, dtype=torch.int32, device=cuda)
    ctx = torch.tensor(lens, dtype=torch.int32, device=cuda)
    q, k, v = q.to(cuda), k.to(cuda), v.to(cuda)
    a, b = pool.on(cuda), pool.on(cuda)
    pkv.kv_store_fp8(k, v, *a[:4], slots)
    want = pkv.paged_decode_fp8(q, *a, ctx, 0.1, max(lens))
    got = pkv.kv_store_paged_decode_fp8(k, v, slots, q, *b, ctx, 0.1, max(lens))
    assert torch.equal(got, want)
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_cache_beyond_32_bit_offsets(cuda):
    """Rows whose byte offset needs 33 bits, stored and attended to."""
    pkv = U.lib()
    rng = np.random.default_rng(17)
    bs, hkv, d = 256, 8, 128
    nb = (1 << 32) // (bs * hkv * d) + 40
    small = F.Pool([600], bs, hkv, d, seed=9, spare=1)
    kc = torch.empty((nb, bs, hkv, d), dtype=torch.uint8, device=cuda)
    vc = torch.empty_like(kc)
    ks = torch.ones((nb, hkv), device=cuda)
    vs = torch.ones((nb, hkv), device=cuda)
    far = nb - 20
    sk, sv, sks, svs, bt = small.on(cuda)
    for i in range(4):
        kc[far + i], vc[far + i] = sk[i].view(torch.uint8), sv[i].view(torch.uint8)
        ks[far + i], vs[far + i] = sks[i], svs[i]
    args = (kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs)
    bt = torch.where(bt >= 0, bt + far, bt)
    q = F.bf16(rng, 1, 16, d)
    ctx = torch.tensor([600], dtype=torch.int32, device=cuda)
    row = F.bf16(rng, 1, hkv, d)
    slot = torch.tensor([int(small.bt[0, 2]) * bs + 599 % bs + far * bs], dtype=torch.int32,
                        device=cuda)
    pkv.kv_store_fp8(row.to(cuda), row.to(cuda), *args, slot)
    out = pkv.paged_decode_fp8(q.to(cuda), *args, bt, ctx, 0.1, 600)
    ref = ofp.kv_store(U.f64(row), U.f64(row), small.codes["k"], small.codes["v"],
                       small.scale["k"], small.scale["v"], slot.cpu().numpy() - far * bs)
    small.codes, small.scale = {"k": ref[0], "v": ref[1]}, {"k": ref[2], "v": ref[3]}
    _check_decode(out, small, q, 0.1)


# ----------------------------------------------------------------------------
# prefill
# ----------------------------------------------------------------------------
def _prefill(pkv, dev, lq, lp, bs, hkv, group, d, seed, max_k=None, extra=0):
    rng = np.random.default_rng(seed)
    pool = F.Pool(lp, bs, hkv, d, seed=seed, spread=3)
    t = sum(lq)
    q, k, v = (F.bf16(rng, t + extra, h, d) for h in (hkv * group, hkv, hkv))
    cu = lambda x: np.concatenate([[0], np.cumsum(x)]).astype(np.int32)  # noqa: E731
    cu_q, cu_k = cu(lq), cu(np.asarray(lq) + np.asarray(lp))
    scale = 1 / math.sqrt(d)
    st = pkv.new_status(dev)
    kc, vc, ks, vs, bt = pool.on(dev)
    out = torch.full((t + extra, hkv * group, d), 7.0, dtype=torch.bfloat16, device=dev)
    pkv.paged_prefill_varlen_fp8(q.to(dev), k.to(dev), v.to(dev), kc, vc, ks, vs,
                                 torch.from_numpy(cu_q).to(dev), torch.from_numpy(cu_k).to(dev),
                                 max(lq), max_k or int((np.asarray(lq) + lp).max()), bt, scale,
                                 out=out, status=st)
    assert U.status_word(st) == 0
    assert (out[t:] == 7.0).all()                # rows of no sequence: left as they were
    kv, vv = pool.values("k"), pool.values("v")
    ref = oatt.paged_prefill_varlen(U.f64(q[:t]), U.f64(k), U.f64(v), kv, vv, cu_q, cu_k, pool.bt,
                                    scale)
    everything = [np.concatenate([a.reshape(-1, d), U.f64(b).reshape(-1, d)])
                  for a, b in ((kv, k), (vv, v))]
    tol = F.bound(ref, U.f64(q[:t]), everything[0], everything[1], scale, F.PREFILL, 0)
    err = np.abs(U.f64(out[:t]) - ref)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("lq,lp,bs,hkv,group,d", [
    ([1], [1], 16, 1, 1, 64), ([1], [300], 256, 2, 4, 128), ([130], [0], 16, 2, 2, 128),
    ([5, 1, 140], [128, 127, 129], 16, 2, 2, 128), ([5, 0, 70], [0, 50, 513], 64, 1, 8, 64),
    ([33, 200], [100, 7], 24, 3, 3, 64), ([17, 3], [1000, 1], 1024, 1, 4, 128),
    ([129, 1, 1], [255, 256, 257], 128, 2, 1, 128), ([10, 11], [37, 5], 1, 1, 2, 64),
    # few queries on long prefixes: keys split over work items, some rows unsplit
    ([1], [3000], 64, 1, 2, 128), ([20, 160, 5, 300], [2500, 900, 0, 17], 16, 2, 2, 128),
    ([130, 7], [511, 4000], 256, 1, 3, 64), ([1] * 20, [700] * 19 + [5000], 32, 1, 1, 64),
    ([1], [5000], 64, 1, 2, 128), ([20, 160, 5, 300], [6500, 4600, 0, 17], 16, 1, 2, 128),
    ([130, 7], [511, 9000], 256, 1, 3, 64), ([65, 128], [4096, 3968], 128, 2, 1, 128),
])
def test_prefill_is_the_oracles(cuda, lq, lp, bs, hkv, group, d):
    _prefill(U.lib(), cuda, lq, lp, bs, hkv, group, d, seed=bs + sum(lq), extra=3)


def test_prefill_in_groups_of_sequences(cuda):
    """max_seqlen_k so large that the prefixes' workspace holds two of the five
    sequences at a time."""
    pkv = U.lib()
    need = [pkv.paged_prefill_fp8_workspace_bytes(b, 300, 8, 500000, (64, 16, 8, 128))
            for b in (1, 2, 3, 5)]
    # (besides the prefixes, the splits' partial results: a hundredth of them)
    assert need[0] < 0.6 * need[1] and max(need[2:]) < 1.02 * need[1] < 5 << 30
    _prefill(pkv, cuda, [60, 1, 90, 100, 49], [130, 400, 0, 7, 256], 16, 8, 1, 128, seed=3,
             max_k=500000)


def test_prefill_skips_inconsistent_sequences(cuda):
    """More cached keys than the table holds (the table's last block ends inside
    the workspace's), fewer keys than queries, a prefix beyond max_seqlen_k."""
    pkv = U.lib()
    rng = np.random.default_rng(2)
    bs, hkv, d = 16, 1, 64
    pool = F.Pool([48, 48, 48, 48], bs, hkv, d, seed=1)
    lq, lk = [4, 4, 4, 4], [4 + 48, 4 + 49, 3, 4 + 48]     # (the second is over max_seqlen_k too)
    cu = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32,  # noqa: E731,E501
                                device=cuda)
    q, k = F.bf16(rng, 16, 2, d), F.bf16(rng, 16, hkv, d)
    kc, vc, ks, vs, bt = pool.on(cuda)
    st = pkv.new_status(cuda)
    out = torch.full((16, 2, d), 7.0, dtype=torch.bfloat16, device=cuda)
    pkv.paged_prefill_varlen_fp8(q.to(cuda), k.to(cuda), k.to(cuda), kc, vc, ks, vs, cu(lq),
                                 cu(lk), 4, 53, bt, 0.125, out=out, status=st)
    assert U.status_word(st) == pkv.STATUS["BAD_SEQLENS"]
    assert (out[4:12] == 7.0).all()
    kv, vv = pool.values("k"), pool.values("v")
    for i in (0, 3):
        rows = slice(4 * i, 4 * i + 4)
        ref = oatt.paged_prefill_varlen(U.f64(q[rows]), U.f64(k[rows]), U.f64(k[rows]), kv, vv,
                                        [0, 4], [0, 52], pool.bt[i:i + 1], 0.125)
        tol = F.bound(ref, U.f64(q[rows]), np.concatenate([kv.reshape(-1, d),
                                                           U.f64(k).reshape(-1, d)]),
                      np.concatenate([vv.reshape(-1, d), U.f64(k).reshape(-1, d)]), 0.125,
                      F.PREFILL, 0)
        assert (np.abs(U.f64(out[rows]) - ref) <= tol).all()


def test_prefill_skips_a_sequence_beyond_max_seqlen_k(cuda):
    """Its keys would not fit the workspace's splits; the others are attended."""
    pkv = U.lib()
    rng = np.random.default_rng(3)
    bs, hkv, d = 64, 1, 128
    lens, lq = [1000, 1000], [300, 40]
    pool = F.Pool(lens, bs, hkv, d, seed=1)
    q, k = F.bf16(rng, 340, 2, d), F.bf16(rng, 340, hkv, d)
    cu_q = torch.tensor([0, 300, 340], dtype=torch.int32, device=cuda)
    cu_k = torch.tensor([0, 1300, 2340], dtype=torch.int32, device=cuda)
    kc, vc, ks, vs, bt = pool.on(cuda)
    st = pkv.new_status(cuda)
    out = torch.full((340, 2, d), 7.0, dtype=torch.bfloat16, device=cuda)
    pkv.paged_prefill_varlen_fp8(q.to(cuda), k.to(cuda), k.to(cuda), kc, vc, ks, vs, cu_q, cu_k, 300,
                                 1040, bt, 0.09, out=out, status=st)
    assert U.status_word(st) == pkv.STATUS["BAD_SEQLENS"]
    assert (out[:300] == 7.0).all()
    kv, vv = pool.values("k"), pool.values("v")
    ref = oatt.paged_prefill_varlen(U.f64(q[300:]), U.f64(k[300:]), U.f64(k[300:]), kv, vv, [0, 40],
                                    [0, 1040], pool.bt[1:], 0.09)
    both = [np.concatenate([x.reshape(-1, d), U.f64(k).reshape(-1, d)]) for x in (kv, vv)]
    tol = F.bound(ref, U.f64(q[300:]), *both, 0.09, F.PREFILL, 0)
    assert (np.abs(U.f64(out[300:]) - ref) <= tol).all()


def test_split_prefill_gives_up_then_recovers(cuda):
    """The bounded waits of the prefill kernel run out while its keys are split."""
    pkv = U.lib()
    try:
        for polls in (0, 2, 4):
            pkv.set_wait_poll_limit(polls)
            try:
                _prefill(pkv, cuda, [20, 160], [2500, 900], 16, 2, 2, 128, seed=4)
            except AssertionError:
                pass                             # the status said so (or too few polls were few)
            torch.cuda.synchronize()
    finally:
        pkv.set_wait_poll_limit()
    _prefill(pkv, cuda, [20, 160], [2500, 900], 16, 2, 2, 128, seed=4)


def test_split_prefill_skips_a_sequence_beyond_max_seqlen_k(cuda):
    # 4340 keys: two splits of 17 tiles; the longer sequence's rows have no room in them
    pkv = U.lib()
    rng = np.random.default_rng(3)
    hkv, d = 1, 128
    pool = F.Pool([4300, 4300], 64, hkv, d, seed=1)
    q, k = F.bf16(rng, 340, 2, d), F.bf16(rng, 340, hkv, d)
    cu_q = torch.tensor([0, 300, 340], dtype=torch.int32, device=cuda)
    cu_k = torch.tensor([0, 4600, 8940], dtype=torch.int32, device=cuda)
    kc, vc, ks, vs, bt = pool.on(cuda)
    st = pkv.new_status(cuda)
    out = torch.full((340, 2, d), 7.0, dtype=torch.bfloat16, device=cuda)
    pkv.paged_prefill_varlen_fp8(q.to(cuda), k.to(cuda), k.to(cuda), kc, vc, ks, vs, cu_q, cu_k, 300,
                                 4340, bt, 0.09, out=out, status=st)
    assert U.status_word(st) == pkv.STATUS["BAD_SEQLENS"]
    assert (out[:300] == 7.0).all()
    kv, vv = pool.values("k"), pool.values("v")
    ref = oatt.paged_prefill_varlen(U.f64(q[300:]), U.f64(k[300:]), U.f64(k[300:]), kv, vv, [0, 40],
                                    [0, 4340], pool.bt[1:], 0.09)
    both = [np.concatenate([x.reshape(-1, d), U.f64(k).reshape(-1, d)]) for x in (kv, vv)]
    tol = F.bound(ref, U.f64(q[300:]), *both, 0.09, F.PREFILL, 0)
    assert (np.abs(U.f64(out[300:]) - ref) <= tol).all()


@pytest.mark.parametrize("polls", [0, 2, 4])
def test_long_split_prefill_gives_up_then_recovers(cuda, polls):
    pkv = U.lib()
    case = ([20, 160], [5500, 900], 16, 1, 2, 128)
    pkv.set_wait_poll_limit(polls)
    try:
        _prefill(pkv, cuda, *case, seed=4)
    except AssertionError:
        pass                                     # the status said so (or too few polls were few)
    finally:
        pkv.set_wait_poll_limit()
    torch.cuda.synchronize()
    _prefill(pkv, cuda, *case, seed=4)


def test_prefill_unreadable_prefix_rows_are_zeros(cuda):
    pkv = U.lib()
    rng = np.random.default_rng(2)
    bs, hkv, d = 16, 1, 64
    for what, bit in (("id", "BAD_BLOCK_ID"), ("scale", "BAD_SCALE")):
        pool = F.Pool([48], bs, hkv, d, seed=1)
        q, k = F.bf16(rng, 3, 2, d), F.bf16(rng, 3, hkv, d)
        kc, vc, ks, vs, bt = pool.on(cuda)
        blk = int(pool.bt[0, 1])
        if what == "id":
            bt[0, 1] = 10 ** 6
        else:
            ks[blk], vs[blk] = 0.0, math.inf
        cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=cuda)  # noqa: E731
        st = pkv.new_status(cuda)
        out = pkv.paged_prefill_varlen_fp8(q.to(cuda), k.to(cuda), k.to(cuda), kc, vc, ks, vs,
                                           cu(3), cu(51), 3, 51, bt, 0.125, status=st)
        assert U.status_word(st) == pkv.STATUS[bit]
        for c in pool.codes.values():
            c[blk] = 0
        kv, vv = pool.values("k"), pool.values("v")
        ref = oatt.paged_prefill_varlen(U.f64(q), U.f64(k), U.f64(k), kv, vv, [0, 3], [0, 51],
                                        pool.bt, 0.125)
        tol = F.bound(ref, U.f64(q), np.concatenate([kv.reshape(-1, d), U.f64(k).reshape(-1, d)]),
                      np.concatenate([vv.reshape(-1, d), U.f64(k).reshape(-1, d)]), 0.125,
                      F.PREFILL, 0)
        assert (np.abs(U.f64(out) - ref) <= tol).all()


# ----------------------------------------------------------------------------
# together, streams and graphs
# ----------------------------------------------------------------------------
def test_a_conversation_in_the_8_bit_cache(cuda):
    """Two prompts prefilled in two chunks each, then decode steps and sampling
    with penalties, every step against the oracle's own cache."""
    pkv = U.lib()
    rng = np.random.default_rng(20)
    bs, hkv, hq, d, vocab = 16, 2, 6, 64, 300
    scale = 1 / math.sqrt(d)
    tables = np.asarray([[3, 7, 1, 9], [0, 5, 8, 2]], np.int32)
    codes = [np.full((10, bs, hkv, d), 0x7F, np.uint8) for _ in "kv"]
    scales = [np.zeros((10, hkv), np.float32) for _ in "kv"]
    gpu = [torch.from_numpy(c).to(cuda).view(torch.float8_e4m3fn) for c in codes] + \
          [torch.from_numpy(s).to(cuda) for s in scales]
    bt = torch.from_numpy(tables).to(cuda)
    st = pkv.new_status(cuda)
    slots_of = lambda b, a, n: [int(tables[b, p // bs]) * bs + p % bs  # noqa: E731
                                for p in range(a, a + n)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    state = (*codes, *scales)
    done = [0, 0]
    for new in ([20, 9], [14, 22]):
        t = sum(new)
        q, k, v = (F.bf16(rng, t, h, d) for h in (hq, hkv, hkv))
        cu_q = np.concatenate([[0], np.cumsum(new)])
        cu_k = np.concatenate([[0], np.cumsum(np.asarray(new) + done)])
        out = pkv.paged_prefill_varlen_fp8(q.to(cuda), k.to(cuda), v.to(cuda), *gpu, i32(cu_q),
                                           i32(cu_k), max(new), 60, bt, scale, status=st)
        kv, vv = ofp.decode_values(state[0], state[2]), ofp.decode_values(state[1], state[3])
        ref = oatt.paged_prefill_varlen(U.f64(q), U.f64(k), U.f64(v), kv, vv, cu_q, cu_k, tables,
                                        scale)
        tol = F.bound(ref, U.f64(q), np.full((1, d), 6.0), np.full((1, d), 6.0), scale,
                      F.PREFILL, 0)
        assert (np.abs(U.f64(out) - ref) <= tol).all()
        slots = slots_of(0, done[0], new[0]) + slots_of(1, done[1], new[1])
        pkv.kv_store_fp8(k.to(cuda), v.to(cuda), *gpu, i32(slots), status=st)
        state = ofp.kv_store(U.f64(k), U.f64(v), *state, slots)[:4]
        done = [a + n for a, n in zip(done, new)]
    for _ in range(4):
        q, k, v = (F.bf16(rng, 2, h, d) for h in (hq, hkv, hkv))
        slots = slots_of(0, done[0], 1) + slots_of(1, done[1], 1)
        done = [n + 1 for n in done]
        out = pkv.kv_store_paged_decode_fp8(k.to(cuda), v.to(cuda), i32(slots), q.to(cuda), *gpu,
                                            bt, i32(done), scale, 64, status=st)
        state = ofp.kv_store(U.f64(k), U.f64(v), *state, slots)[:4]
        kv, vv = ofp.decode_values(state[0], state[2]), ofp.decode_values(state[1], state[3])
        ref = oatt.paged_decode(U.f64(q), kv, vv, tables, done, scale)
        tol = F.bound(ref, U.f64(q), np.full((1, d), 6.0), np.full((1, d), 6.0), scale,
                      F.DECODE, 64)
        assert (np.abs(U.f64(out) - ref) <= tol).all()
        # the sampler's part of the step: every token but one forbidden or used up
        logits = torch.from_numpy(rng.normal(size=(2, vocab)).astype(np.float32)).to(cuda)
        want = rng.integers(0, vocab, 2)
        mask = np.zeros((2, -(-vocab // 32)), np.uint32)
        for b in range(2):
            mask[b, want[b] // 32] |= np.uint32(1 << (want[b] % 32))
        ruled = pkv.apply_logit_rules(logits, allowed_mask=torch.from_numpy(
            mask.view(np.int32)).to(cuda), status=st)
        ids = pkv.sample(ruled, torch.ones(2, device=cuda),
                         torch.ones((2, vocab), device=cuda), status=st)
        assert ids.tolist() == want.tolist()
    assert U.status_word(st) == 0
    for got, ref in zip(gpu[:2], state[:2]):
        np.testing.assert_array_equal(got.view(torch.uint8).cpu().numpy(), ref)


@pytest.mark.parametrize("bs", [16, 64])
def test_captured_step_replays(cuda, bs):
    """Store, decode and prefill captured in one graph, replayed with new
    contents, equal the eager calls; run on a side stream."""
    pkv = U.lib()
    rng = np.random.default_rng(21)
    lens = [bs + 1, 3 * bs, 7]
    pool = F.Pool(lens, bs, 2, 128, seed=6)
    args = pool.on(cuda)
    twin = [a.clone() for a in args]
    slots = torch.tensor([int(pool.bt[i, (n - 1) // bs]) * bs + (n - 1) % bs
                          for i, n in enumerate(lens)], dtype=torch.int32, device=cuda)
    ctx = torch.tensor(lens, dtype=torch.int32, device=cuda)
    cu_q = torch.tensor([0, 1, 3, 6], dtype=torch.int32, device=cuda)
    cu_k = torch.cumsum(torch.tensor([0] + [n + m for n, m in zip(lens, (1, 2, 3))]), 0).to(
        device=cuda, dtype=torch.int32)
    q, k, v = (torch.zeros((n, h, 128), dtype=torch.bfloat16, device=cuda)
               for n, h in ((6, 4), (6, 2), (6, 2)))

    def step(c, stream=None):
        a = pkv.kv_store_paged_decode_fp8(k[:3], v[:3], slots, q[:3], *c, ctx, 0.1, max(lens),
                                          stream=stream)
        b = pkv.paged_prefill_varlen_fp8(q, k, v, *c[:4], cu_q, cu_k, 3, max(lens) + 3, c[4], 0.1,
                                         stream=stream)
        return a, b

    def refill(seed):
        r = np.random.default_rng(seed)
        for t in (q, k, v):
            t.copy_(F.bf16(r, *t.shape))
    refill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = [a.clone() for a in args]
    torch.cuda.current_stream().synchronize()
    step(warm, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(args)
    for seed in (1, 2):
        refill(seed)
        graph.replay()
        want = step(twin)
        torch.cuda.synchronize()
        for x, y in zip(held, want):
            assert torch.equal(x, y)
        for x, y in zip(args, twin):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_random_cases(cuda):
    """Seeded random geometries of store, decode and prefill."""
    pkv = U.lib()
    rng = np.random.default_rng(99)
    for i in range(30):
        bs = int(rng.choice([1, 3, 8, 16, 20, 32, 64, 96, 128, 256]))
        hkv, group, d = (int(rng.choice(c)) for c in ([1, 2, 3, 8], [1, 2, 5, 8, 12], [64, 128]))
        lens = rng.integers(0, 400, int(rng.integers(1, 6))).tolist()
        pool = F.Pool(lens, bs, hkv, d, seed=1000 + i, spread=6, arbitrary=bool(i % 2))
        q = F.bf16(rng, len(lens), hkv * group, d, mag=2.0)
        out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda),
                                   torch.tensor(lens, dtype=torch.int32, device=cuda), 0.09,
                                   max(max(lens), 1))
        _check_decode(out, pool, q, 0.09)
        n = int(rng.choice([1, 9, 300, 2100]))
        slots = _store_case(rng, n, pool.codes["k"].shape[0], bs, hkv, d,
                            str(rng.choice(["runs", "shuffled"])))
        _run_store(pkv, cuda, F.bf16(rng, n, hkv, d), F.bf16(rng, n, hkv, d), pool, slots)


@pytest.mark.parametrize("bs,d", [(64, 128), (16, 128), (64, 64)])
def test_decode_gives_up_then_recovers(cuda, bs, d):
    """The split kernels' bounded waits run out: they report, let their copies
    and MMAs finish and return; the next call is the oracle's."""
    pkv = U.lib()
    rng = np.random.default_rng(31)
    lens = [700, 64, 1500, 1]
    pool = F.Pool(lens, bs, 2, d, seed=6)
    q = F.bf16(rng, 4, 8, d)
    args = (q.to(cuda), *pool.on(cuda), torch.tensor(lens, dtype=torch.int32, device=cuda), 0.1,
            1500)
    try:
        for polls in (0, 1, 2, 3, 5):
            pkv.set_wait_poll_limit(polls)
            st = pkv.new_status(cuda)
            pkv.paged_decode_fp8(*args, status=st)
            word = U.status_word(st)
            if polls == 0:
                assert word & pkv.STATUS["WAIT_TIMEOUT"]
            assert word & ~pkv.STATUS["WAIT_TIMEOUT"] == 0
    finally:
        pkv.set_wait_poll_limit()
    st = pkv.new_status(cuda)
    out = pkv.paged_decode_fp8(*args, status=st)
    assert U.status_word(st) == 0
    _check_decode(out, pool, q, 0.1)


@pytest.mark.parametrize("bs", [16, 256])
@pytest.mark.parametrize("group", [2, 4, 8])
def test_decode_many_stages_a_cta(cuda, bs, group):
    """Enough keys that every CTA's ring goes round several times; the call
    reports nothing (a wait at the kernel's end that ran out would)."""
    pkv = U.lib()
    rng = np.random.default_rng(41)
    nb, hkv, d, B = 8192 // bs * 4, 8, 128, 32
    kc = torch.randint(0, 127, (nb, bs, hkv, d), dtype=torch.uint8, device=cuda).view(
        torch.float8_e4m3fn)
    ks = torch.full((nb, hkv), 2.0 ** -9, device=cuda)
    bt = torch.from_numpy(np.stack([rng.permutation(nb)[:8192 // bs] for _ in range(B)]).astype(
        np.int32)).to(cuda)
    ctx = torch.from_numpy(rng.integers(6000, 8193, B).astype(np.int32)).to(cuda)
    q = F.bf16(rng, B, hkv * group, d).to(cuda)
    st = pkv.new_status(cuda)
    out = pkv.paged_decode_fp8(q, kc, kc, ks, ks, bt, ctx, 0.05, 8192, status=st)
    assert U.status_word(st) == 0
    # the same rows attended to through the bf16 decode (exact rows, another kernel)
    rows = (kc.float() * ks[:, None, :, None]).to(torch.bfloat16)
    ref = pkv.paged_decode(q, rows, rows, bt, ctx, 0.05, 8192)
    U.assert_close(U.f64(out), U.f64(ref), "fp8 against bf16 decode")


def _work(cuda, seed):
    """Calls that take every kernel: the list form of the store, a decode with a plan
    kernel and a combine, a prefill whose keys are split.  (inputs, call)"""
    pkv = U.lib()
    rng = np.random.default_rng(seed)
    hkv, d, bs = 2, 128, 16
    lens = [5000, 4600] + rng.integers(0, 60, 130).tolist()
    pool = F.Pool(lens, bs, hkv, d, seed=seed)
    cache = pool.on(cuda)
    n = 2300
    slots = torch.from_numpy(rng.permutation(pool.bt[0][:n // bs + 1])[:, None] * bs +
                             np.arange(bs)).flatten()[:n].to(cuda, torch.int32)
    x = [F.bf16(rng, n, hkv, d).to(cuda) for _ in "kv"]
    qd = F.bf16(rng, len(lens), 4, d).to(cuda)
    ctx = torch.tensor(lens, dtype=torch.int32, device=cuda)
    qp = F.bf16(rng, 150, 4, d).to(cuda)
    cu_q = torch.tensor([0, 130, 150], dtype=torch.int32, device=cuda)
    cu_k = torch.tensor([0, 5130, 9750], dtype=torch.int32, device=cuda)

    def call(c, stream=None):
        pkv.kv_store_fp8(*x, *c[:4], slots, stream=stream)
        a = pkv.paged_decode_fp8(qd, *c, ctx, 0.1, 5000, stream=stream)
        b = pkv.paged_prefill_varlen_fp8(qp, x[0][:150], x[1][:150], *c[:4], cu_q, cu_k, 130, 5130,
                                         c[4][:2].contiguous(), 0.1, stream=stream)
        return a, b
    return cache, call


def test_calls_on_two_streams_at_once(cuda):
    """Their scratch is their own: the results are those of one after the other."""
    work = [_work(cuda, s) for s in (1, 2)]
    want = []
    for cache, call in work:
        c = [t.clone() for t in cache]
        want.append((call(c), c))
    torch.cuda.synchronize()
    for _ in range(5):
        caches = [[t.clone() for t in cache] for cache, _ in work]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in work]
        got = [call(c, s) for (_, call), c, s in zip(work, caches, streams)]
        torch.cuda.synchronize()
        for g, c, (w, wc) in zip(got, caches, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))
            assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                       for x, y in zip(c, wc))


def test_captured_calls_replay_between_eager_ones(cuda):
    work = [_work(cuda, s) for s in (3, 4)]
    want = []
    for cache, call in work:
        c = [t.clone() for t in cache]
        want.append(call(c))
    graphs, held = [], []
    caches = [[t.clone() for t in cache] for cache, _ in work]
    torch.cuda.synchronize()
    for (_, call), c in zip(work, caches):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(call(c))
        graphs.append(g)
    for _ in range(3):
        for i in (0, 1):
            for x in held[i]:
                x.zero_()
            graphs[i].replay()
            eager = work[1 - i][1]([t.clone() for t in work[1 - i][0]])
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(held[i], want[i]))
            assert all(torch.equal(x, y) for x, y in zip(eager, want[1 - i]))


def test_split_prefill_infinities_and_nan(cuda):
    """As the unsplit kernel: a query's NaN or infinity is its head's alone."""
    pkv = U.lib()
    rng = np.random.default_rng(6)
    pool = F.Pool([4600], 64, 1, 128, seed=3)
    kc, vc, ks, vs, bt = pool.on(cuda)
    q = F.bf16(rng, 140, 2, 128).to(cuda)
    k = F.bf16(rng, 140, 1, 128).to(cuda)
    cu = [torch.tensor([0, n], dtype=torch.int32, device=cuda) for n in (140, 4740)]
    run = lambda: pkv.paged_prefill_varlen_fp8(  # noqa: E731
        q, k, k, kc, vc, ks, vs, *cu, 140, 4740, bt, 0.1)
    clean = run()
    q[3, 1, 0], q[131, 0, 77] = math.nan, math.inf
    out = run()
    touched = torch.zeros((140, 2), dtype=torch.bool, device=cuda)
    touched[3, 1] = touched[131, 0] = True
    assert torch.equal(out[~touched], clean[~touched])
    assert out[touched].isnan().all()


@pytest.mark.parametrize("bs", [16, 128])
def test_split_prefill_of_short_sequences(cuda, bs):
    """A stated maximum that asks for splits, and sequences that have none."""
    _prefill(U.lib(), cuda, [3, 200, 1], [50, 0, 700], bs, 1, 2, 64, seed=bs, max_k=100000, extra=2)
