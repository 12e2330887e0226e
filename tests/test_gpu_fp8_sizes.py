"""The 8-bit cache's calls at the ends of their sizes: nothing to do, many sequences, many heads."""
import numpy as np
import pytest
import torch

import fp8_util as F
import gpu_util as U
from oracle import attention as oatt
from oracle import fp8_cache as ofp

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def _check(got, q, pool, scale):
    kv, vv = pool.values("k"), pool.values("v")
    ref = oatt.paged_decode(U.f64(q), kv, vv, pool.bt, pool.lens, scale)
    tol = F.bound(ref, U.f64(q), kv, vv, scale, F.DECODE, max(pool.lens))
    assert (np.abs(U.f64(got) - ref) <= tol).all()


@pytest.mark.parametrize("B", [0, 3])
@pytest.mark.parametrize("n", [0, 2])
def test_store_and_decode_with_nothing_to_store_or_to_decode(cuda, B, n):
    pkv = U.lib()
    rng = np.random.default_rng(B + n)
    bs, hkv, d = 16, 2, 64
    pool = F.Pool([20, 0, 5], bs, hkv, d, seed=1)
    kc, vc, ks, vs, bt = pool.on(cuda)
    q, k, v = (F.bf16(rng, m, h, d) for m, h in ((B, 4), (n, hkv), (n, hkv)))
    slots = np.asarray([pool.bt[0, 1] * bs + 2, pool.bt[2, 0] * bs + 5][:n], np.int32)
    st = pkv.new_status(cuda)
    out = pkv.kv_store_paged_decode_fp8(k.to(cuda), v.to(cuda), _i32(slots, cuda), q.to(cuda), kc, vc,
                                        ks, vs, bt[:B].contiguous(), _i32(pool.lens[:B], cuda), 0.1,
                                        32, status=st)
    assert U.status_word(st) == 0 and out.shape == q.shape
    ref = ofp.kv_store(U.f64(k), U.f64(v), pool.codes["k"], pool.codes["v"], pool.scale["k"],
                       pool.scale["v"], slots)
    for got, want in zip((kc, vc), ref[:2]):
        np.testing.assert_array_equal(got.view(torch.uint8).cpu().numpy(), want)
    if B:
        pool.codes, pool.scale = {"k": ref[0], "v": ref[1]}, {"k": ref[2], "v": ref[3]}
        _check(out, q, pool, 0.1)


def test_decode_of_no_keys_at_all(cuda):
    pkv = U.lib()
    pool = F.Pool([0, 0], 64, 1, 128, seed=1)
    q = F.bf16(np.random.default_rng(0), 2, 4, 128).to(cuda)
    for most in (0, 1, 5000):
        st = pkv.new_status(cuda)
        out = pkv.paged_decode_fp8(q, *pool.on(cuda), _i32([0, 0], cuda), 0.1, most, status=st,
                                   out=torch.full_like(q, 7.0))
        assert U.status_word(st) == 0 and (out == 0).all()


@pytest.mark.parametrize("most", [40, 5000])             # without and with a combine
def test_decode_of_many_sequences(cuda, most):
    """More sequences than a grid's y extent; their tables share a few blocks."""
    pkv = U.lib()
    rng = np.random.default_rng(most)
    B, bs, d = 66000, 16, 64
    pool = F.Pool([40, 33, 7, 1, 0], bs, 1, d, seed=2)
    kind = rng.integers(0, 5, B)
    few = F.bf16(rng, 5, 2, d)
    q = few[torch.from_numpy(kind)].to(cuda)
    bt = pool.bt[kind]
    ctx = np.asarray(pool.lens)[kind]
    st = pkv.new_status(cuda)
    args = pool.on(cuda)[:4]
    width = torch.from_numpy(np.pad(bt, ((0, 0), (0, 40)), constant_values=-1)).to(cuda)
    out = pkv.paged_decode_fp8(q, *args, width, _i32(ctx, cuda), 0.1, most, status=st)
    assert U.status_word(st) == 0
    first = out[torch.from_numpy(np.asarray([np.nonzero(kind == i)[0][0] for i in range(5)]))]
    assert torch.equal(out, first[torch.from_numpy(kind).to(cuda)])
    _check(first, few, pool, 0.1)


@pytest.mark.parametrize("hkv,group,d", [(128, 1, 64), (1, 128, 128), (65, 3, 128), (1, 71, 64)])
@pytest.mark.parametrize("bs", [16, 64])
def test_many_heads(cuda, hkv, group, d, bs):
    pkv = U.lib()
    rng = np.random.default_rng(hkv)
    pool = F.Pool([150, 3], bs, hkv, d, seed=bs)
    cache = pool.on(cuda)
    for n in (3, 2100):
        slots = rng.integers(-1, pool.codes["k"].shape[0] * bs, n).astype(np.int32)
        k, v = F.bf16(rng, n, hkv, d), F.bf16(rng, n, hkv, d)
        pkv.kv_store_fp8(k.to(cuda), v.to(cuda), *cache[:4], _i32(slots, cuda))
        ref = ofp.kv_store(U.f64(k), U.f64(v), pool.codes["k"], pool.codes["v"], pool.scale["k"],
                           pool.scale["v"], slots)
        pool.codes, pool.scale = {"k": ref[0], "v": ref[1]}, {"k": ref[2].astype(np.float32),
                                                              "v": ref[3].astype(np.float32)}
        for got, want in zip(cache[:4], (pool.codes["k"], pool.codes["v"], pool.scale["k"],
                                         pool.scale["v"])):
            got = got.view(torch.uint8) if got.dtype == torch.float8_e4m3fn else got
            got = got.cpu().numpy()
            assert ((got == want) | ((got != got) if got.dtype == np.float32 else
                                     (got & 127 == 127) & (want & 127 == 127))).all()
    # blocks that a row at offset 0 began anew keep old rows' codes: attend to clean ones
    pool = F.Pool([150, 3], bs, hkv, d, seed=bs)
    q = F.bf16(rng, 2, hkv * group, d)
    out = pkv.paged_decode_fp8(q.to(cuda), *pool.on(cuda), _i32([150, 3], cuda), 0.1, 150)
    _check(out, q, pool, 0.1)


def test_prefill_of_nothing(cuda):
    pkv = U.lib()
    rng = np.random.default_rng(0)
    pool = F.Pool([20, 30], 16, 1, 64, seed=1)
    kc, vc, ks, vs, bt = pool.on(cuda)
    empty = F.bf16(rng, 0, 1, 64).to(cuda)
    st = pkv.new_status(cuda)
    for b in (0, 2):
        out = pkv.paged_prefill_varlen_fp8(F.bf16(rng, 0, 2, 64).to(cuda), empty, empty, kc, vc, ks,
                                           vs, _i32([0] * (b + 1), cuda),
                                           _i32([0, 20, 50][:b + 1], cuda), 0, 30,
                                           bt[:b].contiguous(), 0.1, status=st)
        assert out.shape == (0, 2, 64)
    assert U.status_word(st) == 0


def test_prefill_of_many_sequences(cuda):
    """More sequences than one group of the prefix pass takes: one query each on up to 20 cached
    keys, against the bf16 prefill of the same rows."""
    pkv = U.lib()
    rng = np.random.default_rng(5)
    B, bs, d = 66000, 16, 64
    pool = F.Pool([20, 16, 3, 0], bs, 1, d, seed=2)
    kind = rng.integers(0, 4, B)
    lp = np.asarray(pool.lens)[kind]
    q, k, v = (F.bf16(rng, B, h, d).to(cuda) for h in (2, 1, 1))
    cu_q = _i32(np.arange(B + 1), cuda)
    cu_k = _i32(np.concatenate([[0], np.cumsum(lp + 1)]), cuda)
    bt = torch.from_numpy(pool.bt[kind]).to(cuda)
    kc, vc, ks, vs, _ = pool.on(cuda)
    st = pkv.new_status(cuda)
    out = pkv.paged_prefill_varlen_fp8(q, k, v, kc, vc, ks, vs, cu_q, cu_k, 1, 21, bt, 0.1,
                                       status=st)
    rows = [(c.float() * s[:, None, :, None]).to(torch.bfloat16) for c, s in ((kc, ks), (vc, vs))]
    want = pkv.paged_prefill_varlen(q, k, v, *rows, cu_q, cu_k, 1, 21, bt, 0.1, status=st)
    assert U.status_word(st) == 0
    U.assert_close(U.f64(out), U.f64(want), "fp8 against bf16 prefill")


def test_captured_runs_of_one_plan(cuda):
    """Two graphs over one planned workspace, replayed in turn, and a plan for more sequences
    than a warp's own schedule holds."""
    pkv = U.lib()
    rng = np.random.default_rng(9)
    lens = [700] + rng.integers(0, 90, 150).tolist()
    pool = F.Pool(lens, 16, 2, 128, seed=3)
    args, ctx = pool.on(cuda), _i32(lens, cuda)
    ws = pkv.paged_decode_plan_fp8(ctx, 8, 700, args[4].shape[1], args[0])
    qs = [F.bf16(rng, len(lens), 8, 128).to(cuda) for _ in range(2)]
    want = [pkv.paged_decode_fp8(q, *args, ctx, 0.1, 700) for q in qs]
    graphs, held = [], []
    torch.cuda.synchronize()
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(pkv.paged_decode_run_fp8(q, *args, ctx, 0.1, 700, ws))
        graphs.append(g)
    for _ in range(3):
        for g, h, w in zip(graphs, held, want):
            h.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, w)
