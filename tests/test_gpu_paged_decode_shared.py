"""paged_decode_shared against the float64 oracle of paged_decode.

Bound, from the kernel's roundings.  q . K: bf16 products are exact in fp32; sums of at most
128 of them, each partial sum off by at most 2^-23 of the magnitudes summed (a tensor core may
cut instead of round).  With X = scale * max_j sum_d |q_d K_jd| the exponent is off by at most
128 * 2^-23 X, and by 4 * 2^-24 X from the fp32 steps behind it (the scale's product with
log2 e, the product and difference with the maximum).  P is rounded to bf16 for the product
with V, 2^-8 of itself (finfo.eps / 2 is 2^-8); the sum l takes the unrounded P; exp2 is good to 2^-22,
the parts' factors to as much.  The product with V sums n keys in fp32: 2^-23 n of the summed
magnitudes at most, n the keys a part sums, n <= 448 * 128 here and 2^-23 n A below 2^-7 A only in
theory; the sums run in an order that leaves far less, so 2^-23 * 512 A is taken for them.  The
result is rounded to bf16.  With A = max |V| over the keys:
    |out - ref| <= 2^-8 |ref| + A (2^-8 + 2 * (132 * 2^-23 X + 2^-21) + 512 * 2^-23)."""
import math

import numpy as np
import pytest
import torch

from gpu_util import f64, lib, status_word
from oracle import attention as oatt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Batch:
    """Groups of sequences over one pool; NaN in every slot that holds no token."""

    def __init__(self, sizes, prefixes, suffixes, hq, hkv, d, bs, dev, seed=0, mag=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.hq, self.d, self.scale = hq, d, 1 / math.sqrt(d)
        self.offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.prefix = np.asarray(prefixes, np.int32)
        B = int(sum(sizes))
        group = np.repeat(np.arange(len(sizes)), sizes)
        self.ctx = np.asarray([prefixes[group[b]] + suffixes[b] for b in range(B)], np.int32)
        whole = [p // bs for p in prefixes]          # blocks that are common as a whole
        nb = sum(whole) + sum(-(-int(c) // bs) - whole[group[b]]
                              for b, c in enumerate(self.ctx)) + spare
        perm = rng.permutation(nb).tolist()
        common = [[perm.pop() for _ in range(w)] for w in whole]
        width = max(1, max(-(-int(c) // bs) for c in self.ctx))
        self.bt = np.full((B, width), -1, np.int32)
        used = np.zeros((nb, bs), bool)
        self.k = rng.normal(size=(nb, bs, hkv, d)) * mag
        self.v = rng.normal(size=(nb, bs, hkv, d))
        for b in range(B):
            g, n = group[b], -(-int(self.ctx[b]) // bs)
            blocks = common[g] + [perm.pop() for _ in range(n - whole[g])]
            self.bt[b, :n] = blocks
            for i, blk in enumerate(blocks):
                used[blk, :min(bs, self.ctx[b] - i * bs)] = True
            # a prefix that ends inside a block: the members' own copies of its rows
            rest = prefixes[g] - whole[g] * bs
            if rest > 0 and b > self.offsets[g]:
                src = self.bt[self.offsets[g], whole[g]]
                for x in (self.k, self.v):
                    x[blocks[whole[g]], :rest] = x[src, :rest]
        self.k[~used], self.v[~used] = np.nan, np.nan
        self.q = rng.normal(size=(B, hq, d)) * mag
        t = lambda x: torch.from_numpy(x).to(BF).to(dev)  # noqa: E731
        self.tq, self.tk, self.tv = t(self.q), t(self.k), t(self.v)
        i = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
        self.tbt, self.tctx = i(self.bt), i(self.ctx)
        self.toff, self.tpre = i(self.offsets), i(self.prefix)
        self.max_ctx = int(self.ctx.max())

    def run(self, pkv, **kw):
        return pkv.paged_decode_shared(self.tq, self.tk, self.tv, self.tbt, self.tctx, self.toff,
                                       self.tpre, self.scale, self.max_ctx, **kw)

    def check(self, got):
        ref = oatt.paged_decode(f64(self.tq), self.tk.cpu(), self.tv.cpu(), self.bt, self.ctx,
                                self.scale)
        q, k, v = np.abs(f64(self.tq)), np.abs(f64(self.tk)), np.abs(f64(self.tv))
        kmax = np.nanmax(k.reshape(-1, self.d), 0)
        x = self.scale * (q * kmax).sum(-1).max()
        a = np.nanmax(v)
        bound = 2.0 ** -8 * np.abs(ref) + a * (2.0 ** -8 + 2 * (132 * 2.0 ** -23 * x + 2.0 ** -21) +
                                               512 * 2.0 ** -23)
        err = np.abs(f64(got) - ref)
        assert (err <= bound).all(), float((err / bound).max())
        rel = np.linalg.norm(f64(got) - ref) / max(np.linalg.norm(ref), 1e-30)
        assert rel <= 5e-3, rel


CASES = [  # sizes, prefixes, suffixes (or a bound for random ones), hq, hkv, d, block size
    ([2], [1000], [1, 30], 16, 8, 128, 256),
    ([1], [0], [1], 1, 1, 64, 16),                      # one sequence, one key
    ([3], [64], [0, 0, 1], 2, 1, 64, 8),                # nothing but the prefix
    ([5], [256], 300, 4, 2, 128, 16),
    ([64], [512], 200, 16, 8, 128, 256),                # one row tile
    ([70], [640], 150, 16, 8, 128, 64),                 # a pair of row tiles, one sequence over
    ([40], [384], 40, 32, 2, 64, 128),                  # 5 row tiles of 8 sequences
    ([9, 1, 20, 2], [200, 300, 77, 1024], 130, 14, 2, 128, 1),       # G 7, gathered rows
    ([6, 7], [100, 90], 64, 6, 2, 64, 20),              # gathered, prefixes inside a block
    ([6, 7], [100, 90], 64, 6, 2, 128, 24),             # boxes of 24, tiles of 120
    ([4, 4], [130, 260], 90, 5, 1, 64, 48),
    ([3, 5], [777, 300], 900, 8, 1, 128, 192),
    ([2, 2], [500, 129], 260, 40, 40, 64, 40),
    ([2, 3], [200, 300], 50, 160, 1, 64, 16),           # more than 128 heads a kv head
    ([4], [136], 40, 3, 3, 128, 136),
    ([30] + [1] * 8 + [12], [1280] + [50] * 8 + [640], 400, 32, 8, 128, 16),
    # several items a CTA, whole row tiles and single sequences in turn
    ([24] * 4, [300, 200, 700, 65], 150, 16, 8, 64, 20),
    ([30] * 2, [300, 500], 100, 16, 8, 128, 12),
    ([24] * 4, [300, 200, 700, 65], 150, 16, 8, 64, 16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_oracle(cuda, case):
    pkv = lib()
    sizes, prefixes, suffixes, hq, hkv, d, bs = CASES[case]
    if isinstance(suffixes, int):
        suffixes = np.random.default_rng(case).integers(0, suffixes + 1, sum(sizes)).tolist()
    b = Batch(sizes, prefixes, suffixes, hq, hkv, d, bs, cuda, seed=case)
    st = pkv.new_status(cuda)
    got = b.run(pkv, status=st)
    assert status_word(st) == 0
    b.check(got)


def test_sharp_scores(cuda):
    """Scores that spread over hundreds: maxima that rise from tile to tile and parts far apart."""
    pkv = lib()
    b = Batch([20, 3], [700, 300], [120] * 23, 8, 2, 128, 16, cuda, seed=3, mag=6.0)
    order = torch.arange(b.tk.shape[0] * 16, device=cuda).view(-1, 16, 1, 1)
    b.tk *= (1 + (order % 37).to(BF) / 8)
    for g, p in enumerate((700, 300)):         # the members' copies of a common row stay alike
        first, last = b.offsets[g], b.offsets[g + 1]
        rows = b.tk[int(b.bt[first, p // 16]), :p % 16].clone()
        for i in range(first, last):
            b.tk[int(b.bt[i, p // 16]), :p % 16] = rows
    b.check(b.run(pkv))


def test_no_groups_is_paged_decode(cuda):
    pkv = lib()
    b = Batch([7], [0], [1, 127, 128, 129, 500, 0, 1000], 8, 2, 128, 64, cuda, seed=4)
    b.check(b.run(pkv))
    got = pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, b.tctx, None, None, b.scale, b.max_ctx)
    b.check(got)
    assert (got[5] == 0).all()


def test_plan_and_runs_over_layers(cuda):
    """One schedule for several layers, as often as wanted; a workspace of its own size is enough."""
    pkv = lib()
    b = Batch([33, 2], [900, 130], [77] * 35, 8, 2, 128, 16, cuda, seed=5)
    ws = torch.empty(pkv.paged_decode_shared_workspace_bytes(35, 8, b.max_ctx, b.tk),
                     dtype=torch.uint8, device=cuda)
    st = pkv.new_status(cuda)
    got = pkv.paged_decode_plan_shared(b.tctx, b.toff, b.tpre, 8, b.max_ctx, b.tbt.shape[1], b.tk,
                                       workspace=ws, status=st)
    assert got is ws
    one = pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws, status=st)
    b.check(one)
    two = pkv.paged_decode_run_shared(b.tq, b.tv, b.tk, b.tbt, b.scale, b.max_ctx, ws)
    three = pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws)
    assert torch.equal(one, three) and not torch.equal(one, two)
    assert torch.equal(one, b.run(pkv))
    assert status_word(st) == 0


def test_bad_lengths_groups_and_blocks(cuda):
    pkv = lib()
    b = Batch([4, 3, 2], [256, 128, 0], [100] * 9, 4, 2, 64, 16, cuda, seed=6)
    good = b.run(pkv)
    S = pkv.STATUS

    def run(**kw):
        t = {k: getattr(b, k).clone() for k in ("tctx", "toff", "tpre", "tbt")}
        for k, f in kw.items():
            f(t[k])
        st = pkv.new_status(cuda)
        got = pkv.paged_decode_shared(b.tq, b.tk, b.tv, t["tbt"], t["tctx"], t["toff"], t["tpre"],
                                      b.scale, b.max_ctx, status=st)
        return got, status_word(st)

    def put(i, v):
        def f(t):
            t.view(-1)[i] = v
        return f
    # a member shorter than its prefix, negative, too long: zeros; an empty one: zeros, no report
    for n, bit in ((200, S["BAD_CONTEXT_LEN"]), (-1, S["BAD_CONTEXT_LEN"]),
                   (b.max_ctx + 1, S["BAD_CONTEXT_LEN"]), (0, 0)):
        for i in (0, 2):                                 # a group's first member too
            got, st = run(tctx=put(i, n))
            assert st == bit and (got[i] == 0).all()
            keep = [j for j in range(9) if j != i]
            assert torch.equal(got[keep], good[keep])
    # every member empty
    got, st = run(tctx=lambda t: t[:4].zero_())
    assert st == 0 and (got[:4] == 0).all()
    # offsets that decrease, or leave the batch: no group is used, the result is the same
    for i, v in ((1, 8), (3, 10), (0, -1), (2, 2**31 - 1)):
        got, st = run(toff=put(i, v))
        assert st == S["BAD_SEQLENS"]
        b.check(got)
    for v in (-5, b.max_ctx + 1, 2**31 - 1):             # a bad prefix counts as 0
        got, st = run(tpre=put(0, v))
        assert st == S["BAD_SEQLENS"]
        b.check(got)
    # sequences before the first and behind the last group
    got, st = run(toff=lambda t: t.copy_(torch.tensor([1, 4, 7, 8], dtype=torch.int32)))
    assert st == 0
    b.check(got)
    # a block outside the pool: its keys are left out
    for v in (-1, b.tk.shape[0], 2**31 - 1):
        got, st = run(tbt=put(4 * b.bt.shape[1] + 10, v))      # own block of sequence 4
        assert st == S["BAD_BLOCK_ID"]
        keep = [j for j in range(9) if j != 4]
        assert torch.equal(got[keep], good[keep]) and got[4].isfinite().all()
        own_keys = [k for k in range(int(b.ctx[4])) if k // 16 != 10]
        q = f64(b.tq)[4]
        rows = [(b.bt[4, k // 16], k % 16) for k in own_keys]
        kk = np.stack([f64(b.tk[r, o]) for r, o in rows])
        vv = np.stack([f64(b.tv[r, o]) for r, o in rows])
        for h in range(4):
            w = np.exp((kk[:, h // 2] @ q[h]) * b.scale)
            ref = (w[:, None] * vv[:, h // 2]).sum(0) / w.sum()
            assert np.abs(f64(got[4, h]) - ref).max() <= 2.0 ** -8 * (np.abs(ref).max() +
                                                                     2 * np.abs(vv).max())


def test_infinite_and_nan_queries(cuda):
    pkv = lib()
    b = Batch([40], [300], [50] * 40, 4, 2, 64, 16, cuda, seed=7)
    good = b.run(pkv)
    b.tq[3, 1, 5] = float("nan")
    b.tq[38, 2, 0] = float("inf")
    got = b.run(pkv)
    assert got[3, 1].isnan().all() and got[38, 2].isnan().all()
    mask = torch.ones_like(got, dtype=torch.bool)
    mask[3, 1] = mask[38, 2] = False
    assert torch.equal(got[mask], good[mask])


def test_output_alignment_streams_and_capture(cuda):
    pkv = lib()
    b = Batch([20, 1, 5], [512, 30, 200], [70] * 26, 16, 4, 128, 16, cuda, seed=8)
    ref = b.run(pkv)
    store = torch.empty(ref.numel() + 8, dtype=BF, device=cuda)
    out = store[8:].view(ref.shape)                      # 16-byte aligned only
    assert out.data_ptr() % 32 == 16 and torch.equal(b.run(pkv, out=out), ref)
    one = Batch([2], [0], [60, 90], 16, 4, 128, 16, cuda, seed=9)          # direct results
    ref1 = one.run(pkv)
    out = store[8:8 + ref1.numel()].view(ref1.shape)
    assert torch.equal(one.run(pkv, out=out), ref1)
    # two calls at once, on two streams
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [(b.run(pkv), b.run(pkv, stream=side)) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref) for pair in got for x in pair)
    # two graphs of one workspace, replayed with other lengths
    ws = torch.empty(pkv.paged_decode_shared_workspace_bytes(26, 16, b.max_ctx, b.tk),
                     dtype=torch.uint8, device=cuda)
    outs, graphs = [torch.empty_like(ref) for _ in range(2)], []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            b.run(pkv, out=o, workspace=ws)
    b.tctx -= 40
    b.ctx = b.ctx - 40
    b.tpre[1] = 0
    for g in (0, 1, 0):
        graphs[g].replay()
        b.check(outs[g])
        assert torch.equal(outs[g], b.run(pkv))


def test_a_step_of_a_layer(cuda):
    """Norms, rotation and cache write of a step's new tokens, then attention over groups that
    share their prompts: against the oracles, over a cache written by the same call."""
    from oracle import head_rotation as ohr
    pkv = lib()
    rng = np.random.default_rng(11)
    hq, hkv, d, bs = 8, 2, 64, 16
    b = Batch([5, 4], [160, 96], [33] * 9, hq, hkv, d, bs, cuda, seed=12)
    x = torch.from_numpy(rng.normal(size=(9, hq + 2 * hkv, d))).to(BF).to(cuda)
    q, k, v = x.split((hq, hkv, hkv), 1)
    w = torch.from_numpy(1 + 0.2 * rng.normal(size=d)).to(BF).to(cuda)
    pos = b.ctx - 1
    slots = np.asarray([b.bt[i, p // bs] * bs + p % bs for i, p in enumerate(pos)], np.int32)
    st = pkv.new_status(cuda)
    rope = pkv.rotary(d, base=1e6)
    ws = pkv.paged_decode_plan_shared(b.tctx, b.toff, b.tpre, hq, b.max_ctx, b.tbt.shape[1], b.tk,
                                      status=st)
    b.tq = pkv.qk_norm_rope_kv_store(q, k, v, w, w, 1e-6, torch.from_numpy(pos).to(cuda), rope,
                                     b.tk, b.tv, torch.from_numpy(slots).to(cuda), status=st)
    got = pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws, status=st)
    assert status_word(st) == 0
    freq, _ = ohr.frequencies(d, 1e6)
    for have, rows in ((b.tq, q), (b.tk.view(-1, hkv, d)[torch.from_numpy(slots).long()
                                                         .to(cuda)], k)):
        ref = ohr.norm_rope(f64(rows), f64(w), 1e-6, pos, freq)
        # bf16's rounding, and fp32's steps (see test_gpu_qk_norm_rope.py) of two entries
        assert (np.abs(f64(have) - ref) <= 2.0 ** -8 * np.abs(ref) +
                24 * 2.0 ** -24 * 2 * np.abs(ref).max()).all()
    b.check(got)
    # the same by the other operators of the framework
    other = pkv.paged_decode(b.tq, b.tk, b.tv, b.tbt, b.tctx, b.scale, b.max_ctx)
    assert (got.float() - other.float()).abs().max() <= 2e-2


def test_waits_that_run_out_are_reported(cuda):
    """With no polls every wait gives up at once: the call unwinds, and the next one is right."""
    pkv = lib()
    for d, bs in ((128, 16), (64, 20)):
        b = Batch([40, 3], [300, 200], [90] * 43, 8, 2, d, bs, cuda, seed=13)
        ref = b.run(pkv)
        ws = pkv.paged_decode_plan_shared(b.tctx, b.toff, b.tpre, 8, b.max_ctx, b.tbt.shape[1],
                                          b.tk)
        st = pkv.new_status(cuda)
        pkv.set_wait_poll_limit(0)
        try:
            pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws,
                                        status=st)
        finally:
            pkv.set_wait_poll_limit()
        assert status_word(st) & pkv.STATUS["WAIT_TIMEOUT"]
        got = pkv.paged_decode_run_shared(b.tq, b.tk, b.tv, b.tbt, b.scale, b.max_ctx, ws)
        assert torch.equal(got, ref)


PLANS = {  # what the one CTA of the plan does in turns, and runs whose length has a bound
    "1300 sequences": ([600, 700], [128, 70], 60, 2, 1, 64, 16),
    "400 sequences": ([390, 10], [130, 256], 40, 2, 1, 64, 16),
    "1160 groups": ([1] * 1100 + [2] * 60, [70] * 1160, 50, 2, 1, 64, 16),
    "1160 groups, gathered": ([1] * 500 + [3] * 660, [70] * 1160, 30, 2, 1, 64, 5),
    "long own keys": ([1, 2], [500, 100], [30000, 9000, 17000], 2, 1, 64, 16),
    "many rows, no room for short runs": ([40], [6400], 30, 128, 1, 64, 128),
    "two groups of more rows": ([13, 27], [3200, 5000], 30, 128, 1, 64, 64),
}


@pytest.mark.parametrize("name", PLANS)
def test_plans(cuda, name):
    pkv = lib()
    sizes, prefixes, suffixes, hq, hkv, d, bs = PLANS[name]
    if isinstance(suffixes, int):
        suffixes = np.random.default_rng(1).integers(0, suffixes + 1, sum(sizes)).tolist()
    b = Batch(sizes, prefixes, suffixes, hq, hkv, d, bs, cuda, seed=20)
    st = pkv.new_status(cuda)
    got = b.run(pkv, status=st)
    assert status_word(st) == 0
    b.check(got)
    assert torch.equal(got, b.run(pkv))


def test_nothing_to_attend_and_empty_groups(cuda):
    pkv = lib()
    b = Batch([3], [100], [20, 0, 7], 4, 2, 64, 16, cuda, seed=30)
    zero = torch.zeros(3, dtype=torch.int32, device=cuda)
    st = pkv.new_status(cuda)
    for max_len in (0, b.max_ctx):
        got = pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, zero, b.toff, zero[:1], b.scale,
                                      max_len, status=st)
        assert (got == 0).all() and status_word(st) == 0
    e = pkv.paged_decode_shared(b.tq[:0], b.tk, b.tv, b.tbt[:0], b.tctx[:0], b.toff[:1],
                                b.tpre[:0], b.scale, b.max_ctx, status=st)
    assert e.shape == (0, 4, 64)
    # groups without sequences, a group of one, the rest without a group
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    for off, pre in ((i(0, 0, 3, 3), i(50, 100, 7)), (i(0, 0, 1, 1), i(9, 100, 120)),
                     (i(3, 3), i(100)), (i(1, 3), i(100))):
        b.check(pkv.paged_decode_shared(b.tq, b.tk, b.tv, b.tbt, b.tctx, off, pre, b.scale,
                                        b.max_ctx, status=st))
        assert status_word(st) == 0
