"""apply_logit_rules on the GPU against the float64 oracle.

Bound of an entry: the repetition product (a quotient is a product with a
rounded inverse: two roundings), f * n + p, its subtraction and the bias are at
most five fp32 roundings, each off by at most 2^-24 of a value no larger than the
sum of the magnitudes that went in (the oracle's second result); logits of any
type are exact in fp32.  A sixth covers their products."""
import math

import numpy as np
import pytest
import torch

import gpu_util as U
from oracle import logit_rules as olr

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _case(seed, B, V, T, bias, mask, dtype="fp32", pad=0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(B, V + pad)).astype(np.float32) * 3).to(TYPES[dtype])
    c = {"logits": x[:, :V]}
    if T:
        c["token_ids"] = rng.integers(0, max(1, V // 3), (B, T)).astype(np.int32)
        c["token_lens"] = rng.integers(0, T + 1, B).astype(np.int32)
        c["token_lens"][0] = T
        c["prompt_lens"] = (c["token_lens"] * rng.uniform(0, 1, B)).astype(np.int32)
        c["repetition"] = rng.choice([1.0, 1.2, 0.8, 2.0], B).astype(np.float32)
        c["presence"] = rng.choice([0.0, 0.5, -1.0], B).astype(np.float32)
        c["frequency"] = rng.choice([0.0, 0.3, -0.1], B).astype(np.float32)
    if bias:
        n = rng.integers(0, bias + 1, B)
        c["bias_offsets"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        total = int(n.sum())
        c["bias_ids"] = rng.integers(0, max(1, V // 2), total).astype(np.int32)   # repeats
        c["bias_values"] = rng.normal(0, 5, total).astype(np.float32)
    if mask:
        m = rng.integers(0, 2 ** 32, (B, -(-V // 32)), dtype=np.uint64).astype(np.uint32)
        if V % 32:
            m[:, -1] &= np.uint32((1 << (V % 32)) - 1)
        m[0, 0] |= np.uint32(1)
        if B > 1:
            m[1] = 0xFFFFFFFF
        c["allowed_mask"] = m
    return c


NAMES = {"repetition": "repetition_penalties", "presence": "presence_penalties",
         "frequency": "frequency_penalties", "bias_ids": "bias_token_ids"}


def _args(c, dev):
    out = {}
    for k, v in c.items():
        if k != "logits":
            v = v.view(np.int32) if v.dtype == np.uint32 else v
            out[NAMES.get(k, k)] = torch.from_numpy(v).to(dev)
    return out


def _logits(c, dev):
    """On the GPU with the case's row stride."""
    x = c["logits"]
    wide = torch.empty((x.shape[0], x.stride(0)), dtype=x.dtype, device=dev)
    view = wide[:, :x.shape[1]]
    view.copy_(x)
    return view


def _check(got, c):
    ref, spread = olr.apply(U.f64(c["logits"]), **{k: v for k, v in c.items() if k != "logits"})
    got = U.f64(got)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(ref))
    fine = np.isfinite(ref)
    assert np.isfinite(got[fine]).all()
    assert (np.abs(got[fine] - ref[fine]) <= 6 * 2.0 ** -24 * spread[fine]).all()


@pytest.mark.parametrize("B,V,T,bias,mask", [
    (1, 1, 1, 1, True), (3, 31, 5, 0, True), (2, 32, 0, 0, True), (4, 33, 40, 6, True),
    (2, 1000, 300, 20, False), (5, 1024, 0, 9, False), (3, 1028, 64, 0, False),
    (2, 2051, 77, 30, True), (300, 64, 9, 2, True), (2, 300, 1500, 3, True),
])
@pytest.mark.parametrize("dtype,pad", [("fp32", 0), ("fp32", 3), ("bf16", 0), ("bf16", 8),
                                       ("fp16", 1)])
def test_rules_are_the_oracles(cuda, B, V, T, bias, mask, dtype, pad):
    pkv = U.lib()
    c = _case(B * 1000 + V + T, B, V, T, bias, mask, dtype, pad)
    st = pkv.new_status(cuda)
    out = pkv.apply_logit_rules(_logits(c, cuda), **_args(c, cuda), status=st)
    assert U.status_word(st) == 0 and out.is_contiguous() and out.dtype == torch.float32
    _check(out, c)


@pytest.mark.parametrize("V", [*range(1, 24), 8191, 8193, 9217])
@pytest.mark.parametrize("dtype,skew,pad", [("fp32", 0, 0), ("fp32", 1, 2), ("fp32", 3, 5),
                                            ("bf16", 5, 0), ("bf16", 0, 3), ("fp16", 7, 1)])
def test_rows_anywhere_in_their_16_bytes(cuda, V, dtype, skew, pad):
    """Rows of logits and of out that begin at every offset from 16 bytes, alike or not:
    what lies around them is neither written nor read into the result."""
    pkv = U.lib()
    B = 9 if V < 1000 else 2
    c = _case(V + skew, B, V, 12 if V < 1000 else 3, 3, V % 2 == 1, dtype, 0)
    stride = V + pad
    room = torch.full((skew + B * stride + 16,), math.nan, dtype=TYPES[dtype], device=cuda)
    logits = room[skew:skew + B * stride].view(B, stride)[:, :V]
    logits.copy_(c["logits"])
    for lead in range(4):
        wide = torch.full((lead + B * V + 8,), 7.0, device=cuda)
        out = wide[lead:lead + B * V].view(B, V)
        st = pkv.new_status(cuda)
        pkv.apply_logit_rules(logits, **_args(c, cuda), out=out, status=st)
        assert U.status_word(st) in (0, pkv.STATUS["NO_ALLOWED_TOKEN"])
        _check(out, c)
        assert (wide[:lead] == 7.0).all() and (wide[lead + B * V:] == 7.0).all()


@pytest.mark.parametrize("T", [32766, 32767, 32768, 70000])
@pytest.mark.parametrize("V,dtype", [(72, "fp32"), (73, "fp32"), (72, "bf16")])
def test_long_histories(cuda, T, V, dtype):
    """Nearly every generated token is the same, next to entries with prompt tokens,
    single ones and none: counts up to and beyond what 16 bits hold."""
    pkv = U.lib()
    rng = np.random.default_rng(T)
    ids = np.stack([np.full(T, 40), np.full(T, 41), np.full(T, V - 1)]).astype(np.int32)
    ids[:, :4] = [42, 39, 5, V - 2]
    ids[:, -1] = 38
    x = torch.from_numpy(rng.normal(size=(3, V)).astype(np.float32)).to(TYPES[dtype])
    c = {"logits": x, "token_ids": ids, "token_lens": np.full(3, T, np.int32),
         "prompt_lens": np.asarray([4, 0, 2], np.int32),
         "repetition": np.asarray([1.5, 1.0, 0.7], np.float32),
         "presence": np.asarray([0.25, 0.5, 0.0], np.float32),
         "frequency": np.asarray([0.001, 0.01, 0.3], np.float32)}
    st = pkv.new_status(cuda)
    out = pkv.apply_logit_rules(x.to(cuda), **_args(c, cuda), status=st)
    assert U.status_word(st) == 0
    _check(out, c)


@pytest.mark.parametrize("V", [9000, 9003, 40000])
def test_several_segments_of_a_row(cuda, V):
    """Rows of more than one CTA's segment, tokens near every segment's edge
    (checked where the history, the biases and the mask reach)."""
    pkv = U.lib()
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.normal(size=(2, V)).astype(np.float32))
    edges = np.asarray(sorted({0, V - 1, *(e + d for e in range(1024, V, 1024)
                                           for d in (-1, 0, 1))}), np.int32)
    ids = np.stack([edges, np.roll(edges, 3)]).astype(np.int32)
    args = {"token_ids": ids, "repetition_penalties": np.full(2, 1.5, np.float32),
            "bias_offsets": np.asarray([0, len(edges), 2 * len(edges)], np.int32),
            "bias_token_ids": np.concatenate([edges, edges[::-1]]),
            "bias_values": np.ones(2 * len(edges), np.float32)}
    mask = np.full((2, -(-V // 32)), 0xFFFFFFFF, np.uint32)
    mask[0, 1], mask[1, -1] = 0, 0
    out = pkv.apply_logit_rules(x.to(cuda), **{k: torch.from_numpy(v).to(cuda)
                                               for k, v in args.items()},
                                allowed_mask=torch.from_numpy(mask.view(np.int32)).to(cuda))
    want = x.double().numpy()
    for b in range(2):
        w = want[b, edges]
        want[b, edges] = np.where(w > 0, w / 1.5, w * 1.5) + 1
    want[0, 32:64] = -math.inf
    want[1, (V - 1) // 32 * 32:] = -math.inf
    got = U.f64(out)
    np.testing.assert_array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= 4 * 2.0 ** -24 * (np.abs(want[fine]) + 2)).all()


@pytest.mark.parametrize("V", [96, 97, 20000])
@pytest.mark.parametrize("what", ["penalties", "mask", "bias", "all", "none"])
def test_in_place_is_out_of_place(cuda, V, what):
    pkv = U.lib()
    every = what == "all"
    c = _case(V, 3, V, 50 if every or what == "penalties" else 0,
              7 if every or what == "bias" else 0, every or what == "mask")
    x = c["logits"].to(cuda).contiguous()
    want = pkv.apply_logit_rules(x, **_args(c, cuda))
    got = pkv.apply_logit_rules(x, **_args(c, cuda), out=x)
    assert got is x and torch.equal(got, want)


def test_special_values(cuda):
    """Infinities and NaN in the logits, masked and not; the type's lowest value."""
    pkv = U.lib()
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[math.inf, -math.inf, math.nan, low, 1.0, math.nan, math.inf, low]],
                     device=cuda)
    mask = torch.tensor([[0b00011111]], dtype=torch.int32, device=cuda)
    out = pkv.apply_logit_rules(
        x, token_ids=torch.tensor([[0, 1, 2, 3, 3]], dtype=torch.int32, device=cuda),
        repetition_penalties=torch.tensor([2.0], device=cuda),
        frequency_penalties=torch.tensor([0.5], device=cuda),
        bias_offsets=torch.tensor([0, 2], dtype=torch.int32, device=cuda),
        bias_token_ids=torch.tensor([4, 5], dtype=torch.int32, device=cuda),
        bias_values=torch.tensor([math.inf, math.inf], device=cuda), allowed_mask=mask)[0].tolist()
    assert out[0] == math.inf and out[1] == -math.inf and math.isnan(out[2])
    assert out[3] == -math.inf                   # low * 2
    assert out[4] == math.inf
    assert out[5:] == [-math.inf] * 3            # masked: whatever was there


def test_status_bits_and_what_is_left_out(cuda):
    pkv = U.lib()
    x = torch.zeros((2, 64), device=cuda) + 1.0
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda)  # noqa: E731
    f32 = lambda v: torch.tensor(v, device=cuda)  # noqa: E731

    def run(**kw):
        st = pkv.new_status(cuda)
        out = pkv.apply_logit_rules(x, status=st, **kw)
        return out.cpu(), U.status_word(st)
    S = pkv.STATUS
    # ids: padding below 0 is skipped, one past the vocabulary reported
    out, st = run(token_ids=i32([[5, -1, -7], [6, 64, 2 ** 31 - 1]]),
                  repetition_penalties=f32([2.0, 2.0]))
    assert st == S["BAD_TOKEN_ID"]
    assert (out != 1).sum() == 2 and out[0, 5] == 0.5 and out[1, 6] == 0.5
    out, st = run(bias_offsets=i32([0, 2, 3]), bias_token_ids=i32([-1, 3, 64]),
                  bias_values=f32([9.0, 9.0, 9.0]))
    assert st == S["BAD_TOKEN_ID"] and (out != 1).sum() == 1 and out[0, 3] == 10.0
    # lengths
    for kw in ({"token_lens": [4, 3]}, {"token_lens": [-1, 3]}, {"prompt_lens": [4, 0]},
               {"prompt_lens": [-1, 0]}, {"token_lens": [1, 3], "prompt_lens": [2, 0]}):
        out, st = run(token_ids=i32([[1, 2, 3], [1, 2, 3]]), presence_penalties=f32([0.5, 0.5]),
                      **{k: i32(v) for k, v in kw.items()})
        assert st == S["BAD_SEQLENS"] and (out[0] == 1).all() and (out[1, 1:4] == 0.5).all()
    for off in ([-1, 1, 1], [2, 1, 1], [0, 4, 3]):
        out, st = run(bias_offsets=i32(off), bias_token_ids=i32([1, 2, 3]),
                      bias_values=f32([1.0, 1.0, 1.0]))
        assert st == S["BAD_SEQLENS"] and (out[0] == 1).all()
    # penalties
    for name, bad in (("repetition_penalties", [0.0, -1.0, 1e-31, 1e31, math.inf, math.nan]),
                      ("presence_penalties", [math.inf, math.nan]),
                      ("frequency_penalties", [-math.inf, math.nan])):
        for v in bad:
            out, st = run(token_ids=i32([[1], [1]]), **{name: f32([v, 0.5])})
            assert st == S["BAD_PENALTY"] and (out[0] == 1).all() and out[1, 1] != 1
    # a row whose mask leaves nothing (bits past the vocabulary do not count)
    y = x[:, :40].contiguous()
    mask = i32([[0, 1 << 8], [0, 1]])
    st = pkv.new_status(cuda)
    out = pkv.apply_logit_rules(y, allowed_mask=mask, status=st).cpu()
    assert U.status_word(st) == S["NO_ALLOWED_TOKEN"]
    assert torch.isneginf(out[0]).all() and (~torch.isneginf(out[1])).sum() == 1


def test_graph_and_side_stream(cuda):
    pkv = U.lib()
    c = _case(5, 4, 5000, 200, 10, True)
    args, x = _args(c, cuda), c["logits"].to(cuda)
    want = pkv.apply_logit_rules(x, **args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pkv.apply_logit_rules(x, **args, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = pkv.apply_logit_rules(x, **args)
    x.mul_(2)
    graph.replay()
    assert torch.equal(held, pkv.apply_logit_rules(x, **args))


def test_empty_batch_and_many_rows(cuda):
    pkv = U.lib()
    assert pkv.apply_logit_rules(torch.zeros((0, 50), device=cuda)).shape == (0, 50)
    x = torch.arange(70000, device=cuda, dtype=torch.float32)[:, None] + torch.zeros(1, 4,
                                                                                     device=cuda)
    lens = (torch.arange(70000, device=cuda, dtype=torch.int32) % 2).contiguous()
    out = pkv.apply_logit_rules(x, token_ids=torch.full((70000, 1), 2, dtype=torch.int32,
                                                        device=cuda), token_lens=lens,
                                presence_penalties=torch.ones(70000, device=cuda))
    want = x.clone()
    want[:, 2] -= lens.float()
    assert torch.equal(out, want)
