"""Cases for an 8-bit paged KV cache and for the logit rules in front of the sampler.

Four operators of one serving step, each in its plain form and as the
library's call:

  store    K/V rows quantised to e4m3 into a paged cache with one scale for
           each (cache block, kv head)
  decode   one query per sequence against that cache
  prefill  causal varlen chunks whose prefix lies in that cache
  rules    repetition / presence / frequency penalties, biases and an
           allowed-token mask on a step's logits

Lengths are the same set for every seed of a case (work depends on the case
alone); their order, the block tables and all values come from the seed.
"""
import math

import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
SCALE_EXP_LO, SCALE_EXP_HI = -64, 119
LOGIT_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # the cache write of one decode step: one new token per running sequence
        {"name": "store-step", "op": "store", "seqs": 512, "lo": 1, "hi": 1, "hkv": 8, "d": 128,
         "bs": 256, "pad": 0},
        # the cache write of a full prefill round (16384 tokens of 16 prompts)
        {"name": "store-chunk", "op": "store", "seqs": 16, "lo": 512, "hi": 1536, "hkv": 8,
         "d": 128, "bs": 256, "pad": 0},
        # a single user's next token
        {"name": "decode-one", "op": "decode", "batch": 1, "hq": 16, "hkv": 8, "d": 128,
         "bs": 256, "lo": 1000, "hi": 1000, "log": False},
        # a small model's decode step at a moderate batch
        {"name": "decode-64", "op": "decode", "batch": 64, "hq": 16, "hkv": 8, "d": 128,
         "bs": 256, "lo": 512, "hi": 4096, "log": False},
        # a large model's decode step, contexts spread from short to very long
        {"name": "decode-long", "op": "decode", "batch": 96, "hq": 64, "hkv": 8, "d": 128,
         "bs": 256, "lo": 128, "hi": 32768, "log": True},
        # small cache blocks and ragged contexts down to one token
        {"name": "decode-bs16", "op": "decode", "batch": 48, "hq": 32, "hkv": 8, "d": 128,
         "bs": 16, "lo": 1, "hi": 8192, "log": False},
        # chunks of long prompts continued on what earlier rounds cached
        {"name": "prefill-chunk", "op": "prefill", "batch": 4, "hq": 32, "hkv": 8, "d": 128,
         "bs": 256, "qlo": 1024, "qhi": 3000, "plo": 0, "phi": 8192},
        # the next turn of a few conversations: short questions on a cached history
        {"name": "prefill-turn", "op": "prefill", "batch": 3, "hq": 16, "hkv": 8, "d": 128,
         "bs": 16, "qlo": 20, "qhi": 301, "plo": 500, "phi": 6000},
        # one user's logits
        {"name": "rules-one", "op": "rules", "batch": 1, "vocab": 151936, "stride": 151936,
         "type": "fp32", "tlo": 1000, "thi": 1000, "bias": 16, "mask": True, "penalties": True},
        # a full decode step's logits, every rule in use
        {"name": "rules-step", "op": "rules", "batch": 512, "vocab": 151936, "stride": 151936,
         "type": "fp32", "tlo": 16, "thi": 4096, "bias": 8, "mask": True, "penalties": True},
        # 16-bit logits of an odd vocabulary in padded rows, penalties only
        {"name": "rules-odd", "op": "rules", "batch": 64, "vocab": 32003, "stride": 32064,
         "type": "bf16", "tlo": 0, "thi": 2000, "bias": 0, "mask": False, "penalties": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["store", "decode", "decode", "prefill", "rules"])
    bs = rng.choice([8, 16, 24, 32, 48, 64, 128, 192, 256])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "store":
        seqs = _log(rng, 1, 512)
        hi = max(1, min(_log(rng, 1, 1536), 16384 // seqs))
        return {"op": op, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "hkv": hkv, "d": d,
                "bs": bs, "pad": rng.choice([0, 1, 17])}
    if op == "decode":
        batch = _log(rng, 1, 96)
        hi = _log(rng, 1, 32768)
        while batch * hi * hkv * d > 96 * 4096 * 1024:
            hi = max(1, hi // 2)
        return {"op": op, "batch": batch, "hq": hkv * group, "hkv": hkv, "d": d, "bs": bs,
                "lo": rng.randint(0, hi), "hi": hi, "log": False}
    if op == "prefill":
        batch = rng.randint(1, 6)
        qhi = _log(rng, 1, 3000)
        phi = _log(rng, 1, 8192)
        while batch * qhi * (qhi + phi) * hkv * group * d > 3000 * 8192 * 4096:
            qhi, phi = max(1, qhi // 2), max(1, phi // 2)
        return {"op": op, "batch": batch, "hq": hkv * group, "hkv": hkv, "d": d, "bs": bs,
                "qlo": rng.randint(1, qhi), "qhi": qhi, "plo": rng.randint(0, phi), "phi": phi}
    vocab = _log(rng, 100, 151936)
    batch = max(1, min(_log(rng, 1, 512), 512 * 151936 // vocab))
    thi = _log(rng, 1, 4096)
    return {"op": op, "batch": batch, "vocab": vocab, "stride": vocab + rng.choice([0, 0, 5, 64]),
            "type": rng.choice(["fp32", "bf16", "fp16"]), "tlo": rng.randint(0, thi), "thi": thi,
            "bias": rng.choice([0, 1, 8, 100]), "mask": rng.choice([True, False]),
            "penalties": rng.choice([True, True, False])}


def _spread(n, lo, hi, log=False):
    """n lengths from lo to hi, evenly spaced (over the logarithm if asked)."""
    if n == 1:
        return [hi]
    if log:
        return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * i / (n - 1))))
                for i in range(n)]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _prefill_lens(case):
    n = case["batch"]
    lq = _spread(n, case["qlo"], case["qhi"])
    return list(zip(lq, reversed(_spread(n, case["plo"], case["phi"]))))


def work(case):
    op = case["op"]
    if op == "store":
        n = sum(_spread(case["seqs"], case["lo"], case["hi"]))
        row = case["hkv"] * case["d"]
        # bf16 rows in, e4m3 rows out, a slot per token
        return {"bytes": n * (2 * row * 2 + 2 * row + 4), "flops": 2 * n * row * 3}
    if op == "decode":
        ctx = sum(_spread(case["batch"], case["lo"], case["hi"], case["log"]))
        blocks = sum(-(-c // case["bs"])
                     for c in _spread(case["batch"], case["lo"], case["hi"], case["log"]))
        return {"bytes": ctx * case["hkv"] * case["d"] * 2 + blocks * (8 * case["hkv"] + 4) +
                case["batch"] * (case["hq"] * case["d"] * 4 + 4),
                "flops": 4 * ctx * case["hq"] * case["d"]}
    if op == "prefill":
        lens = _prefill_lens(case)
        keys = sum(q * p + q * (q + 1) // 2 for q, p in lens)
        row = case["hkv"] * case["d"]
        return {"bytes": sum(q * (case["hq"] * case["d"] * 4 + row * 4) + p * row * 2
                             for q, p in lens),
                "flops": 4 * keys * case["hq"] * case["d"]}
    esize = 4 if case["type"] == "fp32" else 2
    b, v = case["batch"], case["vocab"]
    tokens = sum(_spread(b, case["tlo"], case["thi"]))
    return {"bytes": b * v * (esize + 4) + (b * ((v + 31) // 32) * 4 if case["mask"] else 0) +
            (tokens * 4 if case["penalties"] else 0) + 8 * sum(_spread(b, 0, 2 * case["bias"])),
            "flops": b * v}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(_dev())


def _tables(rng, blocks_per_seq, num_blocks):
    """Random physical blocks for each sequence; -1 behind the last one."""
    perm = rng.permutation(num_blocks)
    width = max(1, max(blocks_per_seq))
    bt = np.full((len(blocks_per_seq), width), -1, np.int32)
    at = 0
    for i, n in enumerate(blocks_per_seq):
        bt[i, :n] = perm[at:at + n]
        at += n
    return bt


def _pool(g, num_blocks, bs, hkv, d):
    """e4m3 codes of about N(0, 1) rows, and scales a few powers of two apart:
    heads and blocks of a real cache differ in magnitude."""
    dev = _dev()
    codes = (torch.randn((num_blocks, bs, hkv, d), generator=g, device=dev,
                         dtype=torch.bfloat16) * 75).clamp_(-FP8_MAX, FP8_MAX).to(FP8)
    e = torch.randint(-8, -5, (num_blocks, hkv), generator=g, device=dev)
    return codes, ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _stale(codes, bt, lens, bs):
    """NaN codes behind each sequence's last token, as a reused pool has."""
    last = np.asarray([bt[i, -(-n // bs) - 1] if n else 0 for i, n in enumerate(lens)])
    used = np.asarray([(n - 1) % bs + 1 if n else 0 for n in lens])
    keep = np.asarray(lens) > 0
    blk, used = _to_dev(last[keep].astype(np.int64)), _to_dev(used[keep].astype(np.int64))
    raw = codes.view(torch.uint8)
    tail = torch.arange(bs, device=codes.device)[None, :] >= used[:, None]
    raw[blk] = torch.where(tail[:, :, None, None], torch.full_like(raw[:1, :1], 0x7F), raw[blk])


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "rules":
        b, v = case["batch"], case["vocab"]
        lens = rng.permutation(np.asarray(_spread(b, case["tlo"], case["thi"]), np.int32))
        width = max(1, case["thi"])
        x = torch.randn((b, case["stride"]), generator=g, device=dev) * 3
        s["logits"] = x.to(LOGIT_TYPES[case["type"]])[:, :v]
        for k in ("token_ids", "prompt_lens", "token_lens", "repetition", "presence", "frequency",
                  "bias_offsets", "bias_ids", "bias_values", "allowed"):
            s[k] = None
        if case["penalties"]:
            u = torch.rand((b, width), generator=g, device=dev)
            s["token_ids"] = (u ** 3 * v).to(torch.int32).clamp_(max=v - 1)
            s["token_lens"] = _to_dev(lens)
            s["prompt_lens"] = _to_dev((lens * rng.uniform(0, 1, b)).astype(np.int32))
            s["repetition"] = _to_dev(rng.choice([1.0, 1.1, 1.3, 0.9], b).astype(np.float32))
            s["presence"] = _to_dev(rng.choice([0.0, 0.5, -0.25], b).astype(np.float32))
            s["frequency"] = _to_dev(rng.choice([0.0, 0.2, 0.7], b).astype(np.float32))
        if case["bias"]:
            n = rng.permutation(_spread(b, 0, 2 * case["bias"]))
            off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
            s["bias_offsets"] = _to_dev(off)
            total = max(1, int(off[-1]))
            s["bias_ids"] = _to_dev(rng.integers(0, v, total).astype(np.int32))
            s["bias_values"] = _to_dev(rng.normal(0, 4, total).astype(np.float32))
        if case["mask"]:
            words = (v + 31) // 32
            m = torch.randint(-2**31, 2**31, (b, words), generator=g, device=dev).to(torch.int32)
            kind = _to_dev(rng.integers(0, 3, b))[:, None]       # all, about half, a few allowed
            few = torch.where(torch.rand((b, words), generator=g, device=dev) < 0.01, m,
                              torch.zeros_like(m))
            m = torch.where(kind == 0, torch.full_like(m, -1), torch.where(kind == 1, m, few))
            if b > 3:
                m[int(rng.integers(0, b))] = 0                   # a row with nothing allowed
            s["allowed"] = m.contiguous()
        return s
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    if op == "store":
        lens = rng.permutation(_spread(case["seqs"], case["lo"], case["hi"]))
        start = rng.integers(0, bs, case["seqs"])
        per_seq = [int(-(-(a + n) // bs)) for a, n in zip(start, lens)]
        nb = sum(-(-(bs - 1 + int(n)) // bs) for n in lens) + 3
        bt = _tables(rng, per_seq, nb)
        seq = np.repeat(np.arange(case["seqs"]), lens)
        within = np.arange(len(seq)) - np.repeat(np.cumsum(lens) - lens, lens)
        pos = start[seq] + within
        slots = bt[seq, pos // bs].astype(np.int64) * bs + pos % bs
        n = len(slots)
        slots = np.concatenate([slots, np.full(case["pad"], -1)]).astype(np.int32)
        n += case["pad"]
        mag = 2.0 ** torch.randint(-2, 2, (hkv,), generator=g, device=dev)[None, :, None]
        for name in ("k", "v"):
            s[name] = (torch.randn((n, hkv, d), generator=g, device=dev) * mag).to(torch.bfloat16)
            s[name + "c"], s[name + "s"] = _pool(g, nb, bs, hkv, d)
        s["slots"] = _to_dev(slots)
        return s
    hq = case["hq"]
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "decode":
        lens = rng.permutation(_spread(case["batch"], case["lo"], case["hi"], case["log"]))
        lq = None
    else:
        pairs = _prefill_lens(case)
        pairs = [pairs[i] for i in rng.permutation(len(pairs))]
        lens = np.asarray([p for _, p in pairs])
        lq = np.asarray([q for q, _ in pairs])
    per_seq = [int(-(-n // bs)) for n in lens]
    nb = sum(per_seq) + 2
    bt = _tables(rng, per_seq, nb)
    for name in ("k", "v"):
        s[name + "c"], s[name + "s"] = _pool(g, nb, bs, hkv, d)
        _stale(s[name + "c"], bt, [int(n) for n in lens], bs)
    s["bt"] = _to_dev(bt)
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731,E501
    if op == "decode":
        s["q"] = randn(case["batch"], hq, d)
        s["ctx"] = _to_dev(np.asarray(lens, np.int32))
        s["max_ctx"] = int(case["hi"])
    else:
        t = int(lq.sum())
        s["q"], s["k"], s["v"] = randn(t, hq, d), randn(t, hkv, d), randn(t, hkv, d)
        s["cu_q"] = _to_dev(np.concatenate([[0], np.cumsum(lq)]).astype(np.int32))
        s["cu_k"] = _to_dev(np.concatenate([[0], np.cumsum(lq + lens)]).astype(np.int32))
        s["max_q"], s["max_k"] = int(lq.max()), int((lq + lens).max())
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import paged_kv_attention_scatter_gb300 as pkv
    op = s["op"]
    if op == "store":
        pkv.kv_store_fp8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["slots"])
        return {"k_cache": s["kc"], "v_cache": s["vc"], "k_scale": s["ks"], "v_scale": s["vs"]}
    if op == "decode":
        return pkv.paged_decode_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"],
                                    s["scale"], s["max_ctx"])
    if op == "prefill":
        return pkv.paged_prefill_varlen_fp8(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["ks"],
                                            s["vs"], s["cu_q"], s["cu_k"], s["max_q"],
                                            s["max_k"], s["bt"], s["scale"])
    return pkv.apply_logit_rules(
        s["logits"], token_ids=s["token_ids"], prompt_lens=s["prompt_lens"],
        token_lens=s["token_lens"], repetition_penalties=s["repetition"],
        presence_penalties=s["presence"], frequency_penalties=s["frequency"],
        bias_offsets=s["bias_offsets"], bias_token_ids=s["bias_ids"],
        bias_values=s["bias_values"], allowed_mask=s["allowed"])


def _plain(s):
    return {"store": _plain_store, "decode": _plain_decode, "prefill": _plain_prefill,
            "rules": _plain_rules}[s["op"]](s)


def _pow2_scale(amax):
    """The smallest power of two c with amax <= 448 c, exponent in [-64, 119]."""
    m, e = torch.frexp(amax)                                    # amax = m 2^e, m in [0.5, 1)
    # 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_EXP_LO)).clamp(SCALE_EXP_LO,
                                                                         SCALE_EXP_HI)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_store(s):
    slots = s["slots"].long()
    nb, bs, hkv, d = s["kc"].shape
    n = slots.numel()
    # the last token of each slot, -1 where the call stores nothing
    ok = (slots >= 0) & (slots < nb * bs)
    token = torch.where(ok, torch.arange(n, device=slots.device), torch.full_like(slots, -1))
    last = torch.full((nb * bs,), -1, dtype=torch.int64, device=slots.device)
    last = last.scatter_reduce(0, slots.clamp(0, nb * bs - 1), token, "amax").view(nb, bs)
    written = last >= 0
    fresh = written[:, 0]                     # a row at offset 0 begins the block anew
    touched = written.any(1)
    out = {}
    for name, full in (("k", "k_cache"), ("v", "v_cache")):
        codes, scale = s[name + "c"], s[name + "s"]
        rows = s[name].float()[last.clamp(min=0)]                       # [nb, bs, hkv, d]
        size = torch.where(written[:, :, None, None] & torch.isfinite(rows), rows.abs(), 0.0)
        new = _pow2_scale(size.amax((1, 3)))                            # [nb, hkv]
        old = torch.where(fresh[:, None], torch.zeros_like(scale), scale)
        new = torch.where(touched[:, None], torch.maximum(old, new), scale)
        held = codes.float()
        ratio = torch.where(fresh[:, None], torch.ones_like(scale), scale / new)
        grown = held * ratio[:, None, :, None]
        fill = (rows / new[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX)
        value = torch.where(written[:, :, None, None], fill, grown)
        codes.copy_(value.to(FP8))
        scale.copy_(new)
        out[full], out[name + "_scale"] = codes, scale
    return out


def _gathered(codes, scale, bt, keys):
    """Rows of each sequence in order, as 32-bit values: [B, S, hkv, d], zero
    from position keys[b] on."""
    idx = bt.long().clamp(min=0)
    rows = codes.view(torch.uint8)[idx].view(FP8).float() * scale[idx][:, :, None, :, None]
    rows = rows.flatten(1, 2)
    seen = torch.arange(rows.shape[1], device=bt.device)[None, :] < keys[:, None]
    return torch.where(seen[:, :, None, None], rows, 0.0)


def _softmax_av(scores, v):
    """softmax(scores) v over the last axis; a row of -inf gives zeros."""
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(m), m, 0.0))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, torch.matmul(p, v) / total, 0.0)


def _plain_decode(s):
    b, hq, d = s["q"].shape
    hkv = s["kc"].shape[2]
    keys = s["ctx"].long()
    k = _gathered(s["kc"], s["ks"], s["bt"], keys).transpose(1, 2)       # [B, hkv, S, d]
    v = _gathered(s["vc"], s["vs"], s["bt"], keys).transpose(1, 2)
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    scores = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    seen = torch.arange(k.shape[2], device=k.device)[None, :] < keys[:, None]
    scores = torch.where(seen[:, None, None, :], scores, -math.inf)
    return _softmax_av(scores, v).reshape(b, hq, d).to(torch.bfloat16)


def _plain_prefill(s):
    t, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq = cu_q[1:] - cu_q[:-1]
    prefix = cu_k[1:] - cu_k[:-1] - lq
    b, mq = lq.numel(), s["max_q"]
    at = torch.arange(mq, device=lq.device)
    mine = at[None, :] < lq[:, None]                                    # [B, mq]
    row = (cu_q[:-1, None] + at[None, :]).clamp(max=t - 1)
    padded = lambda x: torch.where(mine[:, :, None, None], x.float()[row], 0.0)  # noqa: E731
    q = padded(s["q"]).view(b, mq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k = torch.cat([_gathered(s["kc"], s["ks"], s["bt"], prefix), padded(s["k"])], 1)
    v = torch.cat([_gathered(s["vc"], s["vs"], s["bt"], prefix), padded(s["v"])], 1)
    k, v = k.transpose(1, 2)[:, :, None], v.transpose(1, 2)[:, :, None]  # [B, hkv, 1, S, d]
    cached = k.shape[3] - mq
    seen_p = torch.arange(cached, device=lq.device)[None, :] < prefix[:, None]
    seen_o = at[None, :] <= at[:, None]                                 # causal among its own
    scores = torch.matmul(q, k.transpose(3, 4)) * s["scale"]            # [B, hkv, G, mq, S]
    seen = torch.cat([seen_p[:, None, :].expand(b, mq, cached),
                      seen_o[None].expand(b, mq, mq)], 2)
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    out = _softmax_av(scores, v).permute(0, 3, 1, 2, 4).reshape(b * mq, hq, d)
    owner = torch.searchsorted(cu_q, torch.arange(t, device=lq.device), right=True) - 1
    return out[owner * mq + torch.arange(t, device=lq.device) - cu_q[owner]].to(torch.bfloat16)


def _plain_rules(s):
    x = s["logits"].float()
    b, v = x.shape
    dev = x.device
    if s["token_ids"] is not None:
        ids = s["token_ids"].long()
        at = torch.arange(ids.shape[1], device=dev)[None, :]
        live = (at < s["token_lens"][:, None]) & (ids >= 0) & (ids < v)
        made = live & (at >= s["prompt_lens"][:, None])
        ids = ids.clamp(0, v - 1)
        seen = torch.zeros((b, v), device=dev).scatter_add_(1, ids, live.float()) > 0
        count = torch.zeros((b, v), device=dev).scatter_add_(1, ids, made.float())
        r = s["repetition"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias_offsets"] is not None:
        off = s["bias_offsets"].long()
        entry = torch.arange(s["bias_ids"].numel(), device=dev)
        row = torch.searchsorted(off, entry, right=True) - 1
        live = (row >= 0) & (row < b)
        place = row.clamp(0, b - 1) * v + s["bias_ids"].long()
        # the last entry of a row for a token counts
        last = torch.full((b * v,), -1, dtype=torch.int64, device=dev).scatter_reduce(
            0, place, torch.where(live, entry, torch.full_like(entry, -1)), "amax")
        x = x + torch.where(last >= 0, s["bias_values"][last.clamp(min=0)], 0.0).view(b, v)
    if s["allowed"] is not None:
        at = torch.arange(v, device=dev)
        bit = (s["allowed"][:, at // 32] >> (at % 32)[None, :]) & 1
        x = torch.where(bit != 0, x, -math.inf)
    return x


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "decode": _exact_decode, "prefill": _exact_prefill,
            "rules": _exact_rules}[s["op"]](s)


def _e4m3_values():
    """The 256 values of e4m3 (bias 7, three fraction bits, one NaN a sign)."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = math.nan if (c & 127) == 127 else (-mag if c & 128 else mag)
    return torch.from_numpy(out).to(_dev())


def _pow2_64(e):
    """2^e as 64-bit values, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _to_e4m3(y):
    """The e4m3 value nearest to each y (ties to even, at most 448)."""
    a = y.abs().clamp(max=FP8_MAX)
    _, e = torch.frexp(a)
    step = _pow2_64((e - 1).clamp(min=-6) - 3)
    return torch.copysign(torch.round(a / step) * step, y)


def _exact_store(s):
    nb, bs, hkv, d = s["kc"].shape
    table = _e4m3_values()
    slots = s["slots"].tolist()
    held = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < nb * bs:
            held.setdefault(slot // bs, {})[slot % bs] = t
    out = {}
    for name, full in (("k", "k_cache"), ("v", "v_cache")):
        value = table[s[name + "c"].view(torch.uint8).long()]
        scale = s[name + "s"].double()
        x = s[name].double()
        for blk, rows in held.items():
            off = torch.tensor(sorted(rows), device=x.device)
            new = x[torch.tensor([rows[o] for o in sorted(rows)], device=x.device)]
            need = new.abs().amax((0, 2)) / FP8_MAX
            m, e = torch.frexp(need.clamp(min=2.0 ** SCALE_EXP_LO))
            c = _pow2_64(torch.where(m == 0.5, e - 1, e))       # need rounded up to 2^e
            if 0 not in rows:
                c = torch.maximum(c, scale[blk])
                value[blk] = torch.where((c > scale[blk])[None, :, None],
                                         _to_e4m3(value[blk] * (scale[blk] / c)[None, :, None]),
                                         value[blk])
            value[blk, off] = _to_e4m3(new / c[None, :, None])
            scale[blk] = c
        out[full], out[name + "_scale"] = value, scale
    return out


def _rows64(s, name, table, b, n):
    """The first n rows of sequence b in 64 bits, [n, hkv, d]."""
    bs = s["kc"].shape[1]
    blk = s["bt"][b, :-(-n // bs)].long()
    raw = s[name + "c"].view(torch.uint8)[blk].long()
    rows = table[raw] * s[name + "s"][blk].double()[:, None, :, None]
    return rows.flatten(0, 1)[:n]


def _exact_decode(s):
    table = _e4m3_values()
    b, hq, d = s["q"].shape
    hkv = s["kc"].shape[2]
    out = torch.zeros((b, hkv, hq // hkv, d), dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["ctx"].tolist()):
        if n:
            k, v = (_rows64(s, name, table, i, n).permute(1, 2, 0) for name in ("k", "v"))
            q = s["q"][i].double().view(hkv, hq // hkv, d)
            w = torch.softmax(torch.bmm(q, k) * s["scale"], -1)
            out[i] = torch.bmm(w, v.transpose(1, 2))
    return out.view(b, hq, d)


def _exact_prefill(s):
    table = _e4m3_values()
    t, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    out = torch.zeros((t, hq, d), dtype=torch.float64, device=s["q"].device)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for i in range(len(cu_q) - 1):
        a, e = cu_q[i], cu_q[i + 1]
        p = cu_k[i + 1] - cu_k[i] - (e - a)
        k, v = (torch.cat([_rows64(s, name, table, i, p), s[name][a:e].double()])
                for name in ("k", "v"))
        hidden = torch.arange(k.shape[0], device=k.device)[None, :] > \
            p + torch.arange(e - a, device=k.device)[:, None]
        for h in range(hq):
            w = s["q"][a:e, h].double() @ k[:, h // (hq // hkv)].T * s["scale"]
            w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
            out[a:e, h] = w @ v[:, h // (hq // hkv)]
    return out


def _exact_rules(s):
    x = s["logits"].double().cpu().numpy()
    host = {k: (None if s[k] is None else s[k].cpu().numpy()) for k in s
            if k != "logits" and (isinstance(s[k], torch.Tensor) or s[k] is None)}
    b, v = x.shape
    for i in range(b):
        row = x[i]
        if host["token_ids"] is not None:
            n, p = int(host["token_lens"][i]), int(host["prompt_lens"][i])
            ids = host["token_ids"][i, :n]
            r = float(host["repetition"][i])
            for t in np.unique(ids):
                row[t] = row[t] / r if row[t] > 0 else row[t] * r
            made, count = np.unique(ids[p:], return_counts=True)
            row[made] -= float(host["frequency"][i]) * count + float(host["presence"][i])
        if host["bias_offsets"] is not None:
            a, e = host["bias_offsets"][i:i + 2]
            extra = dict(zip(host["bias_ids"][a:e].tolist(), host["bias_values"][a:e].tolist()))
            for t, w in extra.items():
                row[t] += w
        if host["allowed"] is not None:
            bits = np.unpackbits(host["allowed"][i].view(np.uint8), bitorder="little")[:v]
            row[bits == 0] = -math.inf
    return x
