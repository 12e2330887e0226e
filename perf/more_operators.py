"""Cases for the steps around the paged KV cache that share work between heads and sequences.

Three operators of one serving step, each in its plain form and as the
library's call:

  norm    RMS norm of every query and key head and the rotation of its position,
          in one pass
  store   the same, with the keys and the values written into the paged cache
  shared  one query per sequence against that cache, where the sequences of a
          group have their first keys in common

Lengths are the same set for every seed of a case (work depends on the case
alone); their order, the block tables and all values come from the seed.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # a single user's next token, out of the projection's packed rows
        {"name": "norm-one", "op": "norm", "tokens": 1, "hq": 16, "hkv": 8, "d": 128, "rot": 128,
         "type": "bf16", "inter": False, "norm": True, "scaling": "none", "far": 40960,
         "packed": True},
        # a ragged prefill round of a model with interleaved partial rotation, context stretched
        {"name": "norm-partial", "op": "norm", "tokens": 1777, "hq": 32, "hkv": 8, "d": 128,
         "rot": 64, "type": "fp16", "inter": True, "norm": True, "scaling": "yarn",
         "far": 131072, "packed": True},
        # rotation alone, of heads of 80 in 32 bits, at positions of very long documents
        {"name": "norm-rotate", "op": "norm", "tokens": 8191, "hq": 20, "hkv": 4, "d": 80,
         "rot": 40, "type": "fp32", "inter": False, "norm": False, "scaling": "linear",
         "far": 1 << 20, "packed": False},
        # a single user's next token, into the cache
        {"name": "store-one", "op": "store", "tokens": 1, "hq": 16, "hkv": 8, "d": 128,
         "rot": 128, "type": "bf16", "inter": False, "norm": True, "scaling": "none",
         "far": 40960, "packed": True, "bs": 256, "pad": 0},
        # a full decode step: one token of each running sequence, some rows padding
        {"name": "store-step", "op": "store", "tokens": 512, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "type": "bf16", "inter": False, "norm": True, "scaling": "bands",
         "far": 131072, "packed": True, "bs": 256, "pad": 19},
        # a full prefill round
        {"name": "store-round", "op": "store", "tokens": 16384, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "type": "bf16", "inter": False, "norm": True, "scaling": "none",
         "far": 8192, "packed": True, "bs": 256, "pad": 0},
        # two samples of one prompt
        {"name": "shared-two", "op": "shared", "batch": 2, "groups": 1, "hq": 16, "hkv": 8,
         "d": 128, "bs": 256, "plo": 1000, "phi": 1000, "slo": 30, "shi": 200, "plan": False},
        # a small model's decode step behind one system prompt
        {"name": "shared-64", "op": "shared", "batch": 64, "groups": 1, "hq": 16, "hkv": 8,
         "d": 128, "bs": 256, "plo": 2048, "phi": 2048, "slo": 16, "shi": 2048, "plan": False},
        # a full step behind a long instruction, one layer of many with one schedule
        {"name": "shared-step", "op": "shared", "batch": 256, "groups": 1, "hq": 32, "hkv": 8,
         "d": 128, "bs": 256, "plo": 8192, "phi": 8192, "slo": 1, "shi": 1500, "plan": True},
        # tenants with their own prompts, from a lone user to dozens; small cache blocks
        {"name": "shared-tenants", "op": "shared", "batch": 128, "groups": 12, "hq": 32,
         "hkv": 8, "d": 128, "bs": 16, "plo": 100, "phi": 6000, "slo": 0, "shi": 900,
         "plan": False},
        # questions on two long documents, a large model's heads
        {"name": "shared-document", "op": "shared", "batch": 48, "groups": 2, "hq": 64, "hkv": 8,
         "d": 128, "bs": 64, "plo": 30000, "phi": 65536, "slo": 10, "shi": 500, "plan": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["norm", "store", "shared", "shared"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "shared":
        d = rng.choice([64, 128, 128])
        batch = _log(rng, 2, 256)
        phi = _log(rng, 10, 65536)
        shi = _log(rng, 1, 2048)
        while batch * (phi + shi) * hkv * group * d > 48 * 40000 * 8192 or \
                batch * shi * hkv * d > 256 * 1024 * 1024:
            phi, shi = max(10, phi // 2), max(1, shi // 2)
        return {"op": op, "batch": batch, "groups": rng.randint(1, min(batch, 16)),
                "hq": hkv * group, "hkv": hkv, "d": d,
                "bs": rng.choice([8, 16, 20, 24, 32, 48, 64, 128, 192, 256]),
                "plo": rng.randint(0, phi), "phi": phi, "slo": rng.randint(0, shi), "shi": shi,
                "plan": rng.choice([True, False])}
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    rot = rng.choice([d, d, d // 2, d // 4])
    tokens = _log(rng, 1, 16384)
    while tokens * (group + 2) * hkv * d > 16384 * 48 * 128:
        tokens //= 2
    case = {"op": op, "tokens": tokens, "hq": hkv * group, "hkv": hkv, "d": d, "rot": rot,
            "type": "bf16" if op == "store" else rng.choice(["bf16", "fp16", "fp32"]),
            "inter": rng.choice([True, False]), "norm": rng.choice([True, True, False]),
            "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
            "far": _log(rng, 1000, 1 << 20), "packed": rng.choice([True, False])}
    if op == "store":
        case.update(bs=rng.choice([1, 8, 16, 20, 64, 256]), pad=rng.choice([0, 0, 1, 17]))
    return case


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spaced."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _members(case):
    """Sequences of each group: shares in the ratio 1, 2, 3, ..., one at least."""
    n, g = case["batch"], case["groups"]
    total = g * (g + 1) // 2
    size = [1 + (n - g) * (i + 1) // total for i in range(g)]
    size[-1] += n - sum(size)
    return size


def work(case):
    if case["op"] == "shared":
        prefix = _spread(case["groups"], case["plo"], case["phi"])
        suffix = _spread(case["batch"], case["slo"], case["shi"])
        size = _members(case)
        row = case["hkv"] * case["d"]
        keys = sum(n * p for n, p in zip(size, prefix)) + sum(suffix)
        rows = sum(prefix) + sum(suffix)
        blocks = sum(-(-p // case["bs"]) for p in prefix) + sum(-(-s // case["bs"])
                                                               for s in suffix)
        return {"bytes": rows * row * 4 + blocks * 4 + case["batch"] *
                (case["hq"] * case["d"] * 4 + 4), "flops": 4 * keys * case["hq"] * case["d"]}
    size = 4 if case["type"] == "fp32" else 2
    heads = case["hq"] + case["hkv"] * (2 if case["op"] == "store" else 1)
    # rows in and out, a position (and a slot) for each token; seven operations an element
    return {"bytes": case["tokens"] * (heads * case["d"] * size * 2 + 8),
            "flops": 7 * case["tokens"] * heads * case["d"]}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(_dev())


def _rotary_args(case):
    """What a model's configuration says of its rotation."""
    kind = case["scaling"]
    args = {"rotary_dim": case["rot"], "base": 1e6, "interleaved": case["inter"]}
    if kind != "none":
        args.update(scaling=kind, factor=4.0)
    if kind in ("yarn", "bands"):
        args.update(original_max_position=32768)
    return args


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"op": case["op"], "case": dict(case)}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "shared":
        return _prepare_shared(s, case, rng, g, dev)
    n = case["tokens"] + case.get("pad", 0)
    dtype = TYPES[case["type"]]
    heads = (hq, hkv, hkv)
    # heads of a projection's output differ in magnitude
    mag = 2.0 ** torch.randint(-2, 3, (sum(heads),), generator=g, device=dev)
    x = (torch.randn((n, sum(heads), d), generator=g, device=dev) * mag[None, :, None]).to(dtype)
    if case["packed"]:
        s["q"], s["k"], s["v"] = x.split(heads, dim=1)
    else:
        s["q"], s["k"], s["v"] = (t.contiguous() for t in x.split(heads, dim=1))
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"], s["kw"] = ((1 + 0.3 * torch.randn(d, generator=g, device=dev)).to(dtype)
                            for _ in range(2))
    s["eps"] = 1e-6
    # runs of consecutive positions (prompts), or single ones (a decode step)
    run = max(1, n // 16) if n >= 1024 else 1
    starts = rng.integers(0, max(1, case["far"] - run), -(-n // run))
    s["pos"] = _to_dev((starts[:, None] + np.arange(run)[None, :]).reshape(-1)[:n].astype(np.int32))
    s["rotary"] = _rotary_args(case)
    if case["op"] == "store":
        bs = case["bs"]
        nb = -(-case["tokens"] // bs)
        nb += max(3, nb // 4)
        # runs that start anywhere in blocks of their own, in a pool that holds other rows
        perm = rng.permutation(nb * bs // run)
        slots = (perm[:-(-case["tokens"] // run), None] * run + np.arange(run)[None, :])
        slots = slots.reshape(-1)[:case["tokens"]].astype(np.int32)
        s["slots"] = _to_dev(np.concatenate([slots, np.full(case["pad"], -1, np.int32)]))
        for name in ("kc", "vc"):
            s[name] = torch.randn((nb, bs, hkv, d), generator=g, device=dev,
                                  dtype=torch.bfloat16)
    if own:
        import paged_kv_attention_scatter_gb300 as pkv
        s["rope"] = pkv.rotary(**s["rotary"])
    return s


def _prepare_shared(s, case, rng, g, dev):
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    size = [int(n) for n in rng.permutation(_members(case))]
    # prefixes end where a cache block does, as a prefix cache shares whole blocks
    prefix = [int(p) // bs * bs if p >= bs else 0
              for p in rng.permutation(_spread(case["groups"], case["plo"], case["phi"]))]
    suffix = [int(n) for n in rng.permutation(_spread(case["batch"], case["slo"], case["shi"]))]
    group = np.repeat(np.arange(case["groups"]), size)
    ctx = [prefix[group[b]] + suffix[b] for b in range(case["batch"])]
    own_blocks = [-(-n // bs) for n in suffix]
    nb = sum(prefix) // bs + sum(own_blocks) + 2
    perm = rng.permutation(nb)
    width = max(1, max(-(-c // bs) for c in ctx))
    bt = np.full((case["batch"], width), -1, np.int32)
    at = 0
    shared = []
    for p in prefix:
        shared.append(perm[at:at + p // bs])
        at += p // bs
    tails = []
    for b in range(case["batch"]):
        head = shared[group[b]]
        bt[b, :len(head)] = head
        bt[b, len(head):len(head) + own_blocks[b]] = perm[at:at + own_blocks[b]]
        at += own_blocks[b]
        if suffix[b] % bs:
            tails.append((perm[at - 1], suffix[b] % bs))
    for name in ("kc", "vc"):
        s[name] = torch.randn((nb, bs, hkv, d), generator=g, device=dev, dtype=torch.bfloat16)
    if tails:                                # NaN behind each last token, as a reused pool has
        blk = _to_dev(np.asarray([t[0] for t in tails], np.int64))
        used = _to_dev(np.asarray([t[1] for t in tails], np.int64))
        stale = torch.arange(bs, device=dev)[None, :] >= used[:, None]
        for name in ("kc", "vc"):
            s[name][blk] = torch.where(stale[:, :, None, None], math.nan, s[name][blk])
    s["q"] = torch.randn((case["batch"], hq, d), generator=g, device=dev).to(torch.bfloat16)
    s["bt"], s["ctx"] = _to_dev(bt), _to_dev(np.asarray(ctx, np.int32))
    s["offsets"] = _to_dev(np.concatenate([[0], np.cumsum(size)]).astype(np.int32))
    s["prefix"] = _to_dev(np.asarray(prefix, np.int32))
    s["members"], s["prefixes"] = size, prefix
    s["max_ctx"], s["scale"] = max(ctx), 1.0 / math.sqrt(d)
    if own and case["plan"]:
        import paged_kv_attention_scatter_gb300 as pkv
        s["schedule"] = pkv.paged_decode_plan_shared(s["ctx"], s["offsets"], s["prefix"], hq,
                                                     s["max_ctx"], width, s["kc"])
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import paged_kv_attention_scatter_gb300 as pkv
    if s["op"] == "norm":
        q, k = pkv.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["eps"], s["pos"], s["rope"])
        return {"q": q, "k": k}
    if s["op"] == "store":
        q = pkv.qk_norm_rope_kv_store(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["eps"],
                                      s["pos"], s["rope"], s["kc"], s["vc"], s["slots"])
        return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
    if s["case"]["plan"]:
        return pkv.paged_decode_run_shared(s["q"], s["kc"], s["vc"], s["bt"], s["scale"],
                                           s["max_ctx"], s["schedule"])
    return pkv.paged_decode_shared(s["q"], s["kc"], s["vc"], s["bt"], s["ctx"], s["offsets"],
                                   s["prefix"], s["scale"], s["max_ctx"])


def _plain(s):
    if s["op"] == "shared":
        return _plain_shared(s)
    cos, sin = _plain_angles(s)
    q = _plain_head(s["q"], s["qw"], cos, sin, s)
    k = _plain_head(s["k"], s["kw"], cos, sin, s)
    if s["op"] == "norm":
        return {"q": q, "k": k}
    real = s["case"]["tokens"]                 # the rows behind them are padding
    to = s["slots"][:real].long()
    for cache, rows in ((s["kc"], k), (s["vc"], s["v"])):
        cache.view(-1, *cache.shape[2:]).index_copy_(0, to, rows[:real])
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_frequencies(a):
    """Radians for each position and pair, and the factor of cosines and sines."""
    r, base, kind = a["rotary_dim"], a["base"], a.get("scaling")
    i = torch.arange(r // 2, dtype=torch.float64)
    f = a.get("factor", 1.0)
    if kind == "ntk":
        base = base * f ** (r / (r - 2))
    w = base ** (-2 * i / r)
    if kind == "linear":
        return w / f, 1.0
    if kind == "yarn":
        def dim(rotations):
            return r * math.log(a["original_max_position"] / (rotations * 2 * math.pi)) / \
                (2 * math.log(base))
        lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), r - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1
    if kind == "bands":
        length = 2 * math.pi / w
        old, low, high = a["original_max_position"], 1.0, 4.0
        keep = ((old / length - low) / (high - low)).clamp(0, 1)
        return w * keep + w / f * (1 - keep), 1.0
    return w, 1.0


def _plain_angles(s):
    w, mag = _plain_frequencies(s["rotary"])
    angle = s["pos"].double()[:, None] * w.to(s["pos"].device)[None, :]    # far positions
    return (torch.cos(angle) * mag).float()[:, None], (torch.sin(angle) * mag).float()[:, None]


def _plain_head(x, weight, cos, sin, s):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    r = s["rotary"]["rotary_dim"]
    rest = y[..., r:]
    if s["rotary"]["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1).to(x.dtype)


def _plain_shared(s):
    """Group by group: the scores of the common keys as one product, beside the
    scores of each sequence's own keys."""
    hq, d = s["q"].shape[1:]
    bs, hkv = s["kc"].shape[1:3]
    out = torch.empty_like(s["q"])
    at = 0
    for n, p in zip(s["members"], s["prefixes"]):
        seqs = slice(at, at + n)
        at += n
        q = s["q"][seqs].float().view(n, hkv, hq // hkv, d)
        common = s["bt"][seqs][0, :p // bs].long()
        own_table = s["bt"][seqs][:, p // bs:].long().clamp(min=0)
        left = s["ctx"][seqs].long() - p
        seen = torch.arange(own_table.shape[1] * bs, device=q.device)[None, :] < left[:, None]
        kp, vp = (s[c][common].flatten(0, 1).float().transpose(0, 1) for c in ("kc", "vc"))
        ks, vs = (torch.where(seen[:, :, None, None], s[c][own_table].flatten(1, 2).float(),
                              0.0).transpose(1, 2) for c in ("kc", "vc"))
        rows = q.transpose(0, 1).flatten(1, 2)                     # [hkv, n G, d]
        sp = torch.matmul(rows, kp.transpose(1, 2)).view(hkv, n, hq // hkv, p).transpose(0, 1)
        ss = torch.matmul(q, ks.transpose(2, 3))
        ss = torch.where(seen[:, None, None, :], ss, -math.inf)
        scores = torch.cat([sp, ss], -1) * s["scale"]
        if scores.shape[-1] == 0:
            out[seqs] = 0
            continue
        m = scores.amax(-1, keepdim=True)
        w = torch.exp(scores - torch.where(torch.isfinite(m), m, 0.0))
        total = w.sum(-1, keepdim=True)
        op = torch.matmul(w[..., :p].transpose(0, 1).reshape(hkv, n * (hq // hkv), p), vp)
        o = op.view(hkv, n, hq // hkv, d).transpose(0, 1) + torch.matmul(w[..., p:], vs)
        out[seqs] = torch.where(total > 0, o / total, 0.0).reshape(n, hq, d).to(out.dtype)
    return out


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_shared(s) if s["op"] == "shared" else _exact_heads(s)


def _exact_shared(s):
    """Sequence by sequence, every key through the sequence's own table."""
    b, hq, d = s["q"].shape
    bs, hkv = s["kc"].shape[1:3]
    out = torch.zeros((b, hq, d), dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["ctx"].tolist()):
        if n == 0:
            continue
        blocks = s["bt"][i, :-(-n // bs)].long()
        k, v = (s[c][blocks].flatten(0, 1)[:n].double() for c in ("kc", "vc"))
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            w = torch.softmax(s["q"][i, heads].double() @ k[:, h].T * s["scale"], -1)
            out[i, heads] = w @ v[:, h]
    return out


def _exact_heads(s):
    a = s["rotary"]
    r, half = a["rotary_dim"], a["rotary_dim"] // 2
    f = a.get("factor", 1.0)
    kind, base, mag = a.get("scaling"), a["base"], 1.0
    if kind == "ntk":
        base *= f ** (r / (r - 2.0))
    freq = []
    for i in range(half):
        w = math.exp(-2.0 * i / r * math.log(base))
        if kind == "linear":
            w /= f
        elif kind == "yarn":
            old = a["original_max_position"]
            bound = [half * math.log(old / (2 * math.pi * t)) / math.log(base) for t in (32, 1)]
            lo, hi = max(math.floor(bound[0]), 0), min(math.ceil(bound[1]), r - 1)
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            w = (1 - ramp) * w + ramp * w / f
            mag = 1 + 0.1 * math.log(f)
        elif kind == "bands":
            turns = a["original_max_position"] * w / (2 * math.pi)
            w = w if turns >= 4 else w / f if turns <= 1 else \
                w * ((turns - 1) / 3) + w / f * (1 - (turns - 1) / 3)
        freq.append(w)
    angle = torch.outer(s["pos"].double(), torch.tensor(freq, dtype=torch.float64,
                                                        device=s["pos"].device))
    turn = torch.polar(torch.full_like(angle, mag), angle)[:, None]           # mag e^(i angle)

    def head(x, weight):
        y = x.double()
        if weight is not None:
            y = weight.double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] +
                                                 s["eps"])
        else:
            y = y.clone()
        first, second = (slice(0, r, 2), slice(1, r, 2)) if a["interleaved"] else \
            (slice(0, half), slice(half, r))
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = head(s["q"], s["qw"]), head(s["k"], s["kw"])
    if s["op"] == "norm":
        return {"q": q, "k": k}
    hkv, d = s["kc"].shape[2:]
    kc, vc = s["kc"].double(), s["vc"].double()
    keep = s["slots"] >= 0
    to = s["slots"][keep].long()
    kc.view(-1, hkv, d)[to] = k[keep]
    vc.view(-1, hkv, d)[to] = s["v"][keep].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}
