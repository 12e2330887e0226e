"""Host-side refusals of the 8-bit cache's calls and of the logit rules: the C
entry points answer before any CUDA call, the binding before the library."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_scatter_gb300 import _binding, _build
    _build.build()
    return _binding.load()


P = lambda a: ctypes.c_void_p(a)  # noqa: E731
OK, ODD, HALF = P(1 << 20), P((1 << 20) + 2), P((1 << 20) + 1)
BIG = 1 << 40


def _desc(nb=8, bs=16, hkv=2, d=64):
    from paged_kv_attention_scatter_gb300._binding import CacheDesc
    return CacheDesc(nb, bs, hkv, d)


def test_store(lib):
    f = lib.pkv_kv_store_fp8

    def store(n=3, desc=None, ws=None, size=0, **kw):
        a = {k: OK for k in ("k", "v", "kc", "vc", "ks", "vs", "slots")}
        a.update(kw)
        return f(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["slots"], n, ws, size,
                 desc or _desc(), None, None)
    assert store(n=0, k=None, v=None, kc=None, vc=None, ks=None, vs=None, slots=None) == 0
    assert store(n=-1) == -2
    for bad in (_desc(nb=0), _desc(bs=0), _desc(hkv=0), _desc(bs=1025)):
        assert store(desc=bad) == -2
    assert store(desc=_desc(d=96)) == -3
    assert store(desc=_desc(nb=1 << 30, bs=2)) == -7
    for name in ("k", "v", "kc", "vc", "ks", "vs", "slots"):
        assert store(**{name: None}) == -1
        assert store(**{name: ODD}) == -4
    # the list form needs its workspace
    need = lib.pkv_kv_store_fp8_workspace_bytes(2049, _desc())
    assert need > 0 and lib.pkv_kv_store_fp8_workspace_bytes(2048, _desc()) == 0
    assert store(n=2049) == -1
    assert store(n=2049, ws=ODD, size=need) == -4
    assert store(n=2049, ws=OK, size=need - 1) == -5


def test_decode(lib):
    for f in (lib.pkv_paged_decode_fp8, lib.pkv_paged_decode_run_fp8):
        def decode(batch=2, hq=4, max_ctx=64, desc=None, size=BIG, **kw):
            a = {k: OK for k in ("q", "kc", "vc", "ks", "vs", "bt", "ctx", "out", "ws")}
            a.update(kw)
            return f(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], 4, a["ctx"], batch, hq,
                     max_ctx, 0.1, a["out"], a["ws"], size, desc or _desc(), None, None)
        assert decode(batch=0, q=None, ks=None) == 0
        assert decode(batch=-1) == -2 and decode(hq=3) == -2 and decode(max_ctx=-1) == -2
        assert decode(desc=_desc(bs=2000)) == -2 and decode(desc=_desc(d=80)) == -3
        assert decode(desc=_desc(nb=1 << 28, bs=16)) == -7
        for name in ("q", "kc", "vc", "ks", "vs", "bt", "ctx", "out", "ws"):
            assert decode(**{name: None}) == -1
            assert decode(**{name: ODD}) == -4
        need = lib.pkv_paged_decode_fp8_workspace_bytes(2, 4, 64, _desc())
        assert need > 0 and decode(size=need - 1) == -5


def test_decode_plan(lib):
    f = lib.pkv_paged_decode_plan_fp8

    def plan(ctx=OK, batch=2, hq=4, max_ctx=64, ws=OK, size=BIG, desc=None):
        return f(ctx, batch, hq, max_ctx, 4, ws, size, desc or _desc(), None, None)
    assert plan(batch=0, ctx=None, ws=None) == 0
    assert plan(ctx=None) == -1 and plan(ws=None) == -1
    assert plan(ctx=ODD) == -4 and plan(ws=ODD) == -4
    assert plan(hq=3) == -2 and plan(desc=_desc(d=80)) == -3
    need = lib.pkv_paged_decode_fp8_workspace_bytes(2, 4, 64, _desc())
    assert plan(size=need - 1) == -5
    assert lib.pkv_paged_decode_fp8_workspace_bytes(2, 0, 64, _desc()) == 0


def test_store_and_decode(lib):
    f = lib.pkv_kv_store_paged_decode_fp8
    query = lib.pkv_kv_store_paged_decode_fp8_workspace_bytes
    dec = lib.pkv_paged_decode_fp8_workspace_bytes(2, 4, 64, _desc())
    assert query(3, 2, 4, 64, _desc()) >= dec > 0
    assert query(5000, 2, 4, 64, _desc()) >= dec + lib.pkv_kv_store_fp8_workspace_bytes(5000,
                                                                                        _desc())
    assert query(-1, 2, 4, 64, _desc()) == 0 and query(3, 2, 0, 64, _desc()) == 0

    def call(n=3, batch=2, size=BIG, **kw):
        a = {k: OK for k in ("k", "v", "slots", "q", "kc", "vc", "ks", "vs", "bt", "ctx", "out",
                             "ws")}
        a.update(kw)
        return f(a["k"], a["v"], a["slots"], n, a["q"], a["kc"], a["vc"], a["ks"], a["vs"],
                 a["bt"], 4, a["ctx"], batch, 4, 64, 0.1, a["out"], a["ws"], size, _desc(), None,
                 None)
    for name in ("k", "v", "slots", "q", "kc", "vc", "ks", "vs", "bt", "ctx", "out", "ws"):
        assert call(**{name: None}) == -1
        assert call(**{name: ODD}) == -4
    assert call(n=-1) == -2
    assert call(n=5000, size=query(5000, 2, 4, 64, _desc()) - 1) == -5
    assert call(n=0, batch=0) == 0


def test_prefill(lib):
    f = lib.pkv_paged_prefill_varlen_fp8

    def prefill(batch=1, total=4, hq=4, size=BIG, desc=None, scale=0.1, max_k=9, **kw):
        a = {k: OK for k in ("q", "k", "v", "kc", "vc", "ks", "vs", "cq", "ck", "bt", "out",
                             "ws")}
        a.update(kw)
        return f(a["q"], a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["cq"], a["ck"],
                 batch, total, 4, max_k, hq, a["bt"], 2, scale, a["out"], a["ws"], size,
                 desc or _desc(), None, None)
    assert prefill(total=0) == 0 and prefill(batch=0) == 0
    assert prefill(batch=-1) == -2 and prefill(hq=3) == -2 and prefill(scale=0.0) == -2
    assert prefill(max_k=-1) == -2
    assert prefill(desc=_desc(bs=4096)) == -2 and prefill(desc=_desc(d=32)) == -3
    for name in ("q", "k", "v", "kc", "vc", "ks", "vs", "cq", "ck", "out", "ws"):
        assert prefill(**{name: None}) == -1
    for name in ("q", "k", "v", "kc", "vc", "ks", "vs", "cq", "ck", "bt", "out", "ws"):
        assert prefill(**{name: ODD}) == -4
    need = lib.pkv_paged_prefill_fp8_workspace_bytes(1, 4, 4, 9, _desc())
    assert need > 2 * 128 * 2 * 64 * 2 and prefill(size=need - 1) == -5
    assert lib.pkv_paged_prefill_fp8_workspace_bytes(1, 4, 4, -1, _desc()) == 0


def test_prefill_workspace_grows_with_the_call(lib):
    """A workspace for the largest call holds every smaller one."""
    need = lib.pkv_paged_prefill_fp8_workspace_bytes
    sizes = ([0, 1, 2, 3, 7, 40, 600], [0, 1, 100, 128, 129, 1000, 4000, 20000],
             [0, 1, 127, 128, 3900, 4000, 9000, 50000, 400000, 3000000])
    for hq, desc in ((8, _desc(hkv=8, d=128)), (3, _desc(hkv=1, d=64))):
        at = {(b, n, k): need(b, n, hq, k, desc) for b in sizes[0] for n in sizes[1]
              for k in sizes[2]}
        for (b, n, k), bytes_ in at.items():
            for axis, x in enumerate((b, n, k)):
                bigger = [s for s in sizes[axis] if s > x]
                if bigger:
                    key = [b, n, k]
                    key[axis] = bigger[0]
                    assert at[tuple(key)] >= bytes_, (b, n, k, axis)


def test_prefill_sizes_beyond_any_memory(lib):
    """The product of the sizes passes 64 bits."""
    desc = _desc(hkv=1 << 28, d=128)
    assert lib.pkv_paged_prefill_fp8_workspace_bytes(1, 4, 1 << 28, (1 << 31) - 1, desc) > 1 << 60


def test_rules(lib):
    from paged_kv_attention_scatter_gb300._binding import LogitRules

    def rules(logits=OK, kind=0, stride=100, batch=2, vocab=100, out=P(1 << 24), **kw):
        r = LogitRules()
        for k, v in kw.items():
            setattr(r, k, v.value if isinstance(v, ctypes.c_void_p) else v)
        return lib.pkv_apply_logit_rules(logits, kind, stride, batch, vocab, r, out, None, None)
    assert rules(batch=0, logits=None) == 0
    assert rules(batch=-1) == -2 and rules(vocab=0) == -2 and rules(stride=99) == -2
    assert rules(kind=3) == -7 and rules(kind=-1) == -7
    assert rules(logits=None) == -1 and rules(out=None) == -1
    assert rules(logits=ODD) == -4 and rules(out=ODD) == -4 and rules(kind=1, logits=HALF) == -4
    assert rules(token_ids=OK, max_tokens=-1) == -2
    assert rules(bias_offsets=OK, num_biases=-1) == -2
    assert rules(bias_offsets=OK, num_biases=1) == -1
    for name in ("token_ids", "prompt_lens", "token_lens", "repetition_penalties",
                 "presence_penalties", "frequency_penalties", "bias_offsets", "bias_token_ids",
                 "bias_values", "allowed_mask"):
        assert rules(**{name: ODD}) == -4
    # in place: only fp32 rows that lie as the output's, and no other overlap
    assert rules(out=OK, kind=1) == -7 and rules(out=OK, stride=104) == -7
    assert rules(out=P((1 << 20) + 4 * 150)) == -7
    assert rules(logits=P((1 << 24) + 4 * 199)) == -7


def test_status_names(lib):
    import paged_kv_attention_scatter_gb300 as pkv
    for bit, word in (("BAD_SCALE", b"scale"), ("BAD_TOKEN_ID", b"token"),
                      ("BAD_PENALTY", b"penalty"), ("NO_ALLOWED_TOKEN", b"mask")):
        assert word in lib.pkv_status_string(pkv.STATUS[bit])
        assert pkv.status_names(pkv.STATUS[bit]) == [bit]


def test_binding_checks(lib):
    """Shapes, types and devices are refused before the library is called."""
    import paged_kv_attention_scatter_gb300 as pkv
    f8 = torch.float8_e4m3fn
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.uint8).view(f8)
    s = torch.zeros((4, 2))
    rows = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_scale and v_scale"):
        pkv.kv_store_fp8(rows, rows, kc, kc, s[:3], s, slots)
    with pytest.raises(ValueError, match="k_cache and v_cache"):
        pkv.kv_store_fp8(rows, rows, kc, kc[:3], s, s, slots)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        pkv.kv_store_fp8(rows, rows, kc, kc, s, s, slots)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        pkv.apply_logit_rules(torch.zeros((2, 8)))
    with pytest.raises(ValueError, match="hold a plan"):
        pkv.paged_decode_run_fp8(rows, kc, kc, s, s, slots, slots, 0.1, 8, None)
