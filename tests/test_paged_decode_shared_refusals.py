"""Host-side refusals of paged_decode_shared, its plan and its run, and the workspace query:
the C entry points answer before any CUDA call, the binding before the library."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_scatter_gb300 import _binding, _build
    _build.build()
    return _binding.load()


P = lambda a: ctypes.c_void_p(a)  # noqa: E731
OK, ODD = P(1 << 20), P((1 << 20) + 2)
BIG = 1 << 40


def _desc(nb=8, bs=16, hkv=2, d=64):
    from paged_kv_attention_scatter_gb300._binding import CacheDesc
    return CacheDesc(nb, bs, hkv, d)


def _fields(f, names, extra):
    def call(batch=2, hq=4, max_ctx=64, width=4, scale=0.1, size=BIG, groups=1, desc=None, **kw):
        a = {k: OK for k in names}
        a.update(kw)
        return extra(f, a, batch, hq, max_ctx, width, scale, size, groups, desc or _desc())
    return call


def test_calls(lib):
    need = lib.pkv_paged_decode_shared_workspace_bytes(2, 4, 64, _desc())
    calls = {
        "whole": (lib.pkv_paged_decode_shared,
                  ("q", "kc", "vc", "bt", "ctx", "off", "pre", "out", "ws"),
                  lambda f, a, B, hq, mc, w, sc, size, g, d:
                  f(a["q"], a["kc"], a["vc"], a["bt"], w, a["ctx"], a["off"], a["pre"], g, B, hq,
                    mc, sc, a["out"], a["ws"], size, d, None, None)),
        "plan": (lib.pkv_paged_decode_plan_shared, ("ctx", "off", "pre", "ws"),
                 lambda f, a, B, hq, mc, w, sc, size, g, d:
                 f(a["ctx"], a["off"], a["pre"], g, B, hq, mc, w, a["ws"], size, d, None, None)),
        "run": (lib.pkv_paged_decode_run_shared, ("q", "kc", "vc", "bt", "out", "ws"),
                lambda f, a, B, hq, mc, w, sc, size, g, d:
                f(a["q"], a["kc"], a["vc"], a["bt"], w, B, hq, mc, sc, a["out"], a["ws"], size, d,
                  None, None))}
    for name, (f, names, extra) in calls.items():
        call = _fields(f, names, extra)
        assert call(batch=0, **{k: None for k in names}) == 0
        for bad in (dict(batch=-1), dict(hq=3), dict(hq=0), dict(max_ctx=-1), dict(width=0),
                    dict(desc=_desc(nb=0)), dict(desc=_desc(bs=0)), dict(desc=_desc(hkv=0))):
            assert call(**bad) == -2, (name, bad)
        assert call(desc=_desc(d=80)) == -3
        assert call(desc=_desc(nb=1 << 27, bs=16)) == -7
        for k in names:
            assert call(**{k: None}) == -1, (name, k)
            assert call(**{k: ODD}) == -4, (name, k)
        assert call(size=need - 1) == -5
        if name != "plan":
            for scale in (0.0, -1.0, float("nan"), float("inf")):
                assert call(scale=scale) == -2
        if name != "run":
            assert call(groups=-1) == -2


def test_workspace(lib):
    f = lib.pkv_paged_decode_shared_workspace_bytes
    assert f(2, 4, 64, _desc()) == f(2, 4, 64, _desc()) > 0
    assert f(2, 4, 4096, _desc()) > f(2, 4, 64, _desc())
    for bad in ((-1, 4, 64), (2, 0, 64), (2, 3, 64), (2, 4, -1)):
        assert f(*bad, _desc()) == 0
    for desc in (_desc(bs=0), _desc(hkv=0), _desc(d=0)):
        assert f(2, 4, 64, desc) == 0
    assert f(0, 4, 0, _desc()) > 0
    # a batch far beyond any memory is refused, not wrapped around
    assert f(1 << 30, 4, 1 << 30, _desc()) == 0


def test_binding():
    from paged_kv_attention_scatter_gb300 import _binding as B
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    bt = torch.zeros(2, 4, dtype=torch.int32)
    ctx = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        B.paged_decode_shared(q, cache, cache, bt, ctx, None, None, 0.1, 64)
    with pytest.raises(ValueError, match="must both be"):
        B.paged_decode_shared(q, cache, cache[:4], bt, ctx, None, None, 0.1, 64)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        B.paged_decode_run_shared(q, cache, cache, bt, 0.1, 64, None)


def test_contexts_beyond_2_30(lib):
    f = lib.pkv_paged_decode_shared_workspace_bytes
    d = _desc(hkv=1)
    assert f(1, 1, 1 << 30, d) > 0
    for n in ((1 << 30) + 1, 2**31 - 1):
        assert f(1, 1, n, d) == 0
        assert lib.pkv_paged_decode_plan_shared(OK, OK, OK, 1, 1, 1, n, 4, OK, BIG, d, None,
                                                None) == -7
        assert lib.pkv_paged_decode_run_shared(OK, OK, OK, OK, 4, 1, 1, n, 0.1, OK, OK, BIG, d,
                                               None, None) == -7
