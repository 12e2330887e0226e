"""Host-side refusals of qk_norm_rope, qk_norm_rope_kv_store and the rotary functions: the C
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
MB = 1 << 20


def _rotary(turns=MB, dim=64, interleaved=0, magnitude=1.0):
    from paged_kv_attention_scatter_gb300._binding import RotaryDesc
    return RotaryDesc(turns, dim, interleaved, magnitude)


def _norm(lib, q=1 * MB, qs=256, k=2 * MB, ks=128, type=1, qw=3 * MB, kw=3 * MB, wtype=1, eps=1e-6,
          pos=4 * MB, rot=None, n=3, hq=4, hkv=2, d=64, qo=5 * MB, qos=256, ko=6 * MB, kos=128):
    return lib.pkv_qk_norm_rope(q, qs, k, ks, type, qw, kw, wtype, eps, pos, rot or _rotary(), n,
                                hq, hkv, d, qo, qos, ko, kos, None)


def test_norm_rope(lib):
    assert _norm(lib, n=0, q=None, k=None, pos=None, qo=None, ko=None) == 0
    for bad in (dict(n=-1), dict(hq=0), dict(hkv=0), dict(type=3), dict(type=-1), dict(wtype=3),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qs=255),
                dict(ks=127), dict(qos=200), dict(kos=100), dict(hq=1 << 28),
                dict(rot=_rotary(dim=66)), dict(rot=_rotary(dim=-2)), dict(rot=_rotary(dim=7)),
                dict(rot=_rotary(magnitude=float("inf")))):
        assert _norm(lib, **bad) == -2, bad
    assert _norm(lib, qw=None, kw=None, rot=_rotary(dim=0)) == -2     # nothing to do
    for d in (0, 4, 60, 264):
        assert _norm(lib, d=d, qs=4 * 264, ks=4 * 264, rot=_rotary(dim=0)) == -3
    for name in ("q", "k", "pos", "qo", "ko"):
        assert _norm(lib, **{name: None}) == -1
    assert _norm(lib, rot=_rotary(turns=None)) == -1
    for name in ("q", "k", "qo", "ko"):
        assert _norm(lib, **{name: 9 * MB + 8}) == -4
    for name in ("qs", "ks", "qos", "kos"):
        assert _norm(lib, **{name: 260}) == -4
        assert _norm(lib, **{name: 258, "type": 0}) == -4
    assert _norm(lib, qw=3 * MB + 1) == -4 and _norm(lib, kw=3 * MB + 2, wtype=0) == -4
    assert _norm(lib, pos=4 * MB + 2) == -4 and _norm(lib, rot=_rotary(turns=MB + 4)) == -4


def test_overlaps(lib):
    # a row of q and k packed, 4 + 2 heads of 64; outputs in other rows of the same memory
    q, k = 1 * MB, 1 * MB + 4 * 64 * 2
    packed = dict(q=q, qs=384, k=k, ks=384)
    assert _norm(lib, **packed, qo=q, qos=256) == -7         # in place with another stride
    assert _norm(lib, **packed, qo=q + 128, qos=384) == -7   # across heads
    assert _norm(lib, **packed, qo=k, qos=384) == -7
    assert _norm(lib, **packed, ko=q, kos=384) == -7
    assert _norm(lib, ko=5 * MB + 64, kos=128) == -7         # q_out and k_out
    assert _norm(lib, qo=2 * MB) == -7


def _store(lib, q=1 * MB, qs=256, k=2 * MB, ks=128, v=3 * MB, vs=128, n=3, hq=4, slots=4 * MB,
           qo=5 * MB, qos=256, ko=None, kos=0, kc=6 * MB, vc=7 * MB, desc=(8, 16, 2, 64)):
    from paged_kv_attention_scatter_gb300._binding import CacheDesc
    return lib.pkv_qk_norm_rope_kv_store(q, qs, k, ks, v, vs, None, None, 1, 0.0, 8 * MB,
                                         _rotary(), slots, n, hq, qo, qos, ko, kos, kc, vc,
                                         CacheDesc(*desc), None, None)


def test_store(lib):
    assert _store(lib, n=0, q=None, v=None, slots=None, kc=None) == 0
    for desc in ((0, 16, 2, 64), (8, 0, 2, 64), (8, 16, 0, 64)):
        assert _store(lib, desc=desc) == -2
    assert _store(lib, desc=(8, 16, 2, 68)) == -3
    assert _store(lib, vs=127) == -2 and _store(lib, vs=132) == -4
    for name in ("q", "k", "v", "slots", "qo", "kc", "vc"):
        assert _store(lib, **{name: None}) == -1
        assert _store(lib, **{name: 9 * MB + 2}) == -4
    assert _store(lib, qo=3 * MB) == -7 and _store(lib, ko=3 * MB, kos=128) == -7


def test_frequencies(lib):
    from paged_kv_attention_scatter_gb300._binding import RotaryScaling
    out, mag = (ctypes.c_double * 128)(), ctypes.c_float()

    def f(dim=64, base=1e4, kind=0, old=4096, factor=2.0, low=1.0, high=4.0, dst=out):
        return lib.pkv_rotary_frequencies(dim, base, RotaryScaling(kind, old, factor, low, high),
                                          dst, ctypes.byref(mag))
    for kind in range(5):
        assert f(kind=kind) == 0
    nan, inf = float("nan"), float("inf")
    for bad in (dict(dim=0), dict(dim=63), dict(dim=258), dict(base=1.0), dict(base=nan),
                dict(base=inf), dict(kind=5), dict(kind=-1), dict(kind=1, factor=0.5),
                dict(kind=1, factor=nan), dict(kind=2, dim=2), dict(kind=3, old=0),
                dict(kind=3, low=0.0), dict(kind=4, low=4.0), dict(kind=4, high=inf)):
        assert f(**bad) == -2, bad
    assert f(dst=None) == -1
    t = (ctypes.c_uint64 * 1)()
    for v in (-1.0, 65537.0, nan, inf):
        assert lib.pkv_rotary_turns((ctypes.c_double * 1)(v), 1, t) == -2
    assert lib.pkv_rotary_turns(None, 1, t) == -1 and lib.pkv_rotary_turns(None, 0, None) == 0
    assert lib.pkv_rotary_turns(None, -1, None) == -2


def test_binding():
    from paged_kv_attention_scatter_gb300 import _binding as B
    with pytest.raises(ValueError, match="scaling must be one of"):
        B.rotary_frequencies(64, scaling="other")
    with pytest.raises(ValueError, match="exclude each other"):
        B.rotary(64, scaling="ntk", frequencies=[0.1] * 32, device="cpu")
    with pytest.raises(ValueError, match=r"\[rotary_dim / 2\]"):
        B.rotary(64, frequencies=[0.1] * 31, device="cpu")
    with pytest.raises(RuntimeError, match="out of range"):
        B.rotary(4, frequencies=[0.1, -0.1], device="cpu")
    r = B.rotary(4, frequencies=[0.5, 0.25], magnitude=2.0, interleaved=True, device="cpu")
    assert r.turns.shape == (2,) and r.desc.interleaved == 1 and r.magnitude == 2.0
    q = torch.zeros(3, 4, 64)
    with pytest.raises(ValueError, match="must be on cuda"):
        B.qk_norm_rope(q, q, None, None, 0.0, None, None)
    with pytest.raises(TypeError, match="fp32, bf16 or fp16"):
        B.qk_norm_rope(q.double(), q, None, None, 0.0, None, None)
