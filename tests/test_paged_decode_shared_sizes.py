"""Sizes that paged_decode_shared has no workspace for: the query gives 0, and the calls refuse
the sizes, not the workspace that was not made."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from paged_kv_attention_scatter_gb300 import _binding, _build
    _build.build()
    return _binding.load()


OK = ctypes.c_void_p(1 << 20)


@pytest.mark.parametrize("batch,max_ctx", [(1, (1 << 30) + 1), (2, 2**31 - 1), (1 << 30, 1 << 30)])
def test_sizes_without_a_workspace(lib, batch, max_ctx):
    from paged_kv_attention_scatter_gb300._binding import CacheDesc
    desc = CacheDesc(8, 16, 2, 64)
    assert lib.pkv_paged_decode_shared_workspace_bytes(batch, 4, max_ctx, desc) == 0
    for ws in (None, OK):
        assert lib.pkv_paged_decode_shared(OK, OK, OK, OK, 4, OK, OK, OK, 1, batch, 4, max_ctx,
                                           0.1, OK, ws, 0, desc, None, None) == -7
        assert lib.pkv_paged_decode_plan_shared(OK, OK, OK, 1, batch, 4, max_ctx, 4, ws, 0, desc,
                                                None, None) == -7
        assert lib.pkv_paged_decode_run_shared(OK, OK, OK, OK, 4, batch, 4, max_ctx, 0.1, OK, ws,
                                               0, desc, None, None) == -7
