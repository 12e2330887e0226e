"""ctypes binding of libpagedattn.so: argument marshalling only.

Every function checks the tensors' device, dtype and contiguity, passes raw
device pointers, sizes and the current CUDA stream to the C ABI declared in
include/pagedattn.h, and raises on a non-zero return code.  All arithmetic
runs in the library's CUDA kernels; there is no other implementation here, and
a missing library is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import _build

_LIB = None

PKV_STATUS_BITS = {
    1 << 0: "SLOT_OUT_OF_RANGE",
    1 << 1: "BAD_BLOCK_ID",
    1 << 2: "BAD_CONTEXT_LEN",
    1 << 3: "BAD_SEQLENS",
    1 << 4: "BAD_TEMPERATURE",
    1 << 5: "NO_FINITE_KEY",
    1 << 6: "WORKSPACE_OVERFLOW",
    1 << 7: "WAIT_TIMEOUT",
    1 << 8: "BAD_SCALE",
    1 << 9: "BAD_TOKEN_ID",
    1 << 10: "BAD_PENALTY",
    1 << 11: "NO_ALLOWED_TOKEN",
}
STATUS = {v: k for k, v in PKV_STATUS_BITS.items()}

C_FUNCTIONS = ["pkv_version", "pkv_error_string", "pkv_status_string", "pkv_kv_store",
               "pkv_paged_decode_workspace_bytes", "pkv_paged_decode",
               "pkv_paged_prefill_workspace_bytes", "pkv_paged_prefill_varlen", "pkv_sample",
               "pkv_paged_decode_static_workspace", "pkv_kv_store_paged_decode",
               "pkv_kv_store_paged_prefill_varlen", "pkv_paged_decode_plan",
               "pkv_paged_decode_run", "pkv_paged_attention_varlen_workspace_bytes",
               "pkv_kv_store_paged_attention_varlen",
               "pkv_layer_cache", "pkv_sample_philox", "pkv_set_wait_poll_limit",
               "pkv_kv_store_fp8_workspace_bytes", "pkv_kv_store_fp8", "pkv_paged_decode_fp8",
               "pkv_paged_decode_fp8_workspace_bytes", "pkv_paged_decode_plan_fp8",
               "pkv_paged_decode_run_fp8", "pkv_kv_store_paged_decode_fp8_workspace_bytes",
               "pkv_kv_store_paged_decode_fp8", "pkv_paged_prefill_fp8_workspace_bytes",
               "pkv_paged_prefill_varlen_fp8", "pkv_apply_logit_rules"]

# Size of the scratch array compiled into the library for
# pkv_paged_decode_static_workspace (PKV_STATIC_DECODE_WORKSPACE_BYTES).
STATIC_DECODE_WORKSPACE_BYTES = 16 * 1024 * 1024


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class LogitRules(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("token_ids", "prompt_lens", "token_lens", "repetition_penalties",
                 "presence_penalties", "frequency_penalties", "bias_offsets", "bias_token_ids",
                 "bias_values", "allowed_mask")] + \
               [("max_tokens", ctypes.c_int32), ("num_biases", ctypes.c_int32)]


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None) -> ctypes.CDLL:
    """Loads libpagedattn.so (built by __graft_entry__.build() or
    paged_kv_attention_scatter_gb300._build.build()).  Raises if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run paged_kv_attention_scatter_gb300._build."
                           "build() (or __graft_entry__.build()) first")
    lib = ctypes.CDLL(path)
    P, I32, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    lib.pkv_version.restype = ctypes.c_int
    lib.pkv_version.argtypes = []
    lib.pkv_error_string.restype = ctypes.c_char_p
    lib.pkv_error_string.argtypes = [ctypes.c_int]
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_status_string.argtypes = [ctypes.c_uint32]
    lib.pkv_kv_store.restype = ctypes.c_int
    lib.pkv_kv_store.argtypes = [P, P, P, P, P, I32, CacheDesc, P, P]
    lib.pkv_paged_decode_workspace_bytes.restype = SZ
    lib.pkv_paged_decode_workspace_bytes.argtypes = [I32, I32, I32, CacheDesc]
    lib.pkv_paged_decode.restype = ctypes.c_int
    lib.pkv_paged_decode.argtypes = [P, P, P, P, I32, P, I32, I32, I32, F32, P, P, SZ,
                                     CacheDesc, P, P]
    lib.pkv_paged_decode_plan.restype = ctypes.c_int
    lib.pkv_paged_decode_plan.argtypes = [P, I32, I32, I32, I32, P, SZ, CacheDesc, P, P]
    lib.pkv_paged_decode_run.restype = ctypes.c_int
    lib.pkv_paged_decode_run.argtypes = [P, P, P, P, I32, P, I32, I32, I32, F32, P, P, SZ,
                                         CacheDesc, P, P]
    lib.pkv_paged_prefill_workspace_bytes.restype = SZ
    lib.pkv_paged_prefill_workspace_bytes.argtypes = [I32, I32, I32, CacheDesc]
    lib.pkv_paged_prefill_varlen.restype = ctypes.c_int
    lib.pkv_paged_prefill_varlen.argtypes = [P, P, P, P, P, P, P, I32, I32, I32, I32, I32, P,
                                             I32, F32, P, P, SZ, CacheDesc, P, P]
    lib.pkv_sample.restype = ctypes.c_int
    lib.pkv_sample.argtypes = [P, P, P, I32, I32, P, P, P]
    lib.pkv_kv_store_paged_decode.restype = ctypes.c_int
    lib.pkv_kv_store_paged_decode.argtypes = [P, P, P, I32, P, P, P, P, I32, P, I32, I32, I32,
                                              F32, P, P, SZ, CacheDesc, P, P]
    lib.pkv_kv_store_paged_prefill_varlen.restype = ctypes.c_int
    lib.pkv_kv_store_paged_prefill_varlen.argtypes = [P, P, P, P, P, P, P, P, I32, I32, I32,
                                                      I32, I32, P, I32, F32, P, P, SZ,
                                                      CacheDesc, P, P]
    lib.pkv_paged_attention_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.pkv_paged_attention_varlen_workspace_bytes.argtypes = [I32, I32, I32, I32, CacheDesc]
    lib.pkv_kv_store_paged_attention_varlen.restype = ctypes.c_int
    lib.pkv_kv_store_paged_attention_varlen.argtypes = [P, P, P, P, P, P, P, P, I32, I32, I32,
                                                        I32, I32, P, I32, F32, P, P, SZ,
                                                        CacheDesc, P, P]
    lib.pkv_sample_philox.restype = ctypes.c_int
    lib.pkv_sample_philox.argtypes = [P, P, ctypes.c_uint64, ctypes.c_uint64, I32, I32, P, P, P]
    lib.pkv_layer_cache.restype = ctypes.c_int
    lib.pkv_layer_cache.argtypes = [P, I32, I32, CacheDesc, ctypes.POINTER(ctypes.c_void_p),
                                    ctypes.POINTER(ctypes.c_void_p)]
    lib.pkv_set_wait_poll_limit.restype = ctypes.c_int
    lib.pkv_set_wait_poll_limit.argtypes = [ctypes.c_uint32]
    lib.pkv_kv_store_fp8_workspace_bytes.restype = SZ
    lib.pkv_kv_store_fp8_workspace_bytes.argtypes = [I32, CacheDesc]
    lib.pkv_kv_store_fp8.restype = ctypes.c_int
    lib.pkv_kv_store_fp8.argtypes = [P, P, P, P, P, P, P, I32, P, SZ, CacheDesc, P, P]
    lib.pkv_paged_decode_fp8_workspace_bytes.restype = SZ
    lib.pkv_paged_decode_fp8_workspace_bytes.argtypes = [I32, I32, I32, CacheDesc]
    lib.pkv_paged_decode_plan_fp8.restype = ctypes.c_int
    lib.pkv_paged_decode_plan_fp8.argtypes = [P, I32, I32, I32, I32, P, SZ, CacheDesc, P, P]
    for name in ("pkv_paged_decode_fp8", "pkv_paged_decode_run_fp8"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [P, P, P, P, P, P, I32, P, I32, I32, I32, F32, P, P, SZ, CacheDesc, P, P]
    lib.pkv_kv_store_paged_decode_fp8_workspace_bytes.restype = SZ
    lib.pkv_kv_store_paged_decode_fp8_workspace_bytes.argtypes = [I32, I32, I32, I32, CacheDesc]
    lib.pkv_kv_store_paged_decode_fp8.restype = ctypes.c_int
    lib.pkv_kv_store_paged_decode_fp8.argtypes = [P, P, P, I32, P, P, P, P, P, P, I32, P, I32, I32,
                                                  I32, F32, P, P, SZ, CacheDesc, P, P]
    lib.pkv_paged_prefill_fp8_workspace_bytes.restype = SZ
    lib.pkv_paged_prefill_fp8_workspace_bytes.argtypes = [I32, I32, I32, I32, CacheDesc]
    lib.pkv_paged_prefill_varlen_fp8.restype = ctypes.c_int
    lib.pkv_paged_prefill_varlen_fp8.argtypes = [P, P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32,
                                                 P, I32, F32, P, P, SZ, CacheDesc, P, P]
    lib.pkv_apply_logit_rules.restype = ctypes.c_int
    lib.pkv_apply_logit_rules.argtypes = [P, I32, ctypes.c_int64, I32, I32, LogitRules, P, P, P]
    _LIB = lib
    return lib


# ----------------------------------------------------------------------------
def _check(rc: int, what: str) -> None:
    if rc != 0:
        msg = load().pkv_error_string(rc).decode()
        raise RuntimeError(f"{what}: {msg} (code {rc})")


def _dev(t: torch.Tensor, name: str, dtype, device=None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.data_ptr()


def _ptr_or_null(t, name, dtype, device):
    return None if t is None else _dev(t, name, dtype, device)


def _stream(device, stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    nb, bs, hkv, d = k_cache.shape
    return CacheDesc(nb, bs, hkv, d)


def new_status(device) -> torch.Tensor:
    """A zeroed device status word for the `status=` argument."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def status_names(word: int) -> list[str]:
    return [n for b, n in PKV_STATUS_BITS.items() if word & b]


# ----------------------------------------------------------------------------
def kv_store(k, v, k_cache, v_cache, slot_mapping, status=None, stream=None) -> None:
    """Writes row i of k / v into slot slot_mapping[i] of k_cache / v_cache
    (in place).  k, v: [N, Hkv, D] bf16; caches [NB, bs, Hkv, D] bf16;
    slot_mapping [N] int32 (negative = skip)."""
    lib = load()
    dev = k_cache.device
    n = slot_mapping.numel()
    if k.shape != (n,) + tuple(k_cache.shape[2:]) or v.shape != k.shape:
        raise ValueError("k/v must be [num_tokens, num_kv_heads, head_dim] matching the cache")
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    rc = lib.pkv_kv_store(_dev(k, "k", torch.bfloat16, dev), _dev(v, "v", torch.bfloat16, dev),
                          _dev(k_cache, "k_cache", torch.bfloat16, dev),
                          _dev(v_cache, "v_cache", torch.bfloat16, dev),
                          _dev(slot_mapping, "slot_mapping", torch.int32, dev), n,
                          cache_desc(k_cache), _ptr_or_null(status, "status", torch.int32, dev),
                          _stream(dev, stream))
    _check(rc, "pkv_kv_store")


def paged_decode_workspace_bytes(batch, num_q_heads, max_context_len, k_cache) -> int:
    return int(load().pkv_paged_decode_workspace_bytes(batch, num_q_heads, max_context_len,
                                                       cache_desc(k_cache)))


def paged_decode(q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                 out=None, workspace=None, status=None, stream=None) -> torch.Tensor:
    """Decode attention: q [B, Hq, D] bf16 -> out [B, Hq, D] bf16.
    block_tables [B, MB] int32, context_lens [B] int32, max_context_len a host
    upper bound of context_lens."""
    lib = load()
    dev = k_cache.device
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    need = paged_decode_workspace_bytes(B, Hq, max_context_len, k_cache)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = lib.pkv_paged_decode(_dev(q, "q", torch.bfloat16, dev),
                              _dev(k_cache, "k_cache", torch.bfloat16, dev),
                              _dev(v_cache, "v_cache", torch.bfloat16, dev),
                              _dev(block_tables, "block_tables", torch.int32, dev),
                              block_tables.shape[1],
                              _dev(context_lens, "context_lens", torch.int32, dev), B, Hq,
                              int(max_context_len), float(scale),
                              _dev(out, "out", torch.bfloat16, dev),
                              _dev(workspace, "workspace", torch.uint8, dev), workspace.numel(),
                              cache_desc(k_cache),
                              _ptr_or_null(status, "status", torch.int32, dev),
                              _stream(dev, stream))
    _check(rc, "pkv_paged_decode")
    return out


def paged_decode_plan(context_lens, num_q_heads, max_context_len, max_blocks_per_seq, k_cache,
                      workspace=None, status=None, stream=None) -> torch.Tensor:
    """The chunk schedule of a decode batch, written into `workspace` (made
    here when None), for any number of paged_decode_run calls over layers that
    share these context lengths.  Returns the workspace."""
    lib = load()
    dev = k_cache.device
    B = context_lens.numel()
    need = paged_decode_workspace_bytes(B, num_q_heads, max_context_len, k_cache)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = lib.pkv_paged_decode_plan(_dev(context_lens, "context_lens", torch.int32, dev), B,
                                   int(num_q_heads), int(max_context_len),
                                   int(max_blocks_per_seq),
                                   _dev(workspace, "workspace", torch.uint8, dev),
                                   workspace.numel(), cache_desc(k_cache),
                                   _ptr_or_null(status, "status", torch.int32, dev),
                                   _stream(dev, stream))
    _check(rc, "pkv_paged_decode_plan")
    return workspace


def paged_decode_run(q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                     workspace, out=None, status=None, stream=None) -> torch.Tensor:
    """paged_decode with the schedule a paged_decode_plan call wrote into
    `workspace` (same context lengths and sizes)."""
    lib = load()
    dev = k_cache.device
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    rc = lib.pkv_paged_decode_run(_dev(q, "q", torch.bfloat16, dev),
                                  _dev(k_cache, "k_cache", torch.bfloat16, dev),
                                  _dev(v_cache, "v_cache", torch.bfloat16, dev),
                                  _dev(block_tables, "block_tables", torch.int32, dev),
                                  block_tables.shape[1],
                                  _dev(context_lens, "context_lens", torch.int32, dev), B, Hq,
                                  int(max_context_len), float(scale),
                                  _dev(out, "out", torch.bfloat16, dev),
                                  _dev(workspace, "workspace", torch.uint8, dev),
                                  workspace.numel(), cache_desc(k_cache),
                                  _ptr_or_null(status, "status", torch.int32, dev),
                                  _stream(dev, stream))
    _check(rc, "pkv_paged_decode_run")
    return out


def paged_prefill_workspace_bytes(batch, total_q, num_q_heads, k_cache_shape) -> int:
    nb, bs, hkv, d = k_cache_shape
    return int(load().pkv_paged_prefill_workspace_bytes(batch, total_q, num_q_heads,
                                                        CacheDesc(nb, bs, hkv, d)))


def paged_prefill_varlen(q, k, v, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, block_tables, scale, out=None, workspace=None,
                         status=None, stream=None) -> torch.Tensor:
    """Causal varlen prefill: q [Tq, Hq, D], k/v [Tq, Hkv, D] bf16 -> out
    [Tq, Hq, D] bf16.  k_cache/v_cache and block_tables may be None when no
    sequence has a cached prefix."""
    lib = load()
    dev = q.device
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens_q.numel() - 1
    shape = tuple(k_cache.shape) if k_cache is not None else (1, 1, Hkv, D)
    if out is None:
        out = torch.empty_like(q)
    need = paged_prefill_workspace_bytes(B, T, Hq, shape)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    desc = CacheDesc(*shape)
    rc = lib.pkv_paged_prefill_varlen(
        _dev(q, "q", torch.bfloat16, dev), _dev(k, "k", torch.bfloat16, dev),
        _dev(v, "v", torch.bfloat16, dev),
        _ptr_or_null(k_cache, "k_cache", torch.bfloat16, dev),
        _ptr_or_null(v_cache, "v_cache", torch.bfloat16, dev),
        _dev(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev),
        _dev(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev), B, T, int(max_seqlen_q),
        int(max_seqlen_k), Hq, _ptr_or_null(block_tables, "block_tables", torch.int32, dev),
        block_tables.shape[1] if block_tables is not None else 0, float(scale),
        _dev(out, "out", torch.bfloat16, dev), _dev(workspace, "workspace", torch.uint8, dev),
        workspace.numel(), desc, _ptr_or_null(status, "status", torch.int32, dev),
        _stream(dev, stream))
    _check(rc, "pkv_paged_prefill_varlen")
    return out


def kv_store_paged_prefill_varlen(q, k, v, k_cache, v_cache, slot_mapping, cu_seqlens_q,
                                  cu_seqlens_k, max_seqlen_q, max_seqlen_k, block_tables, scale,
                                  out=None, workspace=None, status=None,
                                  stream=None) -> torch.Tensor:
    """kv_store of the chunk's k/v rows (slot_mapping [Tq] int32) followed by
    paged_prefill_varlen, in one call.  block_tables may be None when no
    sequence has a cached prefix; the cache is always written."""
    lib = load()
    dev = q.device
    T, Hq, D = q.shape
    B = cu_seqlens_q.numel() - 1
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must hold one slot per query token")
    if out is None:
        out = torch.empty_like(q)
    need = paged_prefill_workspace_bytes(B, T, Hq, tuple(k_cache.shape))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = lib.pkv_kv_store_paged_prefill_varlen(
        _dev(q, "q", torch.bfloat16, dev), _dev(k, "k", torch.bfloat16, dev),
        _dev(v, "v", torch.bfloat16, dev), _dev(k_cache, "k_cache", torch.bfloat16, dev),
        _dev(v_cache, "v_cache", torch.bfloat16, dev),
        _dev(slot_mapping, "slot_mapping", torch.int32, dev),
        _dev(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev),
        _dev(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev), B, T, int(max_seqlen_q),
        int(max_seqlen_k), Hq, _ptr_or_null(block_tables, "block_tables", torch.int32, dev),
        block_tables.shape[1] if block_tables is not None else 0, float(scale),
        _dev(out, "out", torch.bfloat16, dev), _dev(workspace, "workspace", torch.uint8, dev),
        workspace.numel(), cache_desc(k_cache), _ptr_or_null(status, "status", torch.int32, dev),
        _stream(dev, stream))
    _check(rc, "pkv_kv_store_paged_prefill_varlen")
    return out


def paged_attention_varlen_workspace_bytes(batch, total_q, num_q_heads, max_seqlen_k,
                                           k_cache_shape) -> int:
    nb, bs, hkv, d = k_cache_shape
    return int(load().pkv_paged_attention_varlen_workspace_bytes(
        batch, total_q, num_q_heads, int(max_seqlen_k), CacheDesc(nb, bs, hkv, d)))


def kv_store_paged_attention_varlen(q, k, v, k_cache, v_cache, slot_mapping, cu_seqlens_q,
                                    cu_seqlens_k, max_seqlen_q, max_seqlen_k, block_tables,
                                    scale, out=None, workspace=None, status=None,
                                    stream=None) -> torch.Tensor:
    """kv_store then attention over a batch mixing prefill chunks and decode
    rows: the result of kv_store_paged_prefill_varlen, with one-query
    sequences run by the split-KV decode kernels (they read their own new key
    back from the cache, so slot_mapping must place it in their block table).
    block_tables is required."""
    lib = load()
    dev = q.device
    T, Hq, D = q.shape
    B = cu_seqlens_q.numel() - 1
    if slot_mapping.shape != (T,):
        raise ValueError("slot_mapping must hold one slot per query token")
    if block_tables is None:
        raise ValueError("block_tables is required")
    if out is None:
        out = torch.empty_like(q)
    need = paged_attention_varlen_workspace_bytes(B, T, Hq, max_seqlen_k, tuple(k_cache.shape))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = lib.pkv_kv_store_paged_attention_varlen(
        _dev(q, "q", torch.bfloat16, dev), _dev(k, "k", torch.bfloat16, dev),
        _dev(v, "v", torch.bfloat16, dev), _dev(k_cache, "k_cache", torch.bfloat16, dev),
        _dev(v_cache, "v_cache", torch.bfloat16, dev),
        _dev(slot_mapping, "slot_mapping", torch.int32, dev),
        _dev(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev),
        _dev(cu_seqlens_k, "cu_seqlens_k", torch.int32, dev), B, T, int(max_seqlen_q),
        int(max_seqlen_k), Hq, _dev(block_tables, "block_tables", torch.int32, dev),
        block_tables.shape[1], float(scale),
        _dev(out, "out", torch.bfloat16, dev), _dev(workspace, "workspace", torch.uint8, dev),
        workspace.numel(), cache_desc(k_cache), _ptr_or_null(status, "status", torch.int32, dev),
        _stream(dev, stream))
    _check(rc, "pkv_kv_store_paged_attention_varlen")
    return out


def sample(logits, temperatures, exp_noise, out=None, status=None, stream=None) -> torch.Tensor:
    """Gumbel-max sampling: logits, exp_noise [B, V] fp32, temperatures [B]
    fp32 -> token ids [B] int32."""
    lib = load()
    dev = logits.device
    B, V = logits.shape
    if exp_noise.shape != logits.shape or temperatures.shape != (B,):
        raise ValueError("shape mismatch between logits, temperatures and exp_noise")
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=dev)
    rc = lib.pkv_sample(_dev(logits, "logits", torch.float32, dev),
                        _dev(temperatures, "temperatures", torch.float32, dev),
                        _dev(exp_noise, "exp_noise", torch.float32, dev), B, V,
                        _dev(out, "out", torch.int32, dev),
                        _ptr_or_null(status, "status", torch.int32, dev), _stream(dev, stream))
    _check(rc, "pkv_sample")
    return out


def paged_decode_static_workspace(q, k_cache, v_cache, block_tables, context_lens, scale,
                                  max_context_len, out=None, status=None,
                                  stream=None) -> torch.Tensor:
    """paged_decode for callers that cannot allocate device memory where they
    call (e.g. a plugin whose host engine owns all device memory, or a loop
    that must not pay for cudaMalloc's implicit synchronisation): the split-KV
    scratch is the library's own fixed array of STATIC_DECODE_WORKSPACE_BYTES,
    so apart from `out` (pass it to avoid the one allocation here) nothing is
    allocated.  Calls share that array: do not let two of them overlap on the
    GPU.  The first call on a device resolves the array's address; make it
    before any stream capture."""
    lib = load()
    fn = lib.pkv_paged_decode_static_workspace
    if fn.restype is not ctypes.c_int or not fn.argtypes:
        P, I32, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        fn.restype = ctypes.c_int
        fn.argtypes = [P, P, P, P, I32, P, I32, I32, I32, F32, P, CacheDesc, P, P]
    dev = k_cache.device
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    rc = fn(_dev(q, "q", torch.bfloat16, dev), _dev(k_cache, "k_cache", torch.bfloat16, dev),
            _dev(v_cache, "v_cache", torch.bfloat16, dev),
            _dev(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
            _dev(context_lens, "context_lens", torch.int32, dev), B, Hq, int(max_context_len),
            float(scale), _dev(out, "out", torch.bfloat16, dev), cache_desc(k_cache),
            _ptr_or_null(status, "status", torch.int32, dev), _stream(dev, stream))
    _check(rc, "pkv_paged_decode_static_workspace")
    return out


def kv_store_paged_decode(k, v, slot_mapping, q, k_cache, v_cache, block_tables, context_lens,
                          scale, max_context_len, out=None, workspace=None, status=None,
                          stream=None) -> torch.Tensor:
    """kv_store of the new tokens followed by paged_decode, in one call."""
    lib = load()
    dev = k_cache.device
    B, Hq, D = q.shape
    n = slot_mapping.numel()
    if k.shape != (n,) + tuple(k_cache.shape[2:]) or v.shape != k.shape:
        raise ValueError("k/v must be [num_tokens, num_kv_heads, head_dim] matching the cache")
    if out is None:
        out = torch.empty_like(q)
    need = paged_decode_workspace_bytes(B, Hq, max_context_len, k_cache)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = lib.pkv_kv_store_paged_decode(
        _dev(k, "k", torch.bfloat16, dev), _dev(v, "v", torch.bfloat16, dev),
        _dev(slot_mapping, "slot_mapping", torch.int32, dev), n,
        _dev(q, "q", torch.bfloat16, dev), _dev(k_cache, "k_cache", torch.bfloat16, dev),
        _dev(v_cache, "v_cache", torch.bfloat16, dev),
        _dev(block_tables, "block_tables", torch.int32, dev), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32, dev), B, Hq, int(max_context_len),
        float(scale), _dev(out, "out", torch.bfloat16, dev),
        _dev(workspace, "workspace", torch.uint8, dev), workspace.numel(), cache_desc(k_cache),
        _ptr_or_null(status, "status", torch.int32, dev), _stream(dev, stream))
    _check(rc, "pkv_kv_store_paged_decode")
    return out


def layer_cache(kv_pool: torch.Tensor, layer: int):
    """(k_cache, v_cache) views of one layer of a [2, L, NB, bs, Hkv, D] bf16 pool.
    The layer's addresses come from pkv_layer_cache (checked against the views)."""
    if kv_pool.dim() != 6 or kv_pool.shape[0] != 2 or not kv_pool.is_contiguous():
        raise ValueError("kv_pool must be a contiguous [2, L, NB, bs, Hkv, D] tensor")
    L, nb, bs, hkv, d = kv_pool.shape[1:]
    kp, vp = ctypes.c_void_p(), ctypes.c_void_p()
    rc = load().pkv_layer_cache(kv_pool.data_ptr(), L, int(layer), CacheDesc(nb, bs, hkv, d),
                                ctypes.byref(kp), ctypes.byref(vp))
    _check(rc, "pkv_layer_cache")
    kc, vc = kv_pool[0, layer], kv_pool[1, layer]
    if kc.data_ptr() != kp.value or vc.data_ptr() != vp.value:
        raise RuntimeError("pkv_layer_cache disagrees with the tensor layout")
    return kc, vc


def sample_philox(logits, temperatures, seed: int, offset: int, out=None, status=None,
                  stream=None) -> torch.Tensor:
    """Gumbel-max sampling with in-kernel Philox4x32-10 Exp(1) noise: logits
    [B, V] fp32, temperatures [B] fp32 -> token ids [B] int32."""
    lib = load()
    dev = logits.device
    B, V = logits.shape
    if temperatures.shape != (B,):
        raise ValueError("temperatures must be [batch]")
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=dev)
    rc = lib.pkv_sample_philox(_dev(logits, "logits", torch.float32, dev),
                               _dev(temperatures, "temperatures", torch.float32, dev),
                               int(seed) & (2**64 - 1), int(offset) & (2**64 - 1), B, V,
                               _dev(out, "out", torch.int32, dev),
                               _ptr_or_null(status, "status", torch.int32, dev),
                               _stream(dev, stream))
    _check(rc, "pkv_sample_philox")
    return out


DEFAULT_WAIT_POLLS = 1 << 20            # PKV_DEFAULT_WAIT_POLLS


def set_wait_poll_limit(polls: int = DEFAULT_WAIT_POLLS) -> None:
    """Polls a bounded in-kernel wait makes before it gives up, for calls
    enqueued afterwards (default DEFAULT_WAIT_POLLS).  A diagnostic: 0 makes
    every such wait give up at once, which exercises the kernels' unwinding."""
    _check(load().pkv_set_wait_poll_limit(int(polls) & 0xFFFFFFFF), "pkv_set_wait_poll_limit")


# ----------------------------------------------------------------------------
# The 8-bit KV cache and the logit rules.  These calls run with the tensors'
# device current, and allocate what they make themselves on `stream` when one is
# given, so that PyTorch's allocator hands that memory out again only behind the
# work enqueued there.
FP8 = torch.float8_e4m3fn


def _on(index, stream, call):
    """call(raw stream) with CUDA device `index` current and, if given, `stream`."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, expected cuda:{index}")
        with torch.cuda.stream(stream):                 # makes its device current too
            return call(stream.cuda_stream)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return call(torch._C._cuda_getCurrentRawStream(index))
    return call(torch._C._cuda_getCurrentRawStream(index))


def _at(t, name, dtype, index) -> int:
    """_dev for a tensor that must be on CUDA device `index`; when it is as it
    must be, a few attribute reads: a small call's time is mostly the host's."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index >= 0 and \
            t.is_contiguous():
        return t.data_ptr()
    return _dev(t, name, dtype, torch.device("cuda", max(index, 0)))


def _maybe(t, name, dtype, index):
    return None if t is None else _at(t, name, dtype, index)


@functools.lru_cache(maxsize=256)
def _desc(*shape) -> CacheDesc:
    return CacheDesc(*shape)


def _scratch(workspace, need, index, stream):
    """(address, bytes, address to give back) of the caller's workspace, or of one
    that lives for the call: taken from PyTorch's allocator on the call's stream
    and given back, by _done, behind the work enqueued there (no tensor is made
    for it, which would cost as much as the call's launches)."""
    if workspace is not None:
        return _at(workspace, "workspace", torch.uint8, index), workspace.numel(), None
    if need == 0:
        return None, 0, None
    p = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, stream)
    return p, need, p


def _done(scratch) -> None:
    if scratch is not None:
        torch._C._cuda_cudaCachingAllocator_raw_delete(scratch)


@functools.lru_cache(maxsize=1024)
def _need(name, *args) -> int:
    """A workspace query (a pure function of the sizes); the last four arguments
    are the cache's."""
    return int(getattr(load(), name)(*args[:-4], CacheDesc(*args[-4:])))


def _fp8_cache(k_cache, v_cache, k_scale, v_scale):
    """Checks an e4m3 cache; returns (device index, the four addresses, descriptor)."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both be [num_blocks, block_size, "
                         "num_kv_heads, head_dim]")
    if k_scale.shape != (shape[0], shape[2]) or v_scale.shape != k_scale.shape:
        raise ValueError("k_scale and v_scale must be [num_blocks, num_kv_heads]")
    index = k_cache.get_device()
    return index, (_at(k_cache, "k_cache", FP8, index), _at(v_cache, "v_cache", FP8, index),
                   _at(k_scale, "k_scale", torch.float32, index),
                   _at(v_scale, "v_scale", torch.float32, index)), _desc(*shape)


def _rows_of(k, v, n, desc, index):
    """Checks bf16 K/V rows [n, num_kv_heads, head_dim]; returns their addresses."""
    if k.shape != (n, desc.num_kv_heads, desc.head_dim) or v.shape != k.shape:
        raise ValueError("k/v must be [num_tokens, num_kv_heads, head_dim] matching the cache")
    return _at(k, "k", torch.bfloat16, index), _at(v, "v", torch.bfloat16, index)


def _decode_batch(q, block_tables, context_lens, desc, index):
    """Checks a decode batch over a cache; returns (B, Hq, table width, addresses)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != desc.head_dim:
        raise ValueError("q must be [batch, num_q_heads, head_dim] matching the cache")
    width = block_tables.shape
    if len(width) != 2 or width[0] != shape[0] or context_lens.shape != shape[:1]:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq] and context_lens "
                         "[batch]")
    return (shape[0], shape[1], width[1], _at(q, "q", torch.bfloat16, index),
            _at(block_tables, "block_tables", torch.int32, index),
            _at(context_lens, "context_lens", torch.int32, index))


def _out_like(out, q, index):
    if out is None:
        return torch.empty_like(q)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    _at(out, "out", q.dtype, index)
    return out


def kv_store_fp8_workspace_bytes(num_tokens, k_cache) -> int:
    return int(load().pkv_kv_store_fp8_workspace_bytes(num_tokens, cache_desc(k_cache)))


def kv_store_fp8(k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, workspace=None,
                 status=None, stream=None) -> None:
    """kv_store into an 8-bit cache (in place): k, v [N, Hkv, D] bf16 rows become
    e4m3 codes in k_cache / v_cache [NB, bs, Hkv, D] float8_e4m3fn, with one
    scale per block and kv head in k_scale / v_scale [NB, Hkv] fp32 (value =
    code * scale).  A block's scale is the smallest power of two that holds
    every row stored since its offset 0 was; where it grows, the block's
    earlier rows are re-scaled.  Of several tokens with one slot the last is
    stored.  Start with zeroed scales."""
    lib = load()
    index, cache, desc = _fp8_cache(k_cache, v_cache, k_scale, v_scale)
    n = slot_mapping.numel()
    rows = _rows_of(k, v, n, desc, index)
    slots = _at(slot_mapping, "slot_mapping", torch.int32, index)
    st = _maybe(status, "status", torch.int32, index)

    def call(s):
        need = 0 if workspace is not None else _need("pkv_kv_store_fp8_workspace_bytes", n,
                                                     *k_cache.shape)
        ws, size, own = _scratch(workspace, need, index, s)
        try:
            _check(lib.pkv_kv_store_fp8(*rows, *cache, slots, n, ws, size, desc, st, s),
                   "pkv_kv_store_fp8")
        finally:
            _done(own)
    _on(index, stream, call)


def _decode_fp8(name, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                max_context_len, out, workspace, status, stream):
    lib = load()
    index, cache, desc = _fp8_cache(k_cache, v_cache, k_scale, v_scale)
    B, Hq, width, qp, bt, ctx = _decode_batch(q, block_tables, context_lens, desc, index)
    st = _maybe(status, "status", torch.int32, index)
    max_len = int(max_context_len)

    def call(s):
        o = _out_like(out, q, index)
        need = 0 if workspace is not None else _need("pkv_paged_decode_fp8_workspace_bytes", B, Hq,
                                                     max_len, *k_cache.shape)
        ws, size, own = _scratch(workspace, need, index, s)
        try:
            _check(getattr(lib, name)(qp, *cache, bt, width, ctx, B, Hq, max_len, float(scale),
                                      o.data_ptr(), ws, size, desc, st, s), name)
        finally:
            _done(own)
        return o
    return _on(index, stream, call)


def paged_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                     max_context_len, out=None, workspace=None, status=None,
                     stream=None) -> torch.Tensor:
    """paged_decode over an 8-bit cache (see kv_store_fp8): q [B, Hq, D] bf16 ->
    out [B, Hq, D] bf16."""
    return _decode_fp8("pkv_paged_decode_fp8", q, k_cache, v_cache, k_scale, v_scale,
                       block_tables, context_lens, scale, max_context_len, out, workspace,
                       status, stream)


def paged_decode_fp8_workspace_bytes(batch, num_q_heads, max_context_len, k_cache) -> int:
    return int(load().pkv_paged_decode_fp8_workspace_bytes(batch, num_q_heads,
                                                           int(max_context_len),
                                                           cache_desc(k_cache)))


def paged_decode_plan_fp8(context_lens, num_q_heads, max_context_len, max_blocks_per_seq, k_cache,
                          workspace=None, status=None, stream=None) -> torch.Tensor:
    """The chunk schedule of a decode batch over an 8-bit cache of k_cache's shape,
    for any number of paged_decode_run_fp8 calls (as paged_decode_plan is for
    paged_decode_run).  Returns the workspace."""
    lib = load()
    index = k_cache.get_device()
    _at(k_cache, "k_cache", FP8, index)
    ctx = _at(context_lens, "context_lens", torch.int32, index)
    st = _maybe(status, "status", torch.int32, index)
    desc = _desc(*k_cache.shape)
    B, Hq, max_len = context_lens.numel(), int(num_q_heads), int(max_context_len)

    def call(s):
        ws = workspace
        if ws is None:
            need = lib.pkv_paged_decode_fp8_workspace_bytes(B, Hq, max_len, desc)
            ws = torch.empty(max(need, 16), dtype=torch.uint8, device=k_cache.device)
        _check(lib.pkv_paged_decode_plan_fp8(ctx, B, Hq, max_len, int(max_blocks_per_seq),
                                             _at(ws, "workspace", torch.uint8, index), ws.numel(),
                                             desc, st, s), "pkv_paged_decode_plan_fp8")
        return ws
    return _on(index, stream, call)


def paged_decode_run_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale,
                         max_context_len, workspace, out=None, status=None,
                         stream=None) -> torch.Tensor:
    """paged_decode_fp8 with the schedule a paged_decode_plan_fp8 call wrote into
    `workspace` (same context lengths and sizes)."""
    if workspace is None:
        raise ValueError("workspace must hold a plan")
    return _decode_fp8("pkv_paged_decode_run_fp8", q, k_cache, v_cache, k_scale, v_scale,
                       block_tables, context_lens, scale, max_context_len, out, workspace,
                       status, stream)


def kv_store_paged_decode_fp8_workspace_bytes(num_tokens, batch, num_q_heads, max_context_len,
                                              k_cache) -> int:
    return int(load().pkv_kv_store_paged_decode_fp8_workspace_bytes(
        num_tokens, batch, num_q_heads, int(max_context_len), cache_desc(k_cache)))


def kv_store_paged_decode_fp8(k, v, slot_mapping, q, k_cache, v_cache, k_scale, v_scale,
                              block_tables, context_lens, scale, max_context_len, out=None,
                              workspace=None, status=None, stream=None) -> torch.Tensor:
    """kv_store_fp8 of the new tokens followed by paged_decode_fp8, in one call."""
    lib = load()
    index, cache, desc = _fp8_cache(k_cache, v_cache, k_scale, v_scale)
    n = slot_mapping.numel()
    rows = _rows_of(k, v, n, desc, index)
    slots = _at(slot_mapping, "slot_mapping", torch.int32, index)
    B, Hq, width, qp, bt, ctx = _decode_batch(q, block_tables, context_lens, desc, index)
    st = _maybe(status, "status", torch.int32, index)
    max_len = int(max_context_len)

    def call(s):
        o = _out_like(out, q, index)
        need = 0 if workspace is not None else _need(
            "pkv_kv_store_paged_decode_fp8_workspace_bytes", n, B, Hq, max_len, *k_cache.shape)
        ws, size, own = _scratch(workspace, need, index, s)
        try:
            _check(lib.pkv_kv_store_paged_decode_fp8(
                *rows, slots, n, qp, *cache, bt, width, ctx, B, Hq, max_len, float(scale),
                o.data_ptr(), ws, size, desc, st, s), "pkv_kv_store_paged_decode_fp8")
        finally:
            _done(own)
        return o
    return _on(index, stream, call)


def paged_prefill_fp8_workspace_bytes(batch, total_q, num_q_heads, max_seqlen_k,
                                      k_cache_shape) -> int:
    nb, bs, hkv, d = k_cache_shape
    return int(load().pkv_paged_prefill_fp8_workspace_bytes(
        batch, total_q, num_q_heads, int(max_seqlen_k), CacheDesc(nb, bs, hkv, d)))


def paged_prefill_varlen_fp8(q, k, v, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q,
                             cu_seqlens_k, max_seqlen_q, max_seqlen_k, block_tables, scale,
                             out=None, workspace=None, status=None,
                             stream=None) -> torch.Tensor:
    """paged_prefill_varlen whose cached prefix lies in an 8-bit cache (see
    kv_store_fp8); the chunk's own k/v [Tq, Hkv, D] are bf16 rows.  block_tables is
    required (without a cached prefix, call paged_prefill_varlen).  Output rows
    of no sequence are left unwritten."""
    lib = load()
    index, cache, desc = _fp8_cache(k_cache, v_cache, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != desc.head_dim:
        raise ValueError("q must be [total_q, num_q_heads, head_dim] matching the cache")
    T, Hq, _ = q.shape
    rows = _rows_of(k, v, T, desc, index)
    B = cu_seqlens_q.numel() - 1
    if B < 0 or cu_seqlens_k.numel() != B + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must both be [batch + 1]")
    if block_tables is None:
        raise ValueError("block_tables is required")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be [batch, max_blocks_per_seq]")
    qp = _at(q, "q", torch.bfloat16, index)
    cu_q = _at(cu_seqlens_q, "cu_seqlens_q", torch.int32, index)
    cu_k = _at(cu_seqlens_k, "cu_seqlens_k", torch.int32, index)
    bt = _at(block_tables, "block_tables", torch.int32, index)
    st = _maybe(status, "status", torch.int32, index)
    max_q, max_k, width = int(max_seqlen_q), int(max_seqlen_k), block_tables.shape[1]

    def call(s):
        o = _out_like(out, q, index)
        need = 0 if workspace is not None else _need("pkv_paged_prefill_fp8_workspace_bytes", B, T,
                                                     Hq, max_k, *k_cache.shape)
        ws, size, own = _scratch(workspace, need, index, s)
        try:
            _check(lib.pkv_paged_prefill_varlen_fp8(
                qp, *rows, *cache, cu_q, cu_k, B, T, max_q, max_k, Hq, bt, width, float(scale),
                o.data_ptr(), ws, size, desc, st, s), "pkv_paged_prefill_varlen_fp8")
        finally:
            _done(own)
        return o
    return _on(index, stream, call)


_LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def apply_logit_rules(logits, token_ids=None, prompt_lens=None, token_lens=None,
                      repetition_penalties=None, presence_penalties=None,
                      frequency_penalties=None, bias_offsets=None, bias_token_ids=None,
                      bias_values=None, allowed_mask=None, out=None, status=None,
                      stream=None) -> torch.Tensor:
    """Penalties, biases and a mask on a step's logits, for sample: logits
    [B, V] fp32, bf16 or fp16 (rows may be strided) -> [B, V] fp32.

    token_ids [B, T] int32 holds each row's prompt and generated tokens, of which
    the first prompt_lens [B] are prompt and token_lens [B] count (None: none, and
    all T); the penalties are [B] fp32 (None: off).  Row b's biases are entries
    bias_offsets[b] .. bias_offsets[b + 1] of bias_token_ids int32 and
    bias_values fp32 (the last one for a token counts).  allowed_mask
    [B, ceil(V / 32)] int32 has bit i % 32 of word i / 32 set where token i may be
    drawn.  Pass out=logits (fp32, contiguous) to work in place."""
    lib = load()
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    kind = _LOGIT_TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be fp32, bf16 or fp16, got {logits.dtype}")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [batch, vocab] with contiguous rows")
    B, V = logits.shape
    stride = logits.stride(0) if B > 1 else V
    if stride < V:
        raise ValueError("rows of logits overlap")
    index = logits.get_device()
    r = LogitRules()
    i32, f32 = torch.int32, torch.float32
    if token_ids is not None:
        if token_ids.dim() != 2 or token_ids.shape[0] != B:
            raise ValueError("token_ids must be [batch, max_tokens]")
        r.token_ids = _at(token_ids, "token_ids", i32, index)
        r.max_tokens = token_ids.shape[1]
    for name, t, dtype in (("prompt_lens", prompt_lens, i32), ("token_lens", token_lens, i32),
                           ("repetition_penalties", repetition_penalties, f32),
                           ("presence_penalties", presence_penalties, f32),
                           ("frequency_penalties", frequency_penalties, f32)):
        if t is None:
            continue
        if token_ids is None:
            raise ValueError(f"{name} needs token_ids")
        if t.shape != (B,):
            raise ValueError(f"{name} must be [batch]")
        setattr(r, name, _at(t, name, dtype, index))
    if not (bias_offsets is None and bias_token_ids is None and bias_values is None):
        if bias_offsets is None or bias_token_ids is None or bias_values is None:
            raise ValueError("bias_offsets, bias_token_ids and bias_values go together")
        if bias_offsets.shape != (B + 1,) or bias_token_ids.dim() != 1 or \
                bias_values.shape != bias_token_ids.shape:
            raise ValueError("bias_offsets must be [batch + 1], the others [num_biases]")
        r.bias_offsets = _at(bias_offsets, "bias_offsets", i32, index)
        r.bias_token_ids = _at(bias_token_ids, "bias_token_ids", i32, index)
        r.bias_values = _at(bias_values, "bias_values", f32, index)
        r.num_biases = bias_token_ids.numel()
    if allowed_mask is not None:
        if allowed_mask.shape != (B, (V + 31) // 32):
            raise ValueError("allowed_mask must be [batch, ceil(vocab / 32)]")
        r.allowed_mask = _at(allowed_mask, "allowed_mask", i32, index)
    if out is not None:
        if out.shape != (B, V):
            raise ValueError("out must be [batch, vocab]")
        _at(out, "out", f32, index)
    st = _maybe(status, "status", torch.int32, index)

    def call(s):
        o = torch.empty((B, V), dtype=f32, device=logits.device) if out is None else out
        _check(lib.pkv_apply_logit_rules(logits.data_ptr(), kind, stride, B, V, r, o.data_ptr(),
                                         st, s), "pkv_apply_logit_rules")
        return o
    return _on(index, stream, call)
