"""ctypes binding of libdsa.so (C ABI in include/dsa.h).

Argument marshalling only: every step of the path runs in the library's CUDA kernels.
The functions keep the C names and take torch tensors (device memory owned by the
caller) plus the current CUDA stream.  If the library is missing or cannot load, the
call raises -- there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

DSA_BF16 = 0
DSA_E4M3 = 1
DSA_E4M3_UE8M0 = 2

DSA_ROPE_HALF = 0
DSA_ROPE_INTERLEAVED = 1
DSA_ROPE_BF16 = 0
DSA_ROPE_FP16 = 1
DSA_ROPE_FP32 = 2

_STATUS = {
    0: "DSA_OK",
    1: "DSA_ERR_INVALID_ARG",
    2: "DSA_ERR_UNSUPPORTED",
    3: "DSA_ERR_WORKSPACE",
    4: "DSA_ERR_CUDA",
    5: "DSA_ERR_DEVICE_TIMEOUT",
    6: "DSA_ERR_DEVICE_BOUNDS",
}

EXPORTED = (
    "dsa_indexer_scores",
    "dsa_topk",
    "dsa_indexer_topk_streaming_workspace_size",
    "dsa_indexer_topk_streaming",
    "dsa_sparse_mla_fwd",
    "dsa_dense_mla_fwd",
    "dsa_forward_workspace_size",
    "dsa_forward",
    "dsa_forward_noalloc",
    "dsa_forward_noalloc_scratch_bytes",
    "dsa_check_device_errors",
    "dsa_cache_write",
    "dsa_cache_write_bounded",
    "dsa_cache_write_fp8",
    "dsa_cache_write_fp8_bounded",
    "dsa_paged_plan",
    "dsa_rope",
    "dsa_rope_frequencies",
    "dsa_sparse_mla_fp8_workspace_size",
    "dsa_sparse_mla_fp8_fwd",
    "dsa_set_debug_checks",
    "dsa_selftest_bounded_wait",
    "dsa_status_string",
    "dsa_abi_version",
)


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {_STATUS.get(code, code)} ({msg})")
        self.code = code


class DsaProblem(ctypes.Structure):
    """Mirror of ``dsa_problem_t``."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("cu_q", ctypes.c_void_p),
        ("cu_k", ctypes.c_void_p),
        ("total_q", ctypes.c_int32),
        ("total_k", ctypes.c_int32),
        ("max_len_q", ctypes.c_int32),
        ("max_len_k", ctypes.c_int32),
        ("n_idx_heads", ctypes.c_int32),
        ("idx_dim", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("idx_dtype", ctypes.c_int32),
        ("sm_scale", ctypes.c_float),
        ("block_table", ctypes.c_void_p),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
    ]


class DsaRope(ctypes.Structure):
    """Mirror of ``dsa_rope_desc_t``."""

    _fields_ = [
        ("n_tokens", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rope_begin", ctypes.c_int32),
        ("rope_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("x_token_stride", ctypes.c_int64),
        ("x_head_stride", ctypes.c_int64),
        ("out_token_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("transposed", ctypes.c_int32),
    ]


_lib: Optional[ctypes.CDLL] = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libdsa.so (building it first when it is missing or stale and nvcc exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and _build.needs_build():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"libdsa.so not found at {_build.LIB}; run python -m attention_lightning_indexer_b200.build")
    lib = ctypes.CDLL(_build.LIB)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    pp = ctypes.POINTER(DsaProblem)
    lib.dsa_indexer_scores.argtypes = [pp, P, P, P, P, P, P, i64, i32, i32, P]
    lib.dsa_topk.argtypes = [pp, P, i64, i32, i32, P, P]
    lib.dsa_indexer_topk_streaming_workspace_size.argtypes = [pp, i32]
    lib.dsa_indexer_topk_streaming_workspace_size.restype = sz
    lib.dsa_indexer_topk_streaming.argtypes = [pp, P, P, P, P, P, i32, i32, i32, P, P, sz, P]
    lib.dsa_sparse_mla_fwd.argtypes = [pp, P, P, P, P, P, P]
    lib.dsa_dense_mla_fwd.argtypes = [pp, P, P, P, P, P, P]
    lib.dsa_forward_workspace_size.argtypes = [pp, i32]
    lib.dsa_forward_workspace_size.restype = sz
    lib.dsa_forward.argtypes = [pp, P, P, P, P, P, P, P, i32, P, P, P, P, sz, P]
    lib.dsa_forward_noalloc.argtypes = [pp, P, P, P, P, P, P, P, P, P, P, P]
    lib.dsa_forward_noalloc_scratch_bytes.argtypes = []
    lib.dsa_forward_noalloc_scratch_bytes.restype = sz
    lib.dsa_check_device_errors.argtypes = [P]
    lib.dsa_selftest_bounded_wait.argtypes = [ctypes.c_uint32, P]
    lib.dsa_cache_write.argtypes = [i32, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P]
    lib.dsa_cache_write_bounded.argtypes = [i32, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, i32, P]
    lib.dsa_cache_write_fp8.argtypes = [i32, P, P, P, P, P, P, P, P, ctypes.c_float, ctypes.c_int, P, P, P, P, P]
    lib.dsa_cache_write_fp8_bounded.argtypes = [i32, P, P, P, P, P, P, P, P, ctypes.c_float, ctypes.c_int, P, P, P, P, i32, P]
    lib.dsa_paged_plan.argtypes = [i32, P, P, P, i32, P, i32, P, i32, P, P, P, P, i32, P, P]
    lib.dsa_rope.argtypes = [ctypes.POINTER(DsaRope), P, P, P, P, P]
    dbl = ctypes.c_double
    lib.dsa_rope_frequencies.argtypes = [i32, dbl, dbl, dbl, dbl, dbl, P, ctypes.POINTER(dbl)]
    lib.dsa_sparse_mla_fp8_workspace_size.argtypes = [pp]
    lib.dsa_sparse_mla_fp8_workspace_size.restype = sz
    lib.dsa_sparse_mla_fp8_fwd.argtypes = [pp, P, P, P, P, P, P, P, sz, P]
    lib.dsa_set_debug_checks.argtypes = [i32]
    lib.dsa_set_debug_checks.restype = None
    lib.dsa_status_string.argtypes = [ctypes.c_int]
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_abi_version.restype = i32
    for name in ("dsa_indexer_scores", "dsa_topk", "dsa_indexer_topk_streaming", "dsa_sparse_mla_fwd", "dsa_dense_mla_fwd", "dsa_forward",
                 "dsa_forward_noalloc",
                 "dsa_check_device_errors", "dsa_selftest_bounded_wait", "dsa_cache_write", "dsa_cache_write_fp8",
                 "dsa_cache_write_bounded", "dsa_cache_write_fp8_bounded",
                 "dsa_paged_plan", "dsa_rope", "dsa_rope_frequencies", "dsa_sparse_mla_fp8_fwd"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _check(code: int, where: str) -> None:
    if code != 0:
        raise DsaError(code, where, load().dsa_status_string(code).decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libdsa takes device tensors only")
    if not t.is_contiguous():
        raise ValueError("libdsa takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_problem(batch: int, total_q: int, total_k: int, max_len_q: int, max_len_k: int, topk: int,
                 cu_q: Optional[torch.Tensor] = None, cu_k: Optional[torch.Tensor] = None,
                 idx_dtype: int = DSA_BF16, sm_scale: float = 1.0 / 192 ** 0.5,
                 n_idx_heads: int = 64, idx_dim: int = 128, n_heads: int = 128, d_qk: int = 576,
                 d_v: int = 512, block_table: Optional[torch.Tensor] = None, page_size: int = 64) -> DsaProblem:
    if cu_q is not None:
        assert cu_q.dtype == torch.int32 and cu_k is not None and cu_k.dtype == torch.int32
    max_pages = 0
    if block_table is not None:
        assert block_table.dtype == torch.int32 and block_table.dim() == 2
        max_pages = block_table.shape[1]
    return DsaProblem(batch, _ptr(cu_q), _ptr(cu_k), total_q, total_k, max_len_q, max_len_k, n_idx_heads,
                      idx_dim, n_heads, d_qk, d_v, topk, idx_dtype, sm_scale, _ptr(block_table), page_size,
                      max_pages)


def problem_from_inputs(inp: dict, sm_scale: float = 1.0 / 192 ** 0.5) -> DsaProblem:
    """dsa_problem_t for a dict produced by the seeded input generators (tensors on the GPU)."""
    fp8 = "q_idx8" in inp
    blocks = "q_scale_ue8m0" in inp
    paged = "block_table" in inp
    cu_q = inp.get("cu_q") if inp["batch"] > 1 or paged else None
    cu_k = inp.get("cu_k") if inp["batch"] > 1 or paged else None
    total_k = inp["phys_k"] if paged else inp["total_k"]
    return make_problem(inp["batch"], inp["total_q"], total_k, inp["max_len_q"], inp["max_len_k"],
                        inp["topk"], cu_q=cu_q, cu_k=cu_k,
                        idx_dtype=(DSA_E4M3_UE8M0 if blocks else DSA_E4M3) if fp8 else DSA_BF16,
                        sm_scale=sm_scale, block_table=inp.get("block_table"), page_size=inp.get("page_size", 64))


def scores_ld(max_len_k: int) -> int:
    return max(4, (max_len_k + 3) // 4 * 4)


# ---------------------------------------------------------------- entry points

def dsa_indexer_scores(p: DsaProblem, q_idx, k_idx, w, scores, row_begin: int = 0, row_count: Optional[int] = None,
                       q_scale=None, k_scale=None, stream=None) -> None:
    lib = load()
    if row_count is None:
        row_count = p.total_q - row_begin
    _check(lib.dsa_indexer_scores(ctypes.byref(p), _ptr(q_idx), _ptr(q_scale), _ptr(k_idx), _ptr(k_scale), _ptr(w),
                                  _ptr(scores), scores.stride(0), row_begin, row_count, _stream(stream)),
           "dsa_indexer_scores")


def dsa_topk(p: DsaProblem, scores, idx, row_begin: int = 0, row_count: Optional[int] = None, stream=None) -> None:
    lib = load()
    if row_count is None:
        row_count = p.total_q - row_begin
    _check(lib.dsa_topk(ctypes.byref(p), _ptr(scores), scores.stride(0), row_begin, row_count, _ptr(idx),
                        _stream(stream)), "dsa_topk")


def dsa_indexer_topk_streaming_workspace_size(p: DsaProblem, chunk_q: int = 0) -> int:
    return int(load().dsa_indexer_topk_streaming_workspace_size(ctypes.byref(p), chunk_q))


def dsa_indexer_topk_streaming(p: DsaProblem, q_idx, k_idx, w, idx, workspace, row_begin: int = 0,
                               row_count: Optional[int] = None, chunk_q: int = 0, q_scale=None, k_scale=None,
                               stream=None) -> None:
    """Indexer and top-k without score rows: the same idx as dsa_indexer_scores + dsa_topk."""
    lib = load()
    if row_count is None:
        row_count = p.total_q - row_begin
    _check(lib.dsa_indexer_topk_streaming(ctypes.byref(p), _ptr(q_idx), _ptr(q_scale), _ptr(k_idx), _ptr(k_scale),
                                          _ptr(w), row_begin, row_count, chunk_q, _ptr(idx), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)),
           "dsa_indexer_topk_streaming")


def dsa_sparse_mla_fwd(p: DsaProblem, q, kv, idx, out, lse, stream=None) -> None:
    lib = load()
    _check(lib.dsa_sparse_mla_fwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(out), _ptr(lse),
                                  _stream(stream)), "dsa_sparse_mla_fwd")


def dsa_dense_mla_fwd(p: DsaProblem, q, kv, idx, out, lse, stream=None) -> None:
    """Dense (masked MHA) form: all causal keys, restricted to idx's keys when idx is given."""
    lib = load()
    _check(lib.dsa_dense_mla_fwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(out), _ptr(lse),
                                 _stream(stream)), "dsa_dense_mla_fwd")


def dsa_forward_workspace_size(p: DsaProblem, chunk_q: int = 0) -> int:
    return int(load().dsa_forward_workspace_size(ctypes.byref(p), chunk_q))


def dsa_forward(p: DsaProblem, q_idx, k_idx, w, q, kv, out, lse, workspace, chunk_q: int = 0, idx_out=None,
                q_scale=None, k_scale=None, stream=None) -> None:
    lib = load()
    _check(lib.dsa_forward(ctypes.byref(p), _ptr(q_idx), _ptr(q_scale), _ptr(k_idx), _ptr(k_scale), _ptr(w), _ptr(q),
                           _ptr(kv), chunk_q, _ptr(idx_out), _ptr(out), _ptr(lse), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream)), "dsa_forward")


def dsa_forward_noalloc(p: DsaProblem, q_idx, k_idx, w, q, kv, idx_out, out, lse, q_scale=None, k_scale=None,
                        stream=None) -> None:
    """dsa_forward with the library's fixed scratch array instead of a caller workspace (no
    device allocation by the call; see include/dsa.h for the size limit and sharing rules)."""
    lib = load()
    _check(lib.dsa_forward_noalloc(ctypes.byref(p), _ptr(q_idx), _ptr(q_scale), _ptr(k_idx), _ptr(k_scale), _ptr(w),
                                   _ptr(q), _ptr(kv), _ptr(idx_out), _ptr(out), _ptr(lse), _stream(stream)),
           "dsa_forward_noalloc")


def dsa_forward_noalloc_scratch_bytes() -> int:
    return int(load().dsa_forward_noalloc_scratch_bytes())


def dsa_check_device_errors(stream=None) -> None:
    _check(load().dsa_check_device_errors(_stream(stream)), "dsa_check_device_errors")


_MOST_ROWS = 2 ** 31 - 1


def dsa_cache_write(k_idx_raw, kv_raw, positions, rows, k_norm_w, k_norm_b, kv_norm_w, inv_freq, k_idx_cache,
                    kv_cache, eps: float = 1e-6, stream=None) -> None:
    """Indexer-key and latent cache rows of new tokens (norms + RoPE; see include/dsa.h).  Rows past
    the end of either cache are passed over and reported by dsa_check_device_errors."""
    lib = load()
    n_rows = min(k_idx_cache.numel() // 128, kv_cache.numel() // 576, _MOST_ROWS)
    _check(lib.dsa_cache_write_bounded(int(positions.numel()), _ptr(k_idx_raw), _ptr(kv_raw), _ptr(positions), _ptr(rows),
                                       _ptr(k_norm_w), _ptr(k_norm_b), _ptr(kv_norm_w), _ptr(inv_freq), eps,
                                       _ptr(k_idx_cache), _ptr(kv_cache), n_rows, _stream(stream)), "dsa_cache_write")


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _addresses(where: str, *tensors_and_types):
    """Addresses of contiguous tensors of the given types (None: no tensor), all on the current
    device: the launch goes there, and a stream of another device would not order it."""
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else None   # None: no tensor's device
    for t, dtype in tensors_and_types:
        if t is not None and (t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous()):
            raise ValueError(f"{where}: expected a contiguous {dtype} tensor on the current CUDA device, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
    return [None if t is None else t.data_ptr() for t, _ in tensors_and_types]


# The current stream's handle without the Stream object around it (3 us of a call's 13)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _current_raw_stream(torch.cuda.current_device())


_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


def dsa_paged_plan(len_cached, len_new, block_table, free_pages, cu_q, cu_k, positions, rows, counts, n_pages: int,
                   free_head=None, stream=None) -> None:
    """Sequence offsets, slot map and block-table entries of one step, from the requests'
    lengths (see include/dsa.h).  ``positions`` and ``rows`` may be longer than the step's
    tokens (padding gets position 0 and row -1); ``counts`` [4] receives the new tokens, the
    pages taken, the longest sequence and the error bits."""
    a = _addresses("dsa_paged_plan", (len_cached, _I32), (len_new, _I32), (block_table, _I32), (free_pages, _I32),
                   (free_head, _I32), (cu_q, _I32), (cu_k, _I32), (positions, _I32), (rows, _I32), (counts, _I32))
    B, T = len_cached.numel(), positions.numel()
    _need(len_new.numel() == B and cu_q.numel() == B + 1 and cu_k.numel() == B + 1 and counts.numel() == 4
          and rows.numel() == T and block_table.dim() == 2 and block_table.shape[0] == B
          and (free_head is None or free_head.numel() == 1), "dsa_paged_plan: shapes do not agree")
    _check(load().dsa_paged_plan(B, a[0], a[1], a[2], block_table.shape[1], a[3], free_pages.numel(), a[4], n_pages, a[5],
                                 a[6], a[7], a[8], T, a[9], _raw_stream(stream)), "dsa_paged_plan")


_ROPE_TYPES = {torch.bfloat16: DSA_ROPE_BF16, torch.float16: DSA_ROPE_FP16, torch.float32: DSA_ROPE_FP32}


def dsa_rope(x, positions, inv_freq, out, layout: int = DSA_ROPE_INTERLEAVED, rope_begin: int = 0,
             rope_dim: Optional[int] = None, scale: float = 1.0, transposed: bool = False, stream=None) -> None:
    """Rotary positions on dims ``rope_begin .. + rope_dim`` of ``x`` [tokens, heads, head_dim]
    into ``out`` (same shape and type; ``out`` may be ``x``).  Both may be slices of wider
    tensors: only the last dimension has to be dense."""
    a = _addresses("dsa_rope", (positions, _I32), (inv_freq, _F32))
    dev = positions.get_device()
    _need(x.get_device() == dev and out.get_device() == dev, "dsa_rope: every tensor must be on the current CUDA device")
    _need(x.dim() == 3 and x.shape == out.shape, "dsa_rope takes x and out [tokens, heads, head_dim]")
    dtype = _ROPE_TYPES.get(x.dtype)
    _need(dtype is not None and out.dtype is x.dtype, "dsa_rope takes bf16, fp16 or fp32, the same for x and out")
    T, H, D = x.shape
    xs, os_ = x.stride(), out.stride()
    if rope_dim is None:
        rope_dim = D - rope_begin
    _need(xs[2] == 1 and os_[2] == 1 or D == 1, "dsa_rope: the last dimension must be dense")
    _need(positions.numel() == T, "dsa_rope: positions must be int32 [tokens]")
    _need(2 * inv_freq.numel() == rope_dim, "dsa_rope: inv_freq must be fp32 [rope_dim / 2]")
    r = DsaRope(T, H, D, rope_begin, rope_dim, layout, dtype, xs[0], xs[1], os_[0], os_[1], scale, 1 if transposed else 0)
    _check(load().dsa_rope(ctypes.byref(r), x.data_ptr(), a[0], a[1], out.data_ptr(), _raw_stream(stream)), "dsa_rope")


def dsa_rope_frequencies(rope_dim: int, base: float = 10000.0, factor: float = 1.0, original_len: float = 4096.0,
                         beta_fast: float = 32.0, beta_slow: float = 1.0):
    """RoPE frequencies (a host fp32 tensor [rope_dim / 2]) and the attention factor; ``factor``
    > 1 stretches them for long contexts.  The factor belongs on queries and keys both; the cache
    writes do not scale keys, so a model that uses it gives its square as ``scale`` of dsa_rope
    (see include/dsa.h)."""
    freq = torch.empty(max(rope_dim, 0) // 2, dtype=torch.float32)
    att = ctypes.c_double()
    _check(load().dsa_rope_frequencies(rope_dim, base, factor, original_len, beta_fast, beta_slow,
                                       ctypes.c_void_p(freq.data_ptr()), ctypes.byref(att)), "dsa_rope_frequencies")
    return freq, att.value


_KEY_TYPES = {DSA_BF16: (torch.bfloat16, None), DSA_E4M3: (torch.uint8, torch.float32), DSA_E4M3_UE8M0: (torch.uint8, torch.uint8)}


def dsa_cache_write_fp8(k_idx_raw, kv_raw, positions, rows, k_norm_w, k_norm_b, kv_norm_w, inv_freq, k_idx_cache,
                        k_scale_cache, kv_cache, kv_scale_cache, idx_dtype: int = DSA_E4M3_UE8M0, eps: float = 1e-6,
                        stream=None) -> None:
    """dsa_cache_write into an 8-bit cache: the indexer key as ``idx_dtype`` says, the latent as
    640 e4m3 codes and one ue8m0 scale per row (see include/dsa.h).  Rows past the end of either
    cache are passed over and reported by dsa_check_device_errors."""
    n = positions.numel()
    key, scale = _KEY_TYPES.get(idx_dtype, (None, None))
    _need(key is not None, "dsa_cache_write_fp8: idx_dtype must be DSA_BF16, DSA_E4M3 or DSA_E4M3_UE8M0")
    _need((k_scale_cache is None) == (scale is None), "dsa_cache_write_fp8: k_scale_cache does not fit idx_dtype")
    a = _addresses("dsa_cache_write_fp8", (k_idx_raw, _BF16), (kv_raw, _BF16), (positions, _I32), (rows, _I32), (k_norm_w, _F32),
                   (k_norm_b, _F32), (kv_norm_w, _F32), (inv_freq, _F32), (k_idx_cache, key), (k_scale_cache, scale),
                   (kv_cache, _U8), (kv_scale_cache, _U8))
    _need(rows.numel() == n and k_idx_raw.numel() == 128 * n and kv_raw.numel() == 576 * n,
          "dsa_cache_write_fp8: k_idx_raw [n, 128], kv_raw [n, 576], positions and rows [n]")
    _need(k_norm_w.numel() == 128 and k_norm_b.numel() == 128 and kv_norm_w.numel() == 512 and inv_freq.numel() == 32,
          "dsa_cache_write_fp8: k_norm_w, k_norm_b [128], kv_norm_w [512], inv_freq [32]")
    _need(k_idx_cache.shape[-1] == 128 and kv_cache.shape[-1] == 640
          and kv_scale_cache.numel() * 640 == kv_cache.numel()
          and (scale is None or k_scale_cache.numel() * 128 == k_idx_cache.numel()), "dsa_cache_write_fp8: cache shapes")
    n_rows = min(k_idx_cache.numel() // 128, kv_scale_cache.numel(), _MOST_ROWS)
    _check(load().dsa_cache_write_fp8_bounded(n, a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], eps, idx_dtype, a[8], a[9],
                                              a[10], a[11], n_rows, _raw_stream(stream)), "dsa_cache_write_fp8")


def dsa_sparse_mla_fp8_workspace_size(p: DsaProblem) -> int:
    return int(load().dsa_sparse_mla_fp8_workspace_size(ctypes.byref(p)))


def dsa_sparse_mla_fp8_fwd(p: DsaProblem, q, kv, kv_scale, idx, out, lse, workspace=None, stream=None) -> None:
    """dsa_sparse_mla_fwd over the 8-bit latent cache (kv uint8 [S, 640], kv_scale uint8 [S])."""
    a = _addresses("dsa_sparse_mla_fp8_fwd", (q, _BF16), (kv, _U8), (kv_scale, _U8), (idx, _I32), (out, _BF16), (lse, _F32),
                   (workspace, _U8))
    T, S = p.total_q, p.total_k
    _need(q.numel() == T * 128 * 576 and out.numel() == T * 128 * 512 and lse.numel() == T * 128
          and idx.numel() == T * p.topk and kv.numel() >= S * 640 and kv_scale.numel() >= S,
          "dsa_sparse_mla_fp8_fwd: shapes do not fit the problem")
    _check(load().dsa_sparse_mla_fp8_fwd(ctypes.byref(p), a[0], a[1], a[2], a[3], a[4], a[5], a[6],
                                         0 if workspace is None else workspace.numel(), _raw_stream(stream)),
           "dsa_sparse_mla_fp8_fwd")


def dsa_set_debug_checks(enable: bool) -> None:
    """Per-row input checks in every kernel (see include/dsa.h)."""
    load().dsa_set_debug_checks(1 if enable else 0)


def dsa_selftest_bounded_wait(limit_us: int = 1000, stream=None) -> None:
    """Launch the one-CTA kernel whose bounded wait runs out (see include/dsa.h)."""
    _check(load().dsa_selftest_bounded_wait(limit_us, _stream(stream)), "dsa_selftest_bounded_wait")
