"""Python binding of the C ABI in include/pa.h (argument marshalling only).

Each function here has the name of the C entry point it calls, takes torch tensors,
checks that they are CUDA tensors of the expected dtype and layout, and passes their
device pointers through ctypes.  All arithmetic runs in the library's kernels; there
is no fallback: if ``_build/libpa.so`` is missing the first call raises.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import build as _build

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_SCRATCH_LIMIT = 0, 1, 2, 3, 4
PA_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024
PA_KV_BF16, PA_KV_INT8, PA_KV_E4M3 = 0, 1, 2
PA_Q_MODE_NONE, PA_Q_MODE_CUMSUM, PA_Q_MODE_STRIDED = 0, 1, 2
PA_PRODUCER_AUTO, PA_PRODUCER_FMA, PA_PRODUCER_MMA = 0, 1, 2
DEVERR_PAGE_OUT_OF_RANGE = 0x1
DEVERR_POOL_ROW_OUT_OF_RANGE = 0x2
DEVERR_SLOT_OUT_OF_RANGE = 0x4
DEVERR_WAIT_TIMEOUT = 0x8
DEVERR_SEQLEN_OUT_OF_RANGE = 0x10
DEVERR_KEPT_OUT_OF_RANGE = 0x20
DEVERR_TREE_PARENT = 0x40
DEVERR_TOKEN_OUT_OF_RANGE = 0x80
DEVERR_NO_PROBABILITY = 0x100
DEVERR_OUT_OF_PAGES = 0x200
DEVERR_PAGE_REFS = 0x400
PA_ROPE_PLAIN, PA_ROPE_LINEAR, PA_ROPE_BASE, PA_ROPE_BY_PARTS, PA_ROPE_WAVELENGTH = range(5)

_lock = threading.Lock()
_lib: Optional[ctypes.CDLL] = None


class PAError(RuntimeError):
    def __init__(self, func: str, status: int, lib=None):
        self.status = status
        detail = ""
        if status == PA_ERR_CUDA:
            detail = ": " + (lib or load()).pa_last_error_string().decode()
        super().__init__(f"{func} failed: {status_string(status)} ({status}){detail}")


def library_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """Load libpa.so (built by ``build.build()``, or the file named by the PA_LIBRARY
    environment variable); raise if it is not there."""
    global _lib
    with _lock:
        if _lib is None:
            path = os.environ.get("PA_LIBRARY") or _build.LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(
                    f"CUDA library {path} is missing; build it with "
                    "`python -m paged_kv_decode_metadata_gb300.build`")
            _lib = _declare(ctypes.CDLL(path))
    return _lib


_ts_lib: Optional[ctypes.CDLL] = None


def load_instrumented() -> ctypes.CDLL:
    """Load the timestamp-instrumented build ``_build/libpa_ts.so`` (same entry points
    plus pa_set_timestamp_buffer, include/pa_timestamps.h); raise if it is missing."""
    global _ts_lib
    with _lock:
        if _ts_lib is None:
            path = _build.TS_LIB_PATH
            if not os.path.exists(path):
                raise RuntimeError(f"instrumented library {path} is missing; build it with "
                                   "`python -m paged_kv_decode_metadata_gb300.build --ts`")
            lib = _declare(ctypes.CDLL(path))
            lib.pa_set_timestamp_buffer.argtypes = [ctypes.c_void_p]
            lib.pa_set_timestamp_buffer.restype = ctypes.c_int
            lib.pa_set_test_hold_loads.argtypes = [ctypes.c_int32]
            lib.pa_set_test_hold_loads.restype = ctypes.c_int
            lib.pa_set_test_no_persist.argtypes = [ctypes.c_int32]
            lib.pa_set_test_no_persist.restype = ctypes.c_int
            _ts_lib = lib
    return _ts_lib


def _declare(lib):
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.pa_build_metadata.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp, vp, vp, i64, vp, i64,
                                      i32, i32, i32, i32, vp, i32]
    lib.pa_build_metadata_full.argtypes = [vp, vp, i32, vp, i64, i64, vp, i64, vp, i64, vp, vp,
                                           vp, vp, vp, i64, vp, i64, vp, i64, i32, i32, i32,
                                           i32, i32, i32, vp, i32]
    lib.pa_decode_splitk.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, vp, i32, i32, i32, i32,
                                     i32, i64, i32, i32, f32, vp, vp, vp, vp, i32]
    lib.pa_decode_splitk_multi.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, vp, vp, i32, i32,
                                           i32, i32, i32, i32, i64, i32, i32, f32, vp, vp, vp,
                                           vp, i32]
    lib.pa_decode_splitk_window.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, vp, vp, i32, i32,
                                            i32, i32, i32, i32, i64, i32, i32, i32, f32, vp, vp,
                                            vp, vp, i32]
    lib.pa_window_pages.argtypes = [i32, i32, i32, i32]
    lib.pa_window_pages.restype = i32
    lib.pa_reduce.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, i32]
    lib.pa_decode_step.argtypes = [vp, vp, vp, i64, i64, vp, i64, i32, i32, vp, vp, vp, i64,
                                   vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                   i64, i32, f32, vp, sz, vp, vp, vp, i32]
    lib.pa_decode_step_host.argtypes = [vp, vp, vp, vp, vp] + lib.pa_decode_step.argtypes
    step = lib.pa_decode_step.argtypes
    lib.pa_decode_step_host_packed.argtypes = [vp, vp, vp, vp] + step[2:15] + step[16:31] + \
        step[33:35]
    lib.pa_packed_input_bytes.argtypes = [i32, i32, i32]
    lib.pa_packed_input_bytes.restype = sz
    lib.pa_packed_output_bytes.argtypes = [i32, i32, i32]
    lib.pa_packed_output_bytes.restype = sz
    lib.pa_decode_step_multi.argtypes = [vp, vp, vp, i64, i64, vp, i64, i32, i32, vp, vp, vp,
                                         i64, vp, i64, vp, i32, i32, vp, vp, i32, i32, vp, vp,
                                         vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, f32, vp,
                                         sz, vp, vp, vp, i32]
    lib.pa_decode_step_window.argtypes = [vp, vp, vp, i64, i64, vp, i64, i32, i32, vp, vp, vp,
                                          i64, vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                          i32, i32, i64, i32, i32, f32, vp, sz, vp, vp, vp, i32]
    lib.pa_decode_step_static_scratch.argtypes = [vp, vp, vp, i64, i64, vp, i64, i32, i32, vp,
                                                  vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, i32,
                                                  i32, i32, i32, i32, i32, i64, i32, f32, vp, vp,
                                                  vp, i32]
    lib.pa_decode_step_static_scratch.restype = ctypes.c_int
    f64 = ctypes.c_double
    lib.pa_rope_frequencies.argtypes = [vp, i32, f64, i32, f64, i64, f64, f64]
    lib.pa_rope_append.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, i32, i32, f32, i32, i32,
                                   i32, i32, vp, i64, vp, vp, vp, vp, i32, i32, i64, vp, i32]
    lib.pa_rope_append_weights.argtypes = [*lib.pa_rope_append.argtypes[:22], vp,
                                           *lib.pa_rope_append.argtypes[22:]]
    lib.pa_build_tree_mask.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp, i32]
    lib.pa_tree_attention.argtypes = [vp, vp, vp, vp, vp, i32, vp, i64, vp, vp, vp, i32, i32, i32,
                                      i32, i32, i32, i32, i32, i64, i32, i32, f32, vp, sz, vp, vp,
                                      vp, i32]
    lib.pa_decode_step_tree.argtypes = [vp, vp, vp, i64, i64, vp, i64, i32, i32, vp, vp, vp, i64,
                                        vp, i64, vp, i32, i32, vp, vp, i32, vp, i32, i32, vp, vp,
                                        vp, vp, i32, i32, i32, i32, i32, i32, i64, i32, f32, vp,
                                        sz, vp, vp, vp, i32]
    lib.pa_choose_tree_splits.argtypes = [i32] * 7
    lib.pa_choose_tree_splits.restype = i32
    lib.pa_tree_workspace_bytes.argtypes = [i32] * 8
    lib.pa_tree_workspace_bytes.restype = sz
    lib.pa_accumulate_weights.argtypes = [vp, vp, vp, vp, i32, vp, i64, vp, vp, i32, i32, i32, i32,
                                          i32, i64, i32, f32, vp, i32]
    lib.pa_compact_cache.argtypes = [vp, i64, vp, i32, vp, i32, i64, vp, vp, i32, vp, vp, vp, vp,
                                     i32, vp, vp, i64, i32, vp, i32, i32, i32, i32, i64, vp, i32]
    lib.pa_evict.argtypes = [vp, i64, vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, i32,
                             vp, vp, i32, i32, i32, i32, i64, vp, i32]
    lib.pa_rope_append_blocks.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i32, i32, f32, vp, vp,
                                          vp, i64, i32, i32, i32, i32, i32, i32, i32, vp, i64, vp,
                                          vp, vp, vp, i32, i32, i32, i64, vp, i32]
    lib.pa_block_attention.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, i64, vp, vp, i32, i32, i32,
                                       i32, i32, i32, i32, i64, i32, i32, f32, vp, sz, vp, vp, vp,
                                       i32]
    lib.pa_decode_step_block.argtypes = [vp, vp, vp, i64, i64, vp, i64, i32, i32, vp, vp, vp, i64,
                                         vp, i64, vp, i32, i32, vp, vp, i32, i32, vp, vp, vp, vp,
                                         i32, i32, i32, i32, i32, i32, i32, i64, i32, f32, vp, sz,
                                         vp, vp, vp, i32]
    lib.pa_choose_block_splits.argtypes = [i32] * 7
    lib.pa_choose_block_splits.restype = i32
    lib.pa_block_workspace_bytes.argtypes = [i32] * 8
    lib.pa_block_workspace_bytes.restype = sz
    lib.pa_verify_drafts.argtypes = [vp, i64, vp, i64, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                     vp, i64, vp, vp, vp, vp, i32]
    lib.pa_pages_workspace_bytes.argtypes = [i64, i32]
    lib.pa_pages_workspace_bytes.restype = sz
    lib.pa_pages_copy.argtypes = [vp, vp, i32, i64, i64, vp, vp, i32, vp, i32]
    table = [vp, i64, i64, vp, i64, i32, i32]
    lib.pa_pages_fork.argtypes = table + [vp, vp, vp, i32, vp, i32, vp, vp, sz, vp, i32]
    lib.pa_pages_extend.argtypes = table + [vp, vp, vp, i32, vp, vp, sz, vp, i32]
    lib.pa_pages_free.argtypes = table + [vp, vp, vp, i32, vp, i32]
    lib.pa_pages_compact.argtypes = table + [vp, vp, i32, vp, i32, vp, vp, vp, sz, vp, i32]
    lib.pa_workspace_bytes.argtypes = [i32, i32, i32, i32]
    lib.pa_workspace_bytes.restype = sz
    lib.pa_choose_splits.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.pa_choose_splits.restype = i32
    lib.pa_select_producer.argtypes = [i32]
    lib.pa_select_producer.restype = i32
    lib.pa_last_error_string.argtypes = []
    lib.pa_last_error_string.restype = ctypes.c_char_p
    lib.pa_status_string.argtypes = [i32]
    lib.pa_status_string.restype = ctypes.c_char_p
    lib.pa_read_error_flags.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    for name in ("pa_build_metadata", "pa_build_metadata_full", "pa_decode_splitk",
                 "pa_decode_splitk_multi", "pa_decode_splitk_window", "pa_reduce",
                 "pa_decode_step", "pa_decode_step_host", "pa_decode_step_host_packed",
                 "pa_decode_step_multi",
                 "pa_decode_step_window", "pa_rope_frequencies", "pa_rope_append",
                 "pa_rope_append_weights",
                 "pa_build_tree_mask", "pa_tree_attention", "pa_decode_step_tree",
                 "pa_accumulate_weights", "pa_compact_cache", "pa_evict",
                 "pa_rope_append_blocks", "pa_block_attention", "pa_decode_step_block",
                 "pa_verify_drafts", "pa_pages_copy", "pa_pages_fork", "pa_pages_extend",
                 "pa_pages_free", "pa_pages_compact",
                 "pa_read_error_flags"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


def status_string(status: int) -> str:
    return load().pa_status_string(int(status)).decode()


def _check(func: str, status: int, lib=None):
    if status != PA_OK:
        raise PAError(func, status, lib)


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _io_ptr(t: Optional[torch.Tensor], dtype=None, name="tensor"):
    """Pointer of a step input or output that the kernels may also reach in pinned host
    memory (q, req_pool_indices, seq_lens, out, lse): a CUDA tensor, or a pinned CPU
    tensor, which the kernels then read or write over the host link (no copy)."""
    if t is not None and not t.is_cuda:
        if not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()
    return _ptr(t, dtype, name)


def _row_stride(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return t.stride(0)


def _ptr2d(t: torch.Tensor, dtype, name: str) -> int:
    """Pointer of a row-strided 2-D CUDA tensor (rows may be padded)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    _row_stride(t, name)
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def pa_build_metadata(req_pool_indices, seq_lens, req_to_token, cache_seqlens, cu_seqlens_k,
                      page_table, *, seqlen_offset: int, max_seq_pages: int, page_size: int,
                      full_to_swa_mapping=None, swa_page_table=None, stream=None,
                      use_pdl: bool = True):
    """Fused metadata update; see include/pa.h.  Outputs are written in place."""
    return pa_build_metadata_full(req_pool_indices, seq_lens, req_to_token, cache_seqlens,
                                  cu_seqlens_k, page_table, seqlen_offset=seqlen_offset,
                                  max_seq_pages=max_seq_pages, page_size=page_size,
                                  full_to_swa_mapping=full_to_swa_mapping,
                                  swa_page_table=swa_page_table, stream=stream, use_pdl=use_pdl)


def pa_build_metadata_full(req_pool_indices, seq_lens, req_to_token, cache_seqlens,
                           cu_seqlens_k, page_table, *, seqlen_offset: int, max_seq_pages: int,
                           page_size: int, full_to_swa_mapping=None, swa_page_table=None,
                           cu_seqlens_q=None, qlens=None, q_mode: int = PA_Q_MODE_NONE,
                           q_stride: int = 0, out_cache_loc=None, swa_out_cache_loc=None,
                           stream=None, use_pdl: bool = True):
    lib = load()
    bs = req_pool_indices.shape[0]
    pt_stride = _row_stride(page_table, "page_table")
    swa_stride = _row_stride(swa_page_table, "swa_page_table") if swa_page_table is not None else 0
    idx_dtype = req_pool_indices.dtype
    if idx_dtype not in (torch.int64, torch.int32):
        raise ValueError("req_pool_indices must be int64 or int32")
    st = lib.pa_build_metadata_full(
        _io_ptr(req_pool_indices, idx_dtype, "req_pool_indices"),
        _io_ptr(seq_lens, idx_dtype, "seq_lens"), 64 if idx_dtype == torch.int64 else 32,
        _ptr2d(req_to_token, torch.int32, "req_to_token"),
        req_to_token.shape[0], req_to_token.stride(0),
        _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
        full_to_swa_mapping.numel() if full_to_swa_mapping is not None else 0,
        _ptr(out_cache_loc, torch.int64, "out_cache_loc"),
        out_cache_loc.numel() if out_cache_loc is not None else 0,
        _ptr(qlens, idx_dtype, "qlens"),
        _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"),
        _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"),
        _ptr2d(page_table, torch.int32, "page_table"), pt_stride,
        _ptr2d(swa_page_table, torch.int32, "swa_page_table") if swa_page_table is not None else None,
        swa_stride,
        _ptr(swa_out_cache_loc, torch.int64, "swa_out_cache_loc"),
        swa_out_cache_loc.numel() if swa_out_cache_loc is not None else 0,
        bs, int(seqlen_offset), int(max_seq_pages), int(page_size), int(q_mode), int(q_stride),
        _stream(stream), int(bool(use_pdl)))
    _check("pa_build_metadata_full", st)


def _kv_args(k_cache, v_cache, k_scale, v_scale):
    if k_cache.dtype == torch.bfloat16:
        return PA_KV_BF16, None, None
    if k_cache.dtype == torch.int8:
        if k_scale is None or v_scale is None:
            raise ValueError("int8 KV needs k_scale and v_scale")
        return PA_KV_INT8, _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale")
    raise ValueError(f"unsupported KV dtype {k_cache.dtype}")


def pa_decode_splitk(q, k_cache, v_cache, page_table, cache_seqlens, scratch_m, scratch_l,
                     scratch_acc, *, max_seq_pages: int, num_splits: int, sm_scale: float,
                     k_scale=None, v_scale=None, stream=None, use_pdl: bool = True):
    """Split-K producer: writes per-split (m, l, acc) partials; see include/pa.h."""
    lib = load()
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    bs, hq, d = q.shape
    num_pages, hkv, page_size, _ = k_cache.shape
    st = lib.pa_decode_splitk(
        _io_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"),
        ks, vs, kv_dtype, _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"),
        _ptr(cache_seqlens, torch.int32, "cache_seqlens"), bs, hq, hkv, d, page_size, num_pages,
        int(max_seq_pages), int(num_splits), float(sm_scale),
        _ptr(scratch_m, torch.float32, "scratch_m"), _ptr(scratch_l, torch.float32, "scratch_l"),
        _ptr(scratch_acc, torch.float32, "scratch_acc"), _stream(stream), int(bool(use_pdl)))
    _check("pa_decode_splitk", st)


def pa_decode_splitk_multi(q, k_cache, v_cache, page_table, cache_seqlens, cu_seqlens_q,
                           scratch_m, scratch_l, scratch_acc, *, max_q_len: int,
                           max_seq_pages: int, num_splits: int, sm_scale: float, k_scale=None,
                           v_scale=None, stream=None, use_pdl: bool = True):
    """Split-K producer for several query tokens per request (rows from cu_seqlens_q,
    causal within the request's newest tokens); see include/pa.h."""
    lib = load()
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    total_q, hq, d = q.shape
    bs = cache_seqlens.shape[0]
    num_pages, hkv, page_size, _ = k_cache.shape
    st = lib.pa_decode_splitk_multi(
        _io_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"),
        ks, vs, kv_dtype, _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"), _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"), bs, int(max_q_len), hq, hkv, d,
        page_size, num_pages, int(max_seq_pages), int(num_splits), float(sm_scale),
        _ptr(scratch_m, torch.float32, "scratch_m"), _ptr(scratch_l, torch.float32, "scratch_l"),
        _ptr(scratch_acc, torch.float32, "scratch_acc"), _stream(stream), int(bool(use_pdl)))
    _check("pa_decode_splitk_multi", st)


def pa_decode_splitk_window(q, k_cache, v_cache, page_table, cache_seqlens, scratch_m,
                            scratch_l, scratch_acc, *, sliding_window: int, max_seq_pages: int,
                            num_splits: int, sm_scale: float, cu_seqlens_q=None,
                            max_q_len: int = 1, k_scale=None, v_scale=None, stream=None,
                            use_pdl: bool = True):
    """Split-K producer of a sliding-window layer: reads the sliding-window pool
    (``k_cache``/``v_cache``) through the sliding-window page table; one query per
    request, or the rows ``cu_seqlens_q`` assigns.  See include/pa.h."""
    lib = load()
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    rows, hq, d = q.shape
    bs = cache_seqlens.shape[0]
    num_pages, hkv, page_size, _ = k_cache.shape
    st = lib.pa_decode_splitk_window(
        _io_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"),
        ks, vs, kv_dtype, _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"), _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"), bs, int(max_q_len), hq, hkv, d,
        page_size, num_pages, int(max_seq_pages), int(sliding_window), int(num_splits),
        float(sm_scale), _ptr(scratch_m, torch.float32, "scratch_m"),
        _ptr(scratch_l, torch.float32, "scratch_l"), _ptr(scratch_acc, torch.float32, "scratch_acc"),
        _stream(stream), int(bool(use_pdl)))
    _check("pa_decode_splitk_window", st)


def pa_window_pages(sliding_window: int, max_q_len: int, page_size: int,
                    max_seq_pages: int) -> int:
    """Pages a sliding-window split partition spans; see include/pa.h."""
    return int(load().pa_window_pages(int(sliding_window), int(max_q_len), int(page_size),
                                      int(max_seq_pages)))


def pa_reduce(scratch_m, scratch_l, scratch_acc, out, lse=None, *, stream=None,
              use_pdl: bool = True):
    """Log-sum-exp reducer: writes out (bf16) and lse (fp32); see include/pa.h."""
    lib = load()
    bs, hq, s = scratch_m.shape
    d = scratch_acc.shape[-1]
    st = lib.pa_reduce(_ptr(scratch_m, torch.float32, "scratch_m"),
                       _ptr(scratch_l, torch.float32, "scratch_l"),
                       _ptr(scratch_acc, torch.float32, "scratch_acc"), bs, hq, d, s,
                       _io_ptr(out, torch.bfloat16, "out"), _io_ptr(lse, torch.float32, "lse"),
                       _stream(stream), int(bool(use_pdl)))
    _check("pa_reduce", st)


def pa_decode_step(*, lib=None, **kw):
    """Metadata + split-K producer + reducer in one call; see include/pa.h.  ``lib``
    selects another build of the library (e.g. ``load_instrumented()``).  Keyword
    arguments: those of ``_decode_step_args``."""
    lib = lib or load()
    _check("pa_decode_step", lib.pa_decode_step(*_decode_step_args(**kw)), lib)


def _decode_step_args(*, req_pool_indices, seq_lens, req_to_token, seqlen_offset: int,
                      max_seq_pages: int, cache_seqlens, cu_seqlens_k, page_table, q, k_cache,
                      v_cache, num_splits: int, sm_scale: float, workspace, out, lse=None,
                      k_scale=None, v_scale=None, full_to_swa_mapping=None, swa_page_table=None,
                      stream=None, use_pdl: bool = True):
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    bs, hq, d = q.shape
    num_pages, hkv, page_size, _ = k_cache.shape
    return (
        _io_ptr(req_pool_indices, torch.int64, "req_pool_indices"),
        _io_ptr(seq_lens, torch.int64, "seq_lens"), _ptr2d(req_to_token, torch.int32, "req_to_token"),
        req_to_token.shape[0], req_to_token.stride(0),
        _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
        full_to_swa_mapping.numel() if full_to_swa_mapping is not None else 0,
        int(seqlen_offset), int(max_seq_pages), _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"), _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"),
        _ptr2d(swa_page_table, torch.int32, "swa_page_table") if swa_page_table is not None else None,
        _row_stride(swa_page_table, "swa_page_table") if swa_page_table is not None else 0,
        _io_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"),
        _ptr(v_cache, None, "v_cache"), ks, vs, kv_dtype, bs, hq, hkv, d, page_size, num_pages,
        int(num_splits), float(sm_scale), _ptr(workspace, None, "workspace"),
        workspace.numel() * workspace.element_size(), _io_ptr(out, torch.bfloat16, "out"),
        _io_ptr(lse, torch.float32, "lse"), _stream(stream), int(bool(use_pdl)))


def _host_ptr(t, dtype, name):
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _decode_step_host_args(*, h_q, h_req_pool_indices, h_seq_lens, h_out, h_lse=None, **kw):
    return (_host_ptr(h_q, torch.bfloat16, "h_q"),
            _host_ptr(h_req_pool_indices, torch.int64, "h_req_pool_indices"),
            _host_ptr(h_seq_lens, torch.int64, "h_seq_lens"),
            _host_ptr(h_out, torch.bfloat16, "h_out"),
            _host_ptr(h_lse, torch.float32, "h_lse")) + _decode_step_args(**kw)


def pa_decode_step_host(*, lib=None, **kw):
    """pa_decode_step with host inputs (h_q, h_req_pool_indices, h_seq_lens) and host
    outputs (h_out, h_lse), copies enqueued on the same stream; see include/pa.h.  The
    other keyword arguments are those of ``pa_decode_step``."""
    lib = lib or load()
    _check("pa_decode_step_host", lib.pa_decode_step_host(*_decode_step_host_args(**kw)), lib)


def _decode_step_host_packed_args(*, h_inputs, inputs, h_outputs, outputs, **kw):
    """``kw``: the arguments of ``pa_decode_step``, whose q, req_pool_indices and
    seq_lens must be the views of ``inputs``, and out and lse those of ``outputs``, that
    the packed layout defines (their pointers are not passed; only shapes are read)."""
    a = _decode_step_args(**kw)
    bs, hq, d = a[21], a[22], a[24]
    lib = load()
    for t, name, n in ((h_inputs, "h_inputs", lib.pa_packed_input_bytes(bs, hq, d)),
                       (h_outputs, "h_outputs", lib.pa_packed_output_bytes(bs, hq, d))):
        if t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < n:
            raise ValueError(f"{name} must be a contiguous host buffer of {n} bytes")
    for t, name, n in ((inputs, "inputs", lib.pa_packed_input_bytes(bs, hq, d)),
                       (outputs, "outputs", lib.pa_packed_output_bytes(bs, hq, d))):
        if not t.is_cuda or not t.is_contiguous() or t.numel() * t.element_size() < n:
            raise ValueError(f"{name} must be a contiguous device buffer of {n} bytes")
    if a[15] != inputs.data_ptr() or a[0] != inputs.data_ptr() + d * hq * bs * 2 or \
            a[31] != outputs.data_ptr() or (a[32] is not None and
                                            a[32] != outputs.data_ptr() + d * hq * bs * 2):
        raise ValueError("q / req_pool_indices / seq_lens and out / lse must be the packed views")
    return (h_inputs.data_ptr(), inputs.data_ptr(), h_outputs.data_ptr(),
            outputs.data_ptr()) + a[2:15] + a[16:31] + a[33:35]


def pa_decode_step_multi(*, req_pool_indices, seq_lens, req_to_token, seqlen_offset: int,
                         max_seq_pages: int, cache_seqlens, cu_seqlens_k, page_table,
                         cu_seqlens_q, q, max_q_len: int, k_cache, v_cache, num_splits: int,
                         sm_scale: float, workspace, out, lse=None, qlens=None,
                         q_mode: int = PA_Q_MODE_CUMSUM, q_stride: int = 0, k_scale=None,
                         v_scale=None, full_to_swa_mapping=None, swa_page_table=None,
                         stream=None, use_pdl: bool = True):
    """Metadata (with cu_seqlens_q) + multi-query producer + reducer over the q rows;
    see include/pa.h."""
    lib = load()
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    total_q, hq, d = q.shape
    bs = cache_seqlens.shape[0]
    num_pages, hkv, page_size, _ = k_cache.shape
    st = lib.pa_decode_step_multi(
        _io_ptr(req_pool_indices, torch.int64, "req_pool_indices"),
        _io_ptr(seq_lens, torch.int64, "seq_lens"), _ptr2d(req_to_token, torch.int32, "req_to_token"),
        req_to_token.shape[0], req_to_token.stride(0),
        _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
        full_to_swa_mapping.numel() if full_to_swa_mapping is not None else 0,
        int(seqlen_offset), int(max_seq_pages), _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"), _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"),
        _ptr2d(swa_page_table, torch.int32, "swa_page_table") if swa_page_table is not None else None,
        _row_stride(swa_page_table, "swa_page_table") if swa_page_table is not None else 0,
        _ptr(qlens, torch.int64, "qlens"), int(q_mode), int(q_stride),
        _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"), _io_ptr(q, torch.bfloat16, "q"), total_q,
        int(max_q_len), _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"), ks, vs,
        kv_dtype, bs, hq, hkv, d, page_size, num_pages, int(num_splits), float(sm_scale),
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
        _io_ptr(out, torch.bfloat16, "out"), _io_ptr(lse, torch.float32, "lse"), _stream(stream),
        int(bool(use_pdl)))
    _check("pa_decode_step_multi", st)


def pa_decode_step_window(*, lib=None, **kw):
    """Metadata + sliding-window producer + reducer in one call; see include/pa.h.
    Keyword arguments: those of ``_decode_step_window_args``."""
    lib = lib or load()
    _check("pa_decode_step_window", lib.pa_decode_step_window(*_decode_step_window_args(**kw)),
           lib)


def _decode_step_window_args(*, req_pool_indices, seq_lens, req_to_token, seqlen_offset: int,
                             max_seq_pages: int, cache_seqlens, cu_seqlens_k, page_table,
                             full_to_swa_mapping, swa_page_table, q, k_swa, v_swa,
                             sliding_window: int, num_splits: int, sm_scale: float, workspace,
                             out, lse=None, k_swa_scale=None, v_swa_scale=None, stream=None,
                             use_pdl: bool = True):
    kv_dtype, ks, vs = _kv_args(k_swa, v_swa, k_swa_scale, v_swa_scale)
    bs, hq, d = q.shape
    num_pages, hkv, page_size, _ = k_swa.shape
    return (
        _io_ptr(req_pool_indices, torch.int64, "req_pool_indices"),
        _io_ptr(seq_lens, torch.int64, "seq_lens"), _ptr2d(req_to_token, torch.int32, "req_to_token"),
        req_to_token.shape[0], req_to_token.stride(0),
        _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
        full_to_swa_mapping.numel(), int(seqlen_offset), int(max_seq_pages),
        _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"), _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"), _ptr2d(swa_page_table, torch.int32, "swa_page_table"),
        _row_stride(swa_page_table, "swa_page_table"), _io_ptr(q, torch.bfloat16, "q"),
        _ptr(k_swa, None, "k_swa"), _ptr(v_swa, None, "v_swa"), ks, vs, kv_dtype, bs, hq, hkv, d,
        page_size, num_pages, int(sliding_window), int(num_splits), float(sm_scale),
        _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
        _io_ptr(out, torch.bfloat16, "out"), _io_ptr(lse, torch.float32, "lse"), _stream(stream),
        int(bool(use_pdl)))


class PreparedCall:
    """One entry point with its arguments marshalled once: calling it repeats the call
    on the same tensors, stream and options, without re-validating or re-converting the
    Python arguments.  The call holds references to the tensors it was prepared with
    (``keep``), so their memory stays allocated; they must stay in place (in-place
    updates are fine)."""

    def __init__(self, name: str, args: tuple, lib=None, keep: tuple = ()):
        self.lib = lib or load()
        self.name = name
        self.fn = getattr(self.lib, name)
        self.args = tuple(t(a) if a is not None else None
                          for t, a in zip(self.fn.argtypes, args))
        # (and to host arrays, and the tensors of a list of pools)
        flat = [x for k in keep for x in (k if isinstance(k, (list, tuple)) else (k,))]
        self._keep = tuple(k for k in flat if isinstance(k, (torch.Tensor, ctypes.Array)))

    def __call__(self):
        st = self.fn(*self.args)
        if st != PA_OK:
            raise PAError(self.name, st, self.lib)


def prepare_decode_step(*, lib=None, **kw) -> PreparedCall:
    """``pa_decode_step`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_decode_step", _decode_step_args(**kw), lib, keep=tuple(kw.values()))


def prepare_decode_step_host(*, lib=None, **kw) -> PreparedCall:
    """``pa_decode_step_host`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_decode_step_host", _decode_step_host_args(**kw), lib, keep=tuple(kw.values()))


def prepare_decode_step_host_packed(*, lib=None, **kw) -> PreparedCall:
    """``pa_decode_step_host_packed`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_decode_step_host_packed", _decode_step_host_packed_args(**kw), lib, keep=tuple(kw.values()))


def prepare_decode_step_window(*, lib=None, **kw) -> PreparedCall:
    """``pa_decode_step_window`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_decode_step_window", _decode_step_window_args(**kw), lib, keep=tuple(kw.values()))


def pa_decode_step_static_scratch(*, req_pool_indices, seq_lens, req_to_token,
                                  seqlen_offset: int, max_seq_pages: int, cache_seqlens,
                                  cu_seqlens_k, page_table, q, k_cache, v_cache,
                                  num_splits: int, sm_scale: float, out, lse=None, k_scale=None,
                                  v_scale=None, full_to_swa_mapping=None, swa_page_table=None,
                                  stream=None, use_pdl: bool = True):
    """pa_decode_step without a workspace argument, for callers that cannot allocate:
    the split-K scratch is the library's built-in array (see include/pa.h).  Calls
    share that array, so calls must not overlap on the GPU."""
    lib = load()
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    bs, hq, d = q.shape
    num_pages, hkv, page_size, _ = k_cache.shape
    st = lib.pa_decode_step_static_scratch(
        _io_ptr(req_pool_indices, torch.int64, "req_pool_indices"),
        _io_ptr(seq_lens, torch.int64, "seq_lens"), _ptr2d(req_to_token, torch.int32, "req_to_token"),
        req_to_token.shape[0], req_to_token.stride(0),
        _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
        full_to_swa_mapping.numel() if full_to_swa_mapping is not None else 0,
        int(seqlen_offset), int(max_seq_pages), _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
        _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"), _ptr2d(page_table, torch.int32, "page_table"),
        _row_stride(page_table, "page_table"),
        _ptr2d(swa_page_table, torch.int32, "swa_page_table") if swa_page_table is not None else None,
        _row_stride(swa_page_table, "swa_page_table") if swa_page_table is not None else 0,
        _io_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"),
        _ptr(v_cache, None, "v_cache"), ks, vs, kv_dtype, bs, hq, hkv, d, page_size, num_pages,
        int(num_splits), float(sm_scale), _io_ptr(out, torch.bfloat16, "out"),
        _io_ptr(lse, torch.float32, "lse"), _stream(stream), int(bool(use_pdl)))
    _check("pa_decode_step_static_scratch", st)


def pa_workspace_bytes(bs: int, num_q_heads: int, head_dim: int, num_splits: int) -> int:
    return int(load().pa_workspace_bytes(bs, num_q_heads, head_dim, num_splits))


def pa_choose_splits(bs: int, num_kv_heads: int, max_seq_pages: int, page_size: int,
                     kv_dtype: int = 0, sm_count: int = 0) -> int:
    """Split count heuristic; kv_dtype PA_KV_BF16 (0) or PA_KV_INT8 (1)."""
    return int(load().pa_choose_splits(bs, num_kv_heads, max_seq_pages, page_size, kv_dtype,
                                       sm_count))


def pa_select_producer(producer: int) -> int:
    """Choose the split-K producer implementation (PA_PRODUCER_AUTO / _FMA / _MMA) for
    later calls; returns the previous choice."""
    return int(load().pa_select_producer(int(producer)))


class producer:
    """Context manager: run a block with one producer implementation selected."""

    def __init__(self, which: int):
        self.which = which

    def __enter__(self):
        self.prev = pa_select_producer(self.which)
        return self

    def __exit__(self, *exc):
        pa_select_producer(self.prev)


def pa_status_string(status: int) -> str:
    return status_string(status)


def pa_read_error_flags(reset: bool = True, lib=None) -> int:
    """Device error word (synchronises the device); see include/pa.h.  ``lib`` reads the
    word of another build of the library (each build has its own)."""
    v = ctypes.c_uint32(0)
    lib = lib or load()
    _check("pa_read_error_flags", lib.pa_read_error_flags(ctypes.byref(v), int(bool(reset))), lib)
    return int(v.value)


# ---- the cache operators: rotary append, tree attention, weights, eviction ------------------


def _on_device(**tensors):
    """The named tensors are CUDA tensors of the current device (whose context the launch
    uses); None entries pass."""
    current = torch.cuda.current_device() if torch.cuda.is_available() else None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device.index != current:
            raise ValueError(f"{name} is on cuda:{t.device.index}, the current device is "
                             f"cuda:{current}")


def _shape(t: torch.Tensor, shape: tuple, name: str):
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _table(t: torch.Tensor, bs: int, columns: int, name: str):
    """Pointer and row stride of a [bs, >= columns] int32 page table."""
    stride = _row_stride(t, name)
    if t.shape[0] != bs or t.shape[1] < columns:
        raise ValueError(f"{name} must be [{bs}, >= {columns}], got {tuple(t.shape)}")
    return _ptr2d(t, torch.int32, name), stride if bs > 1 else max(stride, t.shape[1])


def _pools(k_cache, v_cache, k_scale, v_scale):
    """(kv_dtype, scale pointers, pool shape) of pools of equal type and shape."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, num_kv_heads, page_size, head_dim]")
    if v_cache.dtype != k_cache.dtype:
        raise ValueError(f"v_cache must be {k_cache.dtype}, got {v_cache.dtype}")
    _shape(v_cache, tuple(k_cache.shape), "v_cache")
    kv_dtype, ks, vs = _kv_args(k_cache, v_cache, k_scale, v_scale)
    if kv_dtype == PA_KV_INT8:
        _shape(k_scale, tuple(k_cache.shape[:3]), "k_scale")
        _shape(v_scale, tuple(k_cache.shape[:3]), "v_scale")
    return kv_dtype, ks, vs, tuple(k_cache.shape)


def pa_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = PA_ROPE_PLAIN, *,
                        factor: float = 1.0, original_length: int = 0, low: float = 0.0,
                        high: float = 0.0) -> torch.Tensor:
    """Radians per position of each rotated pair, a CPU tensor [rotary_dim / 2] float64;
    see include/pa.h."""
    out = torch.empty(max(int(rotary_dim) // 2, 1), dtype=torch.float64)
    _check("pa_rope_frequencies", load().pa_rope_frequencies(
        out.data_ptr(), int(rotary_dim), float(base), int(scaling), float(factor),
        int(original_length), float(low), float(high)))
    return out


def _token_rows(t: torch.Tensor, tokens: int, name: str):
    """(pointer, token stride, heads) of [tokens, heads, 128] bf16 rows whose heads are
    contiguous (a view of a wider projection row is fine)."""
    if t.dim() != 3 or t.shape[0] != tokens or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be [{tokens}, heads, head_dim] bf16")
    heads, d = t.shape[1], t.shape[2]
    if (d > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), t.stride(0) if tokens > 1 else heads * d, heads


def _rope_append_args(*, q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache,
                      k_scale=None, v_scale=None, weights=None, interleaved: bool = False,
                      amplitude: float = 1.0, stream=None, use_pdl: bool = True):
    _on_device(q=q, k=k, v=v, positions=positions, slots=slots, inv_freq=inv_freq, q_out=q_out,
               k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
               weights=weights)
    kv_dtype, ks, vs, (num_pages, hkv, page_size, d) = _pools(k_cache, v_cache, k_scale, v_scale)
    tokens = q.shape[0]
    qp, q_stride, hq = _token_rows(q, tokens, "q")
    kp, k_stride, k_heads = _token_rows(k, tokens, "k")
    vp, v_stride, v_heads = _token_rows(v, tokens, "v")
    op, o_stride, _ = _token_rows(q_out, tokens, "q_out")
    _shape(q_out, tuple(q.shape), "q_out")
    if k_heads != hkv or v_heads != hkv or not q.shape[2] == k.shape[2] == v.shape[2] == d:
        raise ValueError("k and v must have the pools' heads, and all rows their head_dim")
    _shape(positions, (tokens,), "positions")
    _shape(slots, (tokens,), "slots")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rotary_dim / 2]")
    if weights is not None:
        _shape(weights, (num_pages, hkv, page_size), "weights")
    return (qp, q_stride, kp, k_stride, vp, v_stride, _ptr(positions, torch.int64, "positions"),
            _ptr(slots, torch.int64, "slots"), _ptr(inv_freq, torch.float64, "inv_freq"),
            2 * inv_freq.numel(), int(bool(interleaved)), float(amplitude), tokens, hq, hkv, d, op,
            o_stride, _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"), ks, vs,
            _ptr(weights, torch.float32, "weights"), kv_dtype, page_size, num_pages, _stream(stream),
            int(bool(use_pdl)))


def pa_rope_append(**kw):
    """Rotary positions on q (into q_out) and k, and the new k and v rows written to their
    slots of the pools, the written rows' accumulated ``weights`` (if given) set to 0; see
    include/pa.h.  Keyword arguments: those of ``_rope_append_args``."""
    _check("pa_rope_append", load().pa_rope_append_weights(*_rope_append_args(**kw)))


def prepare_rope_append(*, lib=None, **kw) -> PreparedCall:
    """``pa_rope_append`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_rope_append_weights", _rope_append_args(**kw), lib,
                        keep=tuple(kw.values()))


def pa_build_tree_mask(parents, cu_seqlens_q, tree_mask, *, max_q_len: int, stream=None,
                       use_pdl: bool = True):
    """Ancestor masks of drafted trees from parent indices; see include/pa.h."""
    _on_device(parents=parents, cu_seqlens_q=cu_seqlens_q, tree_mask=tree_mask)
    _shape(parents, (tree_mask.shape[0],), "parents")
    if tree_mask.dim() != 2:
        raise ValueError("tree_mask must be [total_q, mask_words]")
    _check("pa_build_tree_mask", load().pa_build_tree_mask(
        _ptr(parents, torch.int32, "parents"), _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"),
        cu_seqlens_q.numel() - 1, tree_mask.shape[0], int(max_q_len),
        _ptr(tree_mask, torch.int64, "tree_mask"), tree_mask.shape[1], _stream(stream),
        int(bool(use_pdl))))


def pa_choose_tree_splits(bs: int, max_q_len: int, num_q_heads: int, num_kv_heads: int,
                          page_size: int, max_seq_pages: int, sm_count: int = 0) -> int:
    """Split count of a tree attention; see include/pa.h."""
    return int(load().pa_choose_tree_splits(bs, max_q_len, num_q_heads, num_kv_heads, page_size,
                                            max_seq_pages, sm_count))


def pa_tree_workspace_bytes(bs: int, total_q: int, max_q_len: int, num_q_heads: int,
                            num_kv_heads: int, head_dim: int, page_size: int,
                            max_seq_pages: int) -> int:
    """Workspace of a tree attention with the library's split count; see include/pa.h."""
    return int(load().pa_tree_workspace_bytes(bs, total_q, max_q_len, num_q_heads, num_kv_heads,
                                              head_dim, page_size, max_seq_pages))


def _workspace(workspace):
    if workspace is None:
        return None, 0
    return _ptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size()


def _tree_rows(q, tree_mask, cu_seqlens_q, cache_seqlens, out, lse, d: int):
    """Shapes shared by the tree calls; returns (total_q, num_q_heads, bs, mask_words)."""
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [total_q, num_q_heads, {d}]")
    total_q, hq, _ = q.shape
    bs = cache_seqlens.shape[0]
    _shape(cu_seqlens_q, (bs + 1,), "cu_seqlens_q")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != total_q:
        raise ValueError("tree_mask must be [total_q, mask_words]")
    _shape(out, tuple(q.shape), "out")
    if lse is not None:
        _shape(lse, (total_q, hq), "lse")
    return total_q, hq, bs, tree_mask.shape[1]


def _tree_attention_args(*, q, k_cache, v_cache, page_table, cache_seqlens, cu_seqlens_q,
                         tree_mask, max_q_len: int, max_seq_pages: int, sm_scale: float, out,
                         lse=None, num_splits: int = 0, workspace=None, k_scale=None,
                         v_scale=None, stream=None, use_pdl: bool = True):
    _on_device(q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table,
               cache_seqlens=cache_seqlens, cu_seqlens_q=cu_seqlens_q, tree_mask=tree_mask,
               out=out, lse=lse, workspace=workspace, k_scale=k_scale, v_scale=v_scale)
    kv_dtype, ks, vs, (num_pages, hkv, page_size, d) = _pools(k_cache, v_cache, k_scale, v_scale)
    total_q, hq, bs, words = _tree_rows(q, tree_mask, cu_seqlens_q, cache_seqlens, out, lse, d)
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    ws, ws_bytes = _workspace(workspace)
    return (_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"),
            _ptr(v_cache, None, "v_cache"), ks, vs, kv_dtype, pt, pt_stride,
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
            _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"),
            _ptr(tree_mask, torch.int64, "tree_mask"), words, bs, total_q, int(max_q_len), hq, hkv,
            d, page_size, num_pages, int(max_seq_pages), int(num_splits), float(sm_scale), ws,
            ws_bytes, _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
            _stream(stream), int(bool(use_pdl)))


def pa_tree_attention(**kw):
    """Attention of drafted trees over the cache; see include/pa.h.  Keyword arguments:
    those of ``_tree_attention_args``."""
    _check("pa_tree_attention", load().pa_tree_attention(*_tree_attention_args(**kw)))


def prepare_tree_attention(*, lib=None, **kw) -> PreparedCall:
    """``pa_tree_attention`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_tree_attention", _tree_attention_args(**kw), lib,
                        keep=tuple(kw.values()))


def _decode_step_tree_args(*, req_pool_indices, seq_lens, req_to_token, seqlen_offset: int,
                           max_seq_pages: int, cache_seqlens, cu_seqlens_k, page_table,
                           cu_seqlens_q, tree_mask, q, max_q_len: int, k_cache, v_cache,
                           sm_scale: float, out, lse=None, num_splits: int = 0, workspace=None,
                           qlens=None, q_mode: int = PA_Q_MODE_CUMSUM, q_stride: int = 0,
                           k_scale=None, v_scale=None, full_to_swa_mapping=None,
                           swa_page_table=None, stream=None, use_pdl: bool = True):
    _on_device(req_pool_indices=req_pool_indices, seq_lens=seq_lens, req_to_token=req_to_token,
               cache_seqlens=cache_seqlens, cu_seqlens_k=cu_seqlens_k, page_table=page_table,
               cu_seqlens_q=cu_seqlens_q, tree_mask=tree_mask, q=q, k_cache=k_cache,
               v_cache=v_cache, out=out, lse=lse, workspace=workspace, qlens=qlens,
               k_scale=k_scale, v_scale=v_scale, full_to_swa_mapping=full_to_swa_mapping,
               swa_page_table=swa_page_table)
    kv_dtype, ks, vs, (num_pages, hkv, page_size, d) = _pools(k_cache, v_cache, k_scale, v_scale)
    total_q, hq, bs, words = _tree_rows(q, tree_mask, cu_seqlens_q, cache_seqlens, out, lse, d)
    _shape(req_pool_indices, (bs,), "req_pool_indices")
    _shape(seq_lens, (bs,), "seq_lens")
    _shape(cu_seqlens_k, (bs + 1,), "cu_seqlens_k")
    if qlens is not None:
        _shape(qlens, (bs,), "qlens")
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    swa, swa_stride = (None, 0) if swa_page_table is None else \
        _table(swa_page_table, bs, int(max_seq_pages), "swa_page_table")
    ws, ws_bytes = _workspace(workspace)
    return (_ptr(req_pool_indices, torch.int64, "req_pool_indices"),
            _ptr(seq_lens, torch.int64, "seq_lens"),
            _ptr2d(req_to_token, torch.int32, "req_to_token"), req_to_token.shape[0],
            req_to_token.stride(0), _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
            full_to_swa_mapping.numel() if full_to_swa_mapping is not None else 0,
            int(seqlen_offset), int(max_seq_pages),
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
            _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"), pt, pt_stride, swa, swa_stride,
            _ptr(qlens, torch.int64, "qlens"), int(q_mode), int(q_stride),
            _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"),
            _ptr(tree_mask, torch.int64, "tree_mask"), words, _ptr(q, torch.bfloat16, "q"),
            total_q, int(max_q_len), _ptr(k_cache, None, "k_cache"),
            _ptr(v_cache, None, "v_cache"), ks, vs, kv_dtype, bs, hq, hkv, d, page_size, num_pages,
            int(num_splits), float(sm_scale), ws, ws_bytes, _ptr(out, torch.bfloat16, "out"),
            _ptr(lse, torch.float32, "lse"), _stream(stream), int(bool(use_pdl)))


def pa_decode_step_tree(*, lib=None, **kw):
    """Metadata (with cu_seqlens_q) + tree attention in one call; see include/pa.h.
    Keyword arguments: those of ``_decode_step_tree_args``."""
    lib = lib or load()
    _check("pa_decode_step_tree", lib.pa_decode_step_tree(*_decode_step_tree_args(**kw)), lib)


def prepare_decode_step_tree(*, lib=None, **kw) -> PreparedCall:
    """``pa_decode_step_tree`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_decode_step_tree", _decode_step_tree_args(**kw), lib,
                        keep=tuple(kw.values()))


def _accumulate_weights_args(*, q, lse, k_cache, page_table, cache_seqlens, weights,
                             max_seq_pages: int, sm_scale: float, k_scale=None, stream=None,
                             use_pdl: bool = True):
    _on_device(q=q, lse=lse, k_cache=k_cache, page_table=page_table, cache_seqlens=cache_seqlens,
               weights=weights, k_scale=k_scale)
    kv_dtype, ks, _, (num_pages, hkv, page_size, d) = _pools(k_cache, k_cache, k_scale, k_scale)
    bs = cache_seqlens.shape[0]
    if q.dim() != 3 or q.shape[0] != bs or q.shape[2] != d:
        raise ValueError(f"q must be [{bs}, num_q_heads, {d}]")
    hq = q.shape[1]
    _shape(lse, (bs, hq), "lse")
    _shape(weights, (num_pages, hkv, page_size), "weights")
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    return (_ptr(q, torch.bfloat16, "q"), _ptr(lse, torch.float32, "lse"),
            _ptr(k_cache, None, "k_cache"), ks, kv_dtype, pt, pt_stride,
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
            _ptr(weights, torch.float32, "weights"), bs, hq, hkv, d, page_size, num_pages,
            int(max_seq_pages), float(sm_scale), _stream(stream), int(bool(use_pdl)))


def pa_accumulate_weights(**kw):
    """Attention weights of a decode step added to the cached rows' totals; see
    include/pa.h.  Keyword arguments: those of ``_accumulate_weights_args``."""
    _check("pa_accumulate_weights",
           load().pa_accumulate_weights(*_accumulate_weights_args(**kw)))


def prepare_accumulate_weights(*, lib=None, **kw) -> PreparedCall:
    """``pa_accumulate_weights`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_accumulate_weights", _accumulate_weights_args(**kw), lib,
                        keep=tuple(kw.values()))


def _destination(page_table, dst_page_table, bs: int):
    """(pointer, stride, columns) of the destination table; None means in place."""
    dst = page_table if dst_page_table is None else dst_page_table
    return (*_table(dst, bs, 1, "dst_page_table"), dst.shape[1])


def _compact_cache_args(*, page_table, cache_seqlens, kept, counts, k_cache, v_cache,
                        max_seq_pages: int, dst_page_table=None, begin=None, new_seqlens=None,
                        weights=None, k_scale=None, v_scale=None, stream=None,
                        use_pdl: bool = True):
    _on_device(page_table=page_table, cache_seqlens=cache_seqlens, kept=kept, counts=counts,
               k_cache=k_cache, v_cache=v_cache, dst_page_table=dst_page_table, begin=begin,
               new_seqlens=new_seqlens, weights=weights, k_scale=k_scale, v_scale=v_scale)
    kv_dtype, ks, vs, (num_pages, hkv, page_size, d) = _pools(k_cache, v_cache, k_scale, v_scale)
    bs = cache_seqlens.shape[0]
    if kept.dim() != 3 or kept.shape[0] != bs or kept.shape[1] not in (1, hkv):
        raise ValueError(f"kept must be [{bs}, 1 or {hkv}, max_kept]")
    for name, t in (("counts", counts), ("begin", begin), ("new_seqlens", new_seqlens)):
        if t is not None:
            _shape(t, (bs,), name)
    if weights is not None:
        _shape(weights, (num_pages, hkv, page_size), "weights")
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    dst, dst_stride, dst_pages = _destination(page_table, dst_page_table, bs)
    return (pt, pt_stride, _ptr(cache_seqlens, torch.int32, "cache_seqlens"), int(max_seq_pages),
            _ptr(kept, torch.int32, "kept"), kept.shape[1], kept.shape[2],
            _ptr(counts, torch.int32, "counts"), _ptr(begin, torch.int32, "begin"), kept.shape[2],
            _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"), ks, vs, kv_dtype,
            _ptr(weights, torch.float32, "weights"), dst, dst_stride, dst_pages,
            _ptr(new_seqlens, torch.int32, "new_seqlens"), bs, hkv, d, page_size, num_pages,
            _stream(stream), int(bool(use_pdl)))


def pa_compact_cache(**kw):
    """Kept rows of the cache moved to the front, in order, in place or to the pages of
    ``dst_page_table``; see include/pa.h.  Keyword arguments: those of
    ``_compact_cache_args``."""
    _check("pa_compact_cache", load().pa_compact_cache(*_compact_cache_args(**kw)))


def prepare_compact_cache(*, lib=None, **kw) -> PreparedCall:
    """``pa_compact_cache`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_compact_cache", _compact_cache_args(**kw), lib,
                        keep=tuple(kw.values()))


def _evict_args(*, page_table, cache_seqlens, weights, k_cache, v_cache, max_seq_pages: int,
                budget: int, kept, new_seqlens, num_first: int = 0, num_recent: int = 0,
                dst_page_table=None, k_scale=None, v_scale=None, stream=None,
                use_pdl: bool = True):
    _on_device(page_table=page_table, cache_seqlens=cache_seqlens, weights=weights,
               k_cache=k_cache, v_cache=v_cache, dst_page_table=dst_page_table, kept=kept,
               new_seqlens=new_seqlens, k_scale=k_scale, v_scale=v_scale)
    kv_dtype, ks, vs, (num_pages, hkv, page_size, d) = _pools(k_cache, v_cache, k_scale, v_scale)
    bs = cache_seqlens.shape[0]
    _shape(weights, (num_pages, hkv, page_size), "weights")
    _shape(kept, (bs, hkv, int(budget)), "kept")
    _shape(new_seqlens, (bs,), "new_seqlens")
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    dst, dst_stride, dst_pages = _destination(page_table, dst_page_table, bs)
    return (pt, pt_stride, _ptr(cache_seqlens, torch.int32, "cache_seqlens"), int(max_seq_pages),
            _ptr(weights, torch.float32, "weights"), _ptr(k_cache, None, "k_cache"),
            _ptr(v_cache, None, "v_cache"), ks, vs, kv_dtype, int(budget), int(num_first),
            int(num_recent), dst, dst_stride, dst_pages, _ptr(kept, torch.int32, "kept"),
            _ptr(new_seqlens, torch.int32, "new_seqlens"), bs, hkv, d, page_size, num_pages,
            _stream(stream), int(bool(use_pdl)))


def pa_evict(**kw):
    """Each request's cache shrunk to ``budget`` rows per kv head by accumulated weight;
    see include/pa.h.  Keyword arguments: those of ``_evict_args``."""
    _check("pa_evict", load().pa_evict(*_evict_args(**kw)))


def prepare_evict(*, lib=None, **kw) -> PreparedCall:
    """``pa_evict`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_evict", _evict_args(**kw), lib, keep=tuple(kw.values()))


# ---- block-scaled caches: e4m3 codes, a scale per block of tokens and head --------------------


def _block_pools(k_cache, v_cache, k_scale, v_scale):
    """(scale_block, pool shape) of e4m3 pools and their scales."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, num_kv_heads, page_size, head_dim]")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dtype != torch.float8_e4m3fn:
            raise ValueError(f"{name} must be {torch.float8_e4m3fn}, got {t.dtype}")
    _shape(v_cache, tuple(k_cache.shape), "v_cache")
    num_pages, hkv, page_size, _ = k_cache.shape
    if k_scale.dim() != 3 or k_scale.shape[2] < 1 or page_size % k_scale.shape[2] != 0:
        raise ValueError("k_scale must be [num_pages, num_kv_heads, page_size / scale_block]")
    _shape(k_scale, (num_pages, hkv, k_scale.shape[2]), "k_scale")
    _shape(v_scale, tuple(k_scale.shape), "v_scale")
    return page_size // k_scale.shape[2], tuple(k_cache.shape)


def _rope_append_blocks_args(*, k, v, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q,
                             cache_seqlens, page_table, max_seq_pages: int, q=None, q_out=None,
                             positions=None, inv_freq=None, max_q_len: Optional[int] = None,
                             interleaved: bool = False, amplitude: float = 1.0, stream=None,
                             use_pdl: bool = True):
    _on_device(q=q, k=k, v=v, positions=positions, inv_freq=inv_freq, q_out=q_out, k_cache=k_cache,
               v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, cu_seqlens_q=cu_seqlens_q,
               cache_seqlens=cache_seqlens, page_table=page_table)
    block, (num_pages, hkv, page_size, d) = _block_pools(k_cache, v_cache, k_scale, v_scale)
    tokens = k.shape[0]
    kp, k_stride, k_heads = _token_rows(k, tokens, "k")
    vp, v_stride, v_heads = _token_rows(v, tokens, "v")
    qp, q_stride, hq, op, o_stride = None, 0, 0, None, 0
    if q is not None:
        qp, q_stride, hq = _token_rows(q, tokens, "q")
        if q_out is None or q.shape[2] != d:
            raise ValueError(f"q needs q_out, and rows of {d} channels")
        _shape(q_out, tuple(q.shape), "q_out")
        op, o_stride, _ = _token_rows(q_out, tokens, "q_out")
    if k_heads != hkv or v_heads != hkv or not k.shape[2] == v.shape[2] == d:
        raise ValueError("k and v must have the pools' heads and head_dim")
    bs = cache_seqlens.shape[0]
    _shape(cu_seqlens_q, (bs + 1,), "cu_seqlens_q")
    if inv_freq is not None:
        if inv_freq.dim() != 1 or positions is None:
            raise ValueError("inv_freq must be [rotary_dim / 2], with positions")
        _shape(positions, (tokens,), "positions")
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    return (qp, q_stride, kp, k_stride, vp, v_stride, _ptr(positions, torch.int64, "positions"),
            _ptr(inv_freq, torch.float64, "inv_freq"),
            2 * inv_freq.numel() if inv_freq is not None else 0, int(bool(interleaved)),
            float(amplitude), _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"),
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"), pt, pt_stride, int(max_seq_pages),
            bs, tokens, max(tokens, 1) if max_q_len is None else int(max_q_len), hq, hkv, d, op,
            o_stride, _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"),
            _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale"),
            PA_KV_E4M3, block, page_size, num_pages, _stream(stream), int(bool(use_pdl)))


def pa_rope_append_blocks(**kw):
    """Rotary positions on q (into q_out) and k, and each request's new k and v rows written
    to a block-scaled cache; see include/pa.h.  Without ``inv_freq`` rows are taken as they
    are, without ``q`` there are only k and v.  Keyword arguments: those of
    ``_rope_append_blocks_args``."""
    _check("pa_rope_append_blocks",
           load().pa_rope_append_blocks(*_rope_append_blocks_args(**kw)))


def prepare_rope_append_blocks(*, lib=None, **kw) -> PreparedCall:
    """``pa_rope_append_blocks`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_rope_append_blocks", _rope_append_blocks_args(**kw), lib,
                        keep=tuple(kw.values()))


def pa_choose_block_splits(bs: int, max_q_len: int, num_q_heads: int, num_kv_heads: int,
                           page_size: int, max_seq_pages: int, sm_count: int = 0) -> int:
    """Split count of a block attention; see include/pa.h."""
    return int(load().pa_choose_block_splits(bs, max_q_len, num_q_heads, num_kv_heads, page_size,
                                             max_seq_pages, sm_count))


def pa_block_workspace_bytes(bs: int, total_q: int, max_q_len: int, num_q_heads: int,
                             num_kv_heads: int, head_dim: int, page_size: int,
                             max_seq_pages: int) -> int:
    """Workspace of a block attention with the library's split count; see include/pa.h."""
    return int(load().pa_block_workspace_bytes(bs, total_q, max_q_len, num_q_heads, num_kv_heads,
                                               head_dim, page_size, max_seq_pages))


def _block_rows(q, cu_seqlens_q, cache_seqlens, max_q_len, out, lse, d: int):
    """Shapes shared by the block calls; returns (total_q, num_q_heads, bs, max_q_len)."""
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [total_q, num_q_heads, {d}]")
    total_q, hq, _ = q.shape
    bs = cache_seqlens.shape[0]
    if cu_seqlens_q is not None:
        _shape(cu_seqlens_q, (bs + 1,), "cu_seqlens_q")
    elif total_q != bs or max_q_len != 1:
        raise ValueError("without cu_seqlens_q there is one query per request")
    _shape(out, tuple(q.shape), "out")
    if lse is not None:
        _shape(lse, (total_q, hq), "lse")
    return total_q, hq, bs, int(max_q_len)


def _block_attention_args(*, q, k_cache, v_cache, k_scale, v_scale, page_table, cache_seqlens,
                          max_seq_pages: int, sm_scale: float, out, cu_seqlens_q=None,
                          max_q_len: int = 1, lse=None, num_splits: int = 0, workspace=None,
                          stream=None, use_pdl: bool = True):
    _on_device(q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table,
               cache_seqlens=cache_seqlens, cu_seqlens_q=cu_seqlens_q, out=out, lse=lse,
               workspace=workspace, k_scale=k_scale, v_scale=v_scale)
    block, (num_pages, hkv, page_size, d) = _block_pools(k_cache, v_cache, k_scale, v_scale)
    total_q, hq, bs, mql = _block_rows(q, cu_seqlens_q, cache_seqlens, max_q_len, out, lse, d)
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    ws, ws_bytes = _workspace(workspace)
    return (_ptr(q, torch.bfloat16, "q"), _ptr(k_cache, None, "k_cache"),
            _ptr(v_cache, None, "v_cache"), _ptr(k_scale, torch.float32, "k_scale"),
            _ptr(v_scale, torch.float32, "v_scale"), PA_KV_E4M3, block, pt, pt_stride,
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
            _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"), bs, total_q, mql, hq, hkv, d,
            page_size, num_pages, int(max_seq_pages), int(num_splits), float(sm_scale), ws,
            ws_bytes, _ptr(out, torch.bfloat16, "out"), _ptr(lse, torch.float32, "lse"),
            _stream(stream), int(bool(use_pdl)))


def pa_block_attention(**kw):
    """Attention over a block-scaled cache; see include/pa.h.  Keyword arguments: those of
    ``_block_attention_args``."""
    _check("pa_block_attention", load().pa_block_attention(*_block_attention_args(**kw)))


def prepare_block_attention(*, lib=None, **kw) -> PreparedCall:
    """``pa_block_attention`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_block_attention", _block_attention_args(**kw), lib,
                        keep=tuple(kw.values()))


def _decode_step_block_args(*, req_pool_indices, seq_lens, req_to_token, seqlen_offset: int,
                            max_seq_pages: int, cache_seqlens, cu_seqlens_k, page_table, q,
                            k_cache, v_cache, k_scale, v_scale, sm_scale: float, out,
                            cu_seqlens_q=None, max_q_len: int = 1, lse=None, num_splits: int = 0,
                            workspace=None, qlens=None, q_mode: int = PA_Q_MODE_NONE,
                            q_stride: int = 0, full_to_swa_mapping=None, swa_page_table=None,
                            stream=None, use_pdl: bool = True):
    _on_device(req_pool_indices=req_pool_indices, seq_lens=seq_lens, req_to_token=req_to_token,
               cache_seqlens=cache_seqlens, cu_seqlens_k=cu_seqlens_k, page_table=page_table,
               cu_seqlens_q=cu_seqlens_q, q=q, k_cache=k_cache, v_cache=v_cache, out=out, lse=lse,
               workspace=workspace, qlens=qlens, k_scale=k_scale, v_scale=v_scale,
               full_to_swa_mapping=full_to_swa_mapping, swa_page_table=swa_page_table)
    block, (num_pages, hkv, page_size, d) = _block_pools(k_cache, v_cache, k_scale, v_scale)
    total_q, hq, bs, mql = _block_rows(q, cu_seqlens_q, cache_seqlens, max_q_len, out, lse, d)
    _shape(req_pool_indices, (bs,), "req_pool_indices")
    _shape(seq_lens, (bs,), "seq_lens")
    _shape(cu_seqlens_k, (bs + 1,), "cu_seqlens_k")
    if qlens is not None:
        _shape(qlens, (bs,), "qlens")
    pt, pt_stride = _table(page_table, bs, int(max_seq_pages), "page_table")
    swa, swa_stride = (None, 0) if swa_page_table is None else \
        _table(swa_page_table, bs, int(max_seq_pages), "swa_page_table")
    ws, ws_bytes = _workspace(workspace)
    return (_ptr(req_pool_indices, torch.int64, "req_pool_indices"),
            _ptr(seq_lens, torch.int64, "seq_lens"),
            _ptr2d(req_to_token, torch.int32, "req_to_token"), req_to_token.shape[0],
            req_to_token.stride(0), _ptr(full_to_swa_mapping, torch.int64, "full_to_swa_mapping"),
            full_to_swa_mapping.numel() if full_to_swa_mapping is not None else 0,
            int(seqlen_offset), int(max_seq_pages),
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
            _ptr(cu_seqlens_k, torch.int32, "cu_seqlens_k"), pt, pt_stride, swa, swa_stride,
            _ptr(qlens, torch.int64, "qlens"), int(q_mode), int(q_stride),
            _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"), _ptr(q, torch.bfloat16, "q"),
            total_q, mql, _ptr(k_cache, None, "k_cache"), _ptr(v_cache, None, "v_cache"),
            _ptr(k_scale, torch.float32, "k_scale"), _ptr(v_scale, torch.float32, "v_scale"),
            PA_KV_E4M3, block, bs, hq, hkv, d, page_size, num_pages, int(num_splits),
            float(sm_scale), ws, ws_bytes, _ptr(out, torch.bfloat16, "out"),
            _ptr(lse, torch.float32, "lse"), _stream(stream), int(bool(use_pdl)))


def pa_decode_step_block(*, lib=None, **kw):
    """Metadata + block attention in one call; see include/pa.h.  Keyword arguments: those
    of ``_decode_step_block_args``."""
    lib = lib or load()
    _check("pa_decode_step_block", lib.pa_decode_step_block(*_decode_step_block_args(**kw)), lib)


def prepare_decode_step_block(*, lib=None, **kw) -> PreparedCall:
    """``pa_decode_step_block`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_decode_step_block", _decode_step_block_args(**kw), lib,
                        keep=tuple(kw.values()))


# ---- verification of drafted tokens -------------------------------------------------------------


def _verify_drafts_args(*, target_probs, tokens, cu_seqlens_q, uniforms, final_uniforms, kept,
                        counts, next_tokens, max_q_len: int, draft_probs=None, parents=None,
                        cache_seqlens=None, begin=None, stream=None, use_pdl: bool = True):
    _on_device(target_probs=target_probs, draft_probs=draft_probs, tokens=tokens, parents=parents,
               cu_seqlens_q=cu_seqlens_q, cache_seqlens=cache_seqlens, uniforms=uniforms,
               final_uniforms=final_uniforms, kept=kept, counts=counts, begin=begin,
               next_tokens=next_tokens)
    tp = _ptr2d(target_probs, torch.float32, "target_probs")
    total_q, vocab = target_probs.shape
    bs = final_uniforms.shape[0]
    dp, d_stride = None, 0
    if draft_probs is not None:
        dp, d_stride = _ptr2d(draft_probs, torch.float32, "draft_probs"), draft_probs.stride(0)
        _shape(draft_probs, (total_q, vocab), "draft_probs")
        d_stride = d_stride if total_q > 1 else max(d_stride, vocab)
    _shape(tokens, (total_q,), "tokens")
    _shape(uniforms, (total_q,), "uniforms")
    _shape(cu_seqlens_q, (bs + 1,), "cu_seqlens_q")
    for name, t in (("counts", counts), ("next_tokens", next_tokens), ("begin", begin),
                    ("cache_seqlens", cache_seqlens)):
        if t is not None:
            _shape(t, (bs,), name)
    if parents is not None:
        _shape(parents, (total_q,), "parents")
    kp, k_stride = _table(kept, bs, int(max_q_len), "kept")
    stride = target_probs.stride(0)
    return (tp, stride if total_q > 1 else max(stride, vocab), dp, d_stride, vocab,
            _ptr(tokens, torch.int64, "tokens"), _ptr(parents, torch.int32, "parents"),
            _ptr(cu_seqlens_q, torch.int32, "cu_seqlens_q"),
            _ptr(cache_seqlens, torch.int32, "cache_seqlens"),
            _ptr(uniforms, torch.float32, "uniforms"),
            _ptr(final_uniforms, torch.float32, "final_uniforms"), bs, total_q, int(max_q_len), kp,
            k_stride, _ptr(counts, torch.int32, "counts"), _ptr(begin, torch.int32, "begin"),
            _ptr(next_tokens, torch.int64, "next_tokens"), _stream(stream), int(bool(use_pdl)))


def pa_verify_drafts(**kw):
    """Drafted tokens accepted or rejected by the target's probabilities and given random
    numbers, and the token that follows; see include/pa.h.  Keyword arguments: those of
    ``_verify_drafts_args``."""
    _check("pa_verify_drafts", load().pa_verify_drafts(*_verify_drafts_args(**kw)))


def prepare_verify_drafts(*, lib=None, **kw) -> PreparedCall:
    """``pa_verify_drafts`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_verify_drafts", _verify_drafts_args(**kw), lib,
                        keep=tuple(kw.values()))


# ---- pages: copied, forked, extended, freed, compacted --------------------------------------------


class _PagePool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64)]


def _page_pools(pools, num_pages: int, name: str, pinned: bool = False):
    """Host array of the pools' base addresses and page sizes: tensors [num_pages, ...],
    contiguous, on the current device (``pinned``: or in pinned host memory)."""
    array = (_PagePool * max(len(pools), 1))()
    for i, t in enumerate(pools):
        if t.dim() < 2 or t.shape[0] != num_pages or not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be a contiguous tensor of {num_pages} pages")
        if pinned and not t.is_cuda:
            if not t.is_pinned():
                raise ValueError(f"{name}[{i}] must be a CUDA tensor or pinned host memory")
        else:
            _on_device(**{f"{name}[{i}]": t})
        array[i].base = t.data_ptr()
        array[i].page_bytes = t.numel() // max(num_pages, 1) * t.element_size()
    return array


def _slot_table(req_to_token, page_refs, page_size: int, max_seq_pages: int, rows, lens):
    """The page operators' common arguments and the length of their lists."""
    num_rows, width = req_to_token.shape if req_to_token.dim() == 2 else (0, 0)
    stride = _row_stride(req_to_token, "req_to_token")
    stride = stride if num_rows > 1 else width
    if page_refs.dim() != 1:
        raise ValueError("page_refs must be [num_pages]")
    count = rows.numel()
    _shape(rows, (count,), "rows")
    _shape(lens, (count,), "lens")
    # a row's last page may end past the row only where the row is all that its stride covers: its
    # slots are written up to the stride
    room = width if stride > width else width + int(page_size) - 1
    if int(max_seq_pages) * int(page_size) > room:
        raise ValueError(f"req_to_token has room for fewer than {max_seq_pages} pages a row")
    return (_ptr2d(req_to_token, torch.int32, "req_to_token"), req_to_token.shape[0], stride,
            _ptr(page_refs, torch.int32, "page_refs"), page_refs.numel(), int(page_size),
            int(max_seq_pages)), count


def pa_pages_workspace_bytes(num_pages: int, count: int) -> int:
    """Workspace of a fork, extension or compaction; see include/pa.h."""
    return int(load().pa_pages_workspace_bytes(int(num_pages), int(count)))


def _pages_copy_args(*, src_pools, src_pages, dst_pages, dst_pools=None, stream=None,
                     use_pdl: bool = True):
    _on_device(src_pages=src_pages, dst_pages=dst_pages)
    count = src_pages.numel()
    _shape(src_pages, (count,), "src_pages")
    _shape(dst_pages, (count,), "dst_pages")
    num_src = src_pools[0].shape[0] if src_pools else 0
    src = _page_pools(src_pools, num_src, "src_pools", pinned=True)
    dst, num_dst = src, num_src
    if dst_pools is not None:
        if len(dst_pools) != len(src_pools):
            raise ValueError("src_pools and dst_pools must be lists of one length")
        num_dst = dst_pools[0].shape[0] if dst_pools else 0
        dst = _page_pools(dst_pools, num_dst, "dst_pools", pinned=True)
    return (ctypes.addressof(src), ctypes.addressof(dst), len(src_pools), num_src, num_dst,
            _ptr(src_pages, torch.int32, "src_pages"), _ptr(dst_pages, torch.int32, "dst_pages"),
            count, _stream(stream), int(bool(use_pdl))), (src, dst)


def pa_pages_copy(**kw):
    """Pages copied within or between pools; see include/pa.h.  Keyword arguments: those of
    ``_pages_copy_args``."""
    args, _arrays = _pages_copy_args(**kw)
    _check("pa_pages_copy", load().pa_pages_copy(*args))


def prepare_pages_copy(*, lib=None, **kw) -> PreparedCall:
    """``pa_pages_copy`` with the given keyword arguments, marshalled once."""
    args, arrays = _pages_copy_args(**kw)
    return PreparedCall("pa_pages_copy", args, lib, keep=(*kw.values(), *arrays))


def _pages_fork_args(*, req_to_token, page_refs, page_size: int, max_seq_pages: int, parents,
                     children, lens, pools, child_lens, workspace, stream=None,
                     use_pdl: bool = True):
    _on_device(req_to_token=req_to_token, page_refs=page_refs, parents=parents, children=children,
               lens=lens, child_lens=child_lens, workspace=workspace)
    table, count = _slot_table(req_to_token, page_refs, page_size, max_seq_pages, parents, lens)
    _shape(children, (count,), "children")
    _shape(child_lens, (count,), "child_lens")
    array = _page_pools(pools, page_refs.numel(), "pools")
    return (*table, _ptr(parents, torch.int64, "parents"), _ptr(children, torch.int64, "children"),
            _ptr(lens, torch.int32, "lens"), count, ctypes.addressof(array), len(pools),
            _ptr(child_lens, torch.int32, "child_lens"), *_workspace(workspace), _stream(stream),
            int(bool(use_pdl))), (array,)


def pa_pages_fork(**kw):
    """Requests forked: full pages shared, the last one copied; see include/pa.h.  Keyword
    arguments: those of ``_pages_fork_args``."""
    args, _arrays = _pages_fork_args(**kw)
    _check("pa_pages_fork", load().pa_pages_fork(*args))


def prepare_pages_fork(*, lib=None, **kw) -> PreparedCall:
    """``pa_pages_fork`` with the given keyword arguments, marshalled once."""
    args, arrays = _pages_fork_args(**kw)
    return PreparedCall("pa_pages_fork", args, lib, keep=(*kw.values(), *arrays))


def _pages_extend_args(*, req_to_token, page_refs, page_size: int, max_seq_pages: int, rows, lens,
                       new_lens, granted, workspace, stream=None, use_pdl: bool = True):
    _on_device(req_to_token=req_to_token, page_refs=page_refs, rows=rows, lens=lens,
               new_lens=new_lens, granted=granted, workspace=workspace)
    table, count = _slot_table(req_to_token, page_refs, page_size, max_seq_pages, rows, lens)
    _shape(new_lens, (count,), "new_lens")
    _shape(granted, (count,), "granted")
    return (*table, _ptr(rows, torch.int64, "rows"), _ptr(lens, torch.int32, "lens"),
            _ptr(new_lens, torch.int32, "new_lens"), count,
            _ptr(granted, torch.int32, "granted"), *_workspace(workspace), _stream(stream),
            int(bool(use_pdl)))


def pa_pages_extend(**kw):
    """Free pages handed out to growing requests; see include/pa.h.  Keyword arguments: those
    of ``_pages_extend_args``."""
    _check("pa_pages_extend", load().pa_pages_extend(*_pages_extend_args(**kw)))


def prepare_pages_extend(*, lib=None, **kw) -> PreparedCall:
    """``pa_pages_extend`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_pages_extend", _pages_extend_args(**kw), lib, keep=tuple(kw.values()))


def _pages_free_args(*, req_to_token, page_refs, page_size: int, max_seq_pages: int, rows, lens,
                     keep_lens=None, stream=None, use_pdl: bool = True):
    _on_device(req_to_token=req_to_token, page_refs=page_refs, rows=rows, lens=lens,
               keep_lens=keep_lens)
    table, count = _slot_table(req_to_token, page_refs, page_size, max_seq_pages, rows, lens)
    if keep_lens is not None:
        _shape(keep_lens, (count,), "keep_lens")
    return (*table, _ptr(rows, torch.int64, "rows"), _ptr(lens, torch.int32, "lens"),
            _ptr(keep_lens, torch.int32, "keep_lens"), count, _stream(stream), int(bool(use_pdl)))


def pa_pages_free(**kw):
    """Pages of requests given back; see include/pa.h.  Keyword arguments: those of
    ``_pages_free_args``."""
    _check("pa_pages_free", load().pa_pages_free(*_pages_free_args(**kw)))


def prepare_pages_free(*, lib=None, **kw) -> PreparedCall:
    """``pa_pages_free`` with the given keyword arguments, marshalled once."""
    return PreparedCall("pa_pages_free", _pages_free_args(**kw), lib, keep=tuple(kw.values()))


def _pages_compact_args(*, req_to_token, page_refs, page_size: int, max_seq_pages: int, rows, lens,
                        pools, page_map, num_live, workspace, stream=None, use_pdl: bool = True):
    _on_device(req_to_token=req_to_token, page_refs=page_refs, rows=rows, lens=lens,
               page_map=page_map, num_live=num_live, workspace=workspace)
    table, count = _slot_table(req_to_token, page_refs, page_size, max_seq_pages, rows, lens)
    _shape(page_map, tuple(page_refs.shape), "page_map")
    _shape(num_live, (1,), "num_live")
    array = _page_pools(pools, page_refs.numel(), "pools")
    return (*table, _ptr(rows, torch.int64, "rows"), _ptr(lens, torch.int32, "lens"), count,
            ctypes.addressof(array), len(pools), _ptr(page_map, torch.int32, "page_map"),
            _ptr(num_live, torch.int32, "num_live"), *_workspace(workspace), _stream(stream),
            int(bool(use_pdl))), (array,)


def pa_pages_compact(**kw):
    """The live pages moved to the front of their pools; see include/pa.h.  Keyword arguments:
    those of ``_pages_compact_args``."""
    args, _arrays = _pages_compact_args(**kw)
    _check("pa_pages_compact", load().pa_pages_compact(*args))


def prepare_pages_compact(*, lib=None, **kw) -> PreparedCall:
    """``pa_pages_compact`` with the given keyword arguments, marshalled once."""
    args, arrays = _pages_compact_args(**kw)
    return PreparedCall("pa_pages_compact", args, lib, keep=(*kw.values(), *arrays))
