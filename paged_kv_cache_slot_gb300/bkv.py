"""Thin Python binding of libbkv.so (ctypes).

Argument marshalling only: each function checks the tensors' device, dtype,
shape and contiguity, passes their device pointers and the current CUDA
stream to the C entry point of the same name, and raises :class:`BkvError`
on a non-zero status.  Every step of the path runs in the library's kernels;
there is no fallback of any kind.  If libbkv.so is missing or cannot be
loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

from . import build as _build

BKV_OK, BKV_ERR_INVALID_ARG, BKV_ERR_UNSUPPORTED, BKV_ERR_CUDA = 0, 1, 2, 3
BKV_BF16, BKV_F32 = 0, 1
BKV_MASK_CAUSAL, BKV_MASK_ALL = 0, 1

LIB_PATH = _build.LIB

_lib = None
_lock = threading.Lock()

# The current device and its current stream's handle, without the objects that torch.cuda's functions build
# around them (a call of a few microseconds on the GPU notices those).
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = (torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream")
               else lambda device: torch.cuda.current_stream(device).cuda_stream)


class BkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib = load()
        msg = lib.bkv_status_string(status).decode()
        if status == BKV_ERR_CUDA:
            msg += ": " + lib.bkv_last_cuda_error().decode()
        super().__init__(f"{fn} -> status {status} ({msg})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libbkv.so (built in-tree by ``build()``); raise if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libbkv.so not found at {LIB_PATH}: run paged_kv_cache_slot_gb300.build.build() "
                               "(there is no fallback path)")
        lib = ctypes.CDLL(LIB_PATH)
        i32, i64, vp, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
        cint = ctypes.c_int
        lib.bkv_status_string.restype = ctypes.c_char_p
        lib.bkv_status_string.argtypes = [cint]
        lib.bkv_last_cuda_error.restype = ctypes.c_char_p
        lib.bkv_last_cuda_error.argtypes = []
        lib.bkv_version.restype = ctypes.c_char_p
        lib.bkv_version.argtypes = []
        lib.bkv_compute_slot_mapping.restype = cint
        lib.bkv_compute_slot_mapping.argtypes = [vp, i32, i64, i32, vp, vp, i64, i64, i32, vp, vp, vp]
        lib.bkv_compute_slot_mapping_cp.restype = cint
        lib.bkv_compute_slot_mapping_cp.argtypes = [vp, i32, i64, i32, vp, vp, i64, i64, i32, i32, i32, i32, vp, vp,
                                                    vp]
        lib.bkv_paged_decode_cp.restype = cint
        lib.bkv_paged_decode_cp.argtypes = [vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i32, i32, i32, i32, i64, f32,
                                            cint, i32, i32, i32, cint, vp, vp, vp, sz, vp, vp]
        lib.bkv_paged_attention_ragged.restype = cint
        lib.bkv_paged_attention_ragged.argtypes = [vp, vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i64, i32, i32,
                                                   i32, i32, i64, f32, cint, cint, vp, vp, vp]
        lib.bkv_merge_attn_states.restype = cint
        lib.bkv_merge_attn_states.argtypes = [vp, vp, i32, i64, i32, cint, vp, vp, vp]
        lib.bkv_map_to_kernel_blocks.restype = cint
        lib.bkv_map_to_kernel_blocks.argtypes = [vp, i32, i64, i32, i32, i32, vp, i64, vp]
        lib.bkv_cache_write.restype = cint
        lib.bkv_cache_write.argtypes = [vp, vp, i64, i64, vp, vp, vp, i64, i32, i32, i32, cint, vp, vp]
        lib.bkv_slot_mapping_cache_write_fp8.restype = cint
        lib.bkv_slot_mapping_cache_write_fp8.argtypes = [vp, i32, i64, i32, vp, vp, i64, i64, vp, vp, vp, i64, vp,
                                                         vp, i64, i32, i32, i32, cint, f32, f32, vp, vp]
        lib.bkv_slot_mapping_cache_write.restype = cint
        lib.bkv_slot_mapping_cache_write.argtypes = [vp, i32, i64, i32, vp, vp, i64, i64, vp, vp, vp, i64, vp, vp,
                                                     i64, i32, i32, i32, cint, vp, vp]
        lib.bkv_paged_decode_workspace_size.restype = sz
        lib.bkv_paged_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        dec = [vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i32, i32, i32, i32, i64, f32, cint, i32, cint, vp, vp, sz,
               vp, vp]
        for fn in ("bkv_paged_decode_swa", "bkv_paged_decode_partition", "bkv_paged_decode_merge"):
            getattr(lib, fn).restype = cint
            getattr(lib, fn).argtypes = dec
        # the boundary's own form: no sliding_window argument
        lib.bkv_paged_decode.restype = cint
        lib.bkv_paged_decode.argtypes = dec[:17] + dec[18:]
        lib.bkv_paged_decode_noalloc.restype = cint
        lib.bkv_paged_decode_noalloc.argtypes = dec[:17] + [cint, vp, vp, vp]
        lib.bkv_cache_write_fp8.restype = cint
        lib.bkv_cache_write_fp8.argtypes = [vp, vp, i64, i64, vp, vp, vp, i64, i32, i32, i32, cint, f32, f32, vp, vp]
        dec8 = [vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i32, i32, i32, i32, i64, f32, f32, f32, cint, i32, cint,
                vp, vp, sz, vp, vp]
        for fn in ("bkv_paged_decode_fp8", "bkv_paged_decode_fp8_partition", "bkv_paged_decode_fp8_merge"):
            getattr(lib, fn).restype = cint
            getattr(lib, fn).argtypes = dec8
        rope = [vp, vp, vp, i64, i64, i64, vp, vp, f32, vp, i64, i32, cint, vp, i32, i64, i32, vp, vp, vp, i64, i64, vp,
                vp, vp, vp, i64, i32, i32, i32, i32, cint]
        lib.bkv_qk_norm_rope_cache_write.restype = cint
        lib.bkv_qk_norm_rope_cache_write.argtypes = rope + [vp, vp]
        lib.bkv_qk_norm_rope_cache_write_fp8.restype = cint
        lib.bkv_qk_norm_rope_cache_write_fp8.argtypes = rope + [f32, f32, vp, vp]
        lib.bkv_paged_decode_tree_workspace_size.restype = sz
        lib.bkv_paged_decode_tree_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.bkv_paged_decode_tree.restype = cint
        lib.bkv_paged_decode_tree.argtypes = [vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i32, i32, i32, i32, i64, f32,
                                              vp, i64, cint, vp, vp, sz, vp, vp]
        lib.bkv_verify_draft_chain.restype = cint
        lib.bkv_verify_draft_chain.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
        lib.bkv_verify_draft_tree.restype = cint
        lib.bkv_verify_draft_tree.argtypes = [vp, i64, i64, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp, vp]
        _lib = lib
        return lib


def _check(fn: str, status: int):
    if status != BKV_OK:
        raise BkvError(fn, status)


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(_current_device())
    return stream.cuda_stream


def _dev(t: torch.Tensor, name: str, dtype=None, contiguous=True):
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _opt(t, name, dtype):
    return None if t is None else _dev(t, name, dtype)


def _kv_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BKV_BF16
    if t.dtype == torch.float32:
        return BKV_F32
    raise TypeError(f"KV/Q tensors must be bfloat16 or float32, got {t.dtype}")


def bkv_compute_slot_mapping(block_table, req_indices, positions, block_size, slot_mapping, num_tokens=None,
                             err_count=None, stream=None):
    """slot_mapping[i] = block_table[req, pos // bs] * bs + pos % bs, -1 for padding (see include/bkv.h)."""
    return _slot_mapping("bkv_compute_slot_mapping", (), block_table, req_indices, positions, block_size,
                         slot_mapping, num_tokens, err_count, stream)


def bkv_compute_slot_mapping_cp(block_table, req_indices, positions, block_size, slot_mapping, cp_world, cp_rank,
                                cp_interleave=1, num_tokens=None, err_count=None, stream=None):
    """Rank ``cp_rank``'s slots under decode context parallelism, -1 for other ranks' tokens (see include/bkv.h)."""
    return _slot_mapping("bkv_compute_slot_mapping_cp", (int(cp_world), int(cp_rank), int(cp_interleave)),
                         block_table, req_indices, positions, block_size, slot_mapping, num_tokens, err_count, stream)


def _slot_mapping(fn, cp, block_table, req_indices, positions, block_size, slot_mapping, num_tokens, err_count,
                  stream):
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be 2-D with unit column stride")
    n = positions.numel() if num_tokens is None else int(num_tokens)
    if n > positions.numel() or n > req_indices.numel() or n > slot_mapping.numel():
        raise ValueError("num_tokens exceeds positions / req_indices / slot_mapping")
    _check(fn, getattr(load(), fn)(
        _dev(block_table, "block_table", torch.int32, contiguous=False), block_table.shape[0],
        block_table.stride(0), block_table.shape[1], _dev(req_indices, "req_indices", torch.int32),
        _dev(positions, "positions", torch.int64), n, slot_mapping.numel(), int(block_size), *cp,
        _dev(slot_mapping, "slot_mapping", torch.int64), _opt(err_count, "err_count", torch.int32), _stream(stream)))
    return slot_mapping


def bkv_map_to_kernel_blocks(mgr_table, block_size, kernel_block_size, kernel_table, stream=None):
    """Expand manager block ids into kernel block ids m * bpk + t (see include/bkv.h)."""
    if mgr_table.dim() != 2 or kernel_table.dim() != 2 or mgr_table.stride(1) != 1 or kernel_table.stride(1) != 1:
        raise ValueError("tables must be 2-D with unit column stride")
    if kernel_table.shape[0] != mgr_table.shape[0]:
        raise ValueError("row count mismatch")
    _check("bkv_map_to_kernel_blocks", load().bkv_map_to_kernel_blocks(
        _dev(mgr_table, "mgr_table", torch.int32, contiguous=False), mgr_table.shape[0], mgr_table.stride(0),
        mgr_table.shape[1], int(block_size), int(kernel_block_size),
        _dev(kernel_table, "kernel_table", torch.int32, contiguous=False), kernel_table.stride(0), _stream(stream)))
    return kernel_table


def bkv_cache_write(k_new, v_new, slot_mapping, k_cache, v_cache, num_tokens=None, err_count=None, stream=None):
    """Scatter k_new/v_new rows (num_tokens, H_kv, D) into the caches at slot_mapping (see include/bkv.h)."""
    dt = _check_kv_rows(k_new, v_new, k_cache, v_cache)
    tb, bs, hkv, d = k_cache.shape
    n = k_new.shape[0] if num_tokens is None else int(num_tokens)
    if n > k_new.shape[0] or n > slot_mapping.numel():
        raise ValueError("num_tokens exceeds k_new / slot_mapping")
    _check("bkv_cache_write", load().bkv_cache_write(
        _dev(k_new, "k_new", contiguous=False), _dev(v_new, "v_new", contiguous=False), n, k_new.stride(0),
        _dev(slot_mapping, "slot_mapping", torch.int64), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), tb, bs,
        hkv, d, dt, _opt(err_count, "err_count", torch.int32), _stream(stream)))


def bkv_slot_mapping_cache_write(block_table, req_indices, positions, slot_mapping, k_new, v_new, k_cache, v_cache,
                                 num_tokens=None, err_count=None, stream=None):
    """bkv_compute_slot_mapping then bkv_cache_write in one kernel, with the same results; the caches'
    block size is the table's (see include/bkv.h)."""
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be 2-D with unit column stride")
    dt = _check_kv_rows(k_new, v_new, k_cache, v_cache)
    tb, bs, hkv, d = k_cache.shape
    n = positions.numel() if num_tokens is None else int(num_tokens)
    if n > positions.numel() or n > req_indices.numel() or n > slot_mapping.numel() or n > k_new.shape[0]:
        raise ValueError("num_tokens exceeds positions / req_indices / slot_mapping / k_new")
    _check("bkv_slot_mapping_cache_write", load().bkv_slot_mapping_cache_write(
        _dev(block_table, "block_table", torch.int32, contiguous=False), block_table.shape[0],
        block_table.stride(0), block_table.shape[1], _dev(req_indices, "req_indices", torch.int32),
        _dev(positions, "positions", torch.int64), n, slot_mapping.numel(),
        _dev(slot_mapping, "slot_mapping", torch.int64), _dev(k_new, "k_new", contiguous=False),
        _dev(v_new, "v_new", contiguous=False), k_new.stride(0), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        tb, bs, hkv, d, dt, _opt(err_count, "err_count", torch.int32), _stream(stream)))
    return slot_mapping


def bkv_slot_mapping_cache_write_fp8(block_table, req_indices, positions, slot_mapping, k_new, v_new, k_cache,
                                     v_cache, k_scale, v_scale, num_tokens=None, err_count=None, stream=None):
    """bkv_compute_slot_mapping then bkv_cache_write_fp8 in one kernel, with the same results: k_new / v_new
    (num_tokens, H_kv, D) bf16 or fp32 quantised into uint8 E4M3 caches (see include/bkv.h)."""
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be 2-D with unit column stride")
    dt = _check_kv_rows(k_new, v_new, k_cache, v_cache, fp8=True)
    tb, bs, hkv, d = k_cache.shape
    n = positions.numel() if num_tokens is None else int(num_tokens)
    if n > positions.numel() or n > req_indices.numel() or n > slot_mapping.numel() or n > k_new.shape[0]:
        raise ValueError("num_tokens exceeds positions / req_indices / slot_mapping / k_new")
    _check("bkv_slot_mapping_cache_write_fp8", load().bkv_slot_mapping_cache_write_fp8(
        _dev(block_table, "block_table", torch.int32, contiguous=False), block_table.shape[0],
        block_table.stride(0), block_table.shape[1], _dev(req_indices, "req_indices", torch.int32),
        _dev(positions, "positions", torch.int64), n, slot_mapping.numel(),
        _dev(slot_mapping, "slot_mapping", torch.int64), _dev(k_new, "k_new", contiguous=False),
        _dev(v_new, "v_new", contiguous=False), k_new.stride(0), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        tb, bs, hkv, d, dt, float(k_scale), float(v_scale), _opt(err_count, "err_count", torch.int32),
        _stream(stream)))
    return slot_mapping


def _check_kv_rows(k_new, v_new, k_cache, v_cache, fp8=False):
    """Shape, layout and dtype checks shared by the cache writes; returns the dtype code of the rows.

    Caches (total_blocks, block_size, H_kv, D), equal in shape: bf16 / fp32 like the rows, or uint8 E4M3
    codes when ``fp8``.  Rows (num_tokens, H_kv, D), dense within a row (a row stride is allowed)."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("caches must be (total_blocks, block_size, H_kv, D) and equal in shape")
    _, _, hkv, d = k_cache.shape
    if k_new.dim() != 3 or tuple(k_new.shape[1:]) != (hkv, d) or k_new.shape != v_new.shape:
        raise ValueError("k_new/v_new must be (num_tokens, H_kv, D) matching the cache")
    if k_new.stride(2) != 1 or k_new.stride(1) != d or k_new.stride() != v_new.stride():
        raise ValueError("k_new/v_new rows must be dense (a row stride is allowed)")
    if fp8:
        if k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8:
            raise TypeError("FP8 caches are uint8 tensors of E4M3 codes")
        if k_new.dtype != v_new.dtype:
            raise TypeError("mixed dtypes")
        return _kv_dtype(k_new)
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise TypeError("mixed dtypes")
    return _kv_dtype(k_cache)


def bkv_cache_write_fp8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, num_tokens=None,
                        err_count=None, stream=None):
    """Quantise k_new/v_new rows (num_tokens, H_kv, D; bf16 or fp32) into uint8 E4M3 caches at slot_mapping
    with per-tensor scales (see include/bkv.h)."""
    dt = _check_kv_rows(k_new, v_new, k_cache, v_cache, fp8=True)
    tb, bs, hkv, d = k_cache.shape
    n = k_new.shape[0] if num_tokens is None else int(num_tokens)
    if n > k_new.shape[0] or n > slot_mapping.numel():
        raise ValueError("num_tokens exceeds k_new / slot_mapping")
    _check("bkv_cache_write_fp8", load().bkv_cache_write_fp8(
        _dev(k_new, "k_new", contiguous=False), _dev(v_new, "v_new", contiguous=False), n, k_new.stride(0),
        _dev(slot_mapping, "slot_mapping", torch.int64), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), tb, bs,
        hkv, d, dt, float(k_scale), float(v_scale), _opt(err_count, "err_count", torch.int32), _stream(stream)))


def bkv_paged_decode_workspace_size(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                    max_context_len) -> int:
    return int(load().bkv_paged_decode_workspace_size(int(num_reqs), int(q_len), int(num_q_heads),
                                                      int(num_kv_heads), int(head_dim), int(block_size),
                                                      int(max_context_len)))


def bkv_paged_decode(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace,
                     softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None, stream=None):
    """GQA paged decode attention into ``out`` (num_reqs, q_len, H_q, D) (see include/bkv.h)."""
    return _decode("bkv_paged_decode", q, k_cache, v_cache, block_table, context_lens, max_context_len, out,
                   workspace, softmax_scale, mask_mode, None, err_count, stream)


def bkv_paged_decode_swa(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace,
                         sliding_window, softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None, stream=None):
    """bkv_paged_decode of a sliding-window layer: query t sees the last ``sliding_window`` positions up to its
    own (0: full attention) (see include/bkv.h)."""
    return _decode("bkv_paged_decode_swa", q, k_cache, v_cache, block_table, context_lens, max_context_len, out,
                   workspace, softmax_scale, mask_mode, sliding_window, err_count, stream)


def bkv_paged_decode_noalloc(q, k_cache, v_cache, block_table, context_lens, max_context_len, out,
                             softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None, stream=None):
    """bkv_paged_decode with its scratch in the library's fixed device array instead of a workspace (see
    include/bkv.h)."""
    return _decode("bkv_paged_decode_noalloc", q, k_cache, v_cache, block_table, context_lens, max_context_len, out,
                   False, softmax_scale, mask_mode, None, err_count, stream)


def bkv_paged_decode_partition(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace,
                               softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None, stream=None,
                               sliding_window=0):
    """Phase 1 of bkv_paged_decode: split-KV partials into ``workspace`` (see include/bkv.h)."""
    return _decode("bkv_paged_decode_partition", q, k_cache, v_cache, block_table, context_lens, max_context_len,
                   out, workspace, softmax_scale, mask_mode, sliding_window, err_count, stream)


def bkv_paged_decode_merge(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace,
                           softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None, stream=None,
                           sliding_window=0):
    """Phase 2 of bkv_paged_decode: merge the workspace partials into ``out`` (see include/bkv.h)."""
    return _decode("bkv_paged_decode_merge", q, k_cache, v_cache, block_table, context_lens, max_context_len, out,
                   workspace, softmax_scale, mask_mode, sliding_window, err_count, stream)


def _decode(fn, q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace, softmax_scale,
            mask_mode, sliding_window, err_count, stream, scales=None):
    if q.dim() != 4 or out.shape != q.shape or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("q/out must be (num_reqs, q_len, H_q, D); caches (total_blocks, bs, H_kv, D)")
    nr, ql, hq, d = q.shape
    tb, bs, hkv, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("head_dim mismatch")
    if block_table.dim() != 2 or block_table.shape[0] < nr or block_table.stride(1) != 1:
        raise ValueError("block_table must be (>= num_reqs, cols) with unit column stride")
    dt = _kv_dtype(q)
    cache_dtype = q.dtype if scales is None else torch.uint8
    for t, nm, want in ((k_cache, "k_cache", cache_dtype), (v_cache, "v_cache", cache_dtype), (out, "out", q.dtype)):
        if t.dtype != want:
            raise TypeError(f"{nm} must be {want}, got {t.dtype}")
    # workspace: a uint8 tensor, None (a null pointer), or False (the entry point takes none)
    if workspace is not None and workspace is not False and workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    ws = ()
    if workspace is not False:
        ws = (None, 0) if workspace is None else (_dev(workspace, "workspace"), workspace.numel())
    window = () if sliding_window is None else (int(sliding_window),)
    _check(fn, getattr(load(), fn)(
        _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_table, "block_table", torch.int32, contiguous=False), block_table.stride(0),
        block_table.shape[1], _dev(context_lens, "context_lens", torch.int32), int(max_context_len), nr, ql, hq, hkv,
        d, bs, tb, float(softmax_scale), *(() if scales is None else (float(scales[0]), float(scales[1]))),
        int(mask_mode), *window, dt, _dev(out, "out"), *ws, _opt(err_count, "err_count", torch.int32),
        _stream(stream)))
    return out


def bkv_paged_decode_fp8(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace, k_scale,
                         v_scale, softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None, stream=None,
                         sliding_window=0):
    """bkv_paged_decode over uint8 E4M3 caches with per-tensor scales (see include/bkv.h)."""
    return _decode("bkv_paged_decode_fp8", q, k_cache, v_cache, block_table, context_lens, max_context_len, out,
                   workspace, softmax_scale, mask_mode, sliding_window, err_count, stream, scales=(k_scale, v_scale))


def bkv_paged_decode_fp8_partition(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace,
                                   k_scale, v_scale, softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None,
                                   stream=None, sliding_window=0):
    """Phase 1 of bkv_paged_decode_fp8 (see include/bkv.h)."""
    return _decode("bkv_paged_decode_fp8_partition", q, k_cache, v_cache, block_table, context_lens,
                   max_context_len, out, workspace, softmax_scale, mask_mode, sliding_window, err_count, stream,
                   scales=(k_scale, v_scale))


def bkv_paged_decode_fp8_merge(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, workspace,
                               k_scale, v_scale, softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None,
                               stream=None, sliding_window=0):
    """Phase 2 of bkv_paged_decode_fp8 (see include/bkv.h)."""
    return _decode("bkv_paged_decode_fp8_merge", q, k_cache, v_cache, block_table, context_lens, max_context_len,
                   out, workspace, softmax_scale, mask_mode, sliding_window, err_count, stream,
                   scales=(k_scale, v_scale))


def bkv_paged_decode_cp(q, k_cache, v_cache, block_table, context_lens, max_context_len, out, lse, workspace,
                        cp_world, cp_rank, cp_interleave=1, softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL,
                        err_count=None, stream=None):
    """One rank's part of a context-parallel decode: its normalised ``out`` and fp32 ``lse`` (num_reqs, q_len,
    H_q) over the keys it holds; ``context_lens`` are global lengths (see include/bkv.h).  ``lse`` may be None."""
    if q.dim() != 4 or out.shape != q.shape or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("q/out must be (num_reqs, q_len, H_q, D); caches (total_blocks, bs, H_kv, D)")
    nr, ql, hq, d = q.shape
    tb, bs, hkv, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("head_dim mismatch")
    if block_table.dim() != 2 or block_table.shape[0] < nr or block_table.stride(1) != 1:
        raise ValueError("block_table must be (>= num_reqs, cols) with unit column stride")
    if lse is not None and tuple(lse.shape) != (nr, ql, hq):
        raise ValueError("lse must be (num_reqs, q_len, H_q)")
    dt = _kv_dtype(q)
    for t, nm in ((k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
        if t.dtype != q.dtype:
            raise TypeError(f"{nm} dtype differs from q")
    ws_ptr = None if workspace is None else _dev(workspace, "workspace")
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check("bkv_paged_decode_cp", load().bkv_paged_decode_cp(
        _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_table, "block_table", torch.int32, contiguous=False), block_table.stride(0),
        block_table.shape[1], _dev(context_lens, "context_lens", torch.int32), int(max_context_len), nr, ql, hq, hkv,
        d, bs, tb, float(softmax_scale), int(mask_mode), int(cp_world), int(cp_rank), int(cp_interleave), dt,
        _dev(out, "out"), _opt(lse, "lse", torch.float32), ws_ptr, ws_bytes, _opt(err_count, "err_count", torch.int32),
        _stream(stream)))
    return out, lse


def bkv_paged_attention_ragged(q, query_start_loc, k_cache, v_cache, block_table, context_lens, max_context_len,
                               max_query_len, out, softmax_scale=0.0, mask_mode=BKV_MASK_CAUSAL, err_count=None,
                               stream=None):
    """Attention over a mixed step: q / out packed (num_tokens, H_q, D), request r's tokens at
    [query_start_loc[r], query_start_loc[r+1]) (see include/bkv.h)."""
    if q.dim() != 3 or out.shape != q.shape or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("q/out must be (num_tokens, H_q, D); caches (total_blocks, bs, H_kv, D)")
    nt, hq, d = q.shape
    tb, bs, hkv, d2 = k_cache.shape
    nr = query_start_loc.numel() - 1
    if d2 != d or nr < 0 or context_lens.numel() < nr:
        raise ValueError("head_dim / query_start_loc / context_lens mismatch")
    if block_table.dim() != 2 or block_table.shape[0] < nr or block_table.stride(1) != 1:
        raise ValueError("block_table must be (>= num_reqs, cols) with unit column stride")
    dt = _kv_dtype(q)
    for t, nm in ((k_cache, "k_cache"), (v_cache, "v_cache"), (out, "out")):
        if t.dtype != q.dtype:
            raise TypeError(f"{nm} dtype differs from q")
    _check("bkv_paged_attention_ragged", load().bkv_paged_attention_ragged(
        _dev(q, "q"), _dev(query_start_loc, "query_start_loc", torch.int32), _dev(k_cache, "k_cache"),
        _dev(v_cache, "v_cache"), _dev(block_table, "block_table", torch.int32, contiguous=False),
        block_table.stride(0), block_table.shape[1], _dev(context_lens, "context_lens", torch.int32),
        int(max_context_len), int(max_query_len), nr, nt, hq, hkv, d, bs, tb, float(softmax_scale), int(mask_mode),
        dt, _dev(out, "out"), _opt(err_count, "err_count", torch.int32), _stream(stream)))
    return out


def bkv_merge_attn_states(outs, lses, out, lse_out=None, stream=None):
    """Merge ``parts`` partial results: outs (parts, rows, D), lses fp32 (parts, rows) -> out (rows, D) and
    optionally lse_out (rows) (see include/bkv.h).  Any leading shape with the same element count works."""
    parts = outs.shape[0]
    rows = lses[0].numel()
    d = outs.shape[-1]
    if outs.numel() != parts * rows * d or lses.numel() != parts * rows or out.numel() != rows * d:
        raise ValueError("outs (parts, rows, D), lses (parts, rows), out (rows, D) sizes disagree")
    if out.dtype != outs.dtype:
        raise TypeError("out dtype differs from outs")
    _check("bkv_merge_attn_states", load().bkv_merge_attn_states(
        _dev(outs, "outs"), _dev(lses, "lses", torch.float32), parts, rows, d, _kv_dtype(outs), _dev(out, "out"),
        _opt(lse_out, "lse_out", torch.float32), _stream(stream)))
    return out


_gpus = None   # GPUs of this process, once a call has asked


def _same_device(*tensors):
    """Every tensor on the current device, whose stream the call is enqueued on (with one GPU there is no other)."""
    global _gpus
    if _gpus is None:
        _gpus = torch.cuda.device_count()
    if _gpus == 1:
        return
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on the current device (cuda:{dev}), got {t.device}")


def bkv_qk_norm_rope_cache_write(q, k, v, q_weight, k_weight, norm_eps, cos_sin, block_table, req_indices, positions,
                                 slot_mapping, q_out, k_cache, v_cache, rope_positions=None, interleaved=False,
                                 num_tokens=None, err_count=None, stream=None):
    """Norm of every head of q and k (weights (D,) or None), position rotation by ``cos_sin`` (max_position,
    rot_dim; None: no rotation), slot mapping and K/V write in one kernel: q (num_tokens, H_q, D) -> ``q_out``,
    k / v (num_tokens, H_kv, D) -> the caches (see include/bkv.h).  Returns (q_out, slot_mapping)."""
    return _norm_rope("bkv_qk_norm_rope_cache_write", (), q, k, v, q_weight, k_weight, norm_eps, cos_sin, block_table,
                      req_indices, positions, slot_mapping, q_out, k_cache, v_cache, rope_positions, interleaved,
                      num_tokens, err_count, stream)


def bkv_qk_norm_rope_cache_write_fp8(q, k, v, q_weight, k_weight, norm_eps, cos_sin, block_table, req_indices,
                                     positions, slot_mapping, q_out, k_cache, v_cache, k_scale, v_scale,
                                     rope_positions=None, interleaved=False, num_tokens=None, err_count=None,
                                     stream=None):
    """bkv_qk_norm_rope_cache_write into uint8 E4M3 caches with per-tensor scales (see include/bkv.h)."""
    return _norm_rope("bkv_qk_norm_rope_cache_write_fp8", (float(k_scale), float(v_scale)), q, k, v, q_weight, k_weight,
                      norm_eps, cos_sin, block_table, req_indices, positions, slot_mapping, q_out, k_cache, v_cache,
                      rope_positions, interleaved, num_tokens, err_count, stream)


def _norm_rope(fn, scales, q, k, v, q_weight, k_weight, norm_eps, cos_sin, block_table, req_indices, positions,
               slot_mapping, q_out, k_cache, v_cache, rope_positions, interleaved, num_tokens, err_count, stream):
    cache, qs, ks = k_cache.shape, q.shape, k.shape
    if len(cache) != 4 or cache != v_cache.shape:
        raise ValueError("caches must be (total_blocks, block_size, H_kv, D) and equal in shape")
    tb, bs, hkv, d = cache
    if len(qs) != 3 or qs[2] != d or len(ks) != 3 or ks[1] != hkv or ks[2] != d or ks != v.shape:
        raise ValueError("q must be (num_tokens, H_q, D), k / v (num_tokens, H_kv, D) matching the cache")
    nt, hq, _ = qs
    (q_row, qh, qe), (k_row, kh, ke), (v_row, vh, ve) = q.stride(), k.stride(), v.stride()
    # (a dimension of size 1 may carry any stride)
    if qe != 1 or ke != 1 or ve != 1 or (qh != d and hq > 1) or (hkv > 1 and (kh != d or vh != d)):
        raise ValueError("q, k and v rows must be dense (a row stride is allowed)")
    if nt <= 1:
        q_row = max(q_row, hq * d)
    if ks[0] <= 1:
        k_row, v_row = max(k_row, hkv * d), max(v_row, hkv * d)
    dtype = q.dtype
    dt = _kv_dtype(q)
    cache_dtype = torch.uint8 if scales else dtype
    if k.dtype is not dtype or v.dtype is not dtype:
        raise TypeError("mixed dtypes")
    if k_cache.dtype is not cache_dtype or v_cache.dtype is not cache_dtype or q_out.dtype is not dtype:
        raise TypeError(f"caches must be {cache_dtype} and q_out {dtype}")
    outs = q_out.shape
    if len(outs) != 3 or outs[0] < nt or outs[1] != hq or outs[2] != d:
        raise ValueError("q_out must be (>= num_tokens, H_q, D)")
    if (q_weight is not None and q_weight.numel() != d) or (k_weight is not None and k_weight.numel() != d):
        raise ValueError("q_weight and k_weight must have head_dim elements")
    max_pos, rot = 1 << 62, 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be (max_position, rot_dim)")
        max_pos, rot = cos_sin.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D with unit column stride")
    (rows, cols), (bt_row, bt_col) = block_table.shape, block_table.stride()
    if bt_col != 1 and cols > 1:
        raise ValueError("block_table must be 2-D with unit column stride")
    if rows <= 1:
        bt_row = max(bt_row, cols)
    n, most = positions.numel(), slot_mapping.numel()
    if num_tokens is not None:
        if int(num_tokens) > n:
            raise ValueError("num_tokens exceeds positions")
        n = int(num_tokens)
    if (n > nt or n > ks[0] or n > req_indices.numel() or n > most or
            (rope_positions is not None and n > rope_positions.numel())):
        raise ValueError("num_tokens exceeds q / k / req_indices / slot_mapping / rope_positions")
    args = (_dev(q, "q", None, False), _dev(k, "k", None, False), _dev(v, "v", None, False), q_row, k_row, v_row,
            None if q_weight is None else _dev(q_weight, "q_weight", dtype),
            None if k_weight is None else _dev(k_weight, "k_weight", dtype), norm_eps,
            None if cos_sin is None else _dev(cos_sin, "cos_sin", torch.float32), max_pos, rot, 1 if interleaved else 0,
            _dev(block_table, "block_table", torch.int32, False), rows, bt_row, cols,
            _dev(req_indices, "req_indices", torch.int32), _dev(positions, "positions", torch.int64),
            None if rope_positions is None else _dev(rope_positions, "rope_positions", torch.int64), n, most,
            _dev(slot_mapping, "slot_mapping", torch.int64), _dev(q_out, "q_out"),
            _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), tb, bs, hq, hkv, d, dt, *scales,
            None if err_count is None else _dev(err_count, "err_count", torch.int32))
    _same_device(q, k, v, q_weight, k_weight, cos_sin, block_table, req_indices, positions, rope_positions, slot_mapping,
                 q_out, k_cache, v_cache, err_count)
    _check(fn, getattr(load(), fn)(*args, _stream(stream)))
    return q_out, slot_mapping


def bkv_paged_decode_tree_workspace_size(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                         max_context_len) -> int:
    return int(load().bkv_paged_decode_tree_workspace_size(int(num_reqs), int(q_len), int(num_q_heads),
                                                           int(num_kv_heads), int(head_dim), int(block_size),
                                                           int(max_context_len)))


def bkv_paged_decode_tree(q, k_cache, v_cache, block_table, context_lens, max_context_len, tree_mask, out, workspace,
                          softmax_scale=0.0, err_count=None, stream=None):
    """Paged attention of drafted trees into ``out`` (num_reqs, q_len, H_q, D): a request's q_len tokens are its
    last cached positions, and bit i of token t's words in ``tree_mask`` (int32, (num_reqs, q_len, ceil(q_len /
    32)), or (q_len, ..) for one tree of all requests) lets it see token i (see include/bkv.h)."""
    shape, cache = q.shape, k_cache.shape
    if len(shape) != 4 or out.shape != shape or len(cache) != 4 or cache != v_cache.shape:
        raise ValueError("q/out must be (num_reqs, q_len, H_q, D); caches (total_blocks, bs, H_kv, D)")
    nr, ql, hq, d = shape
    tb, bs, hkv, d2 = cache
    if d2 != d:
        raise ValueError("head_dim mismatch")
    table = block_table.shape
    if len(table) != 2 or table[0] < nr or (block_table.stride(1) != 1 and table[1] > 1):
        raise ValueError("block_table must be (>= num_reqs, cols) with unit column stride")
    bt_row = block_table.stride(0) if table[0] > 1 else max(block_table.stride(0), table[1])
    if context_lens.numel() < nr:
        raise ValueError("context_lens must have num_reqs elements")
    words, ms = (ql + 31) // 32, tree_mask.shape
    if ms[-2:] != (ql, words) or (len(ms) != 2 and (len(ms) != 3 or ms[0] < nr)):
        raise ValueError("tree_mask must be (num_reqs, q_len, ceil(q_len / 32)) or (q_len, ceil(q_len / 32))")
    dt, dtype = _kv_dtype(q), q.dtype
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype or out.dtype is not dtype:
        raise TypeError(f"caches and out must be {dtype}")
    if workspace.dtype is not torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    args = (_dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _dev(block_table, "block_table", torch.int32, contiguous=False), bt_row, table[1],
            _dev(context_lens, "context_lens", torch.int32), int(max_context_len), nr, ql, hq, hkv, d, bs, tb,
            float(softmax_scale), _dev(tree_mask, "tree_mask", torch.int32), ql * words if len(ms) == 3 else 0, dt,
            _dev(out, "out"), _dev(workspace, "workspace"), workspace.numel(), _opt(err_count, "err_count", torch.int32))
    _same_device(q, k_cache, v_cache, block_table, context_lens, tree_mask, out, workspace, err_count)
    _check("bkv_paged_decode_tree", load().bkv_paged_decode_tree(*args, _stream(stream)))
    return out


def bkv_verify_draft_chain(target_probs, draft_probs, draft_tokens, accept_u, sample_u, out_tokens, num_accepted,
                           draft_lens=None, err_count=None, stream=None):
    """Accepts drafted tokens (num_reqs, K) against the target's probabilities (num_reqs, K + 1, V) and the draft
    model's (num_reqs, K, V), both fp32, by the uniform numbers accept_u (num_reqs, K) and sample_u (num_reqs)
    -> out_tokens int64 (num_reqs, K + 1), num_accepted int32 (num_reqs) (see include/bkv.h)."""
    nr, k1, vocab = target_probs.shape
    k = k1 - 1
    if (draft_probs.shape != (nr, k, vocab) or draft_tokens.shape != (nr, k) or accept_u.shape != (nr, k) or
            out_tokens.shape != (nr, k1)):
        raise ValueError("target_probs (R, K + 1, V), draft_probs (R, K, V), draft_tokens / accept_u (R, K) and "
                         "out_tokens (R, K + 1) disagree")
    if sample_u.numel() != nr or num_accepted.numel() != nr or (draft_lens is not None and draft_lens.numel() != nr):
        raise ValueError("sample_u, num_accepted and draft_lens must have num_reqs elements")
    if vocab > 1 and (target_probs.stride(2) != 1 or (k > 0 and draft_probs.stride(2) != 1)):
        raise ValueError("probability rows must be dense")
    args = (_dev(target_probs, "target_probs", torch.float32, contiguous=False), *_row_strides(target_probs),
            _dev(draft_probs, "draft_probs", torch.float32, contiguous=False), *_row_strides(draft_probs),
            _dev(draft_tokens, "draft_tokens", torch.int64), _opt(draft_lens, "draft_lens", torch.int32),
            _dev(accept_u, "accept_u", torch.float32), _dev(sample_u, "sample_u", torch.float32), nr, k, vocab,
            _dev(out_tokens, "out_tokens", torch.int64), _dev(num_accepted, "num_accepted", torch.int32),
            _opt(err_count, "err_count", torch.int32))
    _same_device(target_probs, draft_probs, draft_tokens, draft_lens, accept_u, sample_u, out_tokens, num_accepted,
                 err_count)
    _check("bkv_verify_draft_chain", load().bkv_verify_draft_chain(*args, _stream(stream)))
    return out_tokens, num_accepted


def bkv_verify_draft_tree(target_probs, draft_tokens, parents, accept_u, sample_u, out_tokens, path, num_accepted,
                          err_count=None, stream=None):
    """Accepts a path of a tree of drafted tokens (num_reqs, T; node 0 the root, parents int32) against the
    target's probabilities fp32 (num_reqs, T, V) by the uniform numbers accept_u (num_reqs, T) and sample_u
    (num_reqs) -> out_tokens int64, path int32 (num_reqs, T), num_accepted int32 (num_reqs) (see include/bkv.h)."""
    nr, t, vocab = target_probs.shape
    for x, name in ((draft_tokens, "draft_tokens"), (parents, "parents"), (accept_u, "accept_u"),
                    (out_tokens, "out_tokens"), (path, "path")):
        if x.shape != (nr, t):
            raise ValueError(f"{name} must be (num_reqs, num_nodes)")
    if sample_u.numel() != nr or num_accepted.numel() != nr:
        raise ValueError("sample_u and num_accepted must have num_reqs elements")
    if vocab > 1 and target_probs.stride(2) != 1:
        raise ValueError("probability rows must be dense")
    args = (_dev(target_probs, "target_probs", torch.float32, contiguous=False), *_row_strides(target_probs),
            _dev(draft_tokens, "draft_tokens", torch.int64), _dev(parents, "parents", torch.int32),
            _dev(accept_u, "accept_u", torch.float32), _dev(sample_u, "sample_u", torch.float32), nr, t, vocab,
            _dev(out_tokens, "out_tokens", torch.int64), _dev(path, "path", torch.int32),
            _dev(num_accepted, "num_accepted", torch.int32), _opt(err_count, "err_count", torch.int32))
    _same_device(target_probs, draft_tokens, parents, accept_u, sample_u, out_tokens, path, num_accepted, err_count)
    _check("bkv_verify_draft_tree", load().bkv_verify_draft_tree(*args, _stream(stream)))
    return out_tokens, path, num_accepted


def _row_strides(t):
    """Request and row stride of probabilities (R, rows, V); a dimension of size 1 or 0 may carry any stride."""
    (reqs, rows, vocab), (req, row, _) = t.shape, t.stride()
    return req if reqs > 1 else 0, row if rows > 1 else vocab


def alloc_tree_workspace(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, device=None):
    """Convenience: a uint8 device tensor of the size bkv_paged_decode_tree needs."""
    n = bkv_paged_decode_tree_workspace_size(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                             max_context_len)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def alloc_workspace(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len, device=None):
    """Convenience: a uint8 device tensor of the size bkv_paged_decode needs."""
    n = bkv_paged_decode_workspace_size(num_reqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                        max_context_len)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
