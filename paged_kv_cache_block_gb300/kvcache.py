"""Python binding of libpagedkv.so (the C ABI in include/pagedkv.h).

Argument marshalling only: every step of the path runs in the library's CUDA kernels.  PyTorch
supplies device memory and the current stream.  Importing this module loads the library and
raises if it has not been built (``python -m paged_kv_cache_block_gb300.build``); there is no
fallback implementation.

Same names as the C ABI:
    compute_slot_mapping(...)        kv_compute_slot_mapping
    reshape_and_cache(...)           kv_reshape_and_cache
    paged_attention_workspace_size() kv_paged_attention_workspace_size
    paged_attention_decode(...)      kv_paged_attention_decode
    decode_step(...)                 kv_decode_step
    paged_attention_prefill(...)     kv_paged_attention_prefill
    BlockManager                     kv_bm_* (host block manager, one object per handle)
    apply_block_updates(...)         kv_apply_block_updates
    reshape_and_cache_int4(...)      kv_reshape_and_cache_int4       (include/pagedkv_int4.h)
    paged_attention_decode_int4(...) kv_paged_attention_decode_int4
    decode_step_int4(...)            kv_decode_step_int4
    selftest_bounded_wait(...)       kv_selftest_bounded_wait         (include/pagedkv_selftest.h)
    build_batch(...)                 kv_build_batch                   (include/pagedkv_step.h)
    qk_norm_rope(...)                kv_qk_norm_rope
    qk_norm_rope_and_cache(...)      kv_qk_norm_rope, with the write of K and V into the cache
    paged_attention_tree(...)        kv_paged_attention_tree
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

from . import build as _build

KV_F16, KV_BF16, KV_FP8_E4M3, KV_INT4 = 0, 1, 2, 3
KV_DERR_BAD_BLOCK, KV_DERR_BAD_SLOT, KV_DERR_PAST_TABLE, KV_DERR_TIMEOUT, KV_DERR_BAD_LEN = 1, 2, 4, 8, 16
KV_DERR_BAD_UPDATE = 32
KV_DERR_BAD_POS, KV_DERR_NO_BLOCKS, KV_DERR_BAD_TREE = 64, 128, 256
KV_MAX_TREE = 64
KV_OK, KV_ERR_INVALID_ARG, KV_ERR_UNSUPPORTED, KV_ERR_CUDA, KV_ERR_WORKSPACE, KV_ERR_OUT_OF_BLOCKS = range(6)
KV_MAX_ZERO_CACHES = 128
SIZE_MAX = (1 << 64) - 1

LIB_PATH = _build.LIB


class KVError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{_STATUS.get(status, status)}: {detail}")
        self.status = status


_STATUS = {0: "KV_OK", 1: "KV_ERR_INVALID_ARG", 2: "KV_ERR_UNSUPPORTED", 3: "KV_ERR_CUDA",
           4: "KV_ERR_WORKSPACE", 5: "KV_ERR_OUT_OF_BLOCKS"}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m paged_kv_cache_block_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.kv_compute_slot_mapping.argtypes = [P, i64, i32, i32, P, P, i32, i32, i32, P, P, P]
    lib.kv_compute_slot_mapping.restype = i32
    lib.kv_reshape_and_cache.argtypes = [P, P, i32, i64, i64, i32, i32, i32, P, P, P, i32, i32, i32,
                                         f32, f32, P, P]
    lib.kv_reshape_and_cache.restype = i32
    lib.kv_paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32]
    lib.kv_paged_attention_workspace_size.restype = sz
    lib.kv_paged_attention_plan_info.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, P]
    lib.kv_paged_attention_plan_info.restype = i32
    lib.kv_paged_attention_decode.argtypes = [P, i32, i32, i32, i32, P, P, i32, i32, i32, i32, i32, P,
                                              i64, i32, P, i32, f32, i32, f32, f32, i32, P, sz, P, P,
                                              P, P]
    lib.kv_paged_attention_decode.restype = i32
    lib.kv_decode_step.argtypes = [P, i64, i32, P, P, P, P, P, i64, i64, P, i32, i32, i32, i32, P, P,
                                   i32, i32, i32, i32, i32, P, i32, f32, i32, f32, f32, i32, P, sz, P,
                                   P, P, P]
    lib.kv_decode_step.restype = i32
    lib.kv_paged_attention_decode_noalloc.argtypes = [P, i32, i32, i32, i32, P, P, i32, i32, i32, i32,
                                                      i32, P, i64, i32, P, i32, f32, i32, f32, f32,
                                                      i32, P, P, P, P]
    lib.kv_paged_attention_decode_noalloc.restype = i32
    pi32 = ctypes.POINTER(i32)
    lib.kv_bm_create.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(P)]
    lib.kv_bm_create.restype = i32
    lib.kv_bm_destroy.argtypes = [P]
    lib.kv_bm_destroy.restype = None
    lib.kv_bm_allocate.argtypes = [P, i32, i32]
    lib.kv_bm_allocate.restype = i32
    lib.kv_bm_allocate_batch.argtypes = [P, P, P, i32, P]
    lib.kv_bm_allocate_batch.restype = i32
    lib.kv_bm_free.argtypes = [P, i32]
    lib.kv_bm_free.restype = i32
    lib.kv_bm_share_prefix.argtypes = [P, i32, i32, i32]
    lib.kv_bm_share_prefix.restype = i32
    lib.kv_bm_num_free_blocks.argtypes = [P]
    lib.kv_bm_num_free_blocks.restype = i32
    lib.kv_bm_ref_count.argtypes = [P, i32]
    lib.kv_bm_ref_count.restype = i32
    lib.kv_bm_row.argtypes = [P, i32, pi32, pi32, P, i32]
    lib.kv_bm_row.restype = i32
    lib.kv_bm_pending.argtypes = [P, pi32, pi32]
    lib.kv_bm_pending.restype = i32
    lib.kv_bm_flush.argtypes = [P, P, i32, pi32, P, i32, pi32]
    lib.kv_bm_flush.restype = i32
    lib.kv_paged_attention_prefill.argtypes = [P, i32, P, i32, i32, i32, i32, P, P, i32, i32, i32, i32,
                                               i32, P, i64, i32, P, i32, f32, i32, P, P, P, P]
    lib.kv_paged_attention_prefill.restype = i32
    lib.kv_apply_block_updates.argtypes = [P, i32, P, i64, i32, i32, P, i32, P, i32, i64, i32, P, P]
    lib.kv_apply_block_updates.restype = i32
    lib.kv_reshape_and_cache_int4.argtypes = [P, P, i32, i64, i64, i32, i32, i32, P, P, P, i32, i32, P, P,
                                              i32, P, P]
    lib.kv_reshape_and_cache_int4.restype = i32
    lib.kv_paged_attention_decode_int4.argtypes = [P, i32, i32, i32, i32, P, P, i32, i32, i32, i32, P, i64,
                                                   i32, P, i32, f32, i32, P, P, i32, i32, P, sz, P, P, P, P]
    lib.kv_paged_attention_decode_int4.restype = i32
    lib.kv_decode_step_int4.argtypes = [P, i64, i32, P, P, P, P, P, i64, i64, P, i32, i32, i32, i32, P, P,
                                        i32, i32, i32, i32, P, i32, f32, i32, P, P, i32, i32, P, sz, P, P,
                                        P, P]
    lib.kv_decode_step_int4.restype = i32
    lib.kv_selftest_bounded_wait.argtypes = [i32, P, P, P]
    lib.kv_selftest_bounded_wait.restype = i32
    lib.kv_build_batch.argtypes = [P, P, P, P, i32, i32, P, i64, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P,
                                   P, P]
    lib.kv_build_batch.restype = i32
    lib.kv_qk_norm_rope.argtypes = [P, P, P, i32, i64, i64, i64, i32, i32, i32, i32, P, P, f32, P, P, i32, i32,
                                    i32, P, i64, P, i64, P, P, P, i32, i32, i32, f32, f32, P, P]
    lib.kv_qk_norm_rope.restype = i32
    lib.kv_paged_attention_tree.argtypes = [P, i32, P, i32, i32, i32, i32, P, P, i32, i32, i32, i32, i32, P, i64,
                                            i32, P, i32, f32, i32, P, i32, P, sz, P, P, P, P]
    lib.kv_paged_attention_tree.restype = i32
    lib.kv_paged_attention_tree_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.kv_paged_attention_tree_workspace_size.restype = sz
    lib.kv_status_string.argtypes = [i32]
    lib.kv_status_string.restype = ctypes.c_char_p
    lib.kv_last_error.argtypes = []
    lib.kv_last_error.restype = ctypes.c_char_p
    return lib


lib = _load()


def _check(status: int) -> None:
    if status != 0:
        raise KVError(status, lib.kv_last_error().decode())


def dtype_code(t: torch.dtype) -> int:
    if t == torch.float16:
        return KV_F16
    if t == torch.bfloat16:
        return KV_BF16
    if t in (torch.uint8, torch.float8_e4m3fn):
        return KV_FP8_E4M3
    raise TypeError(f"unsupported dtype {t}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def compute_slot_mapping(block_table: torch.Tensor, query_start_loc: torch.Tensor,
                         positions: torch.Tensor, block_size: int, num_blocks: int,
                         slot_mapping: Optional[torch.Tensor] = None,
                         d_err: Optional[torch.Tensor] = None, max_blocks_per_seq: Optional[int] = None,
                         stream=None) -> torch.Tensor:
    assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.stride(1) == 1
    assert query_start_loc.dtype == torch.int32 and positions.dtype == torch.int32
    T = positions.shape[0]
    if slot_mapping is None:
        slot_mapping = torch.empty(T, dtype=torch.int64, device=positions.device)
    _check(lib.kv_compute_slot_mapping(
        _ptr(block_table), block_table.stride(0), block_table.shape[0],
        block_table.shape[1] if max_blocks_per_seq is None else max_blocks_per_seq,
        _ptr(query_start_loc), _ptr(positions), T, block_size, num_blocks, _ptr(slot_mapping),
        _ptr(d_err), _stream(stream)))
    return slot_mapping


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
                      k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float = 1.0,
                      v_scale: float = 1.0, d_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """key/value [T, Hkv, D] (row stride = stride(0)); caches [NB, bs, Hkv, D]."""
    T, H, D = key.shape
    assert key.stride(2) == 1 and key.stride(1) == D and value.stride(2) == 1 and value.stride(1) == D
    NB, bs = k_cache.shape[0], k_cache.shape[1]
    _check(lib.kv_reshape_and_cache(
        _ptr(key), _ptr(value), dtype_code(key.dtype), key.stride(0), value.stride(0), T, H, D,
        _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), dtype_code(k_cache.dtype), NB, bs,
        float(k_scale), float(v_scale), _ptr(d_err), _stream(stream)))


def paged_attention_workspace_size(num_seqs: int, q_len: int, num_q_heads: int, num_kv_heads: int,
                                   head_dim: int, block_size: int, cache_dtype: int,
                                   max_seq_len: int, window: int = 0, num_workers: int = 0) -> int:
    n = lib.kv_paged_attention_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim,
                                              block_size, cache_dtype, max_seq_len, window,
                                              num_workers)
    if n == SIZE_MAX:
        raise KVError(2, lib.kv_last_error().decode() or "invalid or unsupported sizes")
    return int(n)


PLAN_FIELDS = ("stages", "stage_bytes", "heads_per_cta", "ctas", "threads", "rows_per_warp", "items",
               "workspace_bytes")


def paged_attention_plan_info(num_seqs: int, q_len: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                              block_size: int, cache_dtype: int, max_seq_len: int, window: int = 0,
                              num_workers: int = 0) -> dict:
    """The decode launch geometry for these sizes (kv_paged_attention_plan_info)."""
    info = (ctypes.c_int64 * 8)()
    _check(lib.kv_paged_attention_plan_info(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                            cache_dtype, max_seq_len, window, num_workers, info))
    return dict(zip(PLAN_FIELDS, list(info)))


def paged_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                           q_len: int, scale: float, window: int = 0, k_scale: float = 1.0,
                           v_scale: float = 1.0, num_workers: int = 0,
                           workspace: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                           d_err: Optional[torch.Tensor] = None, max_blocks_per_seq: Optional[int] = None,
                           stream=None) -> torch.Tensor:
    """q [B*q_len, Hq, D]; caches [NB, bs, Hkv, D]; block_table int32 [B, W]; seq_lens int32 [B]."""
    TQ, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    B = seq_lens.shape[0]
    assert TQ == B * q_len and q.is_contiguous() and block_table.stride(1) == 1
    cdt = dtype_code(k_cache.dtype)
    if out is None:
        out = torch.empty_like(q)
    need = paged_attention_workspace_size(B, q_len, Hq, Hkv, D, bs, cdt, max_seq_len, window,
                                          num_workers)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.kv_paged_attention_decode(
        _ptr(q), dtype_code(q.dtype), B, q_len, Hq, _ptr(k_cache), _ptr(v_cache), cdt, Hkv, D, bs, NB,
        _ptr(block_table), block_table.stride(0),
        block_table.shape[1] if max_blocks_per_seq is None else max_blocks_per_seq,
        _ptr(seq_lens), max_seq_len, float(scale), window, float(k_scale), float(v_scale),
        num_workers, _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse_out), _ptr(d_err),
        _stream(stream)))
    return out


def _int4_group(head_dim: int, k_scales: torch.Tensor, v_scales: torch.Tensor) -> int:
    assert k_scales.dtype == torch.float32 and v_scales.dtype == torch.float32
    assert k_scales.is_contiguous() and v_scales.is_contiguous() and k_scales.shape == v_scales.shape
    return head_dim // k_scales.shape[-1]


def reshape_and_cache_int4(key: torch.Tensor, value: torch.Tensor, slot_mapping: torch.Tensor,
                           k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                           v_scales: torch.Tensor, d_err: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """key/value [T, Hkv, D] fp16/bf16; caches uint8 [NB, bs, Hkv, D/2]; scales float32
    [Hkv, D/group_size] (the group size follows from their shape)."""
    T, H, D = key.shape
    assert key.stride(2) == 1 and key.stride(1) == D and value.stride(2) == 1 and value.stride(1) == D
    assert k_cache.dtype == torch.uint8 and k_cache.shape[-1] * 2 == D
    NB, bs = k_cache.shape[0], k_cache.shape[1]
    _check(lib.kv_reshape_and_cache_int4(
        _ptr(key), _ptr(value), dtype_code(key.dtype), key.stride(0), value.stride(0), T, H, D,
        _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), NB, bs, _ptr(k_scales), _ptr(v_scales),
        _int4_group(D, k_scales, v_scales), _ptr(d_err), _stream(stream)))


def paged_attention_decode_int4(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                block_table: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                                q_len: int, scale: float, k_scales: torch.Tensor, v_scales: torch.Tensor,
                                window: int = 0, num_workers: int = 0,
                                workspace: Optional[torch.Tensor] = None,
                                out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                                d_err: Optional[torch.Tensor] = None,
                                max_blocks_per_seq: Optional[int] = None, stream=None) -> torch.Tensor:
    """q [B*q_len, Hq, D]; caches uint8 [NB, bs, Hkv, D/2]; scales float32 [Hkv, D/group_size]."""
    TQ, Hq, D = q.shape
    NB, bs, Hkv, half = k_cache.shape
    B = seq_lens.shape[0]
    assert TQ == B * q_len and q.is_contiguous() and block_table.stride(1) == 1
    assert k_cache.dtype == torch.uint8 and half * 2 == D
    if out is None:
        out = torch.empty_like(q)
    need = paged_attention_workspace_size(B, q_len, Hq, Hkv, D, bs, KV_INT4, max_seq_len, window,
                                          num_workers)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.kv_paged_attention_decode_int4(
        _ptr(q), dtype_code(q.dtype), B, q_len, Hq, _ptr(k_cache), _ptr(v_cache), Hkv, D, bs, NB,
        _ptr(block_table), block_table.stride(0),
        block_table.shape[1] if max_blocks_per_seq is None else max_blocks_per_seq,
        _ptr(seq_lens), max_seq_len, float(scale), window, _ptr(k_scales), _ptr(v_scales),
        _int4_group(D, k_scales, v_scales), num_workers, _ptr(workspace), ws_bytes, _ptr(out),
        _ptr(lse_out), _ptr(d_err), _stream(stream)))
    return out


def selftest_bounded_wait(limit_us: int, d_err: torch.Tensor, d_waited_us: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """kv_selftest_bounded_wait: a kernel whose wait runs out after limit_us (sets
    KV_DERR_TIMEOUT in d_err, the waited microseconds in d_waited_us)."""
    assert d_err.dtype == torch.int32
    _check(lib.kv_selftest_bounded_wait(int(limit_us), _ptr(d_err), _ptr(d_waited_us), _stream(stream)))


def decode_step_int4(block_table: torch.Tensor, query_start_loc: torch.Tensor, positions: torch.Tensor,
                     key: torch.Tensor, value: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, q_len: int,
                     scale: float, k_scales: torch.Tensor, v_scales: torch.Tensor, window: int = 0,
                     num_workers: int = 0, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                     slot_mapping: Optional[torch.Tensor] = None, d_err: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """kv_decode_step_int4: slot mapping, INT4 cache write and attention of one decode step."""
    TQ, Hq, D = q.shape
    NB, bs, Hkv, half = k_cache.shape
    B = seq_lens.shape[0]
    assert TQ == B * q_len and q.is_contiguous() and block_table.stride(1) == 1
    assert key.stride(2) == 1 and key.stride(1) == D and value.stride(2) == 1 and value.stride(1) == D
    assert k_cache.dtype == torch.uint8 and half * 2 == D
    if out is None:
        out = torch.empty_like(q)
    need = paged_attention_workspace_size(B, q_len, Hq, Hkv, D, bs, KV_INT4, max_seq_len, window,
                                          num_workers)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(lib.kv_decode_step_int4(
        _ptr(block_table), block_table.stride(0), block_table.shape[1], _ptr(query_start_loc),
        _ptr(positions), _ptr(slot_mapping), _ptr(key), _ptr(value), key.stride(0), value.stride(0),
        _ptr(q), dtype_code(q.dtype), B, q_len, Hq, _ptr(k_cache), _ptr(v_cache), Hkv, D, bs, NB,
        _ptr(seq_lens), max_seq_len, float(scale), window, _ptr(k_scales), _ptr(v_scales),
        _int4_group(D, k_scales, v_scales), num_workers, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse_out), _ptr(d_err),
        _stream(stream)))
    return out


def decode_step(block_table: torch.Tensor, query_start_loc: torch.Tensor, positions: torch.Tensor,
                key: torch.Tensor, value: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                v_cache: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int, q_len: int,
                scale: float, window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
                num_workers: int = 0, workspace: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, lse_out: Optional[torch.Tensor] = None,
                slot_mapping: Optional[torch.Tensor] = None, d_err: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """kv_decode_step: slot mapping, cache write and attention of one decode step, one launch."""
    TQ, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    B = seq_lens.shape[0]
    assert TQ == B * q_len and q.is_contiguous() and block_table.stride(1) == 1
    assert key.stride(2) == 1 and key.stride(1) == D and value.stride(2) == 1 and value.stride(1) == D
    cdt = dtype_code(k_cache.dtype)
    if out is None:
        out = torch.empty_like(q)
    need = paged_attention_workspace_size(B, q_len, Hq, Hkv, D, bs, cdt, max_seq_len, window,
                                          num_workers)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(lib.kv_decode_step(
        _ptr(block_table), block_table.stride(0), block_table.shape[1], _ptr(query_start_loc),
        _ptr(positions), _ptr(slot_mapping), _ptr(key), _ptr(value), key.stride(0), value.stride(0),
        _ptr(q), dtype_code(q.dtype), B, q_len, Hq, _ptr(k_cache), _ptr(v_cache), cdt, Hkv, D, bs, NB,
        _ptr(seq_lens), max_seq_len, float(scale), window, float(k_scale), float(v_scale),
        num_workers, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
        _ptr(lse_out), _ptr(d_err), _stream(stream)))
    return out


def paged_attention_decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                   block_table: torch.Tensor, seq_lens: torch.Tensor,
                                   max_seq_len: int, q_len: int, scale: float, window: int = 0,
                                   k_scale: float = 1.0, v_scale: float = 1.0, num_workers: int = 0,
                                   out: Optional[torch.Tensor] = None,
                                   lse_out: Optional[torch.Tensor] = None,
                                   d_err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """kv_paged_attention_decode_noalloc: the same attention with the library's static scratch,
    for callers that cannot allocate device memory (pass ``out`` to allocate nothing here)."""
    TQ, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    B = seq_lens.shape[0]
    assert TQ == B * q_len and q.is_contiguous() and block_table.stride(1) == 1
    if out is None:
        out = torch.empty_like(q)
    _check(lib.kv_paged_attention_decode_noalloc(
        _ptr(q), dtype_code(q.dtype), B, q_len, Hq, _ptr(k_cache), _ptr(v_cache),
        dtype_code(k_cache.dtype), Hkv, D, bs, NB, _ptr(block_table), block_table.stride(0),
        block_table.shape[1], _ptr(seq_lens), max_seq_len, float(scale), window, float(k_scale),
        float(v_scale), num_workers, _ptr(out), _ptr(lse_out), _ptr(d_err), _stream(stream)))
    return out


def paged_attention_prefill(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_table: torch.Tensor, seq_lens: torch.Tensor,
                            query_start_loc: torch.Tensor, max_seq_len: int, max_query_len: int,
                            scale: float, window: int = 0, out: Optional[torch.Tensor] = None,
                            lse_out: Optional[torch.Tensor] = None, d_err: Optional[torch.Tensor] = None,
                            max_blocks_per_seq: Optional[int] = None, stream=None) -> torch.Tensor:
    """kv_paged_attention_prefill: q [T, Hq, D] (rows of sequence b are query_start_loc[b] ..
    query_start_loc[b+1]-1, its last positions); caches [NB, bs, Hkv, D]; block_table int32
    [B, W]; seq_lens int32 [B] (including the new rows)."""
    T, Hq, D = q.shape
    NB, bs, Hkv, _ = k_cache.shape
    B = seq_lens.shape[0]
    assert q.is_contiguous() and block_table.stride(1) == 1 and query_start_loc.numel() == B + 1
    if out is None:
        out = torch.empty_like(q)
    _check(lib.kv_paged_attention_prefill(
        _ptr(q), dtype_code(q.dtype), _ptr(query_start_loc), B, T, max_query_len, Hq, _ptr(k_cache),
        _ptr(v_cache), dtype_code(k_cache.dtype), Hkv, D, bs, NB, _ptr(block_table), block_table.stride(0),
        block_table.shape[1] if max_blocks_per_seq is None else max_blocks_per_seq, _ptr(seq_lens),
        max_seq_len, float(scale), window, _ptr(out), _ptr(lse_out), _ptr(d_err), _stream(stream)))
    return out


class BlockManager:
    """Host block manager (kv_bm_*): free pool, reference counts, block-table rows, prefix
    sharing, window release and staged table writes.  allocate / free / share_prefix return the
    C status (0 = OK, KV_ERR_OUT_OF_BLOCKS when the pool is short, KV_ERR_INVALID_ARG for a
    request the manager refuses) instead of raising, since a refusal is an ordinary scheduling
    outcome (kv_last_error() says why); the constructor, row and flush raise KVError."""

    def __init__(self, num_blocks: int, block_size: int, num_rows: int, max_blocks_per_row: int,
                 window: int = 0, zero_fill: bool = True):
        h = ctypes.c_void_p()
        _check(lib.kv_bm_create(num_blocks, block_size, num_rows, max_blocks_per_row, window,
                                int(bool(zero_fill)), ctypes.byref(h)))
        self._h = h
        self.num_blocks, self.block_size = num_blocks, block_size
        self.num_rows, self.max_blocks_per_row, self.window = num_rows, max_blocks_per_row, window

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            lib.kv_bm_destroy(h)
            self._h = None

    def allocate(self, row: int, num_new_tokens: int) -> int:
        return lib.kv_bm_allocate(self._h, row, num_new_tokens)

    def allocate_batch(self, rows, num_new_tokens):
        """kv_bm_allocate_batch over int32 host arrays; returns the per-row statuses."""
        import numpy as np
        r = np.ascontiguousarray(rows, dtype=np.int32)
        n = np.ascontiguousarray(num_new_tokens, dtype=np.int32)
        assert r.shape == n.shape
        st = np.empty(r.shape, dtype=np.int32)
        lib.kv_bm_allocate_batch(self._h, r.ctypes.data, n.ctypes.data, r.size, st.ctypes.data)
        return st

    def free(self, row: int) -> int:
        return lib.kv_bm_free(self._h, row)

    def share_prefix(self, dst_row: int, src_row: int, num_blocks: int) -> int:
        return lib.kv_bm_share_prefix(self._h, dst_row, src_row, num_blocks)

    def num_free_blocks(self) -> int:
        return lib.kv_bm_num_free_blocks(self._h)

    def ref_count(self, block: int) -> int:
        return lib.kv_bm_ref_count(self._h, block)

    def row(self, row: int):
        """(tokens, [physical id per logical block, -1 = released])."""
        import numpy as np
        t, n = ctypes.c_int32(), ctypes.c_int32()
        _check(lib.kv_bm_row(self._h, row, ctypes.byref(t), ctypes.byref(n), None, 0))
        out = np.empty(n.value, dtype=np.int32)
        _check(lib.kv_bm_row(self._h, row, ctypes.byref(t), ctypes.byref(n), out.ctypes.data, out.size))
        return t.value, out.tolist()

    def pending(self):
        u, z = ctypes.c_int32(), ctypes.c_int32()
        _check(lib.kv_bm_pending(self._h, ctypes.byref(u), ctypes.byref(z)))
        return u.value, z.value

    def flush(self, updates=None, zero_ids=None):
        """kv_bm_flush into host int32 arrays (numpy, or pinned torch tensors for an asynchronous
        copy; allocated here when None).  Returns (updates [n, 3], zero_ids [m]) views."""
        import numpy as np
        nu, nz = self.pending()
        if updates is None:
            updates = np.empty((max(nu, 1), 3), dtype=np.int32)
        if zero_ids is None:
            zero_ids = np.empty(max(nz, 1), dtype=np.int32)
        up_ptr = updates.data_ptr() if isinstance(updates, torch.Tensor) else updates.ctypes.data
        z_ptr = zero_ids.data_ptr() if isinstance(zero_ids, torch.Tensor) else zero_ids.ctypes.data
        cap_u = updates.numel() // 3 if isinstance(updates, torch.Tensor) else updates.size // 3
        cap_z = zero_ids.numel() if isinstance(zero_ids, torch.Tensor) else zero_ids.size
        a, b = ctypes.c_int32(), ctypes.c_int32()
        _check(lib.kv_bm_flush(self._h, up_ptr, cap_u, ctypes.byref(a), z_ptr, cap_z, ctypes.byref(b)))
        return updates.reshape(-1)[:3 * a.value].reshape(-1, 3), zero_ids.reshape(-1)[:b.value]


def apply_block_updates(updates: torch.Tensor, block_table: torch.Tensor, zero_ids: torch.Tensor,
                        caches, num_blocks: int, d_err: Optional[torch.Tensor] = None,
                        max_blocks_per_row: Optional[int] = None, stream=None) -> None:
    """kv_apply_block_updates: device int32 updates [n, 3] into block_table [rows, stride];
    zero every cache's block of each id in zero_ids (device int32 [m]).  caches: device tensors
    whose first axis is the block id (e.g. [NB, bs, Hkv, D] K and V of each layer)."""
    assert updates.dtype == torch.int32 and zero_ids.dtype == torch.int32
    assert block_table.dtype == torch.int32 and block_table.stride(1) == 1
    n_up = updates.numel() // 3
    n_zero = zero_ids.numel()
    ptrs = (ctypes.c_void_p * max(len(caches), 1))(*[c.data_ptr() for c in caches])
    block_bytes = 0
    if caches:
        c0 = caches[0]
        block_bytes = c0[0].numel() * c0.element_size()
        for c in caches:
            assert c.is_contiguous() and c.shape[0] == num_blocks
            assert c[0].numel() * c.element_size() == block_bytes
    _check(lib.kv_apply_block_updates(
        _ptr(updates) if n_up else None, n_up, _ptr(block_table), block_table.stride(0),
        block_table.shape[0], block_table.shape[1] if max_blocks_per_row is None else max_blocks_per_row,
        _ptr(zero_ids) if n_zero else None, n_zero, ptrs, len(caches), block_bytes, num_blocks,
        _ptr(d_err), _stream(stream)))


# ---------------------------------------------------------------- a serving step (pagedkv_step.h)
#
# These calls are short next to Python, so their checks are written out in plain expressions (a
# helper call or a message built in advance costs more than the check).
# With stream=, what a call makes (outputs left to it, the workspace) is memory of that stream.

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_i32, _i64, _f32 = torch.int32, torch.int64, torch.float32
_code_of = {torch.float16: KV_F16, torch.bfloat16: KV_BF16, torch.uint8: KV_FP8_E4M3,
            torch.float8_e4m3fn: KV_FP8_E4M3}


def _refuse(what: str) -> None:
    raise KVError(KV_ERR_INVALID_ARG, what)


_DEVICES = "every tensor must be on one CUDA device"


def _on(stream, dev: int):
    """The context of a call on a given stream: what the call allocates is then of that stream's memory,
    so that freeing it hands it to no other stream while the call still runs."""
    if stream.device.index != dev:
        _refuse("the stream must be of the tensors' device")
    return torch.cuda.stream(stream)


def _table(t: torch.Tensor, rows: int, max_blocks: Optional[int]) -> Tuple[int, int]:
    """Row stride and width of a block table [B, W]."""
    shape = t.shape
    if t.dtype is not _i32 or len(shape) != 2 or shape[0] != rows:
        _refuse("block_table: int32 [B, W]")
    width = shape[1]
    stride, step = t.stride()
    if step != 1 and rows and width > 1:
        _refuse("block_table: rows in one piece")
    if rows < 2:
        stride = width
    if max_blocks is None:
        return stride, width
    if not 0 <= max_blocks <= width:
        _refuse("max_blocks_per_seq is past the table's rows")
    return stride, max_blocks


def _error_word(d_err: torch.Tensor, dev: int) -> int:
    if d_err.dtype is not _i32 or d_err.numel() < 1 or d_err.get_device() != dev:
        _refuse("d_err: int32 [1] on the same device")
    return d_err.data_ptr()


class Batch:
    """The metadata of a step, as kv_build_batch fills it (made by batch_buffers or build_batch): views
    of one allocation.  tree_mask is None without parents."""
    FIELDS = ("query_start_loc", "seq_lens", "positions", "slot_mapping", "held_blocks", "free_next", "tree_mask")
    __slots__ = ("_base", "_starts", "_views", "_sizes", "_at", "_pointers")

    def __init__(self, num_seqs: int, num_tokens: int, trees: bool, device):
        if num_tokens < 0:
            _refuse("num_tokens must not be negative")
        words = (num_seqs + 1, num_seqs, num_tokens, 2 * num_tokens, num_seqs, 1, 2 * num_tokens if trees else 0)
        starts, end = [], 0  # of each field, in int32 words, on 16-byte boundaries
        for n in words:
            starts.append(end)
            end += (n + 3) & ~3
        self._base = base = torch.empty(end, dtype=_i32, device=device)
        views = [base[at:at + n] for at, n in zip(starts, words)]
        views[3] = views[3].view(_i64)
        views[6] = views[6].view(_i64) if trees else None
        self._views = tuple(views)
        self._sizes = (num_seqs, num_tokens, trees, base.get_device())
        self._starts = tuple(starts if trees else starts[:6] + [None])
        self._at = None  # of which base _pointers are

    query_start_loc = property(lambda self: self._views[0])
    seq_lens = property(lambda self: self._views[1])
    positions = property(lambda self: self._views[2])
    slot_mapping = property(lambda self: self._views[3])
    held_blocks = property(lambda self: self._views[4])
    free_next = property(lambda self: self._views[5])
    tree_mask = property(lambda self: self._views[6])

    def _asdict(self) -> dict:
        return dict(zip(self.FIELDS, self._views))

    def _place(self, base: int) -> tuple:
        """The fields' addresses for kv_build_batch, once the allocation is at `base`."""
        if not base:
            _refuse("out: its memory has been released")
        self._at = base
        self._pointers = tuple(None if at is None else base + 4 * at for at in self._starts)
        return self._pointers


def batch_buffers(num_seqs: int, num_tokens: int, trees: bool = False, device="cuda") -> Batch:
    """Buffers for build_batch's ``out`` (a loop that chains steps keeps two and swaps them)."""
    return Batch(num_seqs, num_tokens, bool(trees), device)


def build_batch(context_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                free_blocks: torch.Tensor, num_tokens: int, block_size: int, num_blocks: int,
                held_blocks: Optional[torch.Tensor] = None, parents: Optional[torch.Tensor] = None,
                free_start: Optional[torch.Tensor] = None, out: Optional[Batch] = None,
                d_err: Optional[torch.Tensor] = None, max_blocks_per_seq: Optional[int] = None,
                stream=None) -> Batch:
    """kv_build_batch: context_lens, new_lens and held_blocks int32 [B]; block_table int32 [B, W],
    updated in place; free_blocks int32 [F]; parents int32 [num_tokens] for drafted trees;
    free_start int32 [1].  The masks are int64 words (bit j = token j of the request's tree)."""
    dev = context_lens.get_device()
    if dev < 0 or new_lens.get_device() != dev or block_table.get_device() != dev or free_blocks.get_device() != dev:
        _refuse(_DEVICES)
    if stream is not None or dev != _current_device():
        with torch.cuda.device(dev) if stream is None else _on(stream, dev):
            return build_batch(context_lens, new_lens, block_table, free_blocks, num_tokens, block_size, num_blocks,
                               held_blocks, parents, free_start, out, d_err, max_blocks_per_seq)
    B = context_lens.numel()
    if context_lens.dtype is not _i32 or not context_lens.is_contiguous():
        _refuse("context_lens: contiguous int32 [B]")
    if new_lens.dtype is not _i32 or not new_lens.is_contiguous() or new_lens.numel() != B:
        _refuse("new_lens: contiguous int32 [B]")
    if free_blocks.dtype is not _i32 or not free_blocks.is_contiguous():
        _refuse("free_blocks: contiguous int32")
    held = par = start = err = None
    if held_blocks is not None:
        if held_blocks.dtype is not _i32 or not held_blocks.is_contiguous() or held_blocks.numel() != B or \
                held_blocks.get_device() != dev:
            _refuse("held_blocks: contiguous int32 [B] on the same device")
        held = held_blocks.data_ptr()
    if parents is not None:
        if parents.dtype is not _i32 or not parents.is_contiguous() or parents.numel() != num_tokens or \
                parents.get_device() != dev:
            _refuse("parents: contiguous int32 [num_tokens] on the same device")
        par = parents.data_ptr()
    if free_start is not None:
        if free_start.dtype is not _i32 or free_start.numel() != 1 or free_start.get_device() != dev:
            _refuse("free_start: int32 [1] on the same device")
        start = free_start.data_ptr()
    if d_err is not None:
        err = _error_word(d_err, dev)
    bt_stride, width = _table(block_table, B, max_blocks_per_seq)
    if out is None:
        out = Batch(B, num_tokens, parents is not None, context_lens.device)
    elif out._sizes != (B, num_tokens, parents is not None, dev):
        _refuse("out: batch_buffers of these sizes, with trees exactly when parents are given, on this device")
    at = out._base.data_ptr()
    qsl, lens, pos, slots, held_out, free_next, mask = out._pointers if at == out._at else out._place(at)
    status = lib.kv_build_batch(
        context_lens.data_ptr(), new_lens.data_ptr(), held, par, B, num_tokens, block_table.data_ptr(),
        bt_stride, width, block_size, num_blocks, free_blocks.data_ptr(),
        free_blocks.numel(), start, qsl, lens, pos, slots, mask, held_out, free_next, err,
        _raw_stream(dev))
    if status:
        _check(status)
    return out


def _odd_rows(t: torch.Tensor, what: str) -> None:
    """A [T, heads, D] tensor whose strides are not (any, D, 1): an error if they mean something."""
    T, H, _ = t.shape
    if T and (t.stride(2) != 1 or H > 1):
        _refuse(f"{what}: each token's heads in one piece")


def _norm_rope(q, key, value, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight, eps,
               interleaved, k_scale, v_scale, q_out, k_out, d_err):
    dev, dt = q.get_device(), q.dtype
    qshape, kshape = q.shape, key.shape
    if dev < 0 or len(qshape) != 3 or len(kshape) != 3:
        _refuse("q and key: [T, heads, D]; " + _DEVICES)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _norm_rope(q, key, value, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight, eps,
                              interleaved, k_scale, v_scale, q_out, k_out, d_err)
    T, Hq, D = qshape
    if kshape[0] != T or kshape[2] != D:
        _refuse("q and key differ in tokens or head size")
    Hkv = kshape[1]
    # token strides (that of a single token means nothing; it only has to hold the row)
    qs, s1, s2 = q.stride()
    if s2 != 1 or s1 != D:
        _odd_rows(q, "q")
    ks, s1, s2 = key.stride()
    if key.dtype is not dt or key.get_device() != dev:
        _refuse(f"key: {dt} on the same device")
    if s2 != 1 or s1 != D:
        _odd_rows(key, "key")
    if q_out.dtype is not dt or q_out.shape != qshape or q_out.get_device() != dev:
        _refuse(f"q_out: {dt} {list(qshape)} on the same device")
    qos, s1, s2 = q_out.stride()
    if s2 != 1 or s1 != D:
        _odd_rows(q_out, "q_out")
    one_k = -(-Hkv * D // 8) * 8
    if T < 2:
        qs = qos = -(-Hq * D // 8) * 8
        ks = one_k
    pos = cs = wq = wk = kout = err = None
    kos = max_pos = rot = 0
    if k_out is not None:
        if k_out.dtype is not dt or k_out.shape != kshape or k_out.get_device() != dev:
            _refuse(f"k_out: {dt} {list(kshape)} on the same device")
        kos, s1, s2 = k_out.stride()
        if s2 != 1 or s1 != D:
            _odd_rows(k_out, "k_out")
        if T < 2:
            kos = one_k
        kout = k_out.data_ptr()
    if q_weight is not None:
        if q_weight.dtype is not dt or q_weight.numel() != D or not q_weight.is_contiguous() or q_weight.get_device() != dev:
            _refuse(f"q_weight: contiguous {dt} [{D}] on the same device")
        wq = q_weight.data_ptr()
    if k_weight is not None:
        if k_weight.dtype is not dt or k_weight.numel() != D or not k_weight.is_contiguous() or k_weight.get_device() != dev:
            _refuse(f"k_weight: contiguous {dt} [{D}] on the same device")
        wk = k_weight.data_ptr()
    if positions is not None:
        if positions.dtype is not _i32 or positions.numel() != T or not positions.is_contiguous() or \
                positions.get_device() != dev:
            _refuse("positions: contiguous int32 [T] on the same device")
        pos = positions.data_ptr()
    if cos_sin is not None:
        cs_shape = cos_sin.shape
        if cos_sin.dtype is not _f32 or len(cs_shape) != 2 or not cos_sin.is_contiguous() or cos_sin.get_device() != dev:
            _refuse("cos_sin: contiguous float32 [max_position, rotary_dim] on the same device")
        max_pos, rot = cs_shape
        cs = cos_sin.data_ptr()
    if d_err is not None:
        err = _error_word(d_err, dev)
    code = _code_of.get(dt, -1)
    vp = slots = kc = vc = None
    cache_code, NB, bs, vs = code, 0, 1, 0
    if slot_mapping is not None:
        if slot_mapping.dtype is not _i64 or slot_mapping.numel() != T or not slot_mapping.is_contiguous() or \
                slot_mapping.get_device() != dev:
            _refuse("slot_mapping: contiguous int64 [T] on the same device")
        if value.dtype is not dt or value.shape != kshape or value.get_device() != dev:
            _refuse(f"value: {dt} {list(kshape)} on the same device")
        vs, s1, s2 = value.stride()
        if s2 != 1 or s1 != D:
            _odd_rows(value, "value")
        if T < 2:
            vs = one_k
        cshape, cdt = k_cache.shape, k_cache.dtype
        if len(cshape) != 4 or cshape[2] != Hkv or cshape[3] != D or v_cache.shape != cshape or \
                v_cache.dtype is not cdt or not k_cache.is_contiguous() or not v_cache.is_contiguous() or \
                k_cache.get_device() != dev or v_cache.get_device() != dev:
            _refuse("caches: two contiguous [blocks, block_size, heads, D] of one type, heads and D those of key, "
                    "on the same device")
        NB, bs = cshape[0], cshape[1]
        if cdt is not dt:
            cache_code = _code_of.get(cdt, -1)
        vp, slots, kc, vc = value.data_ptr(), slot_mapping.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
        if not slots:  # no tokens: nothing to write (and no slots to say so)
            vp = kc = vc = None
    status = lib.kv_qk_norm_rope(
        q.data_ptr(), key.data_ptr(), vp, code, qs, ks, vs, T, Hq, Hkv, D, wq, wk, eps, pos, cs, max_pos, rot,
        1 if interleaved else 0, q_out.data_ptr(), qos, kout, kos, slots, kc, vc, cache_code, NB, bs, k_scale, v_scale,
        err, _raw_stream(dev))
    if status:
        _check(status)


def qk_norm_rope(q: torch.Tensor, key: torch.Tensor, positions: Optional[torch.Tensor],
                 cos_sin: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 d_err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """kv_qk_norm_rope without the cache: q [T, Hq, D] and key [T, Hkv, D] (views of one
    projection will do; token stride = stride(0)), positions int32 [T], cos_sin float32
    [max_position, rotary_dim].  q_out and k_out may be q and key."""
    if stream is not None:
        with _on(stream, q.get_device()):
            return qk_norm_rope(q, key, positions, cos_sin, q_weight, k_weight, eps, interleaved, q_out, k_out, d_err)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(key.shape, dtype=key.dtype, device=key.device)
    _norm_rope(q, key, None, positions, cos_sin, None, None, None, q_weight, k_weight, eps, interleaved, 1.0, 1.0,
               q_out, k_out, d_err)
    return q_out, k_out


def qk_norm_rope_and_cache(q: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                           positions: Optional[torch.Tensor], cos_sin: Optional[torch.Tensor],
                           slot_mapping: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                           q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                           eps: float = 1e-6, interleaved: bool = False, k_scale: float = 1.0,
                           v_scale: float = 1.0, q_out: Optional[torch.Tensor] = None,
                           k_out: Optional[torch.Tensor] = None, d_err: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """kv_qk_norm_rope with the write of the turned keys and of the values into their slots;
    returns the queries (and fills k_out when it is given)."""
    if stream is not None:
        with _on(stream, q.get_device()):
            return qk_norm_rope_and_cache(q, key, value, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight,
                                          k_weight, eps, interleaved, k_scale, v_scale, q_out, k_out, d_err)
    if slot_mapping is None or value is None or k_cache is None or v_cache is None:
        _refuse("value, slot_mapping and both caches are needed")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _norm_rope(q, key, value, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight, eps, interleaved,
               k_scale, v_scale, q_out, k_out, d_err)
    return q_out


def paged_attention_tree_workspace_size(num_seqs: int, max_query_len: int, num_q_heads: int, num_kv_heads: int,
                                        head_dim: int, num_workers: int = 0) -> int:
    n = lib.kv_paged_attention_tree_workspace_size(num_seqs, max_query_len, num_q_heads, num_kv_heads, head_dim,
                                                   num_workers)
    if n == SIZE_MAX:
        raise KVError(KV_ERR_UNSUPPORTED, lib.kv_last_error().decode() or "invalid or unsupported sizes")
    return int(n)


def paged_attention_tree(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, query_start_loc: torch.Tensor, tree_mask: torch.Tensor,
                         max_seq_len: int, max_query_len: int, scale: float, window: int = 0, num_workers: int = 0,
                         workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         lse_out: Optional[torch.Tensor] = None, d_err: Optional[torch.Tensor] = None,
                         max_blocks_per_seq: Optional[int] = None, stream=None) -> torch.Tensor:
    """kv_paged_attention_tree: q [T, Hq, D] (the drafted tokens of sequence b are rows
    query_start_loc[b] .. query_start_loc[b+1]-1); caches [NB, bs, Hkv, D]; block_table int32 [B, W];
    seq_lens int32 [B] (including the drafted tokens); tree_mask int64 [T].  A workspace that is
    given must hold paged_attention_tree_workspace_size(...) bytes.  A max_query_len of 0 declares an
    empty batch, of which nothing is looked at or written."""
    dev, dt = q.get_device(), q.dtype
    if dev < 0 or q.dim() != 3 or not q.is_contiguous():
        _refuse("q: contiguous [T, heads, D]; " + _DEVICES)
    if stream is not None or dev != _current_device():
        with torch.cuda.device(dev) if stream is None else _on(stream, dev):
            return paged_attention_tree(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, tree_mask, max_seq_len,
                                        max_query_len, scale, window, num_workers, workspace, out, lse_out, d_err,
                                        max_blocks_per_seq)
    T, Hq, D = q.shape
    B = seq_lens.numel()
    cshape, cdt = k_cache.shape, k_cache.dtype
    if len(cshape) != 4 or cshape[3] != D or v_cache.shape != cshape or v_cache.dtype is not cdt or \
            not k_cache.is_contiguous() or not v_cache.is_contiguous() or k_cache.get_device() != dev or \
            v_cache.get_device() != dev:
        _refuse("caches: two contiguous [blocks, block_size, heads, D] of one type, D that of q, on the same device")
    NB, bs, Hkv, _ = cshape
    if seq_lens.dtype is not _i32 or not seq_lens.is_contiguous() or seq_lens.get_device() != dev:
        _refuse("seq_lens: contiguous int32 [B] on the same device")
    if query_start_loc.dtype is not _i32 or not query_start_loc.is_contiguous() or query_start_loc.numel() != B + 1 or \
            query_start_loc.get_device() != dev:
        _refuse("query_start_loc: contiguous int32 [B + 1] on the same device")
    if tree_mask.dtype is not _i64 or not tree_mask.is_contiguous() or tree_mask.numel() != T or \
            tree_mask.get_device() != dev:
        _refuse("tree_mask: contiguous int64 [T] on the same device")
    if block_table.get_device() != dev:
        _refuse(_DEVICES)
    bt_stride, width = _table(block_table, B, max_blocks_per_seq)
    err = lse = None
    if d_err is not None:
        err = _error_word(d_err, dev)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype is not dt or not out.is_contiguous() or out.get_device() != dev:
        _refuse("out: like q")
    if lse_out is not None:
        if lse_out.dtype is not _f32 or lse_out.shape != (T, Hq) or not lse_out.is_contiguous() or \
                lse_out.get_device() != dev:
            _refuse("lse_out: contiguous float32 [T, heads] on the same device")
        lse = lse_out.data_ptr()
    if workspace is None:
        workspace = torch.empty(paged_attention_tree_workspace_size(B, max_query_len, Hq, Hkv, D, num_workers),
                                dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        _refuse("workspace: contiguous, on the same device")
    status = lib.kv_paged_attention_tree(
        q.data_ptr(), _code_of.get(dt, -1), query_start_loc.data_ptr(), B, T, max_query_len, Hq, k_cache.data_ptr(),
        v_cache.data_ptr(), _code_of.get(cdt, -1), Hkv, D, bs, NB, block_table.data_ptr(),
        bt_stride, width, seq_lens.data_ptr(), max_seq_len, scale, window,
        tree_mask.data_ptr(), num_workers, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        out.data_ptr(), lse, err, _raw_stream(dev))
    if status:
        _check(status)
    return out
