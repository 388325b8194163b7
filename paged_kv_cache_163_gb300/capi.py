"""ctypes binding of libpkv.so: the C ABI's calls under the same names.

Argument marshalling only: host arrays become pointers, torch tensors give
their device pointers, shapes and dtypes are read off the tensors.  Every
non-OK status raises ``PkvError`` (``NoBlocksError`` for PKV_ERR_NO_BLOCKS)
with the library's one-line reason.  The library is loaded on first use; if
it has not been built the first call raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_F16, PKV_BF16, PKV_FP8_E4M3, PKV_F32, PKV_FP8_E5M2, PKV_INT8 = 0, 1, 2, 3, 4, 5
PKV_FP8_E4M3_INT4 = 6
DTYPE_NAMES = {"f16": PKV_F16, "bf16": PKV_BF16, "fp8_e4m3": PKV_FP8_E4M3, "f32": PKV_F32,
               "fp8_e5m2": PKV_FP8_E5M2, "int8": PKV_INT8, "fp8_e4m3_int4": PKV_FP8_E4M3_INT4}
# cache types stored as one-byte codes (uint8 tensors) plus fp32 scales
ONE_BYTE_CACHES = ("fp8_e4m3", "fp8_e5m2", "int8")
# cache types with k_scale / v_scale: the one-byte ones, and K FP8 E4M3 + V INT4
# (uint8 tensors; the V rows hold head_dim / 2 bytes)
SCALED_CACHES = ONE_BYTE_CACHES + ("fp8_e4m3_int4",)


def v_row_elems(cache_dtype: str, head_dim: int) -> int:
    """Last dimension of a V cache tensor: head_dim, or head_dim / 2 bytes for 4-bit V."""
    return head_dim // 2 if cache_dtype == "fp8_e4m3_int4" else head_dim
BLOCK_SIZE = 16
MAX_SEQS_PER_CALL = 1024
DEVERR_BAD_SLOT, DEVERR_BAD_BLOCK, DEVERR_BAD_CONTEXT_LEN, DEVERR_WAIT_TIMEOUT = 1, 2, 4, 8
DEVERR_BAD_POSITION = 16

STATUS = {0: "PKV_OK", -1: "PKV_ERR_INVALID", -2: "PKV_ERR_NO_BLOCKS", -3: "PKV_ERR_CUDA",
          -4: "PKV_ERR_UNSUPPORTED", -5: "PKV_ERR_DEVICE_CHECK", -6: "PKV_ERR_WORKSPACE"}


class PkvError(RuntimeError):
    def __init__(self, status: int, where: str, reason: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {reason}")
        self.status = status


class NoBlocksError(PkvError):
    pass


_lib = None


class CopySegment(C.Structure):
    """pkv_copy_segment."""
    _fields_ = [("dst", C.c_void_p), ("src", C.c_void_p), ("bytes", C.c_int64)]


MAX_COPY_SEGMENTS = 8


class PoolDesc(C.Structure):
    """pkv_pool_desc: per-layer pools as base pointers plus byte strides."""
    _fields_ = [("num_layers", C.c_int32), ("num_blocks", C.c_int32), ("num_kv_heads", C.c_int32),
                ("num_q_heads", C.c_int32), ("head_dim", C.c_int32), ("q_dtype", C.c_int),
                ("cache_dtype", C.c_int), ("k_cache", C.c_void_p), ("v_cache", C.c_void_p),
                ("cache_layer_stride", C.c_int64), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("scale_layer_stride", C.c_int64), ("block_size", C.c_int32),
                ("v_cache_layer_stride", C.c_int64)]


_i32p = C.POINTER(C.c_int32)
_i64p = C.POINTER(C.c_int64)
_vp = C.c_void_p

# name: (restype, argtypes)
_PROTOS = {
    "pkv_bm_create": (C.c_int, [C.c_int32, C.c_int32, _i32p, C.POINTER(_vp)]),
    "pkv_bm_destroy": (None, [_vp]),
    "kv_block_alloc": (C.c_int, [_vp, _i32p]),
    "kv_block_free": (C.c_int, [_vp, C.c_int32]),
    "pkv_seq_create": (C.c_int, [_vp, C.c_int64]),
    "pkv_seq_fork": (C.c_int, [_vp, C.c_int64, C.c_int64]),
    "pkv_seq_free": (C.c_int, [_vp, C.c_int64]),
    "pkv_seq_append_slots": (C.c_int, [_vp, _i64p, C.c_int32, _i32p, _i32p, _i32p, _i32p]),
    "pkv_build_block_tables": (C.c_int, [_vp, _i64p, C.c_int32, C.c_int32, _i32p, _i32p]),
    "pkv_bm_num_free": (C.c_int32, [_vp]),
    "pkv_bm_num_blocks": (C.c_int32, [_vp]),
    "pkv_bm_block_size": (C.c_int32, [_vp]),
    "pkv_bm_free_list": (C.c_int, [_vp, _i32p, C.c_int32, _i32p]),
    "pkv_bm_refcount": (C.c_int, [_vp, C.c_int32, _i32p]),
    "pkv_seq_len": (C.c_int, [_vp, C.c_int64, _i32p]),
    "pkv_kv_bytes": (C.c_int64, [C.c_int32, C.c_int32, C.c_int32, C.c_int64, C.c_int]),
    "pkv_pool_blocks": (C.c_int64, [C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int, C.c_int32]),
    "paged_kv_copy_blocks": (C.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, C.c_int32, C.c_int32, C.c_int32,
                                       C.c_int, C.c_int32, C.c_int32, _vp, _vp]),
    "paged_kv_append": (C.c_int, [_vp, _vp, C.c_int, C.c_int32, C.c_int32, C.c_int32, _vp, _vp, _vp,
                                  C.c_int, _vp, _vp, C.c_int32, C.c_int32, _vp, _vp]),
    "paged_attention_workspace_bytes": (C.c_int, [C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int,
                                                  C.c_int, C.POINTER(C.c_size_t)]),
    "paged_attention_decode": (C.c_int, [_vp, C.c_int, _vp, C.c_int, _vp, _vp, C.c_int, _vp, _vp, _vp, C.c_int32,
                                         _vp, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                         C.c_int32, C.c_int32, C.c_float, _vp, C.c_size_t, _vp, _vp]),
    # out, out_dtype, q, q_dtype, k_new, v_new, k_cache, v_cache, cache_dtype, k_scale, v_scale, tables,
    # max_blocks, lens, max_len, num_seqs, hq, hkv, d, num_blocks, block_size, scale, workspace, bytes,
    # d_error, stream
    "paged_attention_decode_append": (C.c_int, [_vp, C.c_int, _vp, C.c_int, _vp, _vp, _vp, _vp, C.c_int, _vp, _vp,
                                                _vp, C.c_int32, _vp, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                                C.c_int32, C.c_int32, C.c_int32, C.c_float, _vp, C.c_size_t, _vp,
                                                _vp]),
    "paged_attention_decode_static": (C.c_int, [_vp, C.c_int, _vp, C.c_int, _vp, _vp, C.c_int, _vp, _vp, _vp,
                                                C.c_int32, _vp, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                                C.c_int32, C.c_int32, C.c_int32, C.c_float, _vp, _vp]),
    "pkv_rope_table": (C.c_int, [_vp, C.c_int32, C.c_int32, C.c_double, C.c_int, C.c_double, C.c_int32, C.c_double,
                                 C.c_double, C.c_double, _vp]),
    # q_out, q, k, v, in_dtype, q_stride, k_stride, v_stride, tokens, hq, hkv, d, positions, slots, cos_sin,
    # max_positions, rot_dim, interleaved, k_cache, v_cache, cache_dtype, k_scale, v_scale, num_blocks,
    # block_size, d_error, stream
    "paged_kv_append_rope": (C.c_int, [_vp, _vp, _vp, _vp, C.c_int, C.c_int64, C.c_int64, C.c_int64, C.c_int32,
                                       C.c_int32, C.c_int32, C.c_int32, _vp, _vp, _vp, C.c_int32, C.c_int32,
                                       C.c_int32, _vp, _vp, C.c_int, _vp, _vp, C.c_int32, C.c_int32, _vp, _vp]),
    # k_out, v_out, out_dtype, num_rows, k_cache, v_cache, cache_dtype, k_scale, v_scale, tables, max_blocks,
    # token_starts, context_lens, out_starts, num_seqs, hkv, d, num_blocks, block_size, d_error, stream
    "paged_kv_gather": (C.c_int, [_vp, _vp, C.c_int, C.c_int32, _vp, _vp, C.c_int, _vp, _vp, _vp, C.c_int32, _vp,
                                  _vp, _vp, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32, _vp, _vp]),
    "paged_attention_extend_workspace_bytes": (C.c_int, [C.c_int32, C.POINTER(C.c_size_t)]),
    # out, out_dtype, q, q_dtype, num_queries, k_cache, v_cache, cache_dtype, k_scale, v_scale, tables, max_blocks,
    # context_lens, query_starts, num_seqs, hq, hkv, d, num_blocks, block_size, scale, window, sinks, workspace,
    # bytes, d_error, stream
    "paged_attention_extend": (C.c_int, [_vp, C.c_int, _vp, C.c_int, C.c_int32, _vp, _vp, C.c_int, _vp, _vp, _vp,
                                         C.c_int32, _vp, _vp, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                         C.c_int32, C.c_float, C.c_int32, C.c_int32, _vp, C.c_size_t, _vp, _vp]),
    "pkv_block_hash": (C.c_uint64, [C.c_uint64, _i32p, C.c_uint64]),
    "pkv_bm_enable_prefix_cache": (C.c_int, [_vp, C.c_uint64]),
    "pkv_seq_admit": (C.c_int, [_vp, C.c_int64, _i32p, C.c_int32, _i32p]),
    "pkv_seq_commit_prefix": (C.c_int, [_vp, C.c_int64, _i32p, C.c_int32, _i32p]),
    "pkv_prefix_cache_stats": (C.c_int, [_vp, C.c_void_p]),
    "pkv_stepper_host_bytes": (C.c_size_t, [C.c_int32, C.c_int32]),
    "pkv_stepper_device_bytes": (C.c_size_t, [C.c_int32, C.c_int32]),
    "pkv_stepper_create": (C.c_int, [C.POINTER(PoolDesc), C.c_int32, C.c_int32, _vp, C.c_size_t, _vp, C.c_size_t,
                                     _vp, C.c_size_t, C.POINTER(_vp)]),
    "pkv_stepper_destroy": (None, [_vp]),
    "pkv_stepper_use_graphs": (C.c_int, [_vp, C.c_int32]),
    "pkv_stepper_use_cascade": (C.c_int, [_vp, C.c_int32]),
    "pkv_stepper_cascade_count": (C.c_int64, [_vp]),
    "pkv_stepper_graph_stats": (C.c_int, [_vp, _i64p, _i64p]),
    # pointer arguments as addresses (ints): the per-step call marshals no ctypes pointer objects
    "pkv_stepper_step": (C.c_int, [_vp, _vp, _vp, C.c_int32, _vp, _vp, C.c_int64, _vp, C.c_int64, _vp, C.c_int,
                                   C.c_int64, C.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pkv_read_device_error": (C.c_int, [_vp, _i32p, C.c_int32, _vp]),
    "pkv_launch_count": (C.c_int64, []),
    "pkv_copy_segments": (C.c_int, [C.c_void_p, C.c_int32, _vp]),
    "pkv_stepper_copy_inputs": (C.c_int, [_vp, C.c_void_p, C.c_int32]),
    "pkv_set_decode_kernel": (C.c_int, [C.c_int]),
    "pkv_set_prefix_kernel": (C.c_int, [C.c_int, C.c_int32]),
    "pkv_get_prefix_kernel": (C.c_int, []),
    "pkv_get_decode_kernel": (C.c_int, []),
    "pkv_status_string": (C.c_char_p, [C.c_int]),
    "pkv_last_error": (C.c_char_p, []),
}


def load(path: str = LIB_PATH):
    """Load libpkv.so once; raises if it is missing (build it first)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m paged_kv_cache_163_gb300.build` (no fallback path exists)")
        lib = C.CDLL(path)
        for name, (res, args) in _PROTOS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def declared_symbols():
    return list(_PROTOS)


def _check(status: int, where: str):
    if status != 0:
        reason = load().pkv_last_error().decode(errors="replace")
        cls = NoBlocksError if status == -2 else PkvError
        raise cls(status, where, reason)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int32)


def _i64(a) -> np.ndarray:
    return np.ascontiguousarray(a, dtype=np.int64)


def _ptr(a: np.ndarray, ctype):
    return a.ctypes.data_as(C.POINTER(ctype))


# ---- host block manager -------------------------------------------------------
def pkv_bm_create(num_blocks: int, block_size: int = BLOCK_SIZE, alloc_order=None):
    h = _vp()
    order = None if alloc_order is None else _i32(alloc_order)
    if order is not None and len(order) != num_blocks:
        raise PkvError(-1, "pkv_bm_create", "alloc_order must have num_blocks entries")
    _check(load().pkv_bm_create(num_blocks, block_size, None if order is None else _ptr(order, C.c_int32),
                                C.byref(h)), "pkv_bm_create")
    return h


def pkv_bm_destroy(bm) -> None:
    load().pkv_bm_destroy(bm)


def kv_block_alloc(bm) -> int:
    out = C.c_int32()
    _check(load().kv_block_alloc(bm, C.byref(out)), "kv_block_alloc")
    return out.value


def kv_block_free(bm, block_id: int) -> None:
    _check(load().kv_block_free(bm, block_id), "kv_block_free")


def pkv_seq_create(bm, seq_id: int) -> None:
    _check(load().pkv_seq_create(bm, seq_id), "pkv_seq_create")


def pkv_seq_fork(bm, parent: int, child: int) -> None:
    _check(load().pkv_seq_fork(bm, parent, child), "pkv_seq_fork")


def pkv_seq_free(bm, seq_id: int) -> None:
    _check(load().pkv_seq_free(bm, seq_id), "pkv_seq_free")


def pkv_seq_append_slots(bm, seq_ids):
    """Returns (slot_mapping int32[n], cow_src int32[k], cow_dst int32[k])."""
    ids = _i64(seq_ids)
    n = len(ids)
    slots = np.empty(n, np.int32)
    src = np.empty(max(n, 1), np.int32)
    dst = np.empty(max(n, 1), np.int32)
    ncow = C.c_int32()
    _check(load().pkv_seq_append_slots(bm, _ptr(ids, C.c_int64), n, _ptr(slots, C.c_int32),
                                       _ptr(src, C.c_int32), _ptr(dst, C.c_int32), C.byref(ncow)),
           "pkv_seq_append_slots")
    return slots, src[:ncow.value].copy(), dst[:ncow.value].copy()


def pkv_build_block_tables(bm, seq_ids, max_blocks: int, tables=None, context_lens=None):
    """Returns (tables int32[n, max_blocks] padded with -1, context_lens int32[n]).

    ``tables`` / ``context_lens`` may be preallocated C-contiguous int32 arrays.
    """
    ids = _i64(seq_ids)
    n = len(ids)
    if tables is None:
        tables = np.empty((n, max_blocks), np.int32)
    if context_lens is None:
        context_lens = np.empty(n, np.int32)
    assert tables.dtype == np.int32 and tables.flags.c_contiguous and tables.size >= n * max_blocks
    assert context_lens.dtype == np.int32 and context_lens.flags.c_contiguous and context_lens.size >= n
    _check(load().pkv_build_block_tables(bm, _ptr(ids, C.c_int64), n, max_blocks, _ptr(tables, C.c_int32),
                                         _ptr(context_lens, C.c_int32)), "pkv_build_block_tables")
    return tables, context_lens


def pkv_bm_num_free(bm) -> int:
    return int(load().pkv_bm_num_free(bm))


def pkv_bm_num_blocks(bm) -> int:
    return int(load().pkv_bm_num_blocks(bm))


def pkv_bm_free_list(bm) -> np.ndarray:
    n = C.c_int32()
    _check(load().pkv_bm_free_list(bm, None, 0, C.byref(n)), "pkv_bm_free_list")
    out = np.empty(max(n.value, 1), np.int32)
    _check(load().pkv_bm_free_list(bm, _ptr(out, C.c_int32), n.value, C.byref(n)), "pkv_bm_free_list")
    return out[:n.value].copy()


def pkv_bm_refcount(bm, block_id: int) -> int:
    out = C.c_int32()
    _check(load().pkv_bm_refcount(bm, block_id, C.byref(out)), "pkv_bm_refcount")
    return out.value


def pkv_seq_len(bm, seq_id: int) -> int:
    out = C.c_int32()
    _check(load().pkv_seq_len(bm, seq_id, C.byref(out)), "pkv_seq_len")
    return out.value


def pkv_kv_bytes(layers, kv_heads, head_dim, tokens, cache_dtype) -> int:
    return int(load().pkv_kv_bytes(layers, kv_heads, head_dim, tokens, _dt(cache_dtype)))


def pkv_pool_blocks(budget_bytes, layers, kv_heads, head_dim, cache_dtype, block_size=BLOCK_SIZE) -> int:
    return int(load().pkv_pool_blocks(budget_bytes, layers, kv_heads, head_dim, _dt(cache_dtype), block_size))


def pkv_bm_block_size(bm) -> int:
    return int(load().pkv_bm_block_size(bm))


# ---- prefix cache --------------------------------------------------------------
class PrefixStats(C.Structure):
    _fields_ = [("lookups", C.c_int64), ("hits", C.c_int64), ("evictions", C.c_int64),
                ("registered", C.c_int64), ("evictable", C.c_int64)]


def pkv_block_hash(parent_hash: int, tokens, config_key: int) -> int:
    t = _i32(tokens)
    if t.size != BLOCK_SIZE:
        raise ValueError("a block hash takes exactly 16 token ids")
    return int(load().pkv_block_hash(parent_hash & 0xFFFFFFFFFFFFFFFF, _ptr(t, C.c_int32),
                                     config_key & 0xFFFFFFFFFFFFFFFF))


def pkv_bm_enable_prefix_cache(bm, config_key: int = 0) -> None:
    _check(load().pkv_bm_enable_prefix_cache(bm, config_key & 0xFFFFFFFFFFFFFFFF), "pkv_bm_enable_prefix_cache")


def pkv_seq_admit(bm, seq_id, tokens) -> int:
    t = _i32(tokens)
    out = C.c_int32()
    _check(load().pkv_seq_admit(bm, int(seq_id), _ptr(t, C.c_int32), t.size, C.byref(out)), "pkv_seq_admit")
    return out.value


def pkv_seq_commit_prefix(bm, seq_id, tokens) -> int:
    t = _i32(tokens)
    out = C.c_int32()
    _check(load().pkv_seq_commit_prefix(bm, int(seq_id), _ptr(t, C.c_int32), t.size, C.byref(out)),
           "pkv_seq_commit_prefix")
    return out.value


def pkv_prefix_cache_stats(bm) -> dict:
    st = PrefixStats()
    _check(load().pkv_prefix_cache_stats(bm, C.byref(st)), "pkv_prefix_cache_stats")
    return {k: int(getattr(st, k)) for k, _ in PrefixStats._fields_}


# ---- device calls --------------------------------------------------------------
def _dt(x) -> int:
    """pkv_dtype of a name ('bf16'), an int, or a torch dtype."""
    if isinstance(x, int):
        return x
    if isinstance(x, str):
        return DTYPE_NAMES[x]
    import torch
    # INT8 caches hold uint8 bytes (code + 128): name them ("int8"), a uint8 tensor reads as FP8 E4M3
    m = {torch.float16: PKV_F16, torch.bfloat16: PKV_BF16, torch.uint8: PKV_FP8_E4M3, torch.float32: PKV_F32}
    if hasattr(torch, "float8_e4m3fn"):
        m[torch.float8_e4m3fn] = PKV_FP8_E4M3
    if hasattr(torch, "float8_e5m2"):
        m[torch.float8_e5m2] = PKV_FP8_E5M2
    return m[x]


def _cdt(k_cache, cache_dtype) -> int:
    """Cache pkv_dtype: given by name, else read off the tensor (uint8 reads as FP8 E4M3)."""
    return _dt(cache_dtype) if cache_dtype is not None else _dt(k_cache.dtype)


def _dp(t):
    """Device pointer of a tensor (or None / an int address)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def paged_kv_copy_blocks(k_cache, v_cache, k_scale, v_scale, src, dst, num_pairs=None,
                         d_error=None, stream=None, cache_dtype=None) -> None:
    nb, hkv, bs, d = k_cache.shape
    n = src.numel() if num_pairs is None else num_pairs
    _check(load().paged_kv_copy_blocks(_dp(k_cache), _dp(v_cache), _dp(k_scale), _dp(v_scale), _dp(src),
                                       _dp(dst), n, hkv, d, _cdt(k_cache, cache_dtype), nb, bs, _dp(d_error),
                                       _stream(stream)), "paged_kv_copy_blocks")


def paged_kv_append(k, v, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None,
                    d_error=None, stream=None, cache_dtype=None) -> None:
    t, hkv, d = k.shape
    nb, bs = k_cache.shape[0], k_cache.shape[2]
    _check(load().paged_kv_append(_dp(k), _dp(v), _dt(k.dtype), t, hkv, d, _dp(slot_mapping), _dp(k_cache),
                                  _dp(v_cache), _cdt(k_cache, cache_dtype), _dp(k_scale), _dp(v_scale), nb, bs,
                                  _dp(d_error), _stream(stream)), "paged_kv_append")


def paged_attention_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, q_dtype,
                                    cache_dtype) -> int:
    out = C.c_size_t()
    _check(load().paged_attention_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, _dt(q_dtype),
                                                  _dt(cache_dtype), C.byref(out)),
           "paged_attention_workspace_bytes")
    return out.value


def paged_attention_decode(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                           max_context_len, scale, workspace, d_error=None, stream=None,
                           num_seqs=None, cache_dtype=None) -> None:
    b, hq, d = q.shape
    if num_seqs is not None:
        b = num_seqs
    nb, hkv, bs = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    _check(load().paged_attention_decode(
        _dp(out), _dt(out.dtype), _dp(q), _dt(q.dtype), _dp(k_cache), _dp(v_cache), _cdt(k_cache, cache_dtype),
        _dp(k_scale),
        _dp(v_scale), _dp(block_tables), block_tables.shape[-1], _dp(context_lens), int(max_context_len), b, hq,
        hkv, d, nb, bs, float(scale), _dp(workspace), workspace.numel() * workspace.element_size(),
        _dp(d_error), _stream(stream)), "paged_attention_decode")


def paged_attention_decode_append(out, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, block_tables,
                                  context_lens, max_context_len, scale, workspace, d_error=None, stream=None,
                                  num_seqs=None, cache_dtype=None) -> None:
    """Append row b of k_new / v_new at position context_lens[b] - 1, then decode (one launch)."""
    b, hq, d = q.shape
    if num_seqs is not None:
        b = num_seqs
    nb, hkv, bs = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    _check(load().paged_attention_decode_append(
        _dp(out), _dt(out.dtype), _dp(q), _dt(q.dtype), _dp(k_new), _dp(v_new), _dp(k_cache), _dp(v_cache),
        _cdt(k_cache, cache_dtype), _dp(k_scale), _dp(v_scale), _dp(block_tables), block_tables.shape[-1],
        _dp(context_lens), int(max_context_len), b, hq, hkv, d, nb, bs, float(scale), _dp(workspace),
        workspace.numel() * workspace.element_size(), _dp(d_error), _stream(stream)), "paged_attention_decode_append")


def paged_attention_decode_static(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                                  max_context_len, scale, d_error=None, stream=None, num_seqs=None,
                                  cache_dtype=None) -> None:
    """paged_attention_decode with the library's static scratch (no workspace, no allocation)."""
    b, hq, d = q.shape
    if num_seqs is not None:
        b = num_seqs
    nb, hkv, bs = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    _check(load().paged_attention_decode_static(
        _dp(out), _dt(out.dtype), _dp(q), _dt(q.dtype), _dp(k_cache), _dp(v_cache), _cdt(k_cache, cache_dtype),
        _dp(k_scale), _dp(v_scale), _dp(block_tables), block_tables.shape[-1], _dp(context_lens),
        int(max_context_len), b, hq, hkv, d, nb, bs, float(scale), _dp(d_error), _stream(stream)),
        "paged_attention_decode_static")


# ---- prompt-side device calls ----------------------------------------------------
# These take whole tensors' shapes from the caller's arguments, so the binding
# checks what the C ABI cannot see: device, type, shape and density.
def _refuse(where, why):
    raise PkvError(-1, where, why)


def _check_tensor(where, name, t, dtype, shape, device, dense=True):
    """t is a tensor of `dtype` (None: any) and `shape` (None entries: any) on `device`."""
    if t.device != device:
        _refuse(where, f"{name} must be on {device}, not {t.device}")
    if dtype is not None and t.dtype != dtype:
        _refuse(where, f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and g != w for g, w in zip(t.shape, shape)):
        _refuse(where, f"{name} must have shape {tuple('*' if w is None else w for w in shape)}, not {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        _refuse(where, f"{name} must be contiguous")


def _cuda_device(where, name, t):
    if not t.is_cuda:
        _refuse(where, f"{name} must be on a CUDA device")
    return t.device


def _check_pool(where, k_cache, v_cache, k_scale, v_scale, cache_dtype, device):
    """Check the cache tensors of one layer; returns (num_blocks, hkv, block_size, head_dim, cache pkv_dtype)."""
    cdt = _cdt(k_cache, cache_dtype)
    name = next(n for n, v in DTYPE_NAMES.items() if v == cdt)
    if k_cache.dim() != 4:
        _refuse(where, "k_cache must have shape [num_blocks, num_kv_heads, block_size, head_dim]")
    nb, hkv, bs, d = k_cache.shape
    if k_cache.element_size() != (1 if name in SCALED_CACHES else 2):
        _refuse(where, f"k_cache has elements of {k_cache.element_size()} bytes, which is not a {name} cache")
    _check_tensor(where, "k_cache", k_cache, None, (nb, hkv, bs, d), device)
    _check_tensor(where, "v_cache", v_cache, k_cache.dtype, (nb, hkv, bs, v_row_elems(name, d)), device)
    if name in SCALED_CACHES:
        import torch
        for n, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None:
                _refuse(where, f"a {name} cache needs {n}")
            _check_tensor(where, n, t, torch.float32, (nb, hkv, bs), device, dense=False)
            if t.numel() and t.stride() != (2 * hkv * bs, 2 * bs, 1):
                _refuse(where, f"{n} must be its half of one [num_blocks, num_kv_heads, 2, block_size] array")
    return nb, hkv, bs, d, cdt


class _on_device:
    """Makes `device` current for a call when it is not already."""

    def __init__(self, device):
        self.index = device.index
        self.back = None

    def __enter__(self):
        import torch
        now = torch.cuda.current_device()
        if now != self.index:
            torch.cuda.set_device(self.index)
            self.back = now

    def __exit__(self, *exc):
        if self.back is not None:
            import torch
            torch.cuda.set_device(self.back)


def _stream_on(stream, device):
    """cudaStream_t: the caller's, or the current stream of `device`."""
    if stream is None:
        return current_stream_handle(device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check_error_word(where, d_error, device):
    if d_error is not None and not isinstance(d_error, int):
        import torch
        _check_tensor(where, "d_error", d_error, torch.int32, (1,), device)


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


def pkv_rope_table(cos_sin, base=10000.0, scaling="none", factor=1.0, original_max=0, slow_turns=1.0,
                   fast_turns=32.0, magnitude=0.0, stream=None) -> None:
    """Fill cos_sin (float32 [max_positions, 2, rot_dim / 2]) with cosines and sines of every position and pair."""
    import torch
    where = "pkv_rope_table"
    dev = _cuda_device(where, "cos_sin", cos_sin)
    _check_tensor(where, "cos_sin", cos_sin, torch.float32, (None, 2, None), dev)
    with _on_device(dev):
        _check(load().pkv_rope_table(_dp(cos_sin), cos_sin.shape[0], 2 * cos_sin.shape[2], float(base),
                                     ROPE_SCALINGS.get(scaling, scaling), float(factor), int(original_max),
                                     float(slow_turns), float(fast_turns), float(magnitude),
                                     _stream_on(stream, dev)), where)


def _token_stride(where, name, t, shape, dtype, device):
    """Elements from one token's rows to the next's of t [tokens, heads, head_dim], whose rows are dense."""
    _check_tensor(where, name, t, dtype, shape, device, dense=False)
    n, h, d = shape
    if n and h and (t.stride(2) != 1 or (h > 1 and t.stride(1) != d)):
        _refuse(where, f"{name}: the rows of one token must be dense")
    return t.stride(0) if n > 1 else h * d


def paged_kv_append_rope(q_out, q, k, v, positions, slot_mapping, cos_sin, k_cache, v_cache, k_scale=None,
                         v_scale=None, interleaved=False, d_error=None, stream=None, cache_dtype=None) -> None:
    """Rotate q (to q_out) and k by cos_sin[positions], and write k and v to their slots, in one launch.

    q [T, Hq, D] and q_out may be None (keys and values only).  The rows of one
    token are dense; q, k and v may be slices of one projection's output.
    """
    import torch
    where = "paged_kv_append_rope"
    dev = _cuda_device(where, "k", k)
    nb, hkv, bs, d, cdt = _check_pool(where, k_cache, v_cache, k_scale, v_scale, cache_dtype, dev)
    t = k.shape[0] if k.dim() else 0
    ks = _token_stride(where, "k", k, (t, hkv, d), None, dev)
    vs = _token_stride(where, "v", v, (t, hkv, d), k.dtype, dev)
    hq, qs = 0, 0
    if k.dtype != torch.float16 and k.dtype != torch.bfloat16:
        _refuse(where, "input rows must be float16 or bfloat16")
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else -1
        qs = _token_stride(where, "q", q, (t, hq, d), k.dtype, dev)
        if q_out is None:
            _refuse(where, "q needs a q_out")
        _check_tensor(where, "q_out", q_out, k.dtype, (t, hq, d), dev)
    _check_tensor(where, "positions", positions, torch.int32, (t,), dev)
    _check_tensor(where, "slot_mapping", slot_mapping, torch.int32, (t,), dev)
    _check_tensor(where, "cos_sin", cos_sin, torch.float32, (None, 2, None), dev)
    _check_error_word(where, d_error, dev)
    with _on_device(dev):
        _check(load().paged_kv_append_rope(
            _dp(q_out) if hq else None, _dp(q) if hq else None, _dp(k), _dp(v), _dt_torch(k.dtype), qs, ks, vs, t, hq,
            hkv, d, _dp(positions), _dp(slot_mapping), _dp(cos_sin), cos_sin.shape[0], 2 * cos_sin.shape[2],
            1 if interleaved else 0, _dp(k_cache), _dp(v_cache), cdt, _dp(k_scale), _dp(v_scale), nb, bs,
            _dp(d_error), _stream_on(stream, dev)), where)


def paged_kv_gather(k_out, v_out, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out_starts,
                    token_starts=None, d_error=None, stream=None, cache_dtype=None) -> None:
    """Cached rows token_starts[b] .. context_lens[b] - 1 of sequence b to rows out_starts[b] .. of k_out, v_out."""
    import torch
    where = "paged_kv_gather"
    dev = _cuda_device(where, "k_out", k_out)
    nb, hkv, bs, d, cdt = _check_pool(where, k_cache, v_cache, k_scale, v_scale, cache_dtype, dev)
    n = k_out.shape[0] if k_out.dim() else 0
    if k_out.dtype not in (torch.float16, torch.bfloat16, torch.float32):
        _refuse(where, "k_out must be float16, bfloat16 or float32")
    _check_tensor(where, "k_out", k_out, None, (n, hkv, d), dev)
    _check_tensor(where, "v_out", v_out, k_out.dtype, (n, hkv, d), dev)
    _check_tensor(where, "block_tables", block_tables, torch.int32, (None, None), dev)
    b = block_tables.shape[0]
    _check_tensor(where, "context_lens", context_lens, torch.int32, (b,), dev)
    _check_tensor(where, "out_starts", out_starts, torch.int32, (b + 1,), dev)
    if token_starts is not None:
        _check_tensor(where, "token_starts", token_starts, torch.int32, (b,), dev)
    _check_error_word(where, d_error, dev)
    with _on_device(dev):
        _check(load().paged_kv_gather(
            _dp(k_out), _dp(v_out), _dt_torch(k_out.dtype), n, _dp(k_cache), _dp(v_cache), cdt, _dp(k_scale),
            _dp(v_scale), _dp(block_tables), block_tables.shape[1], _dp(token_starts), _dp(context_lens),
            _dp(out_starts), b, hkv, d, nb, bs, _dp(d_error), _stream_on(stream, dev)), where)


def paged_attention_extend_workspace_bytes(head_dim) -> int:
    out = C.c_size_t()
    _check(load().paged_attention_extend_workspace_bytes(int(head_dim), C.byref(out)),
           "paged_attention_extend_workspace_bytes")
    return out.value


def paged_attention_extend(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, query_starts,
                           scale, workspace, window=0, sinks=0, d_error=None, stream=None, cache_dtype=None) -> None:
    """Causal attention of each sequence's new tokens (rows query_starts[b] .. of q) over its cache.

    ``window`` (0: none) tokens are visible to a query, its own among them, and
    the first ``sinks``.  ``workspace``: bytes as paged_attention_extend_workspace_bytes, zero-filled once.
    """
    import torch
    where = "paged_attention_extend"
    dev = _cuda_device(where, "q", q)
    nb, hkv, bs, d, cdt = _check_pool(where, k_cache, v_cache, k_scale, v_scale, cache_dtype, dev)
    if q.dtype != torch.float16 and q.dtype != torch.bfloat16:
        _refuse(where, "q must be float16 or bfloat16")
    if q.dim() != 3:
        _refuse(where, "q must have shape [queries, num_q_heads, head_dim]")
    n, hq, _ = q.shape
    _check_tensor(where, "q", q, None, (n, hq, d), dev)
    _check_tensor(where, "out", out, torch.float32 if out.dtype == torch.float32 else q.dtype, (n, hq, d), dev)
    _check_tensor(where, "block_tables", block_tables, torch.int32, (None, None), dev)
    b = block_tables.shape[0]
    _check_tensor(where, "context_lens", context_lens, torch.int32, (b,), dev)
    _check_tensor(where, "query_starts", query_starts, torch.int32, (b + 1,), dev)
    _check_tensor(where, "workspace", workspace, None, (None,), dev)
    _check_error_word(where, d_error, dev)
    with _on_device(dev):
        _check(load().paged_attention_extend(
            _dp(out), _dt_torch(out.dtype), _dp(q), _dt_torch(q.dtype), n, _dp(k_cache), _dp(v_cache), cdt,
            _dp(k_scale), _dp(v_scale), _dp(block_tables), block_tables.shape[1], _dp(context_lens),
            _dp(query_starts), b, hq, hkv, d, nb, bs, float(scale), int(window), int(sinks), _dp(workspace),
            workspace.numel() * workspace.element_size(), _dp(d_error), _stream_on(stream, dev)), where)


def pkv_stepper_host_bytes(max_seqs, max_blocks_per_seq) -> int:
    return int(load().pkv_stepper_host_bytes(max_seqs, max_blocks_per_seq))


def pkv_stepper_device_bytes(max_seqs, max_blocks_per_seq) -> int:
    return int(load().pkv_stepper_device_bytes(max_seqs, max_blocks_per_seq))


def pkv_stepper_create(pool: PoolDesc, max_seqs, max_blocks_per_seq, host_staging, dev_meta, workspace):
    h = _vp()
    _check(load().pkv_stepper_create(C.byref(pool), max_seqs, max_blocks_per_seq, host_staging.data_ptr(),
                                     host_staging.numel() * host_staging.element_size(), _dp(dev_meta),
                                     dev_meta.numel() * dev_meta.element_size(), _dp(workspace),
                                     workspace.numel() * workspace.element_size(), C.byref(h)),
           "pkv_stepper_create")
    return h


def pkv_stepper_destroy(st) -> None:
    load().pkv_stepper_destroy(st)


def pkv_stepper_use_graphs(st, enable: bool) -> None:
    _check(load().pkv_stepper_use_graphs(st, 1 if enable else 0), "pkv_stepper_use_graphs")


def pkv_stepper_use_cascade(st, enable: bool) -> None:
    _check(load().pkv_stepper_use_cascade(st, 1 if enable else 0), "pkv_stepper_use_cascade")


def pkv_stepper_cascade_count(st) -> int:
    return int(load().pkv_stepper_cascade_count(st))


def pkv_stepper_graph_stats(st):
    """(graphs captured, graphs replayed) by this stepper."""
    c, r = C.c_int64(0), C.c_int64(0)
    _check(load().pkv_stepper_graph_stats(st, C.byref(c), C.byref(r)), "pkv_stepper_graph_stats")
    return int(c.value), int(r.value)


def _layer_stride(t, layers):
    """Byte stride between layers of a per-layer tensor ([layers, ...] or one tensor for all: 0)."""
    return t.stride(0) * t.element_size() if t.dim() == 4 and layers > 1 else 0


class StepScratch:
    """Host arrays a step writes its copy pairs into, allocated once per stepper."""

    def __init__(self, max_seqs: int):
        self.src = np.empty(max(max_seqs, 1), np.int32)
        self.dst = np.empty(max(max_seqs, 1), np.int32)
        self.ncow = np.zeros(1, np.int32)
        self.addr = (self.src.ctypes.data, self.dst.ctypes.data, self.ncow.ctypes.data)


def _segments(pairs, where):
    segs = (CopySegment * max(1, len(pairs)))()
    for i, (dst, src) in enumerate(pairs):
        nb = src.numel() * src.element_size()
        if dst.numel() * dst.element_size() != nb:
            raise ValueError(f"{where}: sizes differ")
        segs[i].dst, segs[i].src, segs[i].bytes = dst.data_ptr(), src.data_ptr(), nb
    return segs


def pkv_copy_segments(pairs, stream) -> None:
    """One-launch copy of [(dst tensor, src tensor), ...] (same byte sizes; device or pinned host memory)."""
    _check(load().pkv_copy_segments(_segments(pairs, "pkv_copy_segments"), len(pairs), stream), "pkv_copy_segments")


def pkv_stepper_copy_inputs(st, pairs) -> None:
    """Register [(device tensor, pinned host tensor), ...] copies for the stepper's next step."""
    _check(load().pkv_stepper_copy_inputs(st, _segments(pairs, "pkv_stepper_copy_inputs"), len(pairs)),
           "pkv_stepper_copy_inputs")


def current_stream_handle(device_index: int) -> int:
    """cudaStream_t of torch's current stream on a device."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(device_index)
    return torch.cuda.current_stream(device_index).cuda_stream


_TORCH_DT = None


def _dt_torch(dtype) -> int:
    global _TORCH_DT
    if _TORCH_DT is None:
        import torch
        _TORCH_DT = {torch.float16: PKV_F16, torch.bfloat16: PKV_BF16, torch.float32: PKV_F32,
                     torch.uint8: PKV_FP8_E4M3}
    return _TORCH_DT[dtype]


def pkv_stepper_step(st, bm, seq_ids, k_new, v_new, q, out, scale, layers, d_error=None, events=None,
                     stream=None, scratch: StepScratch | None = None):
    """One decode step; returns (cow_src, cow_dst) of the step.

    ``stream``: a torch stream, a cudaStream_t address, or None for the current
    stream of q's device.  ``scratch``: reusable host arrays (else allocated).
    """
    ids = seq_ids if isinstance(seq_ids, np.ndarray) and seq_ids.dtype == np.int64 else \
        np.asarray(seq_ids, dtype=np.int64)
    if not ids.flags.c_contiguous:
        ids = np.ascontiguousarray(ids)
    n = ids.shape[0]
    if scratch is None or scratch.src.shape[0] < n:
        scratch = StepScratch(n)
    ev0 = ev1 = None
    if events is not None:
        ev0, ev1 = events[0].cuda_event, events[1].cuda_event
    if stream is None:
        sh = current_stream_handle(q.device.index)
    elif isinstance(stream, int):
        sh = stream
    else:
        sh = stream.cuda_stream
    a_src, a_dst, a_n = scratch.addr
    status = load().pkv_stepper_step(
        st, bm, ids.ctypes.data, n, k_new.data_ptr(), v_new.data_ptr(), _layer_stride(k_new, layers),
        q.data_ptr(), _layer_stride(q, layers), out.data_ptr(), _dt_torch(out.dtype), _layer_stride(out, layers),
        float(scale), a_src, a_dst, a_n, _dp(d_error), ev0, ev1, sh)
    if status != 0:
        _check(status, "pkv_stepper_step")
    ncow = int(scratch.ncow[0])
    if ncow == 0:
        return _EMPTY_I32, _EMPTY_I32
    return scratch.src[:ncow].copy(), scratch.dst[:ncow].copy()


_EMPTY_I32 = np.empty(0, np.int32)


def pkv_read_device_error(d_error, clear: bool = True, stream=None, raise_on_error: bool = False) -> int:
    h = C.c_int32()
    st = load().pkv_read_device_error(_dp(d_error), C.byref(h), 1 if clear else 0, _stream(stream))
    if st != -5 or raise_on_error:
        _check(st, "pkv_read_device_error")
    return h.value


DECODE_KERNELS = {"auto": 0, "simt": 1, "mma": 2}


def pkv_set_decode_kernel(kind) -> None:
    """Select the decode kernel process-wide: 'auto', 'simt' or 'mma'."""
    _check(load().pkv_set_decode_kernel(DECODE_KERNELS.get(kind, kind)), "pkv_set_decode_kernel")


def pkv_get_decode_kernel() -> str:
    v = int(load().pkv_get_decode_kernel())
    return {k: n for n, k in DECODE_KERNELS.items()}[v]


PREFIX_KERNELS = {"auto": 0, "mma_sync": 1, "tcgen05": 2}


def pkv_set_prefix_kernel(kind, chunk_tiles: int = 0) -> None:
    """Select the cascade's prefix kernel process-wide: 'auto', 'mma_sync' or 'tcgen05'."""
    _check(load().pkv_set_prefix_kernel(PREFIX_KERNELS.get(kind, kind), int(chunk_tiles)), "pkv_set_prefix_kernel")


def pkv_get_prefix_kernel() -> str:
    v = int(load().pkv_get_prefix_kernel())
    return {k: n for n, k in PREFIX_KERNELS.items()}[v]


def pkv_launch_count() -> int:
    return int(load().pkv_launch_count())


def pkv_status_string(status: int) -> str:
    return load().pkv_status_string(status).decode()
