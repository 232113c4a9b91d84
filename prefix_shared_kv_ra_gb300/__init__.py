"""GB300 (sm_103a) RadixAttention hot path: KV store, extend and decode
attention over a token-granular KV pool shared through a radix-tree prefix
cache.

This module is the thin Python binding of ``libra.so`` (C ABI in
``include/ra.h``).  It only marshals arguments: it checks torch dtypes,
devices, shapes and contiguity, and passes raw device pointers and the
current CUDA stream to the library, where every step of the path runs in
hand-written CUDA kernels.  There is no fallback: if the library is missing
or fails to load, importing the binding raises.

Functions keep the C names: ``ra_kv_store``, ``ra_extend_attention``,
``ra_decode_attention``, ``ra_decode_workspace_bytes``, ... .
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
from typing import Optional

import torch

from . import _build

__all__ = ["RAError", "ra_kv_store", "ra_extend_attention", "ra_extend_workspace_bytes", "ra_decode_attention",
           "ra_decode_workspace_bytes", "ra_decode_attention_store",
           "ra_decode_attention_static", "RA_DECODE_STATIC_SCRATCH_BYTES",
           "ra_kv8_slot_bytes", "ra_kv8_store", "ra_kv8_load", "ra_kv8_decode_attention",
           "ra_qk_norm_rope_store", "ra_qk_norm_rope_kv8_store", "ra_tree_attention", "ra_tree_workspace_bytes",
           "ra_extend_attention_mod", "ra_extend_mod_workspace_bytes", "ra_decode_attention_mod",
           "ra_step_slots", "ra_tree_verify", "ra_tree_verify_greedy", "ra_tree_commit",
           "ra_abi_version", "ra_selftest_bounded_wait", "library_path", "load", "DEVERR_SLOT", "DEVERR_TABLE", "DEVERR_LENGTH",
           "DEVERR_TIMEOUT", "DEVERR_POSITION", "DEVERR_FULL", "DEVERR_VALUE"]

RA_OK = 0
RA_ERR_UNSUPPORTED = 2
RA_DECODE_STATIC_SCRATCH_BYTES = 32 << 20  # size of the library's static decode scratch (include/ra.h)
DEVERR_SLOT, DEVERR_TABLE, DEVERR_LENGTH, DEVERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEVERR_POSITION, DEVERR_FULL, DEVERR_VALUE = 0x10, 0x20, 0x40
_lib = None
_binding = None


class RAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libra.so (building it first only if asked and it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        if not build_if_missing:
            raise ImportError(f"{_build.LIB} is not built; run prefix_shared_kv_ra_gb300._build.build()")
        _build.build()
    lib = ctypes.CDLL(_build.LIB)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.ra_kv_store.argtypes = [P, P, i64, i32, i32, P, P, P, i64, P, P]
    lib.ra_extend_attention.argtypes = [P, P, i64, i32, i32, P, P, i32, f32, P, i64, i64, P, P, P, P, i32, i64,
                                        i32, i32, P, sz, P, P]
    lib.ra_extend_workspace_bytes.argtypes = [i32, i64, i32, i32]
    lib.ra_extend_workspace_bytes.restype = sz
    lib.ra_decode_attention.argtypes = [P, P, i64, i32, i32, P, P, i32, f32, P, i64, i64, P, P, i32, i32, i32,
                                        P, P, P, P, P, i32, i32, i32, P, sz, P, P]
    lib.ra_decode_attention_store.argtypes = [P, P, i64, i32, i32, P, P, P, P, P, i32, f32, P, i64, i64, P, P, i32,
                                              i32, i32, P, P, P, P, P, i32, i32, i32, P, sz, P, P]
    lib.ra_decode_attention_store.restype = ctypes.c_int
    lib.ra_decode_attention_static.argtypes = [P, P, i64, i32, i32, P, P, i32, f32, P, i64, i64, P, P, i32, i32,
                                               i32, P, P, P, P, P, i32, i32, i32, P, P]
    lib.ra_decode_attention_static.restype = ctypes.c_int
    lib.ra_selftest_bounded_wait.argtypes = [i64, P, P]
    lib.ra_selftest_bounded_wait.restype = ctypes.c_int
    lib.ra_kv8_slot_bytes.argtypes = [i32, i32]
    lib.ra_kv8_slot_bytes.restype = sz
    lib.ra_kv8_store.argtypes = [P, i64, i32, i32, P, P, P, i64, P, P]
    lib.ra_kv8_load.argtypes = [P, i64, i32, i32, P, P, P, i64, P, P]
    lib.ra_kv8_decode_attention.argtypes = [P, i64, i32, i32, P, P, i32, f32, P, i64, i64, P, P, i32, i32, P, sz, P, P]
    norm_rope = [P, i64, P, i64, P, i64, i32, i32, i32, P, P, f32, P, P, i64, i32, i32, P, i64]
    lib.ra_qk_norm_rope_store.argtypes = norm_rope + [P, P, i64, P, i64, P, P]
    lib.ra_qk_norm_rope_kv8_store.argtypes = norm_rope + [P, i64, P, i64, P, P]
    lib.ra_tree_attention.argtypes = [P, P, i64, i32, i32, P, P, i32, f32, P, i64, i64, P, P, P, P, P, i32, i32, i64,
                                      i32, i32, P, sz, P, P]
    changed = [P, P, i64, i32, i32, P, P, i32, f32, f32, i32, P, P]
    lib.ra_extend_attention_mod.argtypes = changed + [P, P, i64, i64, P, P, P, P, i32, i64, i32, i32, P, sz, P, P]
    lib.ra_decode_attention_mod.argtypes = changed + [P, i64, i64, P, P, i32, i32, P, sz, P, P]
    lib.ra_extend_mod_workspace_bytes.argtypes = [i32, i64, i32, i32]
    lib.ra_extend_mod_workspace_bytes.restype = sz
    lib.ra_step_slots.argtypes = [P, i64, i64, P, P, P, i32, P, i64, P, P, i32, P, P, i64, P, P, P, P]
    lib.ra_tree_verify.argtypes = [P, i64, P, i64, i32, P, P, P, P, P, P, i32, i64, i32, P, P, P, P, P]
    lib.ra_tree_verify_greedy.argtypes = [P, i32, i64, i32, P, P, P, P, i32, i64, i32, P, P, P, P, P]
    lib.ra_tree_commit.argtypes = [P, i64, i64, P, P, P, P, i32, P, i64, P, i32, P, P, P, i64, P, P, P, P]
    lib.ra_tree_workspace_bytes.argtypes = [i32, i64, i32, i32, i32, i32]
    lib.ra_tree_workspace_bytes.restype = sz
    lib.ra_decode_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32]
    lib.ra_decode_workspace_bytes.restype = sz
    for f in (lib.ra_kv_store, lib.ra_extend_attention, lib.ra_decode_attention, lib.ra_abi_version, lib.ra_kv8_store,
              lib.ra_kv8_load, lib.ra_kv8_decode_attention, lib.ra_qk_norm_rope_store,
              lib.ra_qk_norm_rope_kv8_store, lib.ra_tree_attention, lib.ra_step_slots, lib.ra_tree_verify,
              lib.ra_tree_verify_greedy, lib.ra_tree_commit, lib.ra_extend_attention_mod, lib.ra_decode_attention_mod):
        f.restype = ctypes.c_int
    lib.ra_status_string.argtypes = [ctypes.c_int]
    lib.ra_status_string.restype = ctypes.c_char_p
    lib.ra_last_error_message.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != RA_OK:
        lib = load()
        msg = lib.ra_last_error_message().decode() or lib.ra_status_string(status).decode()
        raise RAError(status, msg)


def _ptr(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, device: torch.device):
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _stream(device: torch.device, stream) -> int:
    if device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got {device}")
    # the raw handle of the current stream: torch.cuda.current_stream builds a Stream object around it, which
    # costs more than the rest of a small call's checks
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)


def ra_selftest_bounded_wait(deadline_cycles: int, device_error: torch.Tensor, stream=None) -> None:
    """One kernel whose waits (an mbarrier nobody arrives at, a counter nobody raises) run out after
    deadline_cycles SM cycles: it must flag DEVERR_TIMEOUT in device_error (int32 [1] on the GPU) and
    return."""
    dev = device_error.device
    _check(load().ra_selftest_bounded_wait(int(deadline_cycles), _ptr(device_error, torch.int32, "device_error", dev),
                                           _stream(dev, stream)))


def ra_abi_version() -> int:
    return int(load().ra_abi_version())


def ra_kv_store(k_pool: torch.Tensor, v_pool: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                out_cache_loc: torch.Tensor, device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """pool[out_cache_loc[i]] = new[i] for K and V (bit copy).  Pools [S, Hkv, D] bf16."""
    dev = k_pool.device
    S, hkv, d = k_pool.shape
    if v_pool.shape != k_pool.shape or k_new.shape != v_new.shape or tuple(k_new.shape[1:]) != (hkv, d):
        raise ValueError("shape mismatch between pools and new rows")
    if out_cache_loc.shape != (k_new.shape[0],):
        raise ValueError("out_cache_loc must be [num_tokens]")
    bf = torch.bfloat16
    _check(load().ra_kv_store(_ptr(k_pool, bf, "k_pool", dev), _ptr(v_pool, bf, "v_pool", dev), S, hkv, d,
                              _ptr(k_new, bf, "k_new", dev), _ptr(v_new, bf, "v_new", dev),
                              _ptr(out_cache_loc, torch.int32, "out_cache_loc", dev), k_new.shape[0],
                              _ptr(device_error, torch.int32, "device_error", dev), _stream(dev, stream)))


def ra_extend_attention(k_pool: torch.Tensor, v_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                        req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, prefix_lens: torch.Tensor,
                        extend_lens: torch.Tensor, qo_indptr: torch.Tensor, *, max_extend_len: int,
                        max_prefix_len: int, sm_scale: float, workspace: torch.Tensor,
                        device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Suffix queries over cached prefix + causal suffix; q, o [total_q, Hq, D] bf16; workspace: uint8,
    at least ra_extend_workspace_bytes(batch, total_q, Hq, Hkv) bytes."""
    dev = k_pool.device
    S, hkv, d = k_pool.shape
    total_q, hq, dq = q.shape
    if dq != d or o.shape != q.shape:
        raise ValueError("q/o shape mismatch")
    batch = req_pool_indices.shape[0]
    bf, i32 = torch.bfloat16, torch.int32
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on the pool's device")
    _check(load().ra_extend_attention(
        _ptr(k_pool, bf, "k_pool", dev), _ptr(v_pool, bf, "v_pool", dev), S, hkv, d, _ptr(q, bf, "q", dev),
        _ptr(o, bf, "o", dev), hq, float(sm_scale), _ptr(req_to_token, i32, "req_to_token", dev),
        req_to_token.shape[1], req_to_token.shape[0], _ptr(req_pool_indices, i32, "req_pool_indices", dev),
        _ptr(prefix_lens, i32, "prefix_lens", dev), _ptr(extend_lens, i32, "extend_lens", dev),
        _ptr(qo_indptr, i32, "qo_indptr", dev), batch, total_q, int(max_extend_len), int(max_prefix_len),
        workspace.data_ptr(), workspace.numel(), _ptr(device_error, i32, "device_error", dev),
        _stream(dev, stream)))


def ra_extend_workspace_bytes(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int) -> int:
    return int(load().ra_extend_workspace_bytes(batch, total_q, num_q_heads, num_kv_heads))


def ra_decode_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
                              num_groups: int = 0, max_group_prefix_len: int = 0, max_group_size: int = 0,
                              max_group_levels: int = 1) -> int:
    return int(load().ra_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len,
                                                num_groups, max_group_prefix_len, max_group_size, max_group_levels))


def ra_decode_attention(k_pool: torch.Tensor, v_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                        req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, seq_lens: torch.Tensor, *,
                        max_seq_len: int, sm_scale: float, workspace: torch.Tensor,
                        group_indptr: Optional[torch.Tensor] = None, group_reqs: Optional[torch.Tensor] = None,
                        group_prefix_len: Optional[torch.Tensor] = None, max_group_prefix_len: int = 0,
                        max_group_size: int = 0, group_prefix_start: Optional[torch.Tensor] = None,
                        group_level: Optional[torch.Tensor] = None, max_group_levels: int = 1,
                        device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """One query per request over its context; q, o [batch, Hq, D] bf16; optional cascade groups (group g
    covers positions group_prefix_start[g] .. group_prefix_len[g]-1 of its members, at group_level[g])."""
    dev = k_pool.device
    S, hkv, d = k_pool.shape
    batch, hq, dq = q.shape
    if dq != d or o.shape != q.shape:
        raise ValueError("q/o shape mismatch")
    bf, i32 = torch.bfloat16, torch.int32
    ng = 0 if group_indptr is None else group_indptr.shape[0] - 1
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on the pool's device")
    _check(load().ra_decode_attention(
        _ptr(k_pool, bf, "k_pool", dev), _ptr(v_pool, bf, "v_pool", dev), S, hkv, d, _ptr(q, bf, "q", dev),
        _ptr(o, bf, "o", dev), hq, float(sm_scale), _ptr(req_to_token, i32, "req_to_token", dev),
        req_to_token.shape[1], req_to_token.shape[0], _ptr(req_pool_indices, i32, "req_pool_indices", dev),
        _ptr(seq_lens, i32, "seq_lens", dev), batch, int(max_seq_len), ng,
        _ptr(group_indptr, i32, "group_indptr", dev), _ptr(group_reqs, i32, "group_reqs", dev),
        _ptr(group_prefix_start, i32, "group_prefix_start", dev), _ptr(group_prefix_len, i32, "group_prefix_len", dev),
        _ptr(group_level, i32, "group_level", dev), int(max_group_prefix_len), int(max_group_size),
        int(max_group_levels), workspace.data_ptr(), workspace.numel(),
        _ptr(device_error, i32, "device_error", dev), _stream(dev, stream)))


def ra_decode_attention_store(k_pool: torch.Tensor, v_pool: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                              out_cache_loc: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                              req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, seq_lens: torch.Tensor, *,
                              max_seq_len: int, sm_scale: float, workspace: torch.Tensor,
                              group_indptr: Optional[torch.Tensor] = None, group_reqs: Optional[torch.Tensor] = None,
                              group_prefix_len: Optional[torch.Tensor] = None, max_group_prefix_len: int = 0,
                              max_group_size: int = 0, group_prefix_start: Optional[torch.Tensor] = None,
                              group_level: Optional[torch.Tensor] = None, max_group_levels: int = 1,
                              device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """The decode step's store and attention in one call: pool[out_cache_loc[b]] = k_new[b] / v_new[b]
    ([batch, Hkv, D] bf16), then ra_decode_attention (same arguments and result)."""
    dev = k_pool.device
    S, hkv, d = k_pool.shape
    batch, hq, dq = q.shape
    if dq != d or o.shape != q.shape:
        raise ValueError("q/o shape mismatch")
    if k_new.shape != (batch, hkv, d) or v_new.shape != k_new.shape or out_cache_loc.shape != (batch,):
        raise ValueError("k_new / v_new must be [batch, Hkv, D] and out_cache_loc [batch]")
    bf, i32 = torch.bfloat16, torch.int32
    ng = 0 if group_indptr is None else group_indptr.shape[0] - 1
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on the pool's device")
    _check(load().ra_decode_attention_store(
        _ptr(k_pool, bf, "k_pool", dev), _ptr(v_pool, bf, "v_pool", dev), S, hkv, d, _ptr(k_new, bf, "k_new", dev),
        _ptr(v_new, bf, "v_new", dev), _ptr(out_cache_loc, i32, "out_cache_loc", dev), _ptr(q, bf, "q", dev),
        _ptr(o, bf, "o", dev), hq, float(sm_scale), _ptr(req_to_token, i32, "req_to_token", dev),
        req_to_token.shape[1], req_to_token.shape[0], _ptr(req_pool_indices, i32, "req_pool_indices", dev),
        _ptr(seq_lens, i32, "seq_lens", dev), batch, int(max_seq_len), ng,
        _ptr(group_indptr, i32, "group_indptr", dev), _ptr(group_reqs, i32, "group_reqs", dev),
        _ptr(group_prefix_start, i32, "group_prefix_start", dev), _ptr(group_prefix_len, i32, "group_prefix_len", dev),
        _ptr(group_level, i32, "group_level", dev), int(max_group_prefix_len), int(max_group_size),
        int(max_group_levels), workspace.data_ptr(), workspace.numel(),
        _ptr(device_error, i32, "device_error", dev), _stream(dev, stream)))


def ra_decode_attention_static(k_pool: torch.Tensor, v_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                               req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, seq_lens: torch.Tensor, *,
                               max_seq_len: int, sm_scale: float, group_indptr: Optional[torch.Tensor] = None,
                               group_reqs: Optional[torch.Tensor] = None,
                               group_prefix_len: Optional[torch.Tensor] = None, max_group_prefix_len: int = 0,
                               max_group_size: int = 0, group_prefix_start: Optional[torch.Tensor] = None,
                               group_level: Optional[torch.Tensor] = None, max_group_levels: int = 1,
                               device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_decode_attention without a workspace argument, for callers that cannot allocate:
    the library's static device scratch (RA_DECODE_STATIC_SCRATCH_BYTES) is used instead."""
    dev = k_pool.device
    S, hkv, d = k_pool.shape
    batch, hq, dq = q.shape
    if dq != d or o.shape != q.shape:
        raise ValueError("q/o shape mismatch")
    bf, i32 = torch.bfloat16, torch.int32
    ng = 0 if group_indptr is None else group_indptr.shape[0] - 1
    # the library resolves its static scratch on the CURRENT device: make it the tensors' device
    with torch.cuda.device(dev):
        _check(load().ra_decode_attention_static(
            _ptr(k_pool, bf, "k_pool", dev), _ptr(v_pool, bf, "v_pool", dev), S, hkv, d, _ptr(q, bf, "q", dev),
            _ptr(o, bf, "o", dev), hq, float(sm_scale), _ptr(req_to_token, i32, "req_to_token", dev),
            req_to_token.shape[1], req_to_token.shape[0], _ptr(req_pool_indices, i32, "req_pool_indices", dev),
            _ptr(seq_lens, i32, "seq_lens", dev), batch, int(max_seq_len), ng,
            _ptr(group_indptr, i32, "group_indptr", dev), _ptr(group_reqs, i32, "group_reqs", dev),
            _ptr(group_prefix_start, i32, "group_prefix_start", dev),
            _ptr(group_prefix_len, i32, "group_prefix_len", dev), _ptr(group_level, i32, "group_level", dev),
            int(max_group_prefix_len), int(max_group_size), int(max_group_levels),
            _ptr(device_error, i32, "device_error", dev), _stream(dev, stream)))


def _native():
    """The C++ side of the calls below: the same checks and the call, without ctypes' cost per argument."""
    global _binding
    if _binding is None:
        lib = load()
        if not os.path.exists(_build.BINDING):
            raise ImportError(f"{_build.BINDING}, the binding for this Python and torch, is not built; run "
                              "prefix_shared_kv_ra_gb300._build.build()")
        spec = importlib.util.spec_from_file_location("_ra_binding", _build.BINDING)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        fns = (lib.ra_kv8_store, lib.ra_kv8_load, lib.ra_kv8_slot_bytes, lib.ra_kv8_decode_attention,
               lib.ra_qk_norm_rope_store, lib.ra_qk_norm_rope_kv8_store, lib.ra_tree_attention, lib.ra_step_slots,
               lib.ra_tree_verify, lib.ra_tree_verify_greedy, lib.ra_tree_commit, lib.ra_extend_attention_mod,
               lib.ra_decode_attention_mod)
        mod.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in fns))
        _binding = mod
    return _binding


@functools.lru_cache(maxsize=None)
def ra_kv8_slot_bytes(num_kv_heads: int, head_dim: int) -> int:
    """Bytes of a quantised pool's record per slot (the layout is in include/ra.h)."""
    n = int(load().ra_kv8_slot_bytes(num_kv_heads, head_dim))
    if n == 0:
        raise RAError(RA_ERR_UNSUPPORTED, f"no quantised pool for {num_kv_heads} kv heads of {head_dim}")
    return n


def ra_kv8_store(kv8_pool: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, out_cache_loc: torch.Tensor,
                 device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise new K/V rows ([num_tokens, Hkv, D] bf16) into the records of slots out_cache_loc."""
    status = (_binding or _native()).kv8_store(kv8_pool, k_new, v_new, out_cache_loc, device_error, stream)
    if status:
        _check(status)


def ra_kv8_load(kv8_pool: torch.Tensor, slots: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor,
                device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Read the records of `slots` back into K/V rows ([num_tokens, Hkv, D] bf16), exactly."""
    status = (_binding or _native()).kv8_load(kv8_pool, slots, k_out, v_out, device_error, stream)
    if status:
        _check(status)


def ra_kv8_decode_attention(kv8_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor, req_to_token: torch.Tensor,
                            req_pool_indices: torch.Tensor, seq_lens: torch.Tensor, *, num_kv_heads: int,
                            max_seq_len: int, sm_scale: float, workspace: torch.Tensor,
                            device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_decode_attention over a quantised pool (uint8 [num_slots, ra_kv8_slot_bytes(Hkv, D)]); q, o
    [batch, Hq, D] bf16; workspace: uint8, ra_decode_workspace_bytes(batch, Hq, Hkv, D, max_seq_len)."""
    status = (_binding or _native()).kv8_decode(kv8_pool, q, o, req_to_token, req_pool_indices, seq_lens, num_kv_heads,
                                                max_seq_len, sm_scale, workspace, device_error, stream)
    if status:
        _check(status)


def ra_qk_norm_rope_store(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight: Optional[torch.Tensor],
                          k_weight: Optional[torch.Tensor], positions: torch.Tensor, cos_sin: torch.Tensor,
                          q_out: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                          out_cache_loc: torch.Tensor, *, eps: float = 1e-6, interleaved: bool = False,
                          device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Per-head RMS norm of q and k, their rotation by cos_sin[positions] (fp32 [max_position, rotary_dim]:
    cosines, then sines), q written to q_out, k and v to pool slots out_cache_loc.  q, k, v, q_out
    [num_tokens, H, D] bf16, any token stride; weights [D] bf16, or None for no norm."""
    status = (_binding or _native()).norm_rope_store(q, k, v, q_weight, k_weight, positions, cos_sin, q_out, k_pool,
                                                     v_pool, out_cache_loc, eps, interleaved, device_error, stream)
    if status:
        _check(status)


def ra_qk_norm_rope_kv8_store(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_weight: Optional[torch.Tensor],
                              k_weight: Optional[torch.Tensor], positions: torch.Tensor, cos_sin: torch.Tensor,
                              q_out: torch.Tensor, kv8_pool: torch.Tensor, out_cache_loc: torch.Tensor, *,
                              eps: float = 1e-6, interleaved: bool = False,
                              device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_qk_norm_rope_store into a quantised pool (uint8 [num_slots, ra_kv8_slot_bytes(Hkv, D)])."""
    status = (_binding or _native()).norm_rope_kv8_store(q, k, v, q_weight, k_weight, positions, cos_sin, q_out,
                                                         kv8_pool, out_cache_loc, eps, interleaved, device_error, stream)
    if status:
        _check(status)


def ra_tree_workspace_bytes(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                            max_draft_len: int, max_prefix_len: int = 0) -> int:
    """Workspace of ra_tree_attention for these bounds (it does not depend on max_prefix_len)."""
    return int(load().ra_tree_workspace_bytes(batch, total_q, num_q_heads, num_kv_heads, head_dim, max_draft_len))


def ra_tree_attention(k_pool: torch.Tensor, v_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                      req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, prefix_lens: torch.Tensor,
                      draft_lens: torch.Tensor, qo_indptr: torch.Tensor, tree_mask: torch.Tensor, *,
                      max_draft_len: int, max_prefix_len: int, sm_scale: float, workspace: torch.Tensor,
                      device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Drafted tokens (q, o [total_q, Hq, D] bf16, request b's rows from qo_indptr[b]) over their request's
    cached prefix and the drafted tokens named by their bit masks (tree_mask int32 [total_q, words], bit c % 32
    of word c / 32 = drafted token c of the request is visible)."""
    status = (_binding or _native()).tree(k_pool, v_pool, q, o, req_to_token, req_pool_indices, prefix_lens, draft_lens,
                                          qo_indptr, tree_mask, max_draft_len, max_prefix_len, sm_scale, workspace,
                                          device_error, stream)
    if status:
        _check(status)


def ra_extend_mod_workspace_bytes(batch: int, total_q: int, num_q_heads: int, num_kv_heads: int) -> int:
    """Workspace of ra_extend_attention_mod."""
    return int(load().ra_extend_mod_workspace_bytes(batch, total_q, num_q_heads, num_kv_heads))


def ra_extend_attention_mod(k_pool: torch.Tensor, v_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                            req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, prefix_lens: torch.Tensor,
                            extend_lens: torch.Tensor, qo_indptr: torch.Tensor, *, max_extend_len: int,
                            max_prefix_len: int, sm_scale: float, workspace: torch.Tensor, score_cap: float = 0.0,
                            window: int = 0, slopes: Optional[torch.Tensor] = None,
                            first_key: Optional[torch.Tensor] = None, full_lens: Optional[torch.Tensor] = None,
                            device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_extend_attention with scores capped (score_cap tanh(s / score_cap)), biased by distance (slopes fp32 [Hq]:
    - slopes[h] |p - j|), and rows that see positions max(first_key[row], p - window + 1) .. p and those below
    full_lens[b] (int32 [total_q], [batch]).  Workspace: uint8, ra_extend_mod_workspace_bytes(batch, total_q, Hq, Hkv)."""
    status = (_binding or _native()).extend_mod(k_pool, v_pool, q, o, req_to_token, req_pool_indices, prefix_lens,
                                                extend_lens, qo_indptr, max_extend_len, max_prefix_len, sm_scale, workspace,
                                                score_cap, window, slopes, first_key, full_lens, device_error, stream)
    if status:
        _check(status)


def ra_decode_attention_mod(k_pool: torch.Tensor, v_pool: torch.Tensor, q: torch.Tensor, o: torch.Tensor,
                            req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, seq_lens: torch.Tensor, *,
                            max_seq_len: int, sm_scale: float, workspace: torch.Tensor, score_cap: float = 0.0,
                            window: int = 0, slopes: Optional[torch.Tensor] = None,
                            first_key: Optional[torch.Tensor] = None, device_error: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """ra_decode_attention (without groups) with the changed scores and masks of ra_extend_attention_mod; first_key int32
    [batch].  Workspace: uint8, ra_decode_workspace_bytes(batch, Hq, Hkv, D, max_seq_len)."""
    status = (_binding or _native()).decode_mod(k_pool, v_pool, q, o, req_to_token, req_pool_indices, seq_lens, max_seq_len,
                                                sm_scale, workspace, score_cap, window, slopes, first_key, device_error,
                                                stream)
    if status:
        _check(status)


def ra_step_slots(req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, seq_lens: torch.Tensor,
                  new_lens: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
                  out_cache_loc: torch.Tensor, positions: torch.Tensor, qo_indptr: torch.Tensor,
                  seq_lens_out: torch.Tensor, *, page_size: int = 1, free_count_out: Optional[torch.Tensor] = None,
                  device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """new_lens[b] new tokens behind the seq_lens[b] of request b: their slots (pages taken from the end of
    free_pages[:free_count]) into req_to_token and out_cache_loc, their positions, the requests' first rows
    (qo_indptr) and new lengths.  All int32; free_count [1] (written in place unless free_count_out is given);
    entries of out_cache_loc and positions [num_tokens] behind the last new token get 0."""
    status = (_binding or _native()).step_slots(req_to_token, req_pool_indices, seq_lens, new_lens, free_pages, free_count,
                                                out_cache_loc, positions, qo_indptr, seq_lens_out, page_size,
                                                free_count_out, device_error, stream)
    if status:
        _check(status)


def ra_tree_verify(target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor], draft_tokens: torch.Tensor,
                   parents: torch.Tensor, draft_lens: torch.Tensor, qo_indptr: torch.Tensor,
                   accept_uniforms: torch.Tensor, final_uniforms: torch.Tensor, path: torch.Tensor,
                   accept_lens: torch.Tensor, next_tokens: torch.Tensor, *, max_draft_len: int,
                   device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Accept or refuse drafted trees against the target's probabilities (fp32 [total_q, vocab], any row stride; row of
    a node: the distribution behind its token) from given uniform numbers: path [batch, max_draft_len] (accepted
    nodes, node 0 first, -1 behind), accept_lens and next_tokens [batch] (int32).  draft_probs: the distributions that
    each node's children were drawn from, or None for drafts taken as given."""
    status = (_binding or _native()).tree_verify(target_probs, draft_probs, draft_tokens, parents, draft_lens, qo_indptr,
                                                 accept_uniforms, final_uniforms, path, accept_lens, next_tokens,
                                                 max_draft_len, device_error, stream)
    if status:
        _check(status)


def ra_tree_verify_greedy(target_logits: torch.Tensor, draft_tokens: torch.Tensor, parents: torch.Tensor,
                          draft_lens: torch.Tensor, qo_indptr: torch.Tensor, path: torch.Tensor,
                          accept_lens: torch.Tensor, next_tokens: torch.Tensor, *, max_draft_len: int,
                          device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """ra_tree_verify at temperature 0: a child is accepted when its token has the largest of its parent's logits
    (bf16 or fp32 [total_q, vocab], any row stride; the lowest token of equal ones)."""
    status = (_binding or _native()).tree_verify_greedy(target_logits, draft_tokens, parents, draft_lens, qo_indptr, path,
                                                        accept_lens, next_tokens, max_draft_len, device_error, stream)
    if status:
        _check(status)


def ra_tree_commit(req_to_token: torch.Tensor, req_pool_indices: torch.Tensor, prefix_lens: torch.Tensor,
                   draft_lens: torch.Tensor, qo_indptr: torch.Tensor, out_cache_loc: torch.Tensor, path: torch.Tensor,
                   accept_lens: torch.Tensor, seq_lens_out: torch.Tensor, free_list: torch.Tensor,
                   free_count: torch.Tensor, *, free_count_out: Optional[torch.Tensor] = None,
                   device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """The accepted path of each verified tree into req_to_token behind the prefix, the new lengths into seq_lens_out,
    the refused tokens' slots to the end of free_list (free_count [1] written in place unless free_count_out is
    given).  A request whose path does not ascend within its tree, or of which a token has no slot (0), is flagged and
    skipped.  All int32."""
    status = (_binding or _native()).tree_commit(req_to_token, req_pool_indices, prefix_lens, draft_lens, qo_indptr,
                                                 out_cache_loc, path, accept_lens, seq_lens_out, free_list, free_count,
                                                 free_count_out, device_error, stream)
    if status:
        _check(status)
