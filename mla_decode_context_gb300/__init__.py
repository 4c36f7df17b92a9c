"""Thin Python binding of libdcp.so (the DCP MLA decode hot path on GB300).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions named like the C entry points take caller-allocated
torch tensors; ``decode_partial`` and ``lse_combine`` allocate their outputs
with torch and call the same entry points.  PyTorch provides device memory
and streams, nothing else (and fills chunk attention's outputs in a step without
requests).

The library is loaded on first use; if it has not been built the call raises
(there is no fallback path).
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from typing import Optional

import torch

from .build_lib import LIB as _LIB_PATH

LATENT_DIM = 512
ROPE_DIM = 64
KV_DIM = 576
MAX_SHARDS = 32
MAX_TREE_ROWS = 256
NOPE_DIM = 128
VALUE_DIM = 128

DEVERR_BAD_BLOCK = 1
DEVERR_SEQ_TOO_LONG = 2
DEVERR_BAD_ROWS = 4
DEVERR_TIMEOUT = 8
DEVERR_NO_BLOCKS = 16
DEVERR_BAD_POSITION = 32

def compute_dtype() -> str:
    """Arithmetic type of the decode contraction: bf16 tensor-core MMAs with
    fp32 accumulation, or fp32 FMA when the CUDA-core kernel is forced
    (DCP_FORCE_SIMT=1) or the layout has no tensor-core tiling."""
    return "f32" if os.environ.get("DCP_FORCE_SIMT", "") == "1" else "bf16"

DTYPE_BF16 = 0
DTYPE_F32 = 1
KV_BF16 = 0
KV_FP8_E4M3 = 1

STATUS = {0: "DCP_OK", 1: "DCP_ERR_INVALID_ARG", 2: "DCP_ERR_UNSUPPORTED_DTYPE",
          3: "DCP_ERR_MISALIGNED", 4: "DCP_ERR_TABLE_TOO_NARROW",
          5: "DCP_ERR_WORKSPACE_TOO_SMALL", 6: "DCP_ERR_CUDA", 7: "DCP_ERR_TIMEOUT"}

# (name, restype, argtypes) of every symbol include/dcp.h declares
_P, _I32, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
EXPORTS = [
    ("dcp_status_str", ctypes.c_char_p, [ctypes.c_int]),
    ("dcp_version", ctypes.c_int, []),
    ("dcp_shard_of", _I32, [_I64, _I32, _I32]),
    ("dcp_local_len", _I32, [_I32, _I32, _I32, _I32]),
    ("dcp_decode_workspace_size", _SZ, [_I32, _I32, _I32, _I32, _I32, _I32]),
    ("dcp_decode_kernel_launches", _I32, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _SZ]),
    ("dcp_mla_decode_partial", ctypes.c_int,
     [_P, _I64, _P, _I32, _I32, _P, _I32, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F,
      _P, _P, _P, _SZ, _P, _P]),
    ("dcp_lse_combine", ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, ctypes.c_int, _P, _P]),
    ("dcp_mla_decode_partial_local", ctypes.c_int,
     [_P, _I64, _P, _I32, _I32, _P, _I32, _I64, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
      _I32, _F, _P, _P, _P, _SZ, _P, _P]),
    ("dcp_mla_decode_partial_v2", ctypes.c_int,
     [_P, _I64, _P, ctypes.c_int, _P, _I32, _I32, _P, _I32, _I64, _I32, _I64, _I32, _I32, _P, _P, _I32, _I32, _I32,
      _I32, _I32, _I32, _I32, _F, _P, ctypes.c_int, _P, _P, _SZ, _P, _P]),
    ("dcp_lse_combine_v2", ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P, _I32, _I32, _I32, _I32, _P, ctypes.c_int, _P,
                                          _P]),
    ("dcp_decode_concat_cache", ctypes.c_int,
     [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _I32, _I32, _P, _I64, _P, _I64, _P, _P]),
    ("dcp_mla_decode_partial_noalloc", ctypes.c_int,
     [_P, _I64, _P, _I32, _I32, _P, _I32, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F,
      _P, _P, _P, _P]),
    ("dcp_decode_concat_cache_v2", ctypes.c_int,
     [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _I32, _I32, _P, _I64, _P, ctypes.c_int, _P, _I64, _P,
      _P]),
    ("dcp_latent_cache_read", ctypes.c_int,
     [_P, ctypes.c_int, _P, _I32, _I32, _P, _I32, _I64, _I32, _I64, _I32, _I32, _I32, _I32, _P, _P, _I32, _I64, _P,
      ctypes.c_int, _I64, _P, _P]),
    ("dcp_mla_decode_partial_window", ctypes.c_int,
     [_P, _I64, _P, ctypes.c_int, _P, _I32, _I32, _P, _I32, _I64, _I32, _I64, _I32, _I32, _P, _P, _I32, _I32, _I32,
      _I32, _I32, _I32, _I32, _F, _I32, _I32, _P, ctypes.c_int, _P, _P, _SZ, _P, _P]),
    ("dcp_mla_decode_partial_tree", ctypes.c_int,
     [_P, _I64, _P, ctypes.c_int, _P, _I32, _I32, _P, _I32, _I64, _I32, _I64, _I32, _I32, _P, _P, _I32, _I32, _I32,
      _I32, _I32, _I32, _I32, _F, _P, _I64, _I32, _I32, _P, ctypes.c_int, _P, _P, _SZ, _P, _P]),
    ("dcp_decode_select_workspace_size", _SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    ("dcp_cache_extend", ctypes.c_int,
     [_P, _I32, _I64, _I32, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P]),
    ("dcp_cache_extend_v2", ctypes.c_int,
     [_P, _I32, _I64, _I32, _I64, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P,
      _P]),
    ("dcp_norm_rope_cache", ctypes.c_int,
     [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _F, _P, _P, _I32, _I32, _P, _I32, _I32,
      _P, ctypes.c_int, _P, _I64, _P, _P]),
    ("dcp_pack_kv_b", ctypes.c_int, [_P, _I32, _P, _P]),
    ("dcp_mla_chunk_attention", ctypes.c_int,
     [_P, _I64, _I64, _P, ctypes.c_int, _P, _I32, _I32, _P, _I32, _I64, _I32, _I64, _I32, _I32, _P, _P, _I32, _I32,
      _I32, _I64, _F, _P, _P, ctypes.c_int, _P, _P, _SZ, _P, _P]),
    ("dcp_chunk_attention_workspace_size", _SZ, [_I32, _I32, _I32, _I64]),
]

_lib = None


class DCPError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__("%s returned %s" % (where, STATUS.get(status, status)))
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded libdcp.so (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libdcp.so is not built (%s); run __graft_entry__.build()" % _LIB_PATH)
        l = ctypes.CDLL(_LIB_PATH)
        for name, res, args in EXPORTS:
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _lib = l
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need_opt(t: Optional[torch.Tensor], name: str, dtype=None, allow_empty=False):
    """Optional device buffers (workspace, dev_error): the kernels write them,
    so a host tensor here would be a host address on the device."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor or None" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.numel() == 0 and not allow_empty:
        raise ValueError("%s must not be empty" % name)


try:  # NVTX ranges name the library calls on profiler timelines
    from torch.cuda import nvtx as _nvtx
except Exception:  # pragma: no cover
    _nvtx = None


class _Range:
    """NVTX range around one library call; a no-op where NVTX is missing
    (it never raises)."""

    def __init__(self, name: str):
        self.name = name
        self.pushed = False

    def __enter__(self):
        if _nvtx is not None:
            try:
                _nvtx.range_push(self.name)
                self.pushed = True
            except Exception:
                pass
        return self

    def __exit__(self, *exc):
        if self.pushed:
            try:
                _nvtx.range_pop()
            except Exception:
                pass
        return False


def _check(st: int, where: str):
    if st != 0:
        raise DCPError(st, where)


def _need(t: torch.Tensor, name: str, dtype, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _decode_geometry(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, D: int,
                     local: bool = False):
    """Validate the decode arguments both decode entry points share and
    return (B, T, H).  Every size the kernels index by is checked here,
    because the C ABI receives bare pointers: a short block table or a
    flattened cache would otherwise be read past its end on the device.
    Shapes are checked before devices, so the checks run on any host."""
    kv_dt = torch.uint8 if isinstance(kv_cache, torch.Tensor) and kv_cache.dtype == torch.uint8 else torch.bfloat16
    o_dt = torch.bfloat16 if isinstance(O_part, torch.Tensor) and O_part.dtype == torch.bfloat16 else torch.float32
    args = (("q", q, torch.bfloat16, False), ("kv_cache", kv_cache, kv_dt, True),
            ("block_table", block_table, torch.int32, False), ("seq_lens", seq_lens, torch.int32, True),
            ("query_start_loc", query_start_loc, torch.int32, True), ("O_part", O_part, o_dt, True),
            ("lse_part", lse_part, torch.float32, True))
    for name, t, dtype, _ in args:
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if q.dim() != 3 or q.shape[2] != KV_DIM or q.stride(2) != 1 or q.stride(1) != KV_DIM:
        raise ValueError("q must be [T, H, 576] with contiguous heads")
    if kv_cache.dim() != 3 or kv_cache.shape[2] != KV_DIM:
        raise ValueError("kv_cache must be [num_blocks, block_size, 576]")
    if local:
        if block_table.dim() != 3 or block_table.stride(2) != 1 or block_table.shape[0] != D:
            raise ValueError("block_table must be [D, B, W] with unit column stride")
    elif block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be [B, W] with unit column stride")
    if seq_lens.dim() != 1 or query_start_loc.dim() != 1:
        raise ValueError("seq_lens and query_start_loc must be 1-D")
    T, H = q.shape[0], q.shape[1]
    B = seq_lens.shape[0]
    if query_start_loc.shape[0] != B + 1 or block_table.shape[-2] != B:
        raise ValueError("seq_lens [B], query_start_loc [B + 1] and block_table [.., B, W] disagree on B")
    if tuple(O_part.shape) != (D, T, H, LATENT_DIM) or tuple(lse_part.shape) != (D, T, H):
        raise ValueError("O_part must be [D, T, H, 512] and lse_part [D, T, H]")
    for name, t, dtype, contiguous in args:
        _need(t, name, dtype, contiguous=contiguous)
    return B, T, H


# ----------------------------------------------------------------------------
# entry points with the C names
# ----------------------------------------------------------------------------
def dcp_version() -> int:
    return lib().dcp_version()


def dcp_status_str(status: int) -> str:
    return lib().dcp_status_str(status).decode()


def dcp_shard_of(pos: int, D: int, interleave: int) -> int:
    return lib().dcp_shard_of(pos, D, interleave)


def dcp_local_len(L: int, d: int, D: int, interleave: int) -> int:
    return lib().dcp_local_len(L, d, D, interleave)


def dcp_decode_workspace_size(B: int, T: int, H: int, D: int, max_seq_len: int, max_q_len: int) -> int:
    n = lib().dcp_decode_workspace_size(B, T, H, D, max_seq_len, max_q_len)
    if n == ctypes.c_size_t(-1).value:
        raise DCPError(1, "dcp_decode_workspace_size")
    return n


def dcp_decode_kernel_launches(B: int, T: int, H: int, D: int, interleave: int, max_seq_len: int,
                               max_q_len: int, workspace_bytes: int) -> int:
    n = lib().dcp_decode_kernel_launches(B, T, H, D, interleave, max_seq_len, max_q_len, workspace_bytes)
    if n < 0:
        raise DCPError(1, "dcp_decode_kernel_launches")
    return n


def dcp_mla_decode_partial(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, *,
                           D: int, interleave: int, scale: float, max_seq_len: int, max_q_len: int,
                           workspace: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None,
                           stream=None) -> None:
    """q bf16 [T, H, 576] (rows may be strided), kv_cache bf16 [NB, bs, 576],
    block_table int32 [B, W] (rows may be strided), seq_lens int32 [B],
    query_start_loc int32 [B + 1]; writes O_part fp32 [D, T, H, 512] and
    lse_part fp32 [D, T, H]."""
    B, T, H = _decode_geometry(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, D)
    _need_opt(workspace, "workspace", allow_empty=True)
    if workspace is not None and workspace.numel() == 0:
        workspace = None
    _need_opt(dev_error, "dev_error", torch.int32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _Range("dcp_mla_decode_partial"):
        st = lib().dcp_mla_decode_partial(
            _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
            block_table.shape[1], block_table.stride(0), _ptr(seq_lens), _ptr(query_start_loc), B, T, H,
            max_seq_len, max_q_len, D, interleave, scale, _ptr(O_part), _ptr(lse_part), _ptr(workspace),
            ws_bytes, _ptr(dev_error), _stream(stream))
    _check(st, "dcp_mla_decode_partial")


def dcp_mla_decode_partial_local(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, *,
                                 D: int, interleave: int, scale: float, max_seq_len: int, max_q_len: int,
                                 shard_begin: int = 0, shard_count: Optional[int] = None,
                                 workspace: Optional[torch.Tensor] = None,
                                 dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """dcp_mla_decode_partial over per-shard tables for shards [shard_begin,
    shard_begin + shard_count) of D (default all): block_table int32
    [shard_count, B, W], shard d's j-th local token of request b in row
    block_table[d - shard_begin, b, j // bs] * bs + j % bs; O_part and
    lse_part have shard_count rows."""
    if shard_count is None:
        shard_count = D - shard_begin
    B, T, H = _decode_geometry(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part,
                               shard_count, local=True)
    _need_opt(workspace, "workspace", allow_empty=True)
    if workspace is not None and workspace.numel() == 0:
        workspace = None
    _need_opt(dev_error, "dev_error", torch.int32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _Range("dcp_mla_decode_partial_local"):
        st = lib().dcp_mla_decode_partial_local(
            _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
            block_table.shape[2], block_table.stride(1), block_table.stride(0), _ptr(seq_lens),
            _ptr(query_start_loc), B, T, H, max_seq_len, max_q_len, D, interleave, shard_begin, shard_count,
            scale, _ptr(O_part), _ptr(lse_part), _ptr(workspace), ws_bytes, _ptr(dev_error), _stream(stream))
    _check(st, "dcp_mla_decode_partial_local")


def dcp_mla_decode_partial_v2(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, *,
                              D: int, interleave: int, scale: float, max_seq_len: int, max_q_len: int,
                              kv_scale: Optional[torch.Tensor] = None, shard_begin: int = 0,
                              shard_count: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                              dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """The general decode: kv_cache bf16, or uint8 FP8 E4M3 codes with
    kv_scale fp32 [num_blocks, block_size]; block_table [B, W] or per-shard
    [shard_count, B, W]; O_part fp32 or bf16 [shard_count, T, H, 512]."""
    if shard_count is None:
        shard_count = D - shard_begin
    local = isinstance(block_table, torch.Tensor) and block_table.dim() == 3
    B, T, H = _decode_geometry(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part,
                               shard_count, local=local)
    fp8 = kv_cache.dtype == torch.uint8
    if fp8:
        _need(kv_scale, "kv_scale", torch.float32)
        if tuple(kv_scale.shape) != tuple(kv_cache.shape[:2]):
            raise ValueError("kv_scale must be [num_blocks, block_size]")
    _need_opt(workspace, "workspace", allow_empty=True)
    if workspace is not None and workspace.numel() == 0:
        workspace = None
    _need_opt(dev_error, "dev_error", torch.int32)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with _Range("dcp_mla_decode_partial_v2"):
        st = lib().dcp_mla_decode_partial_v2(
            _ptr(q), q.stride(0), _ptr(kv_cache), KV_FP8_E4M3 if fp8 else KV_BF16, _ptr(kv_scale if fp8 else None),
            kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table), block_table.shape[-1],
            block_table.stride(-2), 1 if local else 0, block_table.stride(0) if local else 0, shard_begin,
            shard_count, _ptr(seq_lens), _ptr(query_start_loc), B, T, H, max_seq_len, max_q_len, D, interleave,
            scale, _ptr(O_part), DTYPE_BF16 if O_part.dtype == torch.bfloat16 else DTYPE_F32, _ptr(lse_part),
            _ptr(workspace), ws_bytes, _ptr(dev_error), _stream(stream))
    _check(st, "dcp_mla_decode_partial_v2")


def _fits32(bits: int, where: str) -> None:
    """`bits`: a call's whole numbers, ORed.  ctypes cuts a number to its
    parameter's 32 bits.  (One that does not fit may hide behind a negative
    one, which the library refuses.)"""
    if bits >> 31 not in (0, -1):
        raise ValueError("%s: a number does not fit 32 bits" % where)


def dcp_decode_select_workspace_size(B: int, T: int, H: int, D: int, max_seq_len: int, max_q_len: int,
                                     window: int = 0, num_sinks: int = 0) -> int:
    _fits32(B | T | H | D | max_seq_len | max_q_len | window | num_sinks, "dcp_decode_select_workspace_size")
    n = lib().dcp_decode_select_workspace_size(B, T, H, D, max_seq_len, max_q_len, window, num_sinks)
    if n == ctypes.c_size_t(-1).value:
        raise DCPError(1, "dcp_decode_select_workspace_size")
    return n


def _decode_select(where, tree_mask, q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, D,
                   interleave, scale, window, num_sinks, max_seq_len, max_q_len, kv_scale, shard_begin, shard_count,
                   workspace, dev_error, stream) -> None:
    """The two selecting decodes' checks and call.  One expression covers the
    calls that are right; any other goes through _explain_select."""
    if shard_count is None:
        shard_count = D - shard_begin
    _fits32(D | interleave | window | num_sinks | max_seq_len | max_q_len | shard_begin, where)
    tree = where is _TREE
    try:
        T, H, dim = q.shape
        blocks, block_size, row = kv_cache.shape
        B, = seq_lens.shape
        q0, q1, q2 = q.stride()
        table, table_stride = block_table.shape, block_table.stride()
        local = len(table) == 3
        device = q.get_device()
        o_dtype, fp8 = O_part.dtype, kv_cache.dtype is _U8
        good = (
            q.dtype is _BF16 and dim == row == KV_DIM and q1 == KV_DIM and q2 == 1 and device >= 0
            and (fp8 or kv_cache.dtype is _BF16) and kv_cache.get_device() == device and kv_cache.is_contiguous()
            and block_table.dtype is _I32T and block_table.get_device() == device and table_stride[-1] == 1
            and (table[0] == shard_count if local else len(table) == 2) and table[-2] == B
            and seq_lens.dtype is _I32T and seq_lens.get_device() == device and seq_lens.is_contiguous()
            and query_start_loc.dtype is _I32T and query_start_loc.get_device() == device
            and query_start_loc.shape == (B + 1,) and query_start_loc.is_contiguous()
            and (o_dtype is _BF16 or o_dtype is _F32) and O_part.get_device() == device and O_part.is_contiguous()
            and O_part.shape == (shard_count, T, H, LATENT_DIM)
            and lse_part.dtype is _F32 and lse_part.get_device() == device and lse_part.is_contiguous()
            and lse_part.shape == (shard_count, T, H)
            and (_rows_scaled(kv_scale, blocks, block_size, device) if fp8 else kv_scale is None)
            and (workspace is None or (workspace.get_device() == device and workspace.is_contiguous()))
            and (dev_error is None or _flag_word(dev_error, device)))
        if good and tree:
            rows, words = tree_mask.shape
            m0, m1 = tree_mask.stride()
            good = (tree_mask.dtype is _I64T and tree_mask.get_device() == device and rows == T and m1 == 1
                    and words * 64 >= max_q_len)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        T, H, B, local, fp8, device = _explain_select(tree_mask if tree else None, q, kv_cache, block_table, seq_lens,
                                                      query_start_loc, O_part, lse_part, max_q_len, kv_scale,
                                                      shard_count, workspace, dev_error, tree)
        q0, o_dtype = q.stride(0), O_part.dtype
        blocks, block_size, _ = kv_cache.shape
        table, table_stride = block_table.shape, block_table.stride()
        m0 = tree_mask.stride(0) if tree else 0
    extra = (tree_mask.data_ptr(), m0 if T > 1 else (max_q_len + 63) // 64) if tree else ()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    call = getattr(_lib or lib(), where)
    _launch(where, device, call,
            q.data_ptr(), q0 if T > 1 else H * KV_DIM, kv_cache.data_ptr(),
            KV_FP8_E4M3 if fp8 else KV_BF16, kv_scale.data_ptr() if fp8 else None, blocks, block_size,
            block_table.data_ptr(), table[-1], table_stride[-2] if B > 1 else table[-1], 1 if local else 0,
            table_stride[0] if local else 0, shard_begin, shard_count, seq_lens.data_ptr(),
            query_start_loc.data_ptr(), B, T, H, max_seq_len, max_q_len, D, interleave, scale, *extra, window,
            num_sinks, O_part.data_ptr(), DTYPE_BF16 if o_dtype is _BF16 else DTYPE_F32,
            lse_part.data_ptr(), workspace.data_ptr() if ws_bytes else None, ws_bytes,
            None if dev_error is None else dev_error.data_ptr(), _stream_of(stream, device))


def _stream_context(stream, device):
    """`stream` as the current one, for work on tensors of `device`."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    return torch.cuda.stream(stream)


def _explain_select(tree_mask, q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, max_q_len,
                    kv_scale, shard_count, workspace, dev_error, tree):
    """What is wrong with a selecting decode's tensors, shapes before devices
    (as _decode_geometry), or (T, H, B, local, fp8, device) if nothing is."""
    if not isinstance(O_part, torch.Tensor) or O_part.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("O_part must be a bfloat16 or float32 tensor")
    fp8 = _cache_format(kv_cache, kv_scale)
    i32 = torch.int32
    args = [("kv_cache", kv_cache, kv_cache.dtype, True), ("q", q, torch.bfloat16, False),
            ("block_table", block_table, i32, False), ("seq_lens", seq_lens, i32, True),
            ("query_start_loc", query_start_loc, i32, True), ("O_part", O_part, O_part.dtype, True),
            ("lse_part", lse_part, torch.float32, True)]
    if tree:
        args.append(("tree_mask", tree_mask, torch.int64, False))
    if fp8:
        args.append(("kv_scale", kv_scale, torch.float32, True))
    if workspace is not None:
        args.append(("workspace", workspace, getattr(workspace, "dtype", None), True))
    if dev_error is not None:
        args.append(("dev_error", dev_error, i32, False))
    _types(args)
    if q.dim() != 3 or q.shape[2] != KV_DIM or q.stride(2) != 1 or (q.shape[1] > 1 and q.stride(1) != KV_DIM):
        raise ValueError("q must be [T, H, 576] with contiguous heads")
    T, H = q.shape[0], q.shape[1]
    local = block_table.dim() == 3
    if block_table.dim() not in (2, 3) or block_table.stride(-1) != 1 or (local and block_table.shape[0] != shard_count):
        raise ValueError("block_table must be [B, W] or [shard_count, B, W] with unit column stride")
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    if tuple(query_start_loc.shape) != (B + 1,) or block_table.shape[-2] != B:
        raise ValueError("seq_lens [B], query_start_loc [B + 1] and block_table [.., B, W] disagree on B")
    if tuple(O_part.shape) != (shard_count, T, H, LATENT_DIM) or tuple(lse_part.shape) != (shard_count, T, H):
        raise ValueError("O_part must be [D, T, H, 512] and lse_part [D, T, H]")
    words = (max_q_len + 63) // 64
    if tree and (tree_mask.dim() != 2 or tree_mask.shape[0] != T or tree_mask.shape[1] < words or
                 (tree_mask.shape[1] > 1 and tree_mask.stride(1) != 1)):
        raise ValueError("tree_mask must be [T, >= %d] words with unit column stride (see pack_tree_mask)" % words)
    if dev_error is not None and dev_error.numel() == 0:
        raise ValueError("dev_error must not be empty")
    return T, H, B, local, fp8, _placed(args)


_WINDOW, _TREE = "dcp_mla_decode_partial_window", "dcp_mla_decode_partial_tree"


def dcp_mla_decode_partial_window(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, *,
                                  D: int, interleave: int, scale: float, window: int, num_sinks: int = 0,
                                  max_seq_len: int, max_q_len: int, kv_scale: Optional[torch.Tensor] = None,
                                  shard_begin: int = 0, shard_count: Optional[int] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """The decode over a sliding window: each row sees the last ``window``
    tokens of its own context (0: all) and its first ``num_sinks``.  Other
    arguments as for dcp_mla_decode_partial_v2."""
    _decode_select(_WINDOW, None, q, kv_cache, block_table, seq_lens, query_start_loc, O_part,
                   lse_part, D, interleave, scale, window, num_sinks, max_seq_len, max_q_len, kv_scale, shard_begin,
                   shard_count, workspace, dev_error, stream)


def dcp_mla_decode_partial_tree(q, kv_cache, block_table, seq_lens, query_start_loc, tree_mask, O_part, lse_part, *,
                                D: int, interleave: int, scale: float, window: int = 0, num_sinks: int = 0,
                                max_seq_len: int, max_q_len: int, kv_scale: Optional[torch.Tensor] = None,
                                shard_begin: int = 0, shard_count: Optional[int] = None,
                                workspace: Optional[torch.Tensor] = None,
                                dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """The decode of trees of drafted tokens: a request's rows are its tree
    tokens (the last q_len positions of its context), and each sees the
    context before the tree and the rows k of its request whose bit k is set
    in its row of tree_mask (int64 words [T, >= max_q_len / 64], see
    pack_tree_mask).  window and num_sinks as for the window decode, over the
    row's own sequence.  Other arguments as for dcp_mla_decode_partial_v2."""
    _decode_select(_TREE, tree_mask, q, kv_cache, block_table, seq_lens, query_start_loc,
                   O_part, lse_part, D, interleave, scale, window, num_sinks, max_seq_len, max_q_len, kv_scale,
                   shard_begin, shard_count, workspace, dev_error, stream)


def dcp_mla_decode_partial_noalloc(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, *,
                                   D: int, interleave: int, scale: float, max_seq_len: int, max_q_len: int,
                                   dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """The decode for callers that cannot allocate device memory: same
    arguments and results as dcp_mla_decode_partial, but the split-KV scratch
    is a fixed 24 MiB array inside the library (shared by all calls, so calls
    that overlap on the GPU race; the first call on a device must precede
    any stream capture on it)."""
    B, T, H = _decode_geometry(q, kv_cache, block_table, seq_lens, query_start_loc, O_part, lse_part, D)
    _need_opt(dev_error, "dev_error", torch.int32)
    with _Range("dcp_mla_decode_partial_noalloc"):
        st = lib().dcp_mla_decode_partial_noalloc(
            _ptr(q), q.stride(0), _ptr(kv_cache), kv_cache.shape[0], kv_cache.shape[1], _ptr(block_table),
            block_table.shape[1], block_table.stride(0), _ptr(seq_lens), _ptr(query_start_loc), B, T, H,
            max_seq_len, max_q_len, D, interleave, scale, _ptr(O_part), _ptr(lse_part), _ptr(dev_error),
            _stream(stream))
    _check(st, "dcp_mla_decode_partial_noalloc")


def dcp_lse_combine(O_part, lse_part, seq_lens, query_start_loc, out, out_lse, *, stream=None) -> None:
    """O_part fp32 [D, T, H, 512], lse_part fp32 [D, T, H] -> out [T, H, 512]
    (bf16 or fp32, by out.dtype) and out_lse fp32 [T, H].  Shapes are checked
    (on any host) before devices: the kernel reads D*T*H*512 floats of O_part
    and indexes query_start_loc up to B."""
    part_dt = torch.bfloat16 if isinstance(O_part, torch.Tensor) and O_part.dtype == torch.bfloat16 else torch.float32
    args = (("O_part", O_part, part_dt), ("lse_part", lse_part, torch.float32),
            ("seq_lens", seq_lens, torch.int32), ("query_start_loc", query_start_loc, torch.int32),
            ("out_lse", out_lse, torch.float32))
    for name, t, dtype in args:
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor")
    if out.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif out.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    if lse_part.dim() != 3:
        raise ValueError("lse_part must be [D, T, H]")
    D, T, H = lse_part.shape
    if tuple(O_part.shape) != (D, T, H, LATENT_DIM):
        raise ValueError("O_part must be [D, T, H, 512] with lse_part [D, T, H]")
    if tuple(out.shape) != (T, H, LATENT_DIM) or tuple(out_lse.shape) != (T, H):
        raise ValueError("out must be [T, H, 512] and out_lse [T, H]")
    if seq_lens.dim() != 1 or query_start_loc.dim() != 1:
        raise ValueError("seq_lens and query_start_loc must be 1-D")
    B = seq_lens.shape[0]
    if query_start_loc.shape[0] != B + 1:
        raise ValueError("query_start_loc must have B + 1 = %d entries" % (B + 1))
    for name, t, dtype in args:
        _need(t, name, dtype, contiguous=name != "out_lse")
    _need(out, "out", out.dtype)
    if not (out_lse.is_contiguous() or out_lse.data_ptr() == lse_part.data_ptr()):
        raise ValueError("out_lse must be contiguous")
    if part_dt == torch.float32:
        with _Range("dcp_lse_combine"):
            st = lib().dcp_lse_combine(_ptr(O_part), _ptr(lse_part), _ptr(seq_lens), _ptr(query_start_loc), B, T,
                                       H, D, _ptr(out), dt, _ptr(out_lse), _stream(stream))
        _check(st, "dcp_lse_combine")
    else:
        with _Range("dcp_lse_combine_v2"):
            st = lib().dcp_lse_combine_v2(_ptr(O_part), DTYPE_BF16, _ptr(lse_part), _ptr(seq_lens),
                                          _ptr(query_start_loc), B, T, H, D, _ptr(out), dt, _ptr(out_lse),
                                          _stream(stream))
        _check(st, "dcp_lse_combine_v2")


def dcp_decode_concat_cache(ql_nope, q_pe, kv_c, k_pe, slot_mapping, q_out, kv_cache, *,
                            dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """ql_nope bf16 [T, H, 512], q_pe bf16 [T, H, 64] (any token/head strides,
    unit element stride), kv_c bf16 [T, 512], k_pe bf16 [T, 64] (row strides
    allowed), slot_mapping int64 [T]; writes q_out bf16 [T, H, 576] and the
    rows of kv_cache bf16 [num_blocks, block_size, 576] at the non-negative
    slots."""
    for name, t, dt, dims, last in (("ql_nope", ql_nope, torch.bfloat16, 3, LATENT_DIM),
                                    ("q_pe", q_pe, torch.bfloat16, 3, ROPE_DIM),
                                    ("kv_c", kv_c, torch.bfloat16, 2, LATENT_DIM),
                                    ("k_pe", k_pe, torch.bfloat16, 2, ROPE_DIM),
                                    ("q_out", q_out, torch.bfloat16, 3, KV_DIM)):
        if not isinstance(t, torch.Tensor) or t.dtype != dt:
            raise TypeError("%s must be a %s tensor" % (name, dt))
        if t.dim() != dims or t.shape[-1] != last or t.stride(-1) != 1:
            raise ValueError("%s must have %d dims, last of size %d with unit stride" % (name, dims, last))
    T, H = ql_nope.shape[0], ql_nope.shape[1]
    if tuple(q_pe.shape[:2]) != (T, H) or kv_c.shape[0] != T or k_pe.shape[0] != T:
        raise ValueError("ql_nope, q_pe, kv_c and k_pe disagree on T or H")
    if tuple(q_out.shape[:2]) != (T, H) or q_out.stride(1) != KV_DIM:
        raise ValueError("q_out must be [T, H, 576] with dense heads")
    if not isinstance(slot_mapping, torch.Tensor) or slot_mapping.dtype != torch.int64 or \
            tuple(slot_mapping.shape) != (T,):
        raise ValueError("slot_mapping must be an int64 [T] tensor")
    if not isinstance(kv_cache, torch.Tensor) or kv_cache.dtype != torch.bfloat16 or kv_cache.dim() != 3 or \
            kv_cache.shape[2] != KV_DIM:
        raise ValueError("kv_cache must be bf16 [num_blocks, block_size, 576]")
    for name, t in (("ql_nope", ql_nope), ("q_pe", q_pe), ("kv_c", kv_c), ("k_pe", k_pe), ("q_out", q_out)):
        _need(t, name, torch.bfloat16, contiguous=False)
    _need(slot_mapping, "slot_mapping", torch.int64)
    _need(kv_cache, "kv_cache", torch.bfloat16)
    _need_opt(dev_error, "dev_error", torch.int32)
    with _Range("dcp_decode_concat_cache"):
        st = lib().dcp_decode_concat_cache(
            _ptr(ql_nope), ql_nope.stride(0), ql_nope.stride(1), _ptr(q_pe), q_pe.stride(0), q_pe.stride(1),
            _ptr(kv_c), kv_c.stride(0), _ptr(k_pe), k_pe.stride(0), _ptr(slot_mapping), T, H, _ptr(q_out),
            q_out.stride(0), _ptr(kv_cache), kv_cache.shape[0] * kv_cache.shape[1], _ptr(dev_error),
            _stream(stream))
    _check(st, "dcp_decode_concat_cache")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # current_stream() without the object: 0.1 of 3 us


_BF16, _F32, _U8, _I32T, _I64T = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _rows_scaled(kv_scale, blocks: int, block_size: int, device: int) -> bool:
    return (kv_scale.dtype is _F32 and kv_scale.shape == (blocks, block_size) and kv_scale.get_device() == device
            and kv_scale.is_contiguous())


def _flag_word(dev_error, device: int) -> bool:
    return dev_error.dtype is _I32T and dev_error.get_device() == device and dev_error.numel() > 0


try:  # the calls under torch.cuda.nvtx, without its wrappers
    from torch._C import _nvtx as _raw_nvtx
    _push, _pop = _raw_nvtx.rangePushA, _raw_nvtx.rangePop
except Exception:  # pragma: no cover
    _push = _pop = None


def _launch(name: str, device: int, call, *args) -> None:
    """A library call with `device` as the current one (the library launches
    there), named by an NVTX range."""
    if _device_now() != device:
        with torch.cuda.device(device):
            _launch(name, device, call, *args)
        return
    if _push is not None:
        _push(name)
    try:
        st = call(*args)
    finally:
        if _pop is not None:
            _pop()
    if st:
        _check(st, name)


def _stream_of(stream, device: int):
    if stream is None:
        return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _types(args) -> None:
    """args: (name, tensor, dtype, contiguous).  The first half of a call's
    checks; _placed is the second, after the shapes."""
    for name, t, dtype, _ in args:
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _placed(args) -> int:
    """Every tensor on one CUDA device (its index is returned), contiguous
    where it must be."""
    device = args[0][1].get_device()
    for name, t, _, contiguous in args:
        if t.get_device() != device or device < 0:
            if t.get_device() < 0:
                raise ValueError("%s must be a CUDA tensor" % name)
            raise ValueError("%s is on cuda:%d, %s on cuda:%d" % (name, t.get_device(), args[0][0], device))
        if contiguous and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    return device


def _cache_format(kv_cache, kv_scale):
    """Check a paged cache [num_blocks, block_size, 576] (bf16, or uint8 FP8
    E4M3 codes with kv_scale fp32 [num_blocks, block_size]) and return
    whether it is FP8."""
    if not isinstance(kv_cache, torch.Tensor) or kv_cache.dtype not in (torch.bfloat16, torch.uint8):
        raise TypeError("kv_cache must be a bfloat16 or uint8 (FP8 E4M3 codes) tensor")
    if kv_cache.dim() != 3 or kv_cache.shape[2] != KV_DIM:
        raise ValueError("kv_cache must be [num_blocks, block_size, 576]")
    fp8 = kv_cache.dtype == torch.uint8
    if fp8:
        if not isinstance(kv_scale, torch.Tensor) or kv_scale.dtype != torch.float32:
            raise TypeError("an FP8 kv_cache needs kv_scale, a float32 tensor")
        if tuple(kv_scale.shape) != tuple(kv_cache.shape[:2]):
            raise ValueError("kv_scale must be [num_blocks, block_size]")
    elif kv_scale is not None:
        raise ValueError("kv_scale is given for a bf16 kv_cache")
    return fp8


def dcp_decode_concat_cache_v2(ql_nope, q_pe, kv_c, k_pe, slot_mapping, q_out, kv_cache, *,
                               kv_scale: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None,
                               stream=None) -> None:
    """The general form of dcp_decode_concat_cache: kv_cache bf16, or uint8 FP8
    E4M3 codes with kv_scale fp32 [num_blocks, block_size] (each written row
    gets its own power-of-two scale).  ql_nope, q_pe and q_out may all be None
    to write the cache alone."""
    query = ql_nope is not None or q_pe is not None or q_out is not None
    H, strides, q_stride = 0, (0, 0, 0, 0), 0
    try:
        T, latent = kv_c.shape
        blocks, block_size, row = kv_cache.shape
        c0, c1 = kv_c.stride()
        p0, p1 = k_pe.stride()
        device = kv_cache.get_device()
        fp8 = kv_cache.dtype is _U8
        good = (
            device >= 0 and (fp8 or kv_cache.dtype is _BF16) and row == KV_DIM and kv_cache.is_contiguous()
            and kv_c.dtype is _BF16 and kv_c.get_device() == device and latent == LATENT_DIM and c1 == 1
            and k_pe.dtype is _BF16 and k_pe.get_device() == device and k_pe.shape == (T, ROPE_DIM) and p1 == 1
            and slot_mapping.dtype is _I64T and slot_mapping.get_device() == device
            and slot_mapping.shape == (T,) and slot_mapping.is_contiguous()
            and (_rows_scaled(kv_scale, blocks, block_size, device) if fp8 else kv_scale is None)
            and (dev_error is None or _flag_word(dev_error, device)))
        if good and query:
            _, H, _ = ql_nope.shape
            n0, n1, n2 = ql_nope.stride()
            r0, r1, r2 = q_pe.stride()
            q_stride, o1, o2 = q_out.stride()
            strides = (n0, n1, r0, r1)
            good = (
                ql_nope.dtype is _BF16 and ql_nope.get_device() == device
                and ql_nope.shape == (T, H, LATENT_DIM) and n2 == r2 == o2 == 1 and H >= 1 and T > 0
                and q_pe.dtype is _BF16 and q_pe.get_device() == device and q_pe.shape == (T, H, ROPE_DIM)
                and q_out.dtype is _BF16 and q_out.get_device() == device and q_out.shape == (T, H, KV_DIM)
                and o1 == KV_DIM)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        T, H, fp8, device = _explain_write(ql_nope, q_pe, kv_c, k_pe, slot_mapping, q_out, kv_cache, kv_scale,
                                           dev_error, query)
        if query:
            strides = [t.stride(d) for t in (ql_nope, q_pe) for d in (0, 1)]
            q_stride = q_out.stride(0)
        c0, p0 = kv_c.stride(0), k_pe.stride(0)
        blocks, block_size, _ = kv_cache.shape
    if T == 0:
        return
    if T == 1:  # (the stride of a dimension of one element is never used)
        c0 = p0 = 0
        q_stride = H * KV_DIM
    if query and (T == 1 or H == 1):
        many, heads = int(T > 1), int(H > 1)
        strides = (strides[0] * many, strides[1] * heads, strides[2] * many, strides[3] * heads)
    call = (_lib or lib()).dcp_decode_concat_cache_v2
    _launch("dcp_decode_concat_cache_v2", device, call,
            ql_nope.data_ptr() if query else None, strides[0], strides[1], q_pe.data_ptr() if query else None,
            strides[2], strides[3], kv_c.data_ptr(), c0, k_pe.data_ptr(), p0, slot_mapping.data_ptr(), T, H,
            q_out.data_ptr() if query else None, q_stride, kv_cache.data_ptr(),
            KV_FP8_E4M3 if fp8 else KV_BF16, kv_scale.data_ptr() if fp8 else None, blocks * block_size,
            None if dev_error is None else dev_error.data_ptr(), _stream_of(stream, device))


def _explain_write(ql_nope, q_pe, kv_c, k_pe, slot_mapping, q_out, kv_cache, kv_scale, dev_error, query):
    """What is wrong with a cache write's tensors, or (T, H, fp8, device)."""
    bf16 = torch.bfloat16
    fp8 = _cache_format(kv_cache, kv_scale)
    args = [("kv_cache", kv_cache, kv_cache.dtype, True), ("kv_c", kv_c, bf16, False), ("k_pe", k_pe, bf16, False)]
    rows = [("kv_c", kv_c, 2, LATENT_DIM), ("k_pe", k_pe, 2, ROPE_DIM)]
    if query:
        args += [("ql_nope", ql_nope, bf16, False), ("q_pe", q_pe, bf16, False), ("q_out", q_out, bf16, False)]
        rows += [("ql_nope", ql_nope, 3, LATENT_DIM), ("q_pe", q_pe, 3, ROPE_DIM), ("q_out", q_out, 3, KV_DIM)]
    if fp8:
        args.append(("kv_scale", kv_scale, torch.float32, True))
    if dev_error is not None:
        args.append(("dev_error", dev_error, torch.int32, False))
    _types(args)
    for name, t, dims, last in rows:
        if t.dim() != dims or t.shape[-1] != last or t.stride(-1) != 1:
            raise ValueError("%s must have %d dims, last of size %d with unit stride" % (name, dims, last))
    T = kv_c.shape[0]
    H = ql_nope.shape[1] if query else 0
    if k_pe.shape[0] != T or (query and (tuple(ql_nope.shape[:2]) != (T, H) or tuple(q_pe.shape[:2]) != (T, H))):
        raise ValueError("ql_nope, q_pe, kv_c and k_pe disagree on T or H")
    if query and (H < 1 or tuple(q_out.shape[:2]) != (T, H) or (H > 1 and q_out.stride(1) != KV_DIM)):
        raise ValueError("q_out must be [T, H, 576] with dense heads")
    if not isinstance(slot_mapping, torch.Tensor) or slot_mapping.dtype != torch.int64 or \
            tuple(slot_mapping.shape) != (T,):
        raise ValueError("slot_mapping must be an int64 [T] tensor")
    args.append(("slot_mapping", slot_mapping, torch.int64, True))
    if dev_error is not None and dev_error.numel() == 0:
        raise ValueError("dev_error must not be empty")
    return T, H, fp8, _placed(args)


def dcp_latent_cache_read(kv_cache, block_table, cu_lens, out, *, seq_starts: Optional[torch.Tensor] = None,
                          kv_scale: Optional[torch.Tensor] = None, D: int = 1, interleave: int = 1,
                          shard_begin: int = 0, shard_count: Optional[int] = None,
                          dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Read context ranges back out of the paged cache (bf16, or uint8 FP8
    E4M3 codes with kv_scale): out bf16 or fp32 [N, 576] (rows may be strided)
    gets request b's positions seq_starts[b] + i in rows cu_lens[b] + i.
    block_table is [B, W] or per-shard [shard_count, B, W]; rows of positions
    that other shards own are zeros, rows past cu_lens[B] are left alone."""
    if shard_count is None:
        shard_count = D - shard_begin
    if D < 1 or D > MAX_SHARDS or shard_begin < 0 or shard_count < 1 or shard_begin + shard_count > D:
        raise ValueError("shards [shard_begin, shard_begin + shard_count) must lie in [0, D), D <= %d" % MAX_SHARDS)
    _fits32(interleave, "dcp_latent_cache_read")
    try:
        N, dim = out.shape
        out_stride, unit = out.stride()
        blocks, block_size, row = kv_cache.shape
        B = cu_lens.shape[0] - 1
        table, table_stride = block_table.shape, block_table.stride()
        local = len(table) == 3
        device = kv_cache.get_device()
        fp8, o_dtype = kv_cache.dtype is _U8, out.dtype
        good = (
            device >= 0 and (fp8 or kv_cache.dtype is _BF16) and row == dim == KV_DIM and kv_cache.is_contiguous()
            and (o_dtype is _BF16 or o_dtype is _F32) and out.get_device() == device and unit == 1
            and block_table.dtype is _I32T and block_table.get_device() == device and table_stride[-1] == 1
            and (table[0] == shard_count if local else len(table) == 2) and table[-2] == B
            and cu_lens.dtype is _I32T and cu_lens.get_device() == device and cu_lens.shape == (B + 1,)
            and cu_lens.is_contiguous()
            and (seq_starts is None or (seq_starts.dtype is _I32T and seq_starts.get_device() == device
                                        and seq_starts.shape == (B,) and seq_starts.is_contiguous()))
            and (_rows_scaled(kv_scale, blocks, block_size, device) if fp8 else kv_scale is None)
            and (dev_error is None or _flag_word(dev_error, device)))
    except (AttributeError, IndexError, TypeError, ValueError):
        good = False
    if not good:
        B, N, local, fp8, device = _explain_read(kv_cache, block_table, cu_lens, out, seq_starts, kv_scale,
                                                 shard_count, dev_error)
        out_stride, o_dtype = out.stride(0), out.dtype
        blocks, block_size, _ = kv_cache.shape
        table, table_stride = block_table.shape, block_table.stride()
    if B == 0 or N == 0:
        return
    call = (_lib or lib()).dcp_latent_cache_read
    _launch("dcp_latent_cache_read", device, call,
            kv_cache.data_ptr(), KV_FP8_E4M3 if fp8 else KV_BF16, kv_scale.data_ptr() if fp8 else None, blocks,
            block_size, block_table.data_ptr(), table[-1], table_stride[-2] if B > 1 else table[-1],
            1 if local else 0, table_stride[0] if local else 0, D, interleave, shard_begin, shard_count,
            None if seq_starts is None else seq_starts.data_ptr(), cu_lens.data_ptr(), B, N, out.data_ptr(),
            DTYPE_F32 if o_dtype is _F32 else DTYPE_BF16, out_stride if N > 1 else KV_DIM,
            None if dev_error is None else dev_error.data_ptr(), _stream_of(stream, device))


def _explain_read(kv_cache, block_table, cu_lens, out, seq_starts, kv_scale, shard_count, dev_error):
    """What is wrong with a cache read's tensors, or (B, N, local, fp8, device)."""
    fp8 = _cache_format(kv_cache, kv_scale)
    if not isinstance(out, torch.Tensor) or out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be a bfloat16 or float32 tensor")
    args = [("kv_cache", kv_cache, kv_cache.dtype, True), ("block_table", block_table, torch.int32, False),
            ("cu_lens", cu_lens, torch.int32, True), ("out", out, out.dtype, False)]
    if seq_starts is not None:
        args.append(("seq_starts", seq_starts, torch.int32, True))
    if fp8:
        args.append(("kv_scale", kv_scale, torch.float32, True))
    if dev_error is not None:
        args.append(("dev_error", dev_error, torch.int32, False))
    _types(args)
    if out.dim() != 2 or out.shape[1] != KV_DIM or out.stride(1) != 1:
        raise ValueError("out must be [N, 576] with unit column stride")
    if cu_lens.dim() != 1 or cu_lens.shape[0] < 1:
        raise ValueError("cu_lens must be [B + 1]")
    B, N = cu_lens.shape[0] - 1, out.shape[0]
    local = block_table.dim() == 3
    if block_table.dim() not in (2, 3) or block_table.stride(-1) != 1 or block_table.shape[-2] != B or \
            (local and block_table.shape[0] != shard_count):
        raise ValueError("block_table must be [B, W] or [shard_count, B, W] with unit column stride")
    if seq_starts is not None and tuple(seq_starts.shape) != (B,):
        raise ValueError("seq_starts must be [B]")
    if dev_error is not None and dev_error.numel() == 0:
        raise ValueError("dev_error must not be empty")
    return B, N, local, fp8, _placed(args)


def dcp_cache_extend(block_table, seq_lens, query_start_loc, free_blocks, free_count, free_left, positions,
                     slot_mapping, *, block_size: int, D: int = 1, interleave: int = 1, shard_begin: int = 0,
                     shard_count: Optional[int] = None, held: Optional[torch.Tensor] = None,
                     dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Build a step's block tables and slot map: block_table int32 [B, W] or
    per-shard [shard_count, B, W] (extended in place), free_blocks int32 [F],
    free_count and free_left int32 [1] (may be the same), positions int32 [T]
    and slot_mapping int64 [T] (written).  held int32 [B] or [shard_count, B]
    (updated; dcp_cache_extend_v2): how many blocks each table holds, for steps
    whose drafts may be rejected."""
    if shard_count is None:
        shard_count = D - shard_begin
    _fits32(D | interleave | block_size | shard_begin, "dcp_cache_extend")
    try:
        B, = seq_lens.shape
        T, = positions.shape
        num_free, = free_blocks.shape
        table, table_stride = block_table.shape, block_table.stride()
        local = len(table) == 3
        device = block_table.get_device()
        good = (
            device >= 0 and block_table.dtype is _I32T and (table_stride[-1] == 1 or table[-1] == 1)
            and (table[0] == shard_count if local else len(table) == 2) and table[-2] == B
            and seq_lens.dtype is _I32T and seq_lens.get_device() == device and seq_lens.is_contiguous()
            and query_start_loc.dtype is _I32T and query_start_loc.get_device() == device
            and query_start_loc.shape == (B + 1,) and query_start_loc.is_contiguous()
            and free_blocks.dtype is _I32T and free_blocks.get_device() == device and free_blocks.is_contiguous()
            and free_count.dtype is _I32T and free_count.get_device() == device and free_count.numel() == 1
            and free_left.dtype is _I32T and free_left.get_device() == device and free_left.numel() == 1
            and positions.dtype is _I32T and positions.get_device() == device and positions.is_contiguous()
            and slot_mapping.dtype is _I64T and slot_mapping.get_device() == device and slot_mapping.shape == (T,)
            and slot_mapping.is_contiguous()
            and (held is None or (held.dtype is _I32T and held.get_device() == device and held.is_contiguous()
                                  and held.shape == table[:-1]))
            and (dev_error is None or _flag_word(dev_error, device)))
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        B, T, local, device = _explain_extend(block_table, seq_lens, query_start_loc, free_blocks, free_count,
                                              free_left, positions, slot_mapping, shard_count, held, dev_error)
        num_free = free_blocks.shape[0]
        table, table_stride = block_table.shape, block_table.stride()
    call = (_lib or lib()).dcp_cache_extend_v2
    _launch("dcp_cache_extend", device, call,
            block_table.data_ptr(), table[-1], table_stride[-2] if B > 1 else table[-1], 1 if local else 0,
            table_stride[0] if local else 0, seq_lens.data_ptr(), query_start_loc.data_ptr(), B, T, block_size, D,
            interleave, shard_begin, shard_count, free_blocks.data_ptr(), num_free, free_count.data_ptr(),
            free_left.data_ptr(), None if held is None else held.data_ptr(), positions.data_ptr(),
            slot_mapping.data_ptr(),
            None if dev_error is None else dev_error.data_ptr(), _stream_of(stream, device))


def _explain_extend(block_table, seq_lens, query_start_loc, free_blocks, free_count, free_left, positions,
                    slot_mapping, shard_count, held, dev_error):
    """What is wrong with a table extension's tensors, or (B, T, local, device)."""
    i32 = torch.int32
    args = [("block_table", block_table, i32, False), ("seq_lens", seq_lens, i32, True),
            ("query_start_loc", query_start_loc, i32, True), ("free_blocks", free_blocks, i32, True),
            ("free_count", free_count, i32, False), ("free_left", free_left, i32, False),
            ("positions", positions, i32, True), ("slot_mapping", slot_mapping, torch.int64, True)]
    if held is not None:
        args.append(("held", held, i32, True))
    if dev_error is not None:
        args.append(("dev_error", dev_error, i32, False))
    _types(args)
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    local = block_table.dim() == 3
    if block_table.dim() not in (2, 3) or block_table.shape[-2] != B or \
            (block_table.shape[-1] > 1 and block_table.stride(-1) != 1) or (local and block_table.shape[0] != shard_count):
        raise ValueError("block_table must be [B, W] or [shard_count, B, W] with unit column stride")
    if tuple(query_start_loc.shape) != (B + 1,):
        raise ValueError("seq_lens [B] and query_start_loc [B + 1] disagree on B")
    if free_blocks.dim() != 1 or free_count.numel() != 1 or free_left.numel() != 1:
        raise ValueError("free_blocks must be [F], free_count and free_left [1]")
    if positions.dim() != 1 or tuple(slot_mapping.shape) != tuple(positions.shape):
        raise ValueError("positions and slot_mapping must be [T]")
    if held is not None and held.shape != block_table.shape[:-1]:
        raise ValueError("held must be [B] or [shard_count, B], as block_table is")
    if dev_error is not None and dev_error.numel() == 0:
        raise ValueError("dev_error must not be empty")
    return B, positions.shape[0], local, _placed(args)


def dcp_norm_rope_cache(ql_nope, q_pe, q_out, kv_c, k_pe, norm_weight, positions, cos_sin, slot_mapping, kv_cache, *,
                        eps: float = 1e-6, interleaved: bool = True, kv_scale: Optional[torch.Tensor] = None,
                        dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Norm of the latents, rotation of the rope parts and the cache write in
    one launch: kv_c bf16 [T, 512], k_pe bf16 [T, 64] (rows may be strided),
    norm_weight bf16 [512] or None, positions int32 [T], cos_sin fp32
    [max_pos, 64], slot_mapping int64 [T], kv_cache bf16 or FP8 with kv_scale.
    With ql_nope bf16 [T, H, 512] and q_pe [T, H, 64] the decode query goes to
    q_out [T, H, 576]; with q_pe alone its rotated form to q_out [T, H, 64]
    (any token and head strides; q_out may be q_pe)."""
    query, absorbed = q_pe is not None or q_out is not None or ql_nope is not None, ql_nope is not None
    H, strides = 0, (0, 0, 0, 0, 0, 0)
    try:
        T, latent = kv_c.shape
        blocks, block_size, row = kv_cache.shape
        max_pos, angles = cos_sin.shape
        c0, c1 = kv_c.stride()
        p0, p1 = k_pe.stride()
        device = kv_cache.get_device()
        fp8 = kv_cache.dtype is _U8
        good = (
            device >= 0 and (fp8 or kv_cache.dtype is _BF16) and row == KV_DIM and kv_cache.is_contiguous()
            and kv_c.dtype is _BF16 and kv_c.get_device() == device and latent == LATENT_DIM and c1 == 1
            and k_pe.dtype is _BF16 and k_pe.get_device() == device and k_pe.shape == (T, ROPE_DIM) and p1 == 1
            and slot_mapping.dtype is _I64T and slot_mapping.get_device() == device
            and slot_mapping.shape == (T,) and slot_mapping.is_contiguous()
            and positions.dtype is _I32T and positions.get_device() == device and positions.shape == (T,)
            and positions.is_contiguous() and cos_sin.dtype is _F32 and cos_sin.get_device() == device
            and angles == ROPE_DIM and cos_sin.is_contiguous()
            and (norm_weight is None or (norm_weight.dtype is _BF16 and norm_weight.get_device() == device
                                         and norm_weight.shape == (LATENT_DIM,) and norm_weight.is_contiguous()))
            and (_rows_scaled(kv_scale, blocks, block_size, device) if fp8 else kv_scale is None)
            and (dev_error is None or _flag_word(dev_error, device)))
        if good and query:
            _, H, _ = q_pe.shape
            r0, r1, r2 = q_pe.stride()
            o0, o1, o2 = q_out.stride()
            n0 = n1 = 0
            good = (
                q_pe.dtype is _BF16 and q_pe.get_device() == device and q_pe.shape == (T, H, ROPE_DIM) and r2 == o2 == 1
                and q_out.dtype is _BF16 and q_out.get_device() == device and H >= 1 and T > 0
                and q_out.shape == (T, H, KV_DIM if absorbed else ROPE_DIM))
            if good and absorbed:
                n0, n1, n2 = ql_nope.stride()
                good = (ql_nope.dtype is _BF16 and ql_nope.get_device() == device and n2 == 1
                        and ql_nope.shape == (T, H, LATENT_DIM))
            strides = (n0, n1, r0, r1, o0, o1)
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        T, H, fp8, device = _explain_norm_rope(ql_nope, q_pe, q_out, kv_c, k_pe, norm_weight, positions, cos_sin,
                                               slot_mapping, kv_cache, kv_scale, dev_error)
        if query:
            strides = [t.stride(d) if t is not None else 0 for t in (ql_nope, q_pe, q_out) for d in (0, 1)]
        c0, p0 = kv_c.stride(0), k_pe.stride(0)
        blocks, block_size, _ = kv_cache.shape
        max_pos = cos_sin.shape[0]
    _fits32(max_pos, "dcp_norm_rope_cache")
    if T == 0:
        return
    if T == 1:  # (the stride of a dimension of one element is never used)
        c0 = p0 = 0
    if query and (T == 1 or H == 1):
        many, heads = int(T > 1), int(H > 1)
        strides = [s * (heads if i % 2 else many) for i, s in enumerate(strides)]
    call = (_lib or lib()).dcp_norm_rope_cache
    _launch("dcp_norm_rope_cache", device, call,
            ql_nope.data_ptr() if absorbed else None, strides[0], strides[1], q_pe.data_ptr() if query else None,
            strides[2], strides[3], q_out.data_ptr() if query else None, strides[4], strides[5], kv_c.data_ptr(), c0,
            k_pe.data_ptr(), p0, None if norm_weight is None else norm_weight.data_ptr(), eps, positions.data_ptr(),
            cos_sin.data_ptr(), max_pos, 1 if interleaved else 0, slot_mapping.data_ptr(), T, H, kv_cache.data_ptr(),
            KV_FP8_E4M3 if fp8 else KV_BF16, kv_scale.data_ptr() if fp8 else None, blocks * block_size,
            None if dev_error is None else dev_error.data_ptr(), _stream_of(stream, device))


def _explain_norm_rope(ql_nope, q_pe, q_out, kv_c, k_pe, norm_weight, positions, cos_sin, slot_mapping, kv_cache,
                       kv_scale, dev_error):
    """What is wrong with a norm and rotation's tensors, or (T, H, fp8, device)."""
    bf16 = torch.bfloat16
    fp8 = _cache_format(kv_cache, kv_scale)
    args = [("kv_cache", kv_cache, kv_cache.dtype, True), ("kv_c", kv_c, bf16, False), ("k_pe", k_pe, bf16, False),
            ("positions", positions, torch.int32, True), ("cos_sin", cos_sin, torch.float32, True),
            ("slot_mapping", slot_mapping, torch.int64, True)]
    rows = [("kv_c", kv_c, 2, LATENT_DIM), ("k_pe", k_pe, 2, ROPE_DIM)]
    query = q_pe is not None or q_out is not None or ql_nope is not None
    if query:
        args += [("q_pe", q_pe, bf16, False), ("q_out", q_out, bf16, False)]
        rows += [("q_pe", q_pe, 3, ROPE_DIM), ("q_out", q_out, 3, ROPE_DIM if ql_nope is None else KV_DIM)]
        if ql_nope is not None:
            args.append(("ql_nope", ql_nope, bf16, False))
            rows.append(("ql_nope", ql_nope, 3, LATENT_DIM))
    if norm_weight is not None:
        args.append(("norm_weight", norm_weight, bf16, True))
    if fp8:
        args.append(("kv_scale", kv_scale, torch.float32, True))
    if dev_error is not None:
        args.append(("dev_error", dev_error, torch.int32, False))
    _types(args)
    for name, t, dims, last in rows:
        if t.dim() != dims or t.shape[-1] != last or t.stride(-1) != 1:
            raise ValueError("%s must have %d dims, last of size %d with unit stride" % (name, dims, last))
    T = kv_c.shape[0]
    H = q_pe.shape[1] if query else 0
    if k_pe.shape[0] != T or tuple(positions.shape) != (T,) or tuple(slot_mapping.shape) != (T,):
        raise ValueError("kv_c, k_pe, positions and slot_mapping disagree on T")
    if query and (H < 1 or tuple(q_pe.shape[:2]) != (T, H) or tuple(q_out.shape[:2]) != (T, H) or
                  (ql_nope is not None and tuple(ql_nope.shape[:2]) != (T, H))):
        raise ValueError("ql_nope, q_pe and q_out must be [T, H, ..] with H >= 1")
    if norm_weight is not None and tuple(norm_weight.shape) != (LATENT_DIM,):
        raise ValueError("norm_weight must be [512]")
    if cos_sin.dim() != 2 or cos_sin.shape[1] != ROPE_DIM or cos_sin.shape[0] < 1:
        raise ValueError("cos_sin must be [max_pos, 64]")
    if dev_error is not None and dev_error.numel() == 0:
        raise ValueError("dev_error must not be empty")
    return T, H, fp8, _placed(args)


def dcp_pack_kv_b(w_kv_b, packed, *, stream=None) -> None:
    """Lay out the up projection's weight bf16 [H * 256, 512] (a head's 128 key
    rows before its 128 value rows) for chunk attention: packed bf16
    [H, 8, 256, 64]."""
    _types([("w_kv_b", w_kv_b, torch.bfloat16, True), ("packed", packed, torch.bfloat16, True)])
    if w_kv_b.dim() != 2 or w_kv_b.shape[1] != LATENT_DIM or w_kv_b.shape[0] % (NOPE_DIM + VALUE_DIM) or not w_kv_b.shape[0]:
        raise ValueError("w_kv_b must be [H * 256, 512]")
    H = w_kv_b.shape[0] // (NOPE_DIM + VALUE_DIM)
    if tuple(packed.shape) != (H, 8, NOPE_DIM + VALUE_DIM, 64):
        raise ValueError("packed must be [H, 8, 256, 64]")
    device = _placed([("w_kv_b", w_kv_b, torch.bfloat16, True), ("packed", packed, torch.bfloat16, True)])
    _launch("dcp_pack_kv_b", device, lib().dcp_pack_kv_b, w_kv_b.data_ptr(), H, packed.data_ptr(),
            _stream_of(stream, device))


def dcp_chunk_attention_workspace_size(B: int, T: int, H: int, total_len: int) -> int:
    _fits32(B | T | H, "dcp_chunk_attention_workspace_size")
    n = (_lib or lib()).dcp_chunk_attention_workspace_size(B, T, H, min(max(total_len, -1), 1 << 62))
    if n == ctypes.c_size_t(-1).value:
        raise DCPError(1, "dcp_chunk_attention_workspace_size")
    return n


def dcp_mla_chunk_attention(q, kv_cache, block_table, seq_lens, query_start_loc, packed_kv_b, out, lse, workspace, *,
                            scale: float, total_len: int, kv_scale: Optional[torch.Tensor] = None, D: int = 1,
                            interleave: int = 1, dev_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Causal attention of chunks of new tokens over the paged latent cache:
    q bf16 [T, H, 192] (any token and head strides), kv_cache bf16 or FP8 with
    kv_scale, block_table int32 [B, W] or per-shard [D, B, W], packed_kv_b from
    dcp_pack_kv_b; writes out bf16 or fp32 [T, H, 128] and lse fp32 [T, H].
    total_len bounds the sum of seq_lens; workspace has
    dcp_chunk_attention_workspace_size bytes (fewer: more passes).  Without
    requests (B = 0) the rows are zeros and -inf, as other rows of no request."""
    _fits32(D | interleave, "dcp_mla_chunk_attention")
    try:
        T, H, dim = q.shape
        blocks, block_size, row = kv_cache.shape
        B, = seq_lens.shape
        q0, q1, q2 = q.stride()
        table, table_stride = block_table.shape, block_table.stride()
        local = len(table) == 3
        device = q.get_device()
        o_dtype, fp8 = out.dtype, kv_cache.dtype is _U8
        good = (
            q.dtype is _BF16 and dim == NOPE_DIM + ROPE_DIM and q2 == 1 and device >= 0
            and (fp8 or kv_cache.dtype is _BF16) and row == KV_DIM and kv_cache.get_device() == device
            and kv_cache.is_contiguous()
            and block_table.dtype is _I32T and block_table.get_device() == device and table_stride[-1] == 1
            and (table[0] == D if local else len(table) == 2) and table[-2] == B
            and seq_lens.dtype is _I32T and seq_lens.get_device() == device and seq_lens.is_contiguous()
            and query_start_loc.dtype is _I32T and query_start_loc.get_device() == device
            and query_start_loc.shape == (B + 1,) and query_start_loc.is_contiguous()
            and packed_kv_b.dtype is _BF16 and packed_kv_b.get_device() == device and packed_kv_b.is_contiguous()
            and packed_kv_b.shape == (H, 8, NOPE_DIM + VALUE_DIM, 64)
            and (o_dtype is _BF16 or o_dtype is _F32) and out.get_device() == device and out.is_contiguous()
            and out.shape == (T, H, VALUE_DIM)
            and lse.dtype is _F32 and lse.get_device() == device and lse.is_contiguous() and lse.shape == (T, H)
            and (_rows_scaled(kv_scale, blocks, block_size, device) if fp8 else kv_scale is None)
            and (workspace is None or (workspace.get_device() == device and workspace.is_contiguous()))
            and (dev_error is None or _flag_word(dev_error, device)))
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        T, H, B, local, fp8, device = _explain_chunk(q, kv_cache, block_table, seq_lens, query_start_loc, packed_kv_b,
                                                     out, lse, workspace, kv_scale, D, dev_error)
        q0, q1, o_dtype = q.stride(0), q.stride(1), out.dtype
        blocks, block_size, _ = kv_cache.shape
        table, table_stride = block_table.shape, block_table.stride()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    call = (_lib or lib()).dcp_mla_chunk_attention
    _launch("dcp_mla_chunk_attention", device, call,
            q.data_ptr(), q0 if T > 1 else 0, q1 if H > 1 else 0, kv_cache.data_ptr(),
            KV_FP8_E4M3 if fp8 else KV_BF16, kv_scale.data_ptr() if fp8 else None, blocks, block_size,
            block_table.data_ptr(), table[-1], table_stride[-2] if B > 1 else table[-1], 1 if local else 0,
            table_stride[0] if local else 0, D, interleave, seq_lens.data_ptr(), query_start_loc.data_ptr(), B, T, H,
            min(max(total_len, -1), 1 << 62), scale, packed_kv_b.data_ptr(), out.data_ptr(),
            DTYPE_BF16 if o_dtype is _BF16 else DTYPE_F32, lse.data_ptr(),
            workspace.data_ptr() if ws_bytes else None, ws_bytes,
            None if dev_error is None else dev_error.data_ptr(), _stream_of(stream, device))
    if B == 0 and T > 0:  # (the library's call does nothing then)
        with contextlib.nullcontext() if stream is None else _stream_context(stream, q.device):
            out.zero_()
            lse.fill_(-math.inf)


def _explain_chunk(q, kv_cache, block_table, seq_lens, query_start_loc, packed_kv_b, out, lse, workspace, kv_scale, D,
                   dev_error):
    """What is wrong with a chunk attention's tensors, or (T, H, B, local, fp8, device)."""
    if not isinstance(out, torch.Tensor) or out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be a bfloat16 or float32 tensor")
    fp8 = _cache_format(kv_cache, kv_scale)
    i32, bf16 = torch.int32, torch.bfloat16
    args = [("kv_cache", kv_cache, kv_cache.dtype, True), ("q", q, bf16, False),
            ("block_table", block_table, i32, False), ("seq_lens", seq_lens, i32, True),
            ("query_start_loc", query_start_loc, i32, True), ("packed_kv_b", packed_kv_b, bf16, True),
            ("out", out, out.dtype, True), ("lse", lse, torch.float32, True)]
    if fp8:
        args.append(("kv_scale", kv_scale, torch.float32, True))
    if workspace is not None:
        args.append(("workspace", workspace, getattr(workspace, "dtype", None), True))
    if dev_error is not None:
        args.append(("dev_error", dev_error, i32, False))
    _types(args)
    if q.dim() != 3 or q.shape[2] != NOPE_DIM + ROPE_DIM or q.stride(2) != 1:
        raise ValueError("q must be [T, H, 192] with unit stride in the last dim")
    T, H = q.shape[0], q.shape[1]
    local = block_table.dim() == 3
    if block_table.dim() not in (2, 3) or block_table.stride(-1) != 1 or (local and block_table.shape[0] != D):
        raise ValueError("block_table must be [B, W] or [D, B, W] with unit column stride")
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    if tuple(query_start_loc.shape) != (B + 1,) or block_table.shape[-2] != B:
        raise ValueError("seq_lens [B], query_start_loc [B + 1] and block_table [.., B, W] disagree on B")
    if tuple(packed_kv_b.shape) != (H, 8, NOPE_DIM + VALUE_DIM, 64):
        raise ValueError("packed_kv_b must be [H, 8, 256, 64] (see pack_kv_b)")
    if tuple(out.shape) != (T, H, VALUE_DIM) or tuple(lse.shape) != (T, H):
        raise ValueError("out must be [T, H, 128] and lse [T, H]")
    if dev_error is not None and dev_error.numel() == 0:
        raise ValueError("dev_error must not be empty")
    return T, H, B, local, fp8, _placed(args)


# ----------------------------------------------------------------------------
# allocating conveniences
# ----------------------------------------------------------------------------
def decode_workspace(B: int, T: int, H: int, D: int, max_seq_len: int, max_q_len: int,
                     device=None) -> Optional[torch.Tensor]:
    n = dcp_decode_workspace_size(B, T, H, D, max_seq_len, max_q_len)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def decode_partial(q, kv_cache, block_table, seq_lens, query_start_loc, D: int, interleave: int,
                   scale: float, max_seq_len: Optional[int] = None, max_q_len: Optional[int] = None,
                   dev_error: Optional[torch.Tensor] = None, stream=None, kv_scale: Optional[torch.Tensor] = None,
                   out_dtype=torch.float32):
    """Allocating form: returns (O_part fp32 [D, T, H, 512], lse_part fp32 [D, T, H]).
    A 3-D block_table [D, B, W] selects the per-shard layout
    (dcp_mla_decode_partial_local).

    ``max_seq_len``/``max_q_len`` default to the bounds implied by the table
    width and the row count (no device->host copy)."""
    T, H = q.shape[0], q.shape[1]
    B = seq_lens.shape[0]
    local = block_table.dim() == 3
    if max_seq_len is None:
        max_seq_len = block_table.shape[-1] * kv_cache.shape[1] * (D if local else 1)
    if max_q_len is None:
        max_q_len = max(1, T)
    O = torch.empty((D, T, H, LATENT_DIM), dtype=out_dtype, device=q.device)
    lse = torch.empty((D, T, H), dtype=torch.float32, device=q.device)
    ws = decode_workspace(B, T, H, D, max_seq_len, max_q_len, q.device)
    if kv_cache.dtype == torch.uint8 or out_dtype != torch.float32:
        dcp_mla_decode_partial_v2(q, kv_cache, block_table, seq_lens, query_start_loc, O, lse, D=D,
                                  interleave=interleave, scale=scale, max_seq_len=max_seq_len, max_q_len=max_q_len,
                                  kv_scale=kv_scale, workspace=ws, dev_error=dev_error, stream=stream)
        return O, lse
    entry = dcp_mla_decode_partial_local if local else dcp_mla_decode_partial
    entry(q, kv_cache, block_table, seq_lens, query_start_loc, O, lse, D=D, interleave=interleave, scale=scale,
          max_seq_len=max_seq_len, max_q_len=max_q_len, workspace=ws, dev_error=dev_error, stream=stream)
    return O, lse


def lse_combine(O_part, lse_part, seq_lens, query_start_loc, out_dtype=torch.bfloat16, stream=None):
    """Allocating form: returns (out [T, H, 512] of out_dtype, out_lse fp32 [T, H])."""
    D, T, H = lse_part.shape
    out = torch.empty((T, H, LATENT_DIM), dtype=out_dtype, device=O_part.device)
    out_lse = torch.empty((T, H), dtype=torch.float32, device=O_part.device)
    dcp_lse_combine(O_part, lse_part, seq_lens, query_start_loc, out, out_lse, stream=stream)
    return out, out_lse


def decode_concat_cache(ql_nope, q_pe, kv_c, k_pe, slot_mapping, kv_cache, dev_error=None, stream=None,
                        kv_scale: Optional[torch.Tensor] = None):
    """Allocating form: returns the decode query q bf16 [T, H, 576]; writes
    the step's latent rows into kv_cache in place (bf16, or FP8 E4M3 codes and
    their scales with kv_scale)."""
    if kv_scale is not None and stream is not None:  # (as in _decode_select_alloc)
        with _stream_context(stream, ql_nope.device):
            return decode_concat_cache(ql_nope, q_pe, kv_c, k_pe, slot_mapping, kv_cache, dev_error=dev_error,
                                       kv_scale=kv_scale)
    T, H = ql_nope.shape[0], ql_nope.shape[1]
    q = torch.empty((T, H, KV_DIM), dtype=torch.bfloat16, device=ql_nope.device)
    if kv_scale is not None:
        dcp_decode_concat_cache_v2(ql_nope, q_pe, kv_c, k_pe, slot_mapping, q, kv_cache, kv_scale=kv_scale,
                                   dev_error=dev_error)
        return q
    dcp_decode_concat_cache(ql_nope, q_pe, kv_c, k_pe, slot_mapping, q, kv_cache, dev_error=dev_error,
                            stream=stream)
    return q


def latent_cache_write(kv_c, k_pe, slot_mapping, kv_cache, kv_scale: Optional[torch.Tensor] = None, dev_error=None,
                       stream=None) -> None:
    """Write tokens' latent rows into the paged cache in place, without a
    query (a prefill's tokens): kv_cache bf16, or FP8 E4M3 codes with
    kv_scale."""
    dcp_decode_concat_cache_v2(None, None, kv_c, k_pe, slot_mapping, None, kv_cache, kv_scale=kv_scale,
                               dev_error=dev_error, stream=stream)


def latent_cache_read(kv_cache, block_table, cu_lens, num_rows: int, seq_starts: Optional[torch.Tensor] = None,
                      kv_scale: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, D: int = 1,
                      interleave: int = 1, shard_begin: int = 0, shard_count: Optional[int] = None, dev_error=None,
                      stream=None):
    """Allocating form: returns out [num_rows, 576] of out_dtype, num_rows =
    cu_lens[B] (known on the host; rows past cu_lens[B] are undefined)."""
    if stream is not None:  # (as in _decode_select_alloc)
        with _stream_context(stream, kv_cache.device):
            return latent_cache_read(kv_cache, block_table, cu_lens, num_rows, seq_starts=seq_starts,
                                     kv_scale=kv_scale, out_dtype=out_dtype, D=D, interleave=interleave,
                                     shard_begin=shard_begin, shard_count=shard_count, dev_error=dev_error)
    out = torch.empty((num_rows, KV_DIM), dtype=out_dtype, device=kv_cache.device)
    dcp_latent_cache_read(kv_cache, block_table, cu_lens, out, seq_starts=seq_starts, kv_scale=kv_scale, D=D,
                          interleave=interleave, shard_begin=shard_begin, shard_count=shard_count,
                          dev_error=dev_error, stream=stream)
    return out


def pack_tree_mask(visible: torch.Tensor) -> torch.Tensor:
    """Bool [T, n] (row r sees row k of its request) -> the int64 words
    [T, ceil(n / 64)] of the tree decode's mask, on the same device."""
    if visible.dtype != torch.bool or visible.dim() != 2:
        raise TypeError("visible must be a bool [T, n] tensor")
    T, n = visible.shape
    words = max(1, (n + 63) // 64)
    bits = torch.zeros((T, words * 64), dtype=torch.int64, device=visible.device)
    bits[:, :n] = visible.to(torch.int64)
    return (bits.view(T, words, 64) << torch.arange(64, device=visible.device)).sum(-1)


def _decode_select_alloc(where, tree_mask, q, kv_cache, block_table, seq_lens, query_start_loc, D, interleave, scale,
                         window, num_sinks, max_seq_len, max_q_len, kv_scale, out_dtype, workspace, dev_error, stream):
    if stream is not None:  # memory for work on another stream comes from that stream's pool
        with _stream_context(stream, q.device):
            return _decode_select_alloc(where, tree_mask, q, kv_cache, block_table, seq_lens, query_start_loc, D,
                                        interleave, scale, window, num_sinks, max_seq_len, max_q_len, kv_scale,
                                        out_dtype, workspace, dev_error, None)
    T, H = q.shape[0], q.shape[1]
    device = q.device
    if max_seq_len is None:
        max_seq_len = min(block_table.shape[-1] * kv_cache.shape[1] * (D if block_table.dim() == 3 else 1), 0x7fffffff)
    if max_q_len is None:
        max_q_len = max(1, T)
        if where is _TREE:
            max_q_len = max(1, min(T, 64 * tree_mask.shape[-1], MAX_TREE_ROWS))
    O = torch.empty((D, T, H, LATENT_DIM), dtype=out_dtype, device=device)
    lse = torch.empty((D, T, H), dtype=_F32, device=device)
    if workspace is None:
        sizes = seq_lens.shape[0], T, H, D, max_seq_len, max_q_len, window, num_sinks
        index = q.get_device()
        if index < 0 or _device_now() == index:
            n = dcp_decode_select_workspace_size(*sizes)
        else:  # (it goes by the clusters of the device that the call runs on)
            with torch.cuda.device(index):
                n = dcp_decode_select_workspace_size(*sizes)
        workspace = torch.empty(n, dtype=_U8, device=device) if n else None
    _decode_select(where, tree_mask, q, kv_cache, block_table, seq_lens, query_start_loc, O, lse, D, interleave, scale,
                   window, num_sinks, max_seq_len, max_q_len, kv_scale, 0, D, workspace, dev_error, None)
    return O, lse


def decode_partial_window(q, kv_cache, block_table, seq_lens, query_start_loc, D: int, interleave: int, scale: float,
                          window: int, num_sinks: int = 0, max_seq_len: Optional[int] = None,
                          max_q_len: Optional[int] = None, kv_scale: Optional[torch.Tensor] = None,
                          out_dtype=torch.float32, workspace: Optional[torch.Tensor] = None,
                          dev_error: Optional[torch.Tensor] = None, stream=None):
    """Allocating form of dcp_mla_decode_partial_window: returns (O_part
    [D, T, H, 512] of out_dtype, lse_part fp32 [D, T, H]); merge them with
    lse_combine.  max_seq_len and max_q_len default to the bounds that the
    table's width and the row count give; both size the launch, so pass the
    step's own."""
    return _decode_select_alloc(_WINDOW, None, q, kv_cache, block_table, seq_lens,
                                query_start_loc, D, interleave, scale, window, num_sinks, max_seq_len, max_q_len,
                                kv_scale, out_dtype, workspace, dev_error, stream)


def decode_partial_tree(q, kv_cache, block_table, seq_lens, query_start_loc, tree_mask, D: int, interleave: int,
                        scale: float, window: int = 0, num_sinks: int = 0, max_seq_len: Optional[int] = None,
                        max_q_len: Optional[int] = None, kv_scale: Optional[torch.Tensor] = None,
                        out_dtype=torch.float32, workspace: Optional[torch.Tensor] = None,
                        dev_error: Optional[torch.Tensor] = None, stream=None):
    """Allocating form of dcp_mla_decode_partial_tree: returns (O_part
    [D, T, H, 512] of out_dtype, lse_part fp32 [D, T, H]); merge them with
    lse_combine.  Defaults as for decode_partial_window; max_q_len's is also
    bounded by the bits of a mask row and by MAX_TREE_ROWS."""
    return _decode_select_alloc(_TREE, tree_mask, q, kv_cache, block_table, seq_lens,
                                query_start_loc, D, interleave, scale, window, num_sinks, max_seq_len, max_q_len,
                                kv_scale, out_dtype, workspace, dev_error, stream)


def cache_extend(block_table, seq_lens, query_start_loc, free_blocks, free_count, num_tokens: int, block_size: int,
                 free_left: Optional[torch.Tensor] = None, D: int = 1, interleave: int = 1, shard_begin: int = 0,
                 shard_count: Optional[int] = None, dev_error: Optional[torch.Tensor] = None, stream=None,
                 held: Optional[torch.Tensor] = None):
    """Allocating form of dcp_cache_extend: extends block_table in place, writes
    what is left of the free list into free_left (free_count itself by
    default) and returns (positions int32, slot_mapping int64) of the step's
    num_tokens rows.  Steps whose drafts may be rejected give held, int32 zeros
    of block_table's leading dims at first: the blocks that each table holds."""
    if stream is not None:  # (as in _decode_select_alloc)
        with _stream_context(stream, block_table.device):
            return cache_extend(block_table, seq_lens, query_start_loc, free_blocks, free_count, num_tokens,
                                block_size, free_left=free_left, D=D, interleave=interleave, shard_begin=shard_begin,
                                shard_count=shard_count, dev_error=dev_error, held=held)
    positions = torch.empty(num_tokens, dtype=_I32T, device=block_table.device)
    slots = torch.empty(num_tokens, dtype=_I64T, device=block_table.device)
    dcp_cache_extend(block_table, seq_lens, query_start_loc, free_blocks, free_count,
                     free_count if free_left is None else free_left, positions, slots, block_size=block_size, D=D,
                     interleave=interleave, shard_begin=shard_begin, shard_count=shard_count, held=held,
                     dev_error=dev_error)
    return positions, slots


def norm_rope_cache(kv_c, k_pe, slot_mapping, kv_cache, positions, cos_sin,
                    norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    ql_nope: Optional[torch.Tensor] = None, q_pe: Optional[torch.Tensor] = None,
                    q_out: Optional[torch.Tensor] = None, interleaved: bool = True,
                    kv_scale: Optional[torch.Tensor] = None, dev_error: Optional[torch.Tensor] = None, stream=None):
    """Allocating form of dcp_norm_rope_cache: writes the normed and rotated
    latent rows into kv_cache in place and returns the query: the decode's
    [T, H, 576] with ql_nope and q_pe, the rotated rope parts [T, H, 64] with
    q_pe alone (in q_out where it is given), None without."""
    if stream is not None:  # (as in _decode_select_alloc)
        with _stream_context(stream, kv_cache.device):
            return norm_rope_cache(kv_c, k_pe, slot_mapping, kv_cache, positions, cos_sin, norm_weight=norm_weight,
                                   eps=eps, ql_nope=ql_nope, q_pe=q_pe, q_out=q_out, interleaved=interleaved,
                                   kv_scale=kv_scale, dev_error=dev_error)
    if q_out is None and q_pe is not None:
        q_out = torch.empty((q_pe.shape[0], q_pe.shape[1], ROPE_DIM if ql_nope is None else KV_DIM), dtype=_BF16,
                            device=q_pe.device)
    dcp_norm_rope_cache(ql_nope, q_pe, q_out, kv_c, k_pe, norm_weight, positions, cos_sin, slot_mapping, kv_cache,
                        eps=eps, interleaved=interleaved, kv_scale=kv_scale, dev_error=dev_error)
    return q_out


def pack_kv_b(w_kv_b, num_heads: Optional[int] = None, stream=None):
    """Allocating form of dcp_pack_kv_b: the up projection's weight bf16
    [H * 256, 512] as chunk_attention takes it, laid out once per layer."""
    if stream is not None:  # (as in _decode_select_alloc)
        with _stream_context(stream, w_kv_b.device):
            return pack_kv_b(w_kv_b, num_heads)
    H = w_kv_b.shape[0] // (NOPE_DIM + VALUE_DIM)
    if num_heads is not None and num_heads * (NOPE_DIM + VALUE_DIM) != w_kv_b.shape[0]:
        raise ValueError("w_kv_b has %d rows, not 256 for each of %d heads" % (w_kv_b.shape[0], num_heads))
    packed = torch.empty((H, 8, NOPE_DIM + VALUE_DIM, 64), dtype=torch.bfloat16, device=w_kv_b.device)
    dcp_pack_kv_b(w_kv_b, packed)
    return packed


def chunk_attention(q, kv_cache, block_table, seq_lens, query_start_loc, packed_kv_b, scale: float, total_len: int,
                    kv_scale: Optional[torch.Tensor] = None, D: int = 1, interleave: int = 1,
                    out_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                    dev_error: Optional[torch.Tensor] = None, stream=None):
    """Allocating form of dcp_mla_chunk_attention: returns (out [T, H, 128] of
    out_dtype, lse fp32 [T, H])."""
    if stream is not None:  # (as in _decode_select_alloc)
        with _stream_context(stream, q.device):
            return chunk_attention(q, kv_cache, block_table, seq_lens, query_start_loc, packed_kv_b, scale, total_len,
                                   kv_scale=kv_scale, D=D, interleave=interleave, out_dtype=out_dtype,
                                   workspace=workspace, dev_error=dev_error)
    T, H = q.shape[0], q.shape[1]
    out = torch.empty((T, H, VALUE_DIM), dtype=out_dtype, device=q.device)
    lse = torch.empty((T, H), dtype=_F32, device=q.device)
    if workspace is None:
        sizes, index = (seq_lens.shape[0], T, H, total_len), q.get_device()
        if index < 0 or _device_now() == index:
            n = dcp_chunk_attention_workspace_size(*sizes)
        else:  # (it goes by the SMs of the device that the call runs on)
            with torch.cuda.device(index):
                n = dcp_chunk_attention_workspace_size(*sizes)
        workspace = torch.empty(n, dtype=_U8, device=q.device) if n else None
    dcp_mla_chunk_attention(q, kv_cache, block_table, seq_lens, query_start_loc, packed_kv_b, out, lse, workspace,
                            scale=scale, total_len=total_len, kv_scale=kv_scale, D=D, interleave=interleave,
                            dev_error=dev_error)
    return out, lse
