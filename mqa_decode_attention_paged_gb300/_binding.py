"""ctypes binding of ``libmqa_decode.so`` (the C ABI declared in include/mqa_decode.h).

Argument marshalling only: every step of the decode runs in the library's
CUDA kernels.  torch supplies device memory and the current stream.  When the
shared library is missing this module raises at import time instead of falling
back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_WORKSPACE_TOO_SMALL = 3
ERR_CUDA = 4
ERR_DEVICE_CHECK = 5
ERR_DEVICE_TIMEOUT = 6

KV_BF16 = 0
KV_FP8_E4M3 = 1
KV_FP8_E4M3_PER_TOKEN_HEAD = 2
KV_INT8_PER_TOKEN_HEAD = 3
KV_INT4_PER_TOKEN_HEAD = 4
KV_FP8_E4M3_BLOCK = 5
KV_INT8_BLOCK = 6
_KV_NAMES = {"bf16": KV_BF16, "fp8_e4m3": KV_FP8_E4M3, "fp8_e4m3_pth": KV_FP8_E4M3_PER_TOKEN_HEAD,
             "int8_pth": KV_INT8_PER_TOKEN_HEAD, "int4_pth": KV_INT4_PER_TOKEN_HEAD,
             "fp8_e4m3_block": KV_FP8_E4M3_BLOCK, "int8_block": KV_INT8_BLOCK}

LIB_PATH = _build.LIB_PATH


class MqaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = int(code)
        msg = f"{where}: {status_string(code)} (status {code})"
        if self.code == ERR_CUDA:
            msg += f": {lib.mqa_last_cuda_error_string().decode()}"
        super().__init__(msg)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first with `python -m mqa_decode_attention_paged_gb300.build` "
            "(requires nvcc); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.mqa_abi_version.restype = I
    lib.mqa_abi_version.argtypes = []
    lib.mqa_status_string.restype = ctypes.c_char_p
    lib.mqa_status_string.argtypes = [I]
    lib.mqa_device_sm_count.restype = I
    lib.mqa_device_sm_count.argtypes = []
    lib.mqa_last_cuda_error.restype = I
    lib.mqa_last_cuda_error.argtypes = []
    lib.mqa_last_cuda_error_string.restype = ctypes.c_char_p
    lib.mqa_last_cuda_error_string.argtypes = []
    lib.mqa_num_kv_splits.restype = I
    lib.mqa_num_kv_splits.argtypes = [I, I, I]
    lib.mla_decode_workspace_bytes.restype = SZ
    lib.mla_decode_workspace_bytes.argtypes = [I, I, I, I]
    lib.gqa_paged_decode_workspace_bytes.restype = SZ
    lib.gqa_paged_decode_workspace_bytes.argtypes = [I, I, I, I]
    lib.mla_decode.restype = I
    lib.mla_decode.argtypes = [P, P, P, P, F, F, P, P, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.mla_decode_fixed_splits.restype = I
    lib.mla_decode_fixed_splits.argtypes = [P, P, P, P, F, F, P, P, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.mla_decode_multi.restype = I
    lib.mla_decode_multi.argtypes = [P, P, P, P, F, F, P, P, I, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.mla_decode_sparse.restype = I
    lib.mla_decode_sparse.argtypes = [P, P, P, P, P, F, F, P, P, I, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.mla_decode_noalloc.restype = I
    lib.mla_decode_noalloc.argtypes = [P, P, P, P, F, F, P, P, I, I, I, I, I, I, I, I, I, P, P]
    lib.gqa_paged_decode.restype = I
    lib.gqa_paged_decode.argtypes = [P, P, P, P, F, F, F, P, P, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    LL = ctypes.c_longlong
    lib.gqa_window_decode_workspace_bytes.restype = SZ
    lib.gqa_window_decode_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.gqa_window_num_kv_splits.restype = I
    lib.gqa_window_num_kv_splits.argtypes = [I, I, I, I]
    lib.gqa_window_decode.restype = I
    lib.gqa_window_decode.argtypes = [P, P, P, P, P, F, F, F, I, I, P, P, I, I, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.gqa_block_decode.restype = I
    lib.gqa_block_decode.argtypes = [P, P, P, P, P, F, P, P, I, I, I, I, I, I, I, I, I, I, I, P, SZ, P, P]
    lib.gqa_rope_append.restype = I
    lib.gqa_rope_append.argtypes = [P, P, P, P, P, P, P, P, P, P, F, F, I, I, I, I, I, I, I, I, I, I, I, I, I, LL, LL,
                                    LL, LL, P, P]
    lib.mla_rope_append.restype = I
    lib.mla_rope_append.argtypes = [P, P, P, P, P, P, P, P, P, F, I, I, I, I, I, I, I, I, I, I, I, LL, LL, LL, LL, LL,
                                    LL, P, P]
    lib.mqa_lse_merge.restype = I
    lib.mqa_lse_merge.argtypes = [P, P, P, P, I, ctypes.c_longlong, I, P]
    lib.mqa_dcp_shard_max_blocks.restype = I
    lib.mqa_dcp_shard_max_blocks.argtypes = [I, I]
    lib.mqa_dcp_shard.restype = I
    lib.mqa_dcp_shard.argtypes = [P, P, I, I, I, I, I, I, P, I, P]
    lib.mqa_dcp_locate.restype = I
    lib.mqa_dcp_locate.argtypes = [I, I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
    lib.mqa_dcp_scale_shard.restype = I
    lib.mqa_dcp_scale_shard.argtypes = [P, P, P, P, I, I, I, I, I, I, P]
    return lib


lib = _load()


def abi_version() -> int:
    return int(lib.mqa_abi_version())


def status_string(code: int) -> str:
    return lib.mqa_status_string(int(code)).decode()


def device_sm_count() -> int:
    return int(lib.mqa_device_sm_count())


def num_kv_splits(max_seq_len: int, sm_count: int, batch_invariant: bool = False) -> int:
    return int(lib.mqa_num_kv_splits(int(max_seq_len), int(sm_count), int(bool(batch_invariant))))


def mla_decode_workspace_bytes(batch: int, num_heads: int, kv_lora_rank: int, num_kv_splits: int) -> int:
    return int(lib.mla_decode_workspace_bytes(batch, num_heads, kv_lora_rank, num_kv_splits))


def gqa_paged_decode_workspace_bytes(batch: int, num_q_heads: int, head_size: int, num_kv_splits: int) -> int:
    return int(lib.gqa_paged_decode_workspace_bytes(batch, num_q_heads, head_size, num_kv_splits))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(t, name, dtypes=None, shape=None, optional=False, elt=None):
    """Validate the layout of a tensor argument before its pointer is handed to
    the C ABI: dtype (or element size), shape and contiguity.  The library
    reads raw pointers, so a wrong layout would otherwise be read as garbage."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if elt is not None and t.element_size() != elt:
        raise TypeError(f"{name} must have {elt}-byte elements, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(named):
    """Every given tensor must live on the CUDA device of the first."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the call runs on {dev}")


def _check_common(q, kv_cache, code, block_table, seq_lens, out, out_shape, lse, lse_shape, workspace,
                  device_status, extra=()):
    _check(q, "q", (torch.bfloat16,))
    _check(kv_cache, "kv_cache", elt=2 if code == KV_BF16 else 1)
    _check(block_table, "block_table", (torch.int32,))
    if block_table.dim() != 2 or block_table.shape[0] != out_shape[0]:
        raise ValueError("block_table must be int32 [batch, max_blocks]")
    _check(seq_lens, "seq_lens", (torch.int32,), shape=(out_shape[0],))
    _check(out, "out", (torch.bfloat16,), shape=out_shape)
    _check(lse, "lse", (torch.float32,), shape=lse_shape, optional=True)
    _check(workspace, "workspace", optional=True)
    _check(device_status, "device_status", (torch.int32,), optional=True)
    _on_device([("q", q), ("kv_cache", kv_cache), ("block_table", block_table), ("seq_lens", seq_lens),
                ("out", out), ("lse", lse), ("workspace", workspace), ("device_status", device_status),
                *extra])


def _kv_code(kv_cache, kv_dtype):
    if kv_dtype is not None:
        return _KV_NAMES[kv_dtype] if isinstance(kv_dtype, str) else int(kv_dtype)
    if kv_cache.dtype == torch.bfloat16:
        return KV_BF16
    if kv_cache.dtype == torch.float8_e4m3fn:
        return KV_FP8_E4M3
    raise TypeError("kv_cache must be bf16 or float8_e4m3fn (or pass kv_dtype with uint8 storage)")


def mla_decode(q, kv_cache, block_table, seq_lens, scale, k_scale=1.0, *, out=None, lse=None,
               num_kv_splits=1, workspace=None, kv_lora_rank=None, kv_dtype=None,
               device_status=None, stream=None, return_lse=True):
    """MLA decode through the C ABI.  q [B,H,D] bf16, kv_cache [num_blocks, page, D],
    block_table [B, max_blocks] int32, seq_lens [B] int32 (all on one CUDA device).
    Allocates out / lse / workspace with torch when they are not given."""
    return _mla_decode(lib.mla_decode, "mla_decode", q, kv_cache, block_table, seq_lens, scale, k_scale, out,
                       lse, num_kv_splits, workspace, kv_lora_rank, kv_dtype, device_status, stream, return_lse)


def mla_decode_fixed_splits(q, kv_cache, block_table, seq_lens, scale, k_scale=1.0, *, out=None, lse=None,
                            num_kv_splits=1, workspace=None, kv_lora_rank=None, kv_dtype=None,
                            device_status=None, stream=None, return_lse=True):
    """``mla_decode`` with one work unit per (request, split): every request
    cut into num_kv_splits equal page ranges (batch-invariant at any split
    count).  Same arguments and results as :func:`mla_decode`."""
    return _mla_decode(lib.mla_decode_fixed_splits, "mla_decode_fixed_splits", q, kv_cache, block_table,
                       seq_lens, scale, k_scale, out, lse, num_kv_splits, workspace, kv_lora_rank, kv_dtype,
                       device_status, stream, return_lse)


def _mla_decode(fn, name, q, kv_cache, block_table, seq_lens, scale, k_scale, out, lse, num_kv_splits, workspace,
                kv_lora_rank, kv_dtype, device_status, stream, return_lse):
    B, H, D = q.shape
    nb, page, D2 = kv_cache.shape
    if D2 != D:
        raise ValueError("q and kv_cache head sizes differ")
    R = (D - 64) if kv_lora_rank is None else int(kv_lora_rank)
    code = _kv_code(kv_cache, kv_dtype)
    if out is None:
        out = torch.empty((B, H, R), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    need = mla_decode_workspace_bytes(B, H, R, num_kv_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check_common(q, kv_cache, code, block_table, seq_lens, out, (B, H, R), lse, (B, H), workspace,
                  device_status)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = fn(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), float(scale), float(k_scale), _ptr(out),
            _ptr(lse), B, H, D, R, nb, page, block_table.shape[1], code, int(num_kv_splits), _ptr(workspace),
            ws_bytes, _ptr(device_status), _stream(stream))
    if rc != OK:
        raise MqaError(rc, name)
    return out, lse


def mla_decode_multi(q, kv_cache, block_table, seq_lens, scale, k_scale=1.0, *, out=None, lse=None,
                     num_kv_splits=1, workspace=None, kv_lora_rank=None, kv_dtype=None,
                     device_status=None, stream=None, return_lse=True):
    """Multi-token MLA decode through the C ABI.  q [B, q_len, H, D] bf16 (query i of
    request b sits at position seq_lens[b] - q_len + i and sees the keys up to it);
    returns out [B, q_len, H, R] bf16 and lse [B, q_len, H] fp32."""
    B, Lq, H, D = q.shape
    nb, page, D2 = kv_cache.shape
    if D2 != D:
        raise ValueError("q and kv_cache head sizes differ")
    R = (D - 64) if kv_lora_rank is None else int(kv_lora_rank)
    code = _kv_code(kv_cache, kv_dtype)
    if out is None:
        out = torch.empty((B, Lq, H, R), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Lq, H), dtype=torch.float32, device=q.device)
    need = mla_decode_workspace_bytes(B, Lq * H, R, num_kv_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check_common(q, kv_cache, code, block_table, seq_lens, out, (B, Lq, H, R), lse, (B, Lq, H), workspace,
                  device_status)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mla_decode_multi(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), float(scale),
                              float(k_scale), _ptr(out), _ptr(lse), B, Lq, H, D, R, nb, page,
                              block_table.shape[1], code, int(num_kv_splits), _ptr(workspace), ws_bytes,
                              _ptr(device_status), _stream(stream))
    if rc != OK:
        raise MqaError(rc, "mla_decode_multi")
    return out, lse


def mla_decode_sparse(q, kv_cache, block_table, seq_lens, indices, scale, k_scale=1.0, *, out=None,
                      lse=None, num_kv_splits=1, workspace=None, kv_lora_rank=None, kv_dtype=None,
                      device_status=None, stream=None, return_lse=True):
    """Sparse (top-k) MLA decode through the C ABI.  q [B, H, D] bf16, indices [B, topk]
    int32 logical positions (entries outside [0, seq_lens[b]) select nothing); returns
    out [B, H, R] bf16 and lse [B, H] fp32."""
    B, H, D = q.shape
    nb, page, D2 = kv_cache.shape
    if D2 != D:
        raise ValueError("q and kv_cache head sizes differ")
    if indices.dim() != 2 or indices.shape[0] != B or indices.dtype != torch.int32:
        raise ValueError("indices must be int32 [batch, topk]")
    topk = indices.shape[1]
    R = (D - 64) if kv_lora_rank is None else int(kv_lora_rank)
    code = _kv_code(kv_cache, kv_dtype)
    if out is None:
        out = torch.empty((B, H, R), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    need = mla_decode_workspace_bytes(B, H, R, num_kv_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check(indices, "indices", (torch.int32,))
    _check_common(q, kv_cache, code, block_table, seq_lens, out, (B, H, R), lse, (B, H), workspace,
                  device_status, extra=[("indices", indices)])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.mla_decode_sparse(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), _ptr(indices),
                               float(scale), float(k_scale), _ptr(out), _ptr(lse), B, H, D, R, nb, page,
                               block_table.shape[1], topk, code, int(num_kv_splits), _ptr(workspace),
                               ws_bytes, _ptr(device_status), _stream(stream))
    if rc != OK:
        raise MqaError(rc, "mla_decode_sparse")
    return out, lse


def gqa_paged_decode(q, kv_cache, block_table, seq_lens, scale, k_scale=1.0, v_scale=1.0, *,
                     out=None, lse=None, num_kv_splits=1, workspace=None, kv_dtype=None,
                     device_status=None, stream=None, return_lse=True):
    """GQA paged decode through the C ABI.  q [B,Hq,D] bf16; kv_cache
    [num_blocks, 2, page, Hkv, D] bf16 or e4m3 (k_scale / v_scale), or, with
    kv_dtype "fp8_e4m3_pth" / "int8_pth", uint8 [num_blocks, 2, page, Hkv,
    D + 4] rows of D codes followed by their fp32 scale, or "int4_pth", uint8
    [..., D / 2 + 4] rows of packed 4-bit codes followed by the scale."""
    B, Hq, D = q.shape
    nb, two, page, Hkv, D2 = kv_cache.shape
    code = _kv_code(kv_cache, kv_dtype)
    row = {KV_FP8_E4M3_PER_TOKEN_HEAD: D + 4, KV_INT8_PER_TOKEN_HEAD: D + 4,
           KV_INT4_PER_TOKEN_HEAD: D // 2 + 4}.get(code, D)
    if two != 2 or D2 != row:
        raise ValueError(f"kv_cache must be [num_blocks, 2, page, num_kv_heads, {row}]")
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = gqa_paged_decode_workspace_bytes(B, Hq, D, num_kv_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check_common(q, kv_cache, code, block_table, seq_lens, out, (B, Hq, D), lse, (B, Hq), workspace,
                  device_status)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.gqa_paged_decode(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
                              float(scale), float(k_scale), float(v_scale), _ptr(out), _ptr(lse),
                              B, Hq, Hkv, D, nb, page, block_table.shape[1], code,
                              int(num_kv_splits), _ptr(workspace), ws_bytes, _ptr(device_status),
                              _stream(stream))
    if rc != OK:
        raise MqaError(rc, "gqa_paged_decode")
    return out, lse


def lse_merge(shard_out, shard_lse, *, out=None, lse=None, stream=None, return_lse=True):
    """Merge sequence-shard results through the C ABI (decode context
    parallelism, after the caller has gathered the shards): shard_out bf16
    [G, ..., head_dim], shard_lse fp32 [G, ...]; returns (out [..., head_dim]
    bf16, lse [...] fp32)."""
    G = shard_out.shape[0]
    D = shard_out.shape[-1]
    lead = tuple(shard_out.shape[1:-1])
    if tuple(shard_lse.shape) != (G,) + lead:
        raise ValueError("shard_lse must be [num_shards, *shard_out.shape[1:-1]]")
    rows = 1
    for x in lead:
        rows *= int(x)
    if out is None:
        out = torch.empty(lead + (D,), dtype=torch.bfloat16, device=shard_out.device)
    if lse is None and return_lse:
        lse = torch.empty(lead, dtype=torch.float32, device=shard_out.device)
    _check(shard_out, "shard_out", (torch.bfloat16,))
    _check(shard_lse, "shard_lse", (torch.float32,))
    _check(out, "out", (torch.bfloat16,), shape=lead + (D,))
    _check(lse, "lse", (torch.float32,), shape=lead, optional=True)
    _on_device([("shard_out", shard_out), ("shard_lse", shard_lse), ("out", out), ("lse", lse)])
    rc = lib.mqa_lse_merge(_ptr(shard_out), _ptr(shard_lse), _ptr(out), _ptr(lse), int(G), rows, int(D),
                           _stream(stream))
    if rc != OK:
        raise MqaError(rc, "mqa_lse_merge")
    return out, lse


DCP_LAYOUTS = {"round_robin": 0, "contiguous": 1}


def _dcp_layout(layout):
    if layout not in DCP_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(DCP_LAYOUTS)}, got {layout!r}")
    return DCP_LAYOUTS[layout]


def dcp_shard_max_blocks(max_blocks: int, num_ranks: int) -> int:
    n = int(lib.mqa_dcp_shard_max_blocks(int(max_blocks), int(num_ranks)))
    if n < 0:
        raise ValueError("max_blocks and num_ranks must be >= 1")
    return n


def dcp_shard(block_table, seq_lens, page_size, num_ranks, rank, layout="round_robin"):
    """Pages of rank `rank` of `num_ranks` under decode context parallelism
    (host arrays, C ABI ``mqa_dcp_shard``): block_table int32 [B, max_blocks]
    and seq_lens int32 [B] (numpy or CPU tensors) give the whole sequences;
    returns numpy (shard_block_table int32 [B, ceil(max_blocks / num_ranks)],
    shard_seq_lens int32 [B]) for the decode entry points."""
    import numpy as np
    bt = np.ascontiguousarray(np.asarray(block_table), dtype=np.int32)
    sl = np.ascontiguousarray(np.asarray(seq_lens), dtype=np.int32)
    if bt.ndim != 2 or sl.shape != (bt.shape[0],):
        raise ValueError("block_table must be [B, max_blocks] and seq_lens [B]")
    B, mb = bt.shape
    width = dcp_shard_max_blocks(mb, num_ranks)
    table = np.empty((B, width), dtype=np.int32)
    lens = np.empty(B, dtype=np.int32)
    rc = lib.mqa_dcp_shard(bt.ctypes.data, sl.ctypes.data, B, mb, int(page_size), int(num_ranks), int(rank),
                           _dcp_layout(layout), table.ctypes.data, width, lens.ctypes.data)
    if rc != OK:
        raise MqaError(rc, "mqa_dcp_shard")
    return table, lens


def dcp_locate(pos, seq_len, page_size, num_ranks, layout="round_robin"):
    """(rank, position in that rank's shard) of token `pos` of a sequence of
    seq_len tokens (C ABI ``mqa_dcp_locate``)."""
    r, p = ctypes.c_int(), ctypes.c_int()
    rc = lib.mqa_dcp_locate(int(pos), int(seq_len), int(page_size), int(num_ranks), _dcp_layout(layout),
                            ctypes.byref(r), ctypes.byref(p))
    if rc != OK:
        raise MqaError(rc, "mqa_dcp_locate")
    return r.value, p.value


def dcp_scale_shard(shard_out, gathered_lse, rank, *, scaled=None, lse=None, scaled_fp32=True, stream=None,
                    return_lse=True):
    """This rank's share of the merged output, laid out for a sum
    reduce-scatter over the ranks (C ABI ``mqa_dcp_scale_shard``):
    shard_out bf16 [B, H, D], gathered_lse fp32 [G, B, H]; returns (scaled
    [G, B, H / G, D] fp32 or bf16, merged lse [B, H] fp32)."""
    B, H, D = shard_out.shape
    G = gathered_lse.shape[0]
    if H % G != 0:
        raise ValueError("the head count must be a multiple of the number of ranks")
    sdt = torch.float32 if scaled_fp32 else torch.bfloat16
    if scaled is None:
        scaled = torch.empty((G, B, H // G, D), dtype=sdt, device=shard_out.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=shard_out.device)
    _check(shard_out, "shard_out", (torch.bfloat16,))
    _check(gathered_lse, "gathered_lse", (torch.float32,), shape=(G, B, H))
    _check(scaled, "scaled", (sdt,), shape=(G, B, H // G, D))
    _check(lse, "lse", (torch.float32,), shape=(B, H), optional=True)
    _on_device([("shard_out", shard_out), ("gathered_lse", gathered_lse), ("scaled", scaled), ("lse", lse)])
    rc = lib.mqa_dcp_scale_shard(_ptr(shard_out), _ptr(gathered_lse), _ptr(scaled), _ptr(lse), int(G), int(rank),
                                 int(B), int(H), int(D), int(bool(scaled_fp32)), _stream(stream))
    if rc != OK:
        raise MqaError(rc, "mqa_dcp_scale_shard")
    return scaled, lse


NOALLOC_SCRATCH_BYTES = 64 << 20


def mla_decode_noalloc(q, kv_cache, block_table, seq_lens, scale, k_scale=1.0, *, out, lse=None,
                       num_kv_splits=1, kv_lora_rank=None, kv_dtype=None, device_status=None,
                       stream=None):
    """MLA decode without a caller workspace, for callers that cannot allocate
    device memory: the split partials go to the library's own fixed 64 MiB
    device array, so `out` (and `lse`, if wanted) must already exist.  Calls
    share that array: do not let two of them overlap on the GPU."""
    B, H, D = q.shape
    nb, page, _ = kv_cache.shape
    R = (D - 64) if kv_lora_rank is None else int(kv_lora_rank)
    code = _kv_code(kv_cache, kv_dtype)
    _check_common(q, kv_cache, code, block_table, seq_lens, out, (B, H, R), lse, (B, H), None, device_status)
    rc = lib.mla_decode_noalloc(_ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
                                float(scale), float(k_scale), _ptr(out), _ptr(lse), B, H, D, R, nb,
                                page, block_table.shape[1], code,
                                int(num_kv_splits), _ptr(device_status), _stream(stream))
    if rc != OK:
        raise MqaError(rc, "mla_decode_noalloc")
    return out, lse


def gqa_window_decode_workspace_bytes(batch: int, q_len: int, num_q_heads: int, num_kv_heads: int, head_size: int,
                                      num_kv_splits: int) -> int:
    return int(lib.gqa_window_decode_workspace_bytes(batch, q_len, num_q_heads, num_kv_heads, head_size,
                                                     num_kv_splits))


def gqa_window_num_kv_splits(batch: int, q_len: int, num_q_heads: int, num_kv_heads: int) -> int:
    """The smallest num_kv_splits that lets gqa_window_decode / gqa_block_decode fill the current device."""
    n = int(lib.gqa_window_num_kv_splits(batch, q_len, num_q_heads, num_kv_heads))
    if n < 0:
        raise ValueError("no device, or a head layout that gqa_window_decode does not serve")
    return n


_PTH_CODES = (KV_FP8_E4M3_PER_TOKEN_HEAD, KV_INT8_PER_TOKEN_HEAD, KV_INT4_PER_TOKEN_HEAD)


# The calls below run once per layer and token.  Each first asks in one expression whether every tensor is the usual
# kind; only if one is not, _check and its like find out whether the call is wrong, and say how.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _fits(t, dtype, shape, index):
    """Whether t is what _check and _on_device ask for."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _raw(t):
    return None if t is None else t.data_ptr()


def _c_int(x):
    """x as a C int, the nearest where it has none (ctypes would take it modulo 2^32)."""
    return max(-(1 << 31), min(int(x), (1 << 31) - 1))


def _call_stream(stream, index, allocated):
    """The raw stream of a call on device `index`, by default the current one.  Tensors that the call allocated (on
    the current stream) are recorded on a stream that the caller passes, so that their memory is not reused while
    that stream still works on them."""
    raw = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        return raw
    other = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if other != raw and allocated:
        current = torch.cuda.current_stream(index)
        s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(other, device=current.device)
        s.wait_stream(current)
        for t in allocated:
            t.record_stream(s)
    return other


def _block_code(kv_cache, kv_scales, kv_dtype):
    """kv_dtype code of a cache that may have block scales."""
    if kv_dtype is not None or kv_scales is None:
        return _kv_code(kv_cache, kv_dtype)
    if kv_cache.dtype == torch.float8_e4m3fn:
        return KV_FP8_E4M3_BLOCK
    if kv_cache.dtype == torch.int8:
        return KV_INT8_BLOCK
    raise TypeError("a block-scaled kv_cache is float8_e4m3fn or int8 (or pass kv_dtype with uint8 storage)")


def _scale_block(kv_scales, code, nb, page, hkv):
    """Tokens per scale of kv_scales [num_blocks, 2, page / scale_block, num_kv_heads]; 0 for the other formats."""
    if code not in (KV_FP8_E4M3_BLOCK, KV_INT8_BLOCK):
        if kv_scales is not None:
            raise ValueError("kv_scales is for the fp8_e4m3_block and int8_block caches only")
        return 0
    if kv_scales is None:
        raise ValueError("kv_scales is required")
    s = kv_scales.shape
    if len(s) != 4 or s[0] != nb or s[1] != 2 or s[2] < 1 or page % s[2] != 0 or s[3] != hkv:
        raise ValueError(f"kv_scales must be [{nb}, 2, page / scale_block, {hkv}], got {tuple(s)}")
    if kv_scales.dtype is not torch.float32 or not kv_scales.is_contiguous():
        _check(kv_scales, "kv_scales", (torch.float32,))
    return page // s[2]


def gqa_window_decode(q, kv_cache, block_table, seq_lens, scale, window, sinks=0, *, kv_scales=None, k_scale=1.0,
                      v_scale=1.0, out=None, lse=None, num_kv_splits=None, workspace=None, kv_dtype=None,
                      device_status=None, stream=None, return_lse=True):
    """GQA paged decode under a sliding window through the C ABI: the query at position p sees key t iff t <= p and
    (t < sinks or t > p - window).  q bf16 [B, Hq, D], or [B, q_len, Hq, D] for q_len new positions per request
    (the last at seq_lens - 1); kv_cache [num_blocks, 2, page, Hkv, D] bf16 or e4m3 (k_scale / v_scale), or e4m3 /
    int8 codes with kv_scales fp32 [num_blocks, 2, page / scale_block, Hkv].  Returns out like q and lse fp32 like
    q without its last dimension.  num_kv_splits None fills the device; out / lse / workspace are allocated with
    torch when they are not given."""
    return _window_decode("gqa_window_decode", q, kv_cache, kv_scales, block_table, seq_lens, scale, k_scale, v_scale,
                          window, sinks, out, lse, num_kv_splits, workspace, kv_dtype, device_status, stream,
                          return_lse)


def gqa_block_decode(q, kv_cache, kv_scales, block_table, seq_lens, scale, *, out=None, lse=None, num_kv_splits=None,
                     workspace=None, kv_dtype=None, device_status=None, stream=None, return_lse=True):
    """GQA paged decode over a block-scaled 8-bit cache through the C ABI: kv_cache e4m3 or int8 codes
    [num_blocks, 2, page, Hkv, D], kv_scales fp32 [num_blocks, 2, page / scale_block, Hkv].  q and the other
    arguments as for :func:`gqa_window_decode`, without a window."""
    return _window_decode("gqa_block_decode", q, kv_cache, kv_scales, block_table, seq_lens, scale, 1.0, 1.0, None, 0,
                          out, lse, num_kv_splits, workspace, kv_dtype, device_status, stream, return_lse)


def _window_decode(name, q, kv_cache, kv_scales, block_table, seq_lens, scale, k_scale, v_scale, window, sinks, out,
                   lse, num_kv_splits, workspace, kv_dtype, device_status, stream, return_lse):
    shape = q.shape
    if len(shape) not in (3, 4) or kv_cache.dim() != 5:
        raise ValueError("q must be [batch, (q_len,) heads, head_size] and kv_cache have 5 dimensions")
    if len(shape) == 4:
        B, L, Hq, D = shape
    else:
        (B, Hq, D), L = shape, 1
    nb, two, page, Hkv, D2 = kv_cache.shape
    code = _block_code(kv_cache, kv_scales, kv_dtype)
    if two != 2 or D2 != D:
        raise ValueError(f"kv_cache must be [num_blocks, 2, page, num_kv_heads, {D}]")
    index = q.get_device()
    block = _scale_block(kv_scales, code, nb, page, Hkv)
    if window is None and block == 0:
        raise ValueError("gqa_block_decode reads block-scaled caches (fp8_e4m3_block, int8_block)")
    bt_shape = block_table.shape
    if not (index >= 0 and len(bt_shape) == 2 and bt_shape[0] == B and q.dtype is _BF16 and q.is_contiguous()
            and kv_cache.is_contiguous() and kv_cache.get_device() == index
            and kv_cache.element_size() == (2 if code == KV_BF16 else 1)
            and block_table.dtype is _I32 and block_table.get_device() == index and block_table.is_contiguous()
            and seq_lens.dtype is _I32 and seq_lens.shape == bt_shape[:1] and seq_lens.get_device() == index
            and seq_lens.is_contiguous()
            and (kv_scales is None or kv_scales.get_device() == index)
            and (out is None or _fits(out, _BF16, shape, index))
            and (lse is None or _fits(lse, _F32, shape[:-1], index))
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == index))
            and (device_status is None or _fits(device_status, _I32, device_status.shape, index))):
        _check_common(q, kv_cache, code, block_table, seq_lens, q if out is None else out, shape, lse, shape[:-1],
                      workspace, device_status, extra=(("kv_scales", kv_scales),))
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _window_decode(name, q, kv_cache, kv_scales, block_table, seq_lens, scale, k_scale, v_scale,
                                  window, sinks, out, lse, num_kv_splits, workspace, kv_dtype, device_status, stream,
                                  return_lse)
    fresh = []
    if out is None:
        out = torch.empty_like(q)
        fresh.append(out)
    if lse is None and return_lse:
        lse = torch.empty(shape[:-1], dtype=torch.float32, device=q.device)
        fresh.append(lse)
    if num_kv_splits is None:
        num_kv_splits = max(1, lib.gqa_window_num_kv_splits(B, L, Hq, Hkv))
    ws_bytes = 0
    if workspace is None:
        ws_bytes = lib.gqa_window_decode_workspace_bytes(B, L, Hq, Hkv, D, num_kv_splits)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
            fresh.append(workspace)
    else:
        ws_bytes = workspace.nbytes
    raw = _call_stream(stream, index, fresh)
    if window is None:
        rc = lib.gqa_block_decode(q.data_ptr(), kv_cache.data_ptr(), kv_scales.data_ptr(), block_table.data_ptr(),
                                  seq_lens.data_ptr(), float(scale), out.data_ptr(), _raw(lse), B, L, Hq, Hkv, D, nb,
                                  page, bt_shape[1], block, code, int(num_kv_splits), _raw(workspace), ws_bytes,
                                  _raw(device_status), raw)
    else:
        rc = lib.gqa_window_decode(q.data_ptr(), kv_cache.data_ptr(), _raw(kv_scales), block_table.data_ptr(),
                                   seq_lens.data_ptr(), float(scale), float(k_scale), float(v_scale), _c_int(window),
                                   _c_int(sinks), out.data_ptr(), _raw(lse), B, L, Hq, Hkv, D, nb, page, bt_shape[1],
                                   block, code, int(num_kv_splits), _raw(workspace), ws_bytes, _raw(device_status), raw)
    if rc != OK:
        raise MqaError(rc, name)
    return out, lse


def _check_rows(t, name, shape, dense):
    """A bf16 tensor of shape `shape` whose last `dense` dimensions are dense (rows of a wider tensor will do);
    returns its leading strides."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must have dtype torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    st, want = t.stride(), 1
    for i in range(1, dense + 1):
        if shape[-i] != 1 and st[-i] != want:
            raise ValueError(f"the last {dense} dimension(s) of {name} must be contiguous")
        want *= shape[-i]
    # a dimension of one has no stride of its own: any that holds a row will do
    out = []
    for i in range(len(shape) - dense - 1, -1, -1):
        s = st[i] if shape[i] > 1 else want
        out.insert(0, s)
        want = max(want, s * shape[i])
    return tuple(out)


def _head_rows(t, T, width, index):
    """Token stride of bf16 [T, heads, width] on device `index`, dense within a token; 0 if t is anything else."""
    s, st = t.shape, t.stride()
    if (t.dtype is _BF16 and s[0] == T and s[2] == width and st[1] == width and st[2] == 1
            and t.get_device() == index):
        return st[0]
    return 0


def _usual_batch(index, cos_sin, kv_cache, block_table, seq_lens, query_start, device_status):
    """Whether the tensors that describe an append's batch are the usual kind, on device `index`."""
    bt_shape = block_table.shape
    return (index >= 0 and len(bt_shape) == 2 and kv_cache.is_contiguous() and kv_cache.get_device() == index
            and cos_sin.dtype is _F32 and cos_sin.get_device() == index and cos_sin.is_contiguous()
            and block_table.dtype is _I32 and block_table.get_device() == index and block_table.is_contiguous()
            and seq_lens.dtype is _I32 and seq_lens.shape == bt_shape[:1] and seq_lens.get_device() == index
            and seq_lens.is_contiguous()
            and query_start.dtype is _I32 and query_start.shape == (bt_shape[0] + 1,)
            and query_start.get_device() == index and query_start.is_contiguous()
            and (device_status is None or _fits(device_status, _I32, device_status.shape, index)))


def _check_append(cos_sin, width, kv_cache, block_table, seq_lens, query_start, device_status, named):
    _check(cos_sin, "cos_sin", (torch.float32,))
    if cos_sin.dim() != 2 or (width is not None and cos_sin.shape[1] != width):
        raise ValueError(f"cos_sin must be fp32 [max_position, {width or 'rotary_dim'}]")
    _check(kv_cache, "kv_cache")
    _check(block_table, "block_table", (torch.int32,))
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [batch, max_blocks]")
    B = block_table.shape[0]
    _check(seq_lens, "seq_lens", (torch.int32,), shape=(B,))
    _check(query_start, "query_start", (torch.int32,), shape=(B + 1,))
    _check(device_status, "device_status", (torch.int32,), optional=True)
    _on_device([*named, ("cos_sin", cos_sin), ("kv_cache", kv_cache), ("block_table", block_table),
                ("seq_lens", seq_lens), ("query_start", query_start), ("device_status", device_status)])


def gqa_rope_append(k, v, cos_sin, kv_cache, block_table, seq_lens, query_start, *, q=None, q_out=None,
                    kv_scales=None, k_scale=1.0, v_scale=1.0, interleaved=False, kv_dtype=None, device_status=None,
                    stream=None):
    """Append new keys and values to a paged GQA cache through the C ABI, keys (and queries) rotated to their
    positions.  k, v bf16 [T, Hkv, D] and q [T, Hq, D] may be slices of a fused projection (any token stride that
    is a multiple of 8); request b brings tokens query_start[b] .. query_start[b + 1] - 1 (int32 [B + 1]), the last
    at position seq_lens[b] - 1; tokens behind query_start[B] are padding.  cos_sin fp32 [max_position, rotary_dim]
    holds cosines, then sines; interleaved pairs are columns (2i, 2i + 1).  kv_cache is any cache that the GQA
    decode calls read, with kv_scales for the block-scaled formats; both are updated in place.  Returns the rotated
    queries (q_out, which may be q itself; allocated when only q is given), or None."""
    shape, rows, table = k.shape, kv_cache.shape, cos_sin.shape
    if len(shape) != 3 or len(rows) != 5 or len(table) != 2:
        raise ValueError("k must be [tokens, heads, head_size], kv_cache have 5 dimensions and cos_sin 2")
    T, Hkv, D = shape
    nb, two, page, Hkv2, row = rows
    code = _block_code(kv_cache, kv_scales, kv_dtype)
    want = D if code not in _PTH_CODES else D // 2 + 4 if code == KV_INT4_PER_TOKEN_HEAD else D + 4
    if two != 2 or Hkv2 != Hkv or row != want:
        raise ValueError(f"kv_cache must be [num_blocks, 2, page, {Hkv}, {want}]")
    if kv_cache.element_size() != (2 if code == KV_BF16 else 1):
        raise TypeError(f"kv_cache must have {2 if code == KV_BF16 else 1}-byte elements, got {kv_cache.dtype}")
    block = _scale_block(kv_scales, code, nb, page, Hkv)
    index = k.get_device()
    qs = qos = Hq = 0
    if q is not None:
        q_shape = q.shape
        if len(q_shape) != 3:
            raise ValueError("q must be [tokens, heads, head_size]")
        Hq = q_shape[1]
    elif q_out is not None:
        raise ValueError("q_out without q")
    # (a dimension of one has no stride of its own: not the usual kind)
    ks, vs = k.stride(), v.stride()
    if (T > 1 and Hkv > 1 and k.dtype is _BF16 and ks[1] == D and ks[2] == 1
            and v.dtype is _BF16 and v.shape == shape and vs[1] == D and vs[2] == 1 and v.get_device() == index
            and (kv_scales is None or kv_scales.get_device() == index)
            and _usual_batch(index, cos_sin, kv_cache, block_table, seq_lens, query_start, device_status)
            and (q is None or Hq > 1 and (qs := _head_rows(q, T, D, index))
                 and (q_out is None or q_out.shape == q_shape and (qos := _head_rows(q_out, T, D, index))))):
        ks, vs = ks[0], vs[0]
    else:
        ks, = _check_rows(k, "k", (T, Hkv, D), 2)
        vs, = _check_rows(v, "v", (T, Hkv, D), 2)
        if q is not None:
            qs, = _check_rows(q, "q", (T, Hq, D), 2)
            if q_out is not None:
                qos, = _check_rows(q_out, "q_out", (T, Hq, D), 2)
        _check_append(cos_sin, None, kv_cache, block_table, seq_lens, query_start, device_status,
                      (("k", k), ("v", v), ("q", q), ("q_out", q_out), ("kv_scales", kv_scales)))
    B, max_blocks = block_table.shape
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return gqa_rope_append(k, v, cos_sin, kv_cache, block_table, seq_lens, query_start, q=q, q_out=q_out,
                                   kv_scales=kv_scales, k_scale=k_scale, v_scale=v_scale, interleaved=interleaved,
                                   kv_dtype=kv_dtype, device_status=device_status, stream=stream)
    fresh = []
    if q is not None and q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
        qos = Hq * D
        fresh.append(q_out)
    if T == 0:  # (an empty tensor has no address)
        return q_out
    rc = lib.gqa_rope_append(_raw(q), k.data_ptr(), v.data_ptr(), cos_sin.data_ptr(), query_start.data_ptr(),
                             seq_lens.data_ptr(), block_table.data_ptr(), _raw(q_out), kv_cache.data_ptr(),
                             _raw(kv_scales), float(k_scale), float(v_scale), T, B, Hq, Hkv, D, table[1],
                             1 if interleaved else 0, table[0], nb, page, max_blocks, block, code,
                             qs, ks, vs, qos, _raw(device_status), _call_stream(stream, index, fresh))
    if rc != OK:
        raise MqaError(rc, "gqa_rope_append")
    return q_out


def mla_rope_append(kv_c, k_pe, cos_sin, kv_cache, block_table, seq_lens, query_start, *, q_pe=None, q_pe_out=None,
                    k_scale=1.0, interleaved=False, kv_dtype=None, device_status=None, stream=None):
    """Append new latent rows [kv_c | rotated k_pe] to a paged MLA cache (bf16, or e4m3 with k_scale) through the C
    ABI.  kv_c bf16 [T, R] and k_pe [T, 64] may be slices of one projection; q_pe [T, H, 64] is rotated into
    q_pe_out (for instance ``q[..., R:]`` of the absorbed query; may be q_pe itself; allocated when only q_pe is
    given), which is returned (None without q_pe).  cos_sin fp32 [max_position, 64]; the batch is described as for
    :func:`gqa_rope_append`."""
    shape, rows, table = kv_c.shape, kv_cache.shape, cos_sin.shape
    if len(shape) != 2 or len(rows) != 3:
        raise ValueError("kv_c must be [tokens, kv_lora_rank] and kv_cache [num_blocks, page, head_size]")
    T, R = shape
    nb, page, D = rows
    if D != R + 64:
        raise ValueError(f"kv_cache must be [num_blocks, page, {R + 64}]")
    code = _kv_code(kv_cache, kv_dtype)
    if kv_cache.element_size() != (2 if code == KV_BF16 else 1):
        raise TypeError(f"kv_cache must have {2 if code == KV_BF16 else 1}-byte elements, got {kv_cache.dtype}")
    index = kv_c.get_device()
    H = qs = qhs = qos = qohs = 0
    if q_pe is not None:
        q_shape = q_pe.shape
        if len(q_shape) != 3:
            raise ValueError("q_pe must be [tokens, heads, 64]")
        H = q_shape[1]
    elif q_pe_out is not None:
        raise ValueError("q_pe_out without q_pe")
    cs, ps = kv_c.stride(), k_pe.stride()
    if (T > 1 and kv_c.dtype is _BF16 and cs[1] == 1 and k_pe.dtype is _BF16 and k_pe.shape == (T, 64) and ps[1] == 1
            and k_pe.get_device() == index and len(table) == 2 and table[1] == 64
            and _usual_batch(index, cos_sin, kv_cache, block_table, seq_lens, query_start, device_status)
            and (q_pe is None or H > 1 and q_pe.dtype is _BF16 and q_shape[0] == T and q_shape[2] == 64
                 and (qst := q_pe.stride())[2] == 1 and q_pe.get_device() == index
                 and (q_pe_out is None or q_pe_out.dtype is _BF16 and q_pe_out.shape == q_shape
                      and (qost := q_pe_out.stride())[2] == 1 and q_pe_out.get_device() == index))):
        cs, ps = cs[0], ps[0]
        if q_pe is not None:
            qs, qhs, _ = qst
            if q_pe_out is not None:
                qos, qohs, _ = qost
    else:
        cs, = _check_rows(kv_c, "kv_c", (T, R), 1)
        ps, = _check_rows(k_pe, "k_pe", (T, 64), 1)
        if q_pe is not None:
            qs, qhs = _check_rows(q_pe, "q_pe", (T, H, 64), 1)
            if q_pe_out is not None:
                qos, qohs = _check_rows(q_pe_out, "q_pe_out", (T, H, 64), 1)
        _check_append(cos_sin, 64, kv_cache, block_table, seq_lens, query_start, device_status,
                      (("kv_c", kv_c), ("k_pe", k_pe), ("q_pe", q_pe), ("q_pe_out", q_pe_out)))
    B, max_blocks = block_table.shape
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return mla_rope_append(kv_c, k_pe, cos_sin, kv_cache, block_table, seq_lens, query_start, q_pe=q_pe,
                                   q_pe_out=q_pe_out, k_scale=k_scale, interleaved=interleaved, kv_dtype=kv_dtype,
                                   device_status=device_status, stream=stream)
    fresh = []
    if q_pe is not None and q_pe_out is None:
        q_pe_out = torch.empty((T, H, 64), dtype=torch.bfloat16, device=q_pe.device)
        qos, qohs = H * 64, 64
        fresh.append(q_pe_out)
    if T == 0:
        return q_pe_out
    rc = lib.mla_rope_append(kv_c.data_ptr(), k_pe.data_ptr(), _raw(q_pe), cos_sin.data_ptr(),
                             query_start.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), _raw(q_pe_out),
                             kv_cache.data_ptr(), float(k_scale), T, B, H, D, R, 1 if interleaved else 0, table[0],
                             nb, page, max_blocks, code, cs, ps, qs, qhs, qos, qohs, _raw(device_status),
                             _call_stream(stream, index, fresh))
    if rc != OK:
        raise MqaError(rc, "mla_rope_append")
    return q_pe_out
