"""The calls over windowed and block-scaled caches and the cache appends (the C ABI functions of the same names), with
their checks of arguments.  Reached through the package, like the calls of :mod:`._binding`."""
from __future__ import annotations

import torch

from ._binding import (KV_BF16, KV_FP8_E4M3_BLOCK, KV_FP8_E4M3_PER_TOKEN_HEAD, KV_INT4_PER_TOKEN_HEAD, KV_INT8_BLOCK,
                       KV_INT8_PER_TOKEN_HEAD, OK, MqaError, _check, _check_common, _kv_code, _on_device, lib)

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
