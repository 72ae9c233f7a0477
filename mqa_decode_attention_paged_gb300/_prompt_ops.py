"""Prompt attention over paged caches, and forking and compacting their pages (the C ABI functions of the same names),
with their checks of arguments.  Reached through the package, like the calls of :mod:`._binding`."""
from __future__ import annotations

from array import array

import torch

from ._binding import KV_BF16, OK, MqaError, _check, _on_device, lib
from ._cache_ops import (_BF16, _F32, _I32, _NO_WINDOW, _block_code, _c_int, _call_stream, _check_rows, _fits,
                         _head_rows, _raw, _scale_block)


def gqa_prefill(q, kv_cache, block_table, seq_lens, query_start, scale, *, softcap=0.0, slopes=None, window=None,
                sinks=0, prefix_lens=None, kv_scales=None, k_scale=1.0, v_scale=1.0, out=None, lse=None,
                num_kv_splits=None, workspace=None, kv_dtype=None, device_status=None, stream=None, return_lse=True):
    """GQA attention of a ragged batch of new tokens over a paged cache that holds their keys already, through the C
    ABI.  q bf16 [T, Hq, D] may be a slice of a fused projection; request b brings tokens query_start[b] ..
    query_start[b + 1] - 1 (int32 [B + 1]), the last at position seq_lens[b] - 1; rows of tokens outside are padding
    and not written.  The query at position p sees key t iff (t <= p or t < prefix_lens[b]) and (t < sinks or
    t > p - window).  Logits are shaped as by :func:`gqa_score_decode`; kv_cache and its scales are those of
    :func:`gqa_window_decode`.  num_kv_splits None spreads the work evenly over the device, 1 keeps a token's result
    independent of the rest of the batch.  Returns out bf16 [T, Hq, D] and lse fp32 [T, Hq], allocated with torch
    when they are not given."""
    shape, rows = q.shape, kv_cache.shape
    if len(shape) != 3 or len(rows) != 5:
        raise ValueError("q must be [tokens, heads, head_size] and kv_cache have 5 dimensions")
    T, Hq, D = shape
    nb, two, page, Hkv, D2 = rows
    code = _block_code(kv_cache, kv_scales, kv_dtype)
    if two != 2 or D2 != D:
        raise ValueError(f"kv_cache must be [num_blocks, 2, page, num_kv_heads, {D}]")
    block = _scale_block(kv_scales, code, nb, page, Hkv)
    index = q.get_device()
    bt_shape = block_table.shape
    qs = _head_rows(q, T, D, index) if T > 1 and Hq > 1 else 0
    if not (qs and index >= 0 and len(bt_shape) == 2 and kv_cache.is_contiguous() and kv_cache.get_device() == index
            and kv_cache.element_size() == (2 if code == KV_BF16 else 1)
            and block_table.dtype is _I32 and block_table.get_device() == index and block_table.is_contiguous()
            and _fits(seq_lens, _I32, bt_shape[:1], index) and _fits(query_start, _I32, (bt_shape[0] + 1,), index)
            and (prefix_lens is None or _fits(prefix_lens, _I32, bt_shape[:1], index))
            and (kv_scales is None or kv_scales.get_device() == index)
            and (slopes is None or _fits(slopes, _F32, (Hq,), index))
            and (out is None or _fits(out, _BF16, shape, index))
            and (lse is None or _fits(lse, _F32, shape[:2], index))
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == index))
            and (device_status is None or _fits(device_status, _I32, device_status.shape, index))):
        qs, = _check_rows(q, "q", (T, Hq, D), 2)
        _check(kv_cache, "kv_cache", elt=2 if code == KV_BF16 else 1)
        _check(block_table, "block_table", (_I32,))
        if block_table.dim() != 2:
            raise ValueError("block_table must be int32 [batch, max_blocks]")
        B = bt_shape[0]
        _check(seq_lens, "seq_lens", (_I32,), shape=(B,))
        _check(query_start, "query_start", (_I32,), shape=(B + 1,))
        _check(prefix_lens, "prefix_lens", (_I32,), shape=(B,), optional=True)
        _check(slopes, "slopes", (_F32,), shape=(Hq,), optional=True)
        _check(out, "out", (_BF16,), shape=shape, optional=True)
        _check(lse, "lse", (_F32,), shape=shape[:2], optional=True)
        _check(workspace, "workspace", optional=True)
        _check(device_status, "device_status", (_I32,), optional=True)
        _on_device([("q", q), ("kv_cache", kv_cache), ("kv_scales", kv_scales), ("block_table", block_table),
                    ("seq_lens", seq_lens), ("query_start", query_start), ("prefix_lens", prefix_lens),
                    ("slopes", slopes), ("out", out), ("lse", lse), ("workspace", workspace),
                    ("device_status", device_status)])
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return gqa_prefill(q, kv_cache, block_table, seq_lens, query_start, scale, softcap=softcap, slopes=slopes,
                               window=window, sinks=sinks, prefix_lens=prefix_lens, kv_scales=kv_scales,
                               k_scale=k_scale, v_scale=v_scale, out=out, lse=lse, num_kv_splits=num_kv_splits,
                               workspace=workspace, kv_dtype=kv_dtype, device_status=device_status, stream=stream,
                               return_lse=return_lse)
    fresh = []
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
        fresh.append(out)
    if lse is None and return_lse:
        lse = torch.empty(shape[:2], dtype=_F32, device=q.device)
        fresh.append(lse)
    if T == 0:  # (an empty tensor has no address)
        return out, lse
    splits = 2 if num_kv_splits is None else _c_int(num_kv_splits)
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.nbytes
    elif splits > 1:
        ws_bytes = lib.gqa_prefill_workspace_bytes(Hq, Hkv, D)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
            fresh.append(workspace)
    rc = lib.gqa_prefill(q.data_ptr(), kv_cache.data_ptr(), _raw(kv_scales), block_table.data_ptr(),
                         seq_lens.data_ptr(), query_start.data_ptr(), _raw(prefix_lens), float(scale), float(k_scale),
                         float(v_scale), float(softcap), _raw(slopes), _NO_WINDOW if window is None else _c_int(window),
                         _c_int(sinks), out.data_ptr(), _raw(lse), T, bt_shape[0], Hq, Hkv, D, nb, page, bt_shape[1],
                         block, code, qs, splits, _raw(workspace), ws_bytes, _raw(device_status),
                         _call_stream(stream, index, fresh))
    if rc != OK:
        raise MqaError(rc, "gqa_prefill")
    return out, lse


def _pools(caches, num_blocks, index):
    """Addresses and bytes per page of the caches, as arrays of 64-bit words for the C ABI."""
    addresses, sizes = array("Q"), array("Q")
    for t in caches:
        s = t.shape
        if not (len(s) > 0 and s[0] == num_blocks and t.get_device() == index and t.is_contiguous()):
            i = len(addresses)
            _check(t, f"caches[{i}]")
            if len(s) < 1 or s[0] != num_blocks:
                raise ValueError(f"caches[{i}] must have {num_blocks} pages in its first dimension, got {tuple(s)}")
            raise ValueError(f"caches[{i}] is on {t.device}, the call runs on cuda:{index}")
        addresses.append(t.data_ptr())
        sizes.append(t.nbytes // max(1, num_blocks))  # (no pages: refused by the call)
    return addresses, sizes


def _int32(t, shape, index):
    """Whether t is None or an int32 tensor of that shape on device `index`, contiguous."""
    return t is None or (t.dtype is _I32 and t.shape == shape and t.get_device() == index and t.is_contiguous())


def _check_pages(block_table, seq_lens, refs, named, workspace, device_status):
    """The device index of a page operation; raises unless its tensors are what the C ABI takes."""
    _check(block_table, "block_table", (_I32,))
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [rows, max_blocks]")
    _check(seq_lens, "seq_lens", (_I32,), shape=(block_table.shape[0],))
    _check(refs, "refs", (_I32,))
    if refs.dim() != 1:
        raise ValueError("refs must be int32 [num_blocks]")
    for name, t, shape in named:
        _check(t, name, (_I32,), shape=shape, optional=True)
    _check(workspace, "workspace", optional=True)
    _check(device_status, "device_status", (_I32,), optional=True)
    _on_device([("block_table", block_table), ("seq_lens", seq_lens), ("refs", refs), ("workspace", workspace),
                ("device_status", device_status), *((name, t) for name, t, _ in named)])
    return block_table.get_device()


def pages_fork(block_table, seq_lens, parents, refs, caches, page_size, *, new_table=None, new_lens=None,
               new_refs=None, workspace=None, device_status=None, stream=None):
    """New rows of a block table from parents through the C ABI (``mqa_pages_fork``): row r of the result shares the
    pages of row parents[r] (-1: an empty row); a partly filled last page, in which only one row may end, stays with the
    first child, every other one gets the lowest free page with a copy of its data.  block_table int32 [rows, max_blocks],
    seq_lens int32 [rows], parents int32 [new_rows], refs int32 [num_blocks] (holders of each page, 0: free); caches: the
    tensors [num_blocks, ...] whose pages are copied, in place (of every layer; block scales are tensors of their own).
    No parents: every row ends.  Returns new_table [new_rows, max_blocks], new_lens [new_rows] and new_refs
    [num_blocks] (new_refs may be refs itself; allocated with torch when not given)."""
    if parents.dim() != 1:
        raise ValueError("parents must be int32 [new_rows]")
    shape, N, index = block_table.shape, parents.shape[0], block_table.get_device()
    if not (index >= 0 and len(shape) == 2 and refs.dim() == 1 and _int32(block_table, shape, index)
            and _int32(seq_lens, shape[:1], index) and _int32(parents, (N,), index) and _int32(refs, refs.shape, index)
            and _int32(new_table, (N, shape[1]), index) and _int32(new_lens, (N,), index)
            and _int32(new_refs, refs.shape, index)
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == index))
            and (device_status is None or _fits(device_status, _I32, device_status.shape, index))):
        index = _check_pages(block_table, seq_lens, refs,
                             (("parents", parents, (N,)), ("new_table", new_table, (N, shape[-1])),
                              ("new_lens", new_lens, (N,)), ("new_refs", new_refs, refs.shape)), workspace,
                             device_status)
    width, nb = shape[1], refs.shape[0]
    addresses, sizes = _pools(caches, nb, index)
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return pages_fork(block_table, seq_lens, parents, refs, caches, page_size, new_table=new_table,
                              new_lens=new_lens, new_refs=new_refs, workspace=workspace, device_status=device_status,
                              stream=stream)
    fresh = []
    no_rows = (new_table, new_lens) if N == 0 else None
    if no_rows:  # every row ends: one empty row in the place of none, which the C call does not take
        parents, N, new_table, new_lens, workspace = torch.full((1,), -1, dtype=_I32, device=refs.device), 1, None, None, None
        fresh.append(parents)

    def given(t, *size):
        if t is None:
            t = torch.empty(size, dtype=_I32, device=refs.device)
            fresh.append(t)
        return t

    new_table, new_lens, new_refs = given(new_table, N, width), given(new_lens, N), given(new_refs, nb)
    workspace = given(workspace, max(16, lib.mqa_pages_fork_workspace_bytes(N) // 4))
    rc = lib.mqa_pages_fork(block_table.data_ptr(), seq_lens.data_ptr(), parents.data_ptr(), refs.data_ptr(),
                            new_table.data_ptr(), new_lens.data_ptr(), new_refs.data_ptr(), shape[0], N, width, nb,
                            _c_int(page_size), addresses.buffer_info()[0], sizes.buffer_info()[0], len(addresses),
                            workspace.data_ptr(), workspace.nbytes, _raw(device_status),
                            _call_stream(stream, index, fresh))
    if rc != OK:
        raise MqaError(rc, "mqa_pages_fork")
    if no_rows:
        new_table, new_lens = (made[:0] if t is None else t for t, made in zip(no_rows, (new_table, new_lens)))
    return new_table, new_lens, new_refs


def pages_compact(block_table, seq_lens, refs, caches, page_size, *, new_table=None, new_refs=None, moved=None,
                  num_live=None, workspace=None, device_status=None, stream=None):
    """Moves the live pages (refs > 0) of caches to the lowest ids through the C ABI (``mqa_pages_compact``).  Returns
    new_table (the renamed table; may be block_table itself), new_refs (may be refs itself), moved int32 [num_blocks]
    (each page's new id, -1 for free ones) and num_live int32 [1], allocated with torch when not given.  Arguments as
    for :func:`pages_fork`."""
    shape, index = block_table.shape, block_table.get_device()
    if not (index >= 0 and len(shape) == 2 and refs.dim() == 1 and _int32(block_table, shape, index)
            and _int32(seq_lens, shape[:1], index) and _int32(refs, refs.shape, index) and _int32(new_table, shape, index)
            and _int32(new_refs, refs.shape, index) and _int32(moved, refs.shape, index)
            and _int32(num_live, (1,), index)
            and (workspace is None or (workspace.is_contiguous() and workspace.get_device() == index))
            and (device_status is None or _fits(device_status, _I32, device_status.shape, index))):
        index = _check_pages(block_table, seq_lens, refs,
                             (("new_table", new_table, shape), ("new_refs", new_refs, refs.shape),
                              ("moved", moved, refs.shape), ("num_live", num_live, (1,))), workspace, device_status)
    nb = refs.shape[0]
    addresses, sizes = _pools(caches, nb, index)
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return pages_compact(block_table, seq_lens, refs, caches, page_size, new_table=new_table, new_refs=new_refs,
                                 moved=moved, num_live=num_live, workspace=workspace, device_status=device_status,
                                 stream=stream)
    fresh = []

    def given(t, *size):
        if t is None:
            t = torch.empty(size, dtype=_I32, device=refs.device)
            fresh.append(t)
        return t

    new_table, new_refs = given(new_table, *shape), given(new_refs, nb)
    moved, num_live = given(moved, nb), given(num_live, 1)
    workspace = given(workspace, max(16, lib.mqa_pages_compact_workspace_bytes(nb) // 4))
    rc = lib.mqa_pages_compact(block_table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(), new_table.data_ptr(),
                               new_refs.data_ptr(), moved.data_ptr(), num_live.data_ptr(), shape[0], shape[1], nb,
                               _c_int(page_size), addresses.buffer_info()[0], sizes.buffer_info()[0], len(addresses),
                               workspace.data_ptr(), workspace.nbytes, _raw(device_status),
                               _call_stream(stream, index, fresh))
    if rc != OK:
        raise MqaError(rc, "mqa_pages_compact")
    return new_table, new_refs, moved, num_live
