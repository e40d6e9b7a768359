"""Binding of what surrounds attention over the paged cache (include/bole.h): the norm and rotation
of queries and keys, attention behind shared prefixes, and new tokens into the cache. As in bole.py,
only arguments are checked and marshalled here; streams are handled as in delta.py."""
import ctypes
import math

import torch

from .bole import (BOLE_DTYPE_BF16, BOLE_DTYPE_F32, BOLE_FLAG_FORCE_GENERIC, BOLE_FLAG_INTERLEAVED,
                   _need, _ptr, bole_append_dims_t, bole_prefix_dims_t, bole_rotary_dims_t, lib)
from .delta import _allocating_on, _BoundCall, _run, _shaped, _status

_DTYPES = {torch.bfloat16: BOLE_DTYPE_BF16, torch.float32: BOLE_DTYPE_F32}


def _rows(t, name, dtype, device, heads=None, width=None):
    """[T, heads, width], each row contiguous, rows apart by any number of elements that is at
    least a row's (returned)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dim() != 3 or t.shape[1] < 1 or t.shape[2] < 1 or (heads is not None and t.shape[1] != heads) \
            or (width is not None and t.shape[2] != width):
        raise ValueError(f"{name} must be [T, {heads or 'heads'}, {width or 'd'}], got {list(t.shape)}")
    row = t.shape[1] * t.shape[2]
    if t.shape[0] < 1:
        return row
    if (t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2]) or \
            (t.shape[0] > 1 and t.stride(0) < row):
        raise ValueError(f"{name}: heads and their elements must be contiguous, rows apart")
    return t.stride(0) if t.shape[0] > 1 else row


def _span(t):
    """First byte of a tensor's elements, and one past the last."""
    if t.numel() == 0:
        return t.data_ptr(), t.data_ptr()
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(written, others, same=()):
    """Buffers that a call writes may overlap no other buffer of the call, but for the pairs in
    `same`, which may be one and the same."""
    for i, (name, t) in enumerate(written):
        lo, hi = _span(t)
        for other, o in written[i + 1:] + others:
            a, b = _span(o)
            if lo < hi and a < b and lo < b and a < hi and not ((name, other) in same and (lo, hi) == (a, b)):
                raise ValueError(f"{name} overlaps {other}")


def _given(pairs):
    return [(n, t) for n, t in pairs if t is not None]


def _rotary_call(q, k, q_weight, k_weight, inv_freq, first_position, node_offsets, q_out, k_out, eps,
                 parent, interleaved, seq_status, force_generic):
    q_stride = _rows(q, "q", None, None)
    dev, (T, H, d) = q.device, q.shape
    k_stride = _rows(k, "k", q.dtype, dev, None, d)
    if k.shape[0] != T:
        raise ValueError("q and k must have the same rows")
    for name, w in _given([("q_weight", q_weight), ("k_weight", k_weight)]):
        _shaped(w, name, q.dtype, dev, (d,))
    _need(inv_freq, "inv_freq", torch.float32, dev)
    if inv_freq.dim() != 1 or 2 * inv_freq.shape[0] > d:
        raise ValueError("inv_freq must be [rotary_dim / 2], with rotary_dim at most d")
    _need(first_position, "first_position", torch.int32, dev)
    if first_position.dim() != 1:
        raise ValueError("first_position must be [B]")
    B = first_position.shape[0]
    _shaped(node_offsets, "node_offsets", torch.int32, dev, (B + 1,))
    if parent is not None:
        _shaped(parent, "parent", torch.int32, dev, (T,))
    eps = float(eps)
    if not 0.0 <= eps < math.inf:
        raise ValueError("eps must be finite and at least 0")
    q_out = torch.empty((T, H, d), dtype=q.dtype, device=dev) if q_out is None else q_out
    k_out = torch.empty((T, k.shape[1], d), dtype=q.dtype, device=dev) if k_out is None else k_out
    _shaped(q_out, "q_out", q.dtype, dev, (T, H, d))
    _shaped(k_out, "k_out", q.dtype, dev, k.shape)
    others = _given([("q", q), ("k", k), ("q_weight", q_weight), ("k_weight", k_weight),
                     ("inv_freq", inv_freq), ("first_position", first_position),
                     ("node_offsets", node_offsets), ("parent", parent)])
    _apart([("q_out", q_out), ("k_out", k_out)] + _status(seq_status, "seq_status", B, dev), others,
           (("q_out", "q"), ("k_out", "k")))
    dims = bole_rotary_dims_t(B, H, k.shape[1], d, 2 * inv_freq.shape[0], T, _DTYPES[q.dtype],
                              (BOLE_FLAG_FORCE_GENERIC if force_generic else 0) |
                              (BOLE_FLAG_INTERLEAVED if interleaved else 0), q_stride, k_stride, eps)
    args = (_ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq), _ptr(first_position),
            _ptr(parent), _ptr(node_offsets), _ptr(q_out), _ptr(k_out), ctypes.byref(dims),
            _ptr(seq_status))
    return (q_out, k_out), args, (others, q_out, k_out, seq_status, dims)


def bole_qk_norm_rotary(q, k, q_weight, k_weight, inv_freq, first_position, node_offsets, q_out=None,
                        k_out=None, eps=1e-6, parent=None, interleaved=False, seq_status=None,
                        stream=None, force_generic=False):
    """(q_out [T, H, d], k_out [T, H_kv, d]): every head's query and key, divided by its root mean
    square, times its weight ([d]; None: as it is), its first 2 len(inv_freq) dimensions turned by
    position * inv_freq (float32): pairs (j, j + half) or, interleaved, (2 j, 2 j + 1). Row i of
    sequence b (node_offsets int32 [B + 1]) is at first_position[b] + i, with parent (int32 [T]) at
    first_position[b] plus its depth below the tree's roots. Rows of q and k may be apart, as slices
    of one projection are; q_out and k_out are contiguous, and may be q and k themselves."""
    with _allocating_on(stream):
        out, args, _keep = _rotary_call(q, k, q_weight, k_weight, inv_freq, first_position,
                                        node_offsets, q_out, k_out, eps, parent, interleaved,
                                        seq_status, force_generic)
    _run(lib.bole_qk_norm_rotary, "bole_qk_norm_rotary", args, q.device, stream)
    return out


def bind_qk_norm_rotary(q, k, q_weight, k_weight, inv_freq, first_position, node_offsets, q_out, k_out,
                        eps=1e-6, parent=None, interleaved=False, seq_status=None, stream=None,
                        force_generic=False):
    """Same checks as bole_qk_norm_rotary, done once."""
    _, args, keep = _rotary_call(q, k, q_weight, k_weight, inv_freq, first_position, node_offsets,
                                 q_out, k_out, eps, parent, interleaved, seq_status, force_generic)
    return _BoundCall(lib.bole_qk_norm_rotary, "bole_qk_norm_rotary", args, q.device, stream, keep)


def _caches(k_cache, v_cache, dtype, dev, heads, d):
    _need(k_cache, "k_cache", dtype, dev)
    if k_cache.dim() != 4 or k_cache.shape[1] != heads or k_cache.shape[3] != d:
        raise ValueError("k_cache must be [num_pages, H_kv, page_size, d]")
    _shaped(v_cache, "v_cache", dtype, dev, k_cache.shape)


def _tables(page_table, cache_len, dev, table="page_table", length="cache_len", lines="B"):
    _need(page_table, table, torch.int32, dev)
    _need(cache_len, length, torch.int32, dev)
    if page_table.dim() != 2 or tuple(cache_len.shape) != (page_table.shape[0],):
        raise ValueError(f"{table} must be [{lines}, pages] and {length} [{lines}]")


def _prefix_dims(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table, cache_len, scale,
                 force_generic):
    _need(q, "q")
    dev = q.device
    if q.dtype not in _DTYPES:
        raise TypeError(f"q must be bfloat16 or float32, got {q.dtype}")
    if q.dim() != 3 or q.shape[1] < 1 or q.shape[2] < 1:
        raise ValueError("q must be [T, H, d] with d at least 1")
    T, H, d = q.shape
    _need(k, "k", q.dtype, dev)
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != d or k.shape[1] < 1 or H % k.shape[1] != 0:
        raise ValueError("k must be [T, H_kv, d] with H_kv a divisor of H")
    _shaped(v, "v", q.dtype, dev, k.shape)
    _caches(k_cache, v_cache, q.dtype, dev, k.shape[1], d)
    _tables(page_table, cache_len, dev)
    _tables(prefix_table, prefix_len, dev, "prefix_table", "prefix_len", "groups")
    scale = d ** -0.5 if scale is None else float(scale)
    if not abs(scale) < 2.0 ** 127:
        raise ValueError("scale must be finite, and below 2^127 in size")
    return bole_prefix_dims_t(page_table.shape[0], H, k.shape[1], d, T, k_cache.shape[0],
                              k_cache.shape[2], page_table.shape[1], prefix_table.shape[0],
                              prefix_table.shape[1], _DTYPES[q.dtype],
                              BOLE_FLAG_FORCE_GENERIC if force_generic else 0, scale)


def _prefix_call(q, k, v, k_cache, v_cache, prefix_table, prefix_len, group_offsets, page_table,
                 cache_len, node_offsets, out, parent, scale, workspace, seq_status, force_generic):
    dims = _prefix_dims(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table, cache_len,
                        scale, force_generic)
    dev = q.device
    _shaped(group_offsets, "group_offsets", torch.int32, dev, (dims.groups + 1,))
    _shaped(node_offsets, "node_offsets", torch.int32, dev, (dims.batch + 1,))
    if parent is not None:
        _shaped(parent, "parent", torch.int32, dev, (dims.total_rows,))
    out = torch.empty_like(q) if out is None else out
    _shaped(out, "out", q.dtype, dev, q.shape)
    need = lib.bole_prefix_workspace_size(ctypes.byref(dims))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace needs {need} bytes")
    others = _given([("q", q), ("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache),
                     ("prefix_table", prefix_table), ("prefix_len", prefix_len),
                     ("group_offsets", group_offsets), ("page_table", page_table),
                     ("cache_len", cache_len), ("node_offsets", node_offsets), ("parent", parent)])
    _apart([("out", out), ("workspace", workspace)] + _status(seq_status, "seq_status", dims.batch, dev),
           others)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(prefix_table),
            _ptr(prefix_len), _ptr(group_offsets), _ptr(page_table), _ptr(cache_len), _ptr(parent),
            _ptr(node_offsets), _ptr(out), _ptr(workspace), have, ctypes.byref(dims), _ptr(seq_status))
    return out, args, (others, out, workspace, seq_status, dims)


def bole_prefix_workspace_size(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table,
                               cache_len, force_generic=False):
    """Bytes of workspace that bole_prefix_attention needs for these tensors' sizes."""
    dims = _prefix_dims(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table, cache_len,
                        None, force_generic)
    return int(lib.bole_prefix_workspace_size(ctypes.byref(dims)))


def bole_prefix_attention(q, k, v, k_cache, v_cache, prefix_table, prefix_len, group_offsets,
                          page_table, cache_len, node_offsets, out=None, parent=None, scale=None,
                          workspace=None, seq_status=None, stream=None, force_generic=False):
    """out [T, H, d]: each row's attention over the prefix of its group, the cached tokens of its
    sequence behind it, and the rows on its own path. Sequences group_offsets[g] ..
    group_offsets[g + 1] - 1 (int32 [groups + 1]) share the prefix_len[g] tokens in the pages of
    prefix_table[g] (int32 [groups, pages]); the other arguments are those of bole_window_attention.
    The prefix's keys are read once for all rows that share it. scale defaults to d^-1/2. Without a
    workspace one is allocated for the call; calls that may overlap need one each."""
    with _allocating_on(stream):
        out, args, _keep = _prefix_call(q, k, v, k_cache, v_cache, prefix_table, prefix_len,
                                        group_offsets, page_table, cache_len, node_offsets, out,
                                        parent, scale, workspace, seq_status, force_generic)
    _run(lib.bole_prefix_attention, "bole_prefix_attention", args, q.device, stream)
    return out


def bind_prefix_attention(q, k, v, k_cache, v_cache, prefix_table, prefix_len, group_offsets,
                          page_table, cache_len, node_offsets, out, parent=None, scale=None,
                          workspace=None, seq_status=None, stream=None, force_generic=False):
    """Same checks as bole_prefix_attention, done once; the bound call keeps its workspace."""
    with _allocating_on(stream):
        _, args, keep = _prefix_call(q, k, v, k_cache, v_cache, prefix_table, prefix_len,
                                     group_offsets, page_table, cache_len, node_offsets, out, parent,
                                     scale, workspace, seq_status, force_generic)
    return _BoundCall(lib.bole_prefix_attention, "bole_prefix_attention", args, q.device, stream, keep)


def _append_call(k, v, k_cache, v_cache, page_table, cache_len, node_offsets, parent, accepted_idx,
                 accepted_len, new_len, seq_status):
    k_stride = _rows(k, "k", None, None)
    dev, (T, H, d) = k.device, k.shape
    v_stride = _rows(v, "v", k.dtype, dev, H, d)
    if v.shape[0] != T:
        raise ValueError("k and v must have the same rows")
    _caches(k_cache, v_cache, k.dtype, dev, H, d)
    _tables(page_table, cache_len, dev)
    B, max_path = page_table.shape[0], 0
    _shaped(node_offsets, "node_offsets", torch.int32, dev, (B + 1,))
    if (accepted_idx is None) != (accepted_len is None) or (parent is None) != (accepted_idx is None):
        raise ValueError("paths need parent, accepted_idx and accepted_len together")
    if accepted_idx is not None:
        _shaped(parent, "parent", torch.int32, dev, (T,))
        _need(accepted_idx, "accepted_idx", torch.int32, dev)
        if accepted_idx.dim() != 2 or accepted_idx.shape[0] != B:
            raise ValueError("accepted_idx must be [B, max_path]")
        max_path = accepted_idx.shape[1]
        _shaped(accepted_len, "accepted_len", torch.int32, dev, (B,))
    written = [("k_cache", k_cache), ("v_cache", v_cache)] + _status(seq_status, "seq_status", B, dev)
    if new_len is not None:
        _shaped(new_len, "new_len", torch.int32, dev, (B,))
        written.append(("new_len", new_len))
    others = _given([("k", k), ("v", v), ("page_table", page_table), ("cache_len", cache_len),
                     ("node_offsets", node_offsets), ("parent", parent),
                     ("accepted_idx", accepted_idx), ("accepted_len", accepted_len)])
    _apart(written, others)
    dims = bole_append_dims_t(B, H, d, T, k_cache.shape[0], k_cache.shape[2], page_table.shape[1],
                              max_path, _DTYPES[k.dtype], 0, k_stride, v_stride)
    args = (_ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(cache_len),
            _ptr(parent), _ptr(node_offsets), _ptr(accepted_idx), _ptr(accepted_len), _ptr(new_len),
            ctypes.byref(dims), _ptr(seq_status))
    return args, (others, k_cache, v_cache, new_len, seq_status, dims)


def bole_cache_append(k, v, k_cache, v_cache, page_table, cache_len, node_offsets, parent=None,
                      accepted_idx=None, accepted_len=None, new_len=None, seq_status=None,
                      stream=None):
    """Writes k and v [T, H_kv, d] (rows may be apart) behind the cache_len[b] cached tokens of each
    sequence: all its rows, or, with parent, accepted_idx (int32 [B, max_path]) and accepted_len, the
    rows of its tree's accepted path. new_len (int32 [B]) receives the lengths with them; cache_len
    is left, for the other layers' calls. Returns new_len."""
    args, _ = _append_call(k, v, k_cache, v_cache, page_table, cache_len, node_offsets, parent,
                           accepted_idx, accepted_len, new_len, seq_status)
    _run(lib.bole_cache_append, "bole_cache_append", args, k.device, stream)
    return new_len


def bind_cache_append(k, v, k_cache, v_cache, page_table, cache_len, node_offsets, parent=None,
                      accepted_idx=None, accepted_len=None, new_len=None, seq_status=None,
                      stream=None):
    """Same checks as bole_cache_append, done once."""
    args, keep = _append_call(k, v, k_cache, v_cache, page_table, cache_len, node_offsets, parent,
                              accepted_idx, accepted_len, new_len, seq_status)
    return _BoundCall(lib.bole_cache_append, "bole_cache_append", args, k.device, stream, keep)
