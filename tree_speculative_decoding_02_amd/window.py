"""Binding of windowed attention over a paged cache (include/bole.h). As in bole.py, only
arguments are checked and marshalled here; streams are handled as in delta.py."""
import ctypes

import torch

from .bole import (BOLE_DTYPE_BF16, BOLE_DTYPE_F32, BOLE_FLAG_FORCE_GENERIC, _need, _ptr,
                   bole_window_dims_t, lib)
from .delta import _allocating_on, _apart, _BoundCall, _run, _shaped, _status


def _dims(q, k, v, k_cache, v_cache, page_table, cache_len, window, sinks, scale, force_generic):
    _need(q, "q")
    dev = q.device
    dt = {torch.bfloat16: BOLE_DTYPE_BF16, torch.float32: BOLE_DTYPE_F32}.get(q.dtype)
    if dt is None:
        raise TypeError(f"q must be bfloat16 or float32, got {q.dtype}")
    if q.dim() != 3 or q.shape[2] < 1:
        raise ValueError("q must be [T, H, d] with d at least 1")
    T, H, d = q.shape
    _need(k, "k", q.dtype, dev)
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != d or k.shape[1] < 1 or H % k.shape[1] != 0:
        raise ValueError("k must be [T, H_kv, d] with H_kv a divisor of H")
    _shaped(v, "v", q.dtype, dev, k.shape)
    _need(k_cache, "k_cache", q.dtype, dev)
    if k_cache.dim() != 4 or k_cache.shape[1] != k.shape[1] or k_cache.shape[3] != d:
        raise ValueError("k_cache must be [num_pages, H_kv, page_size, d]")
    _shaped(v_cache, "v_cache", q.dtype, dev, k_cache.shape)
    _need(page_table, "page_table", torch.int32, dev)
    _need(cache_len, "cache_len", torch.int32, dev)
    if page_table.dim() != 2 or tuple(cache_len.shape) != (page_table.shape[0],):
        raise ValueError("page_table must be [B, max_pages] and cache_len [B]")
    if not (1 <= window <= 0x7fffffff and 0 <= sinks <= 0x7fffffff):
        raise ValueError("window must be at least 1 and sinks at least 0")
    scale = d ** -0.5 if scale is None else float(scale)
    if not abs(scale) < 2.0 ** 127:
        raise ValueError("scale must be finite, and below 2^127 in size")
    return bole_window_dims_t(page_table.shape[0], H, k.shape[1], d, T, k_cache.shape[0],
                              k_cache.shape[2], page_table.shape[1], window, sinks, dt,
                              BOLE_FLAG_FORCE_GENERIC if force_generic else 0, scale)


def _call(q, k, v, k_cache, v_cache, page_table, cache_len, node_offsets, window, sinks, out,
          parent, scale, workspace, seq_status, force_generic):
    d = _dims(q, k, v, k_cache, v_cache, page_table, cache_len, window, sinks, scale, force_generic)
    dev = q.device
    _shaped(node_offsets, "node_offsets", torch.int32, dev, (d.batch + 1,))
    others = [("q", q), ("k", k), ("v", v), ("k_cache", k_cache), ("v_cache", v_cache),
              ("page_table", page_table), ("cache_len", cache_len), ("node_offsets", node_offsets)]
    if parent is not None:
        _shaped(parent, "parent", torch.int32, dev, (d.total_rows,))
        others.append(("parent", parent))
    if out is None:
        out = torch.empty_like(q)
    _shaped(out, "out", q.dtype, dev, q.shape)
    need = lib.bole_window_workspace_size(ctypes.byref(d))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace needs {need} bytes")
    _apart([("out", out), ("workspace", workspace)] + _status(seq_status, "seq_status", d.batch, dev),
           others)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
            _ptr(cache_len), _ptr(parent), _ptr(node_offsets), _ptr(out), _ptr(workspace), have,
            ctypes.byref(d), _ptr(seq_status))
    return out, args, (others, out, workspace, seq_status, d)


def bole_window_workspace_size(q, k, v, k_cache, v_cache, page_table, cache_len, window, sinks,
                               force_generic=False):
    """Bytes of workspace that bole_window_attention needs for these tensors' sizes."""
    d = _dims(q, k, v, k_cache, v_cache, page_table, cache_len, window, sinks, None, force_generic)
    return int(lib.bole_window_workspace_size(ctypes.byref(d)))


def bole_window_attention(q, k, v, k_cache, v_cache, page_table, cache_len, node_offsets, window,
                          sinks, out=None, parent=None, scale=None, workspace=None,
                          seq_status=None, stream=None, force_generic=False):
    """out [T, H, d]: each row's attention over the cached tokens of its sequence and the rows
    on its own path, as far as the last `window` positions and the first `sinks` reach.
    q [T, H, d], k and v [T, H_kv, d] are this call's rows (node_offsets int32 [B + 1]); with
    parent (int32 [T]) each sequence's rows are a draft tree, without it its next tokens.
    k_cache, v_cache [num_pages, H_kv, page_size, d], page_table int32 [B, max_pages],
    cache_len int32 [B]. scale defaults to d^-1/2. Without a workspace one is allocated for
    the call; calls that may overlap need one each."""
    with _allocating_on(stream):
        out, args, _keep = _call(q, k, v, k_cache, v_cache, page_table, cache_len, node_offsets,
                                 window, sinks, out, parent, scale, workspace, seq_status,
                                 force_generic)
    _run(lib.bole_window_attention, "bole_window_attention", args, q.device, stream)
    return out


def bind_window_attention(q, k, v, k_cache, v_cache, page_table, cache_len, node_offsets, window,
                          sinks, out, parent=None, scale=None, workspace=None, seq_status=None,
                          stream=None, force_generic=False):
    """Same checks as bole_window_attention, done once; the bound call keeps its workspace."""
    with _allocating_on(stream):
        _, args, keep = _call(q, k, v, k_cache, v_cache, page_table, cache_len, node_offsets,
                              window, sinks, out, parent, scale, workspace, seq_status,
                              force_generic)
    return _BoundCall(lib.bole_window_attention, "bole_window_attention", args, q.device, stream,
                      keep)
