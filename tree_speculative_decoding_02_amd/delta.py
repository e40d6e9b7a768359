"""Binding of the gated delta rule (include/bole.h): prompts, single tokens, draft trees and
accepted paths. As in bole.py, only arguments are checked and marshalled here.

Tensors: H0 float32 [B, H, d_k, d_v] (prefill, step and commit update it in place), q and k
[T, H_k, d_k], v [T, H, d_v] (bfloat16 or float32; H_k divides H), gate and beta float32
[T, H], out [T, H, d_v] in the factors' type. All are contiguous and on H0's GPU. With
stream=None a call goes to the stream that is current on that GPU when it is made; a bound
call looks it up each time it is called. A workspace that a bound call made for itself belongs
to `stream`, or to the one that was current when it was bound: as with any tensor, calls on
another stream have to be ordered behind that one, and ahead of it before the bound call is
dropped.
"""
import contextlib
import ctypes

import torch

from .bole import (BOLE_DTYPE_BF16, BOLE_DTYPE_F32, BOLE_FLAG_FORCE_GENERIC, BOLE_OK, _check,
                   _need, _ptr, bole_delta_dims_t, lib)


def _handle(what, device, stream):
    """The stream's handle, checked once; None for the one that is current at each call."""
    if stream is None:
        return None
    if stream.device != device:
        raise ValueError(f"{what}: the stream belongs to {stream.device}, the tensors to {device}")
    return stream.cuda_stream


def _launch(fn, what, args, index, handle):
    """The C call `fn(*args, stream)` on GPU `index`. torch's own accessors stand behind
    torch.cuda.current_device() and current_stream(): those cost a short call as much as its
    kernel takes."""
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index) if handle is None else handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index) if handle is None else handle)
    if st != BOLE_OK:
        _check(st, what)


def _run(fn, what, args, device, stream):
    _launch(fn, what, args, device.index, _handle(what, device, stream))


def _allocating_on(stream):
    """Buffers made for a call belong to the stream that the call runs on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class _BoundCall:
    """A call whose arguments were checked and marshalled once; calling it enqueues the same
    C call again on these buffers, which the object keeps alive."""

    def __init__(self, fn, what, args, device, stream, keep):
        self._a = (fn, what, args, device.index, _handle(what, device, stream))
        self._keep = keep, stream

    def __call__(self):
        _launch(*self._a)


def _shaped(t, name, dtype, device, shape):
    _need(t, name, dtype, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _apart(written, others):
    """Buffers that a call writes may overlap no other buffer of the call."""
    def span(t):
        return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()
    for i, (name, t) in enumerate(written):
        lo, hi = span(t)
        for other, o in written[i + 1:] + others:
            a, b = span(o)
            if lo < hi and a < b and lo < b and a < hi:
                raise ValueError(f"{name} overlaps {other}")


def _dims(H0, q, k, v, gate, beta, max_path=0, force_generic=False):
    _need(H0, "H0", torch.float32)
    if H0.dim() != 4:
        raise ValueError("H0 must be [B, H, d_k, d_v]")
    dev = H0.device
    B, H, d_k, d_v = H0.shape
    _need(k, "k", device=dev)
    fd = {torch.bfloat16: BOLE_DTYPE_BF16, torch.float32: BOLE_DTYPE_F32}.get(k.dtype)
    if fd is None:
        raise TypeError(f"factor dtype must be bfloat16 or float32, got {k.dtype}")
    if k.dim() != 3 or k.shape[2] != d_k or k.shape[1] < 1 or H % k.shape[1] != 0:
        raise ValueError("k must be [T, H_k, d_k] with H_k a divisor of H")
    T = k.shape[0]
    if q is not None:
        _shaped(q, "q", k.dtype, dev, k.shape)
    _shaped(v, "v", k.dtype, dev, (T, H, d_v))
    _shaped(gate, "gate", torch.float32, dev, (T, H))
    _shaped(beta, "beta", torch.float32, dev, (T, H))
    return bole_delta_dims_t(B, H, k.shape[1], d_k, d_v, T, max_path, fd,
                             BOLE_FLAG_FORCE_GENERIC if force_generic else 0)


def _out(out, v):
    if out is None:
        return torch.empty_like(v)
    _shaped(out, "out", v.dtype, v.device, v.shape)
    return out


def _status(t, name, B, dev):
    if t is not None:
        _need(t, name, torch.int32, dev)
        if t.numel() < B:
            raise ValueError(f"{name} needs B entries")
        return [(name, t)]
    return []


def _factors(q, k, v, gate, beta):
    return [(n, t) for n, t in (("q", q), ("k", k), ("v", v), ("gate", gate), ("beta", beta))
            if t is not None]


def _prefill_call(H0, q, k, v, gate, beta, seq_offsets, out, workspace, seq_status, force_generic):
    d = _dims(H0, q, k, v, gate, beta, force_generic=force_generic)
    _shaped(seq_offsets, "seq_offsets", torch.int32, H0.device, (d.batch + 1,))
    out = _out(out, v)
    need = lib.bole_delta_prefill_workspace_size(ctypes.byref(d))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=H0.device)
    _need(workspace, "workspace", device=H0.device)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace needs {need} bytes")
    _apart([("H0", H0), ("out", out), ("workspace", workspace)] +
           _status(seq_status, "seq_status", d.batch, H0.device),
           _factors(q, k, v, gate, beta) + [("seq_offsets", seq_offsets)])
    args = (_ptr(H0), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(seq_offsets),
            _ptr(out), _ptr(workspace), have, ctypes.byref(d), _ptr(seq_status))
    return out, args, (H0, q, k, v, gate, beta, seq_offsets, out, workspace, seq_status, d)


def bole_delta_prefill_workspace_size(H0, q, k, v, gate, beta, force_generic=False):
    """Bytes of workspace that bole_delta_prefill needs for these tensors' sizes."""
    d = _dims(H0, q, k, v, gate, beta, force_generic=force_generic)
    return int(lib.bole_delta_prefill_workspace_size(ctypes.byref(d)))


def bole_delta_prefill(H0, q, k, v, gate, beta, seq_offsets, out=None, workspace=None,
                       seq_status=None, stream=None, force_generic=False):
    """Runs every token of the packed sequences (seq_offsets int32 [B + 1]) through the gated
    delta rule from the states H0, which become the states after each sequence's last token;
    returns out. Without a workspace one is allocated for the call. Calls that may overlap
    need a workspace each."""
    with _allocating_on(stream):
        out, args, _keep = _prefill_call(H0, q, k, v, gate, beta, seq_offsets, out, workspace,
                                         seq_status, force_generic)
    _run(lib.bole_delta_prefill, "bole_delta_prefill", args, H0.device, stream)
    return out


def bind_delta_prefill(H0, q, k, v, gate, beta, seq_offsets, out, workspace=None, seq_status=None,
                       stream=None, force_generic=False):
    """Same checks as bole_delta_prefill, done once; the bound call keeps its workspace."""
    with _allocating_on(stream):
        _, args, keep = _prefill_call(H0, q, k, v, gate, beta, seq_offsets, out, workspace,
                                      seq_status, force_generic)
    return _BoundCall(lib.bole_delta_prefill, "bole_delta_prefill", args, H0.device, stream, keep)


def _step_call(H0, q, k, v, gate, beta, out):
    d = _dims(H0, q, k, v, gate, beta)
    if d.total_tokens != d.batch:
        raise ValueError("a step takes one token per sequence: T must equal B")
    out = _out(out, v)
    _apart([("H0", H0), ("out", out)], _factors(q, k, v, gate, beta))
    args = (_ptr(H0), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(out), ctypes.byref(d))
    return out, args, (H0, q, k, v, gate, beta, out, d)


def bole_delta_step(H0, q, k, v, gate, beta, out=None, stream=None):
    """One token for each sequence (row b belongs to sequence b): H0 in place; returns out."""
    with _allocating_on(stream):
        out, args, _ = _step_call(H0, q, k, v, gate, beta, out)
    _run(lib.bole_delta_step, "bole_delta_step", args, H0.device, stream)
    return out


def bind_delta_step(H0, q, k, v, gate, beta, out, stream=None):
    """Same checks as bole_delta_step, done once."""
    _, args, keep = _step_call(H0, q, k, v, gate, beta, out)
    return _BoundCall(lib.bole_delta_step, "bole_delta_step", args, H0.device, stream, keep)


def _verify_call(H0, q, k, v, gate, beta, parent, node_offsets, out, tree_status, force_generic):
    d = _dims(H0, q, k, v, gate, beta, force_generic=force_generic)
    _shaped(parent, "parent", torch.int32, H0.device, (d.total_tokens,))
    _shaped(node_offsets, "node_offsets", torch.int32, H0.device, (d.batch + 1,))
    out = _out(out, v)
    _apart([("out", out)] + _status(tree_status, "tree_status", d.batch, H0.device),
           [("H0", H0)] + _factors(q, k, v, gate, beta) +
           [("parent", parent), ("node_offsets", node_offsets)])
    args = (_ptr(H0), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(parent),
            _ptr(node_offsets), _ptr(out), ctypes.byref(d), _ptr(tree_status))
    return out, args, (H0, q, k, v, gate, beta, parent, node_offsets, out, tree_status, d)


def bole_delta_tree_verify(H0, q, k, v, gate, beta, parent, node_offsets, out=None,
                           tree_status=None, stream=None, force_generic=False):
    """out[T, H, d_v] = H_i^T q_i for every node of the draft trees (parent int32 [T],
    node_offsets int32 [B + 1]), all nodes in parallel; H0 is not written."""
    with _allocating_on(stream):
        out, args, _ = _verify_call(H0, q, k, v, gate, beta, parent, node_offsets, out, tree_status,
                                    force_generic)
    _run(lib.bole_delta_tree_verify, "bole_delta_tree_verify", args, H0.device, stream)
    return out


def bind_delta_tree_verify(H0, q, k, v, gate, beta, parent, node_offsets, out, tree_status=None,
                           stream=None, force_generic=False):
    """Same checks as bole_delta_tree_verify, done once."""
    _, args, keep = _verify_call(H0, q, k, v, gate, beta, parent, node_offsets, out, tree_status,
                                 force_generic)
    return _BoundCall(lib.bole_delta_tree_verify, "bole_delta_tree_verify", args, H0.device, stream,
                      keep)


def _commit_call(H0, k, v, gate, beta, parent, node_offsets, accepted_idx, accepted_len,
                 path_nodes, tree_status):
    dev = H0.device
    _need(accepted_idx, "accepted_idx", torch.int32, dev)
    if accepted_idx.dim() != 2:
        raise ValueError("accepted_idx must be [B, max_path]")
    d = _dims(H0, None, k, v, gate, beta, max_path=accepted_idx.shape[1])
    _shaped(accepted_idx, "accepted_idx", torch.int32, dev, (d.batch, d.max_path))
    _shaped(accepted_len, "accepted_len", torch.int32, dev, (d.batch,))
    _shaped(parent, "parent", torch.int32, dev, (d.total_tokens,))
    _shaped(node_offsets, "node_offsets", torch.int32, dev, (d.batch + 1,))
    written = [("H0", H0)] + _status(tree_status, "tree_status", d.batch, dev)
    if path_nodes is not None:
        _shaped(path_nodes, "path_nodes", torch.int32, dev, (d.batch, d.max_path))
        written.append(("path_nodes", path_nodes))
    _apart(written, _factors(None, k, v, gate, beta) +
           [("parent", parent), ("node_offsets", node_offsets), ("accepted_idx", accepted_idx),
            ("accepted_len", accepted_len)])
    args = (_ptr(H0), _ptr(k), _ptr(v), _ptr(gate), _ptr(beta), _ptr(parent), _ptr(node_offsets),
            _ptr(accepted_idx), _ptr(accepted_len), ctypes.byref(d), _ptr(path_nodes),
            _ptr(tree_status))
    return args, (H0, k, v, gate, beta, parent, node_offsets, accepted_idx, accepted_len,
                  path_nodes, tree_status, d)


def bole_delta_commit_path(H0, k, v, gate, beta, parent, node_offsets, accepted_idx, accepted_len,
                           path_nodes=None, tree_status=None, stream=None):
    """Commits each tree's accepted path (accepted_idx int32 [B, max_path], accepted_len int32
    [B]) into H0 in place; returns H0."""
    args, _ = _commit_call(H0, k, v, gate, beta, parent, node_offsets, accepted_idx, accepted_len,
                           path_nodes, tree_status)
    _run(lib.bole_delta_commit_path, "bole_delta_commit_path", args, H0.device, stream)
    return H0


def bind_delta_commit_path(H0, k, v, gate, beta, parent, node_offsets, accepted_idx, accepted_len,
                           path_nodes=None, tree_status=None, stream=None):
    """Same checks as bole_delta_commit_path, done once."""
    args, keep = _commit_call(H0, k, v, gate, beta, parent, node_offsets, accepted_idx,
                              accepted_len, path_nodes, tree_status)
    return _BoundCall(lib.bole_delta_commit_path, "bole_delta_commit_path", args, H0.device, stream,
                      keep)
