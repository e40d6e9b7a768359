"""Binding of linear attention with a decay (include/bole.h): prompts and single tokens. As in
bole.py, only arguments are checked and marshalled here; streams are handled as in delta.py.

Tensors: H0 float32 [B, H, d_k, d_v], updated in place; q and k [T, H_k, d_k], v [T, H, d_v]
(bfloat16 or float32; H_k divides H); gate float32 [T, H], or [T, H, d_k] for a decay a key
channel; out [T, H, d_v] in the factors' type. All are contiguous and on H0's GPU.
"""
import ctypes

import torch

from .bole import (BOLE_DTYPE_BF16, BOLE_DTYPE_F32, BOLE_FLAG_FORCE_GENERIC, BOLE_GATE_SCALAR,
                   BOLE_GATE_VECTOR, _need, _ptr, bole_linear_dims_t, lib)
from .delta import _allocating_on, _apart, _BoundCall, _out, _run, _shaped, _status


def _dims(H0, q, k, v, gate, force_generic=False):
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
    _shaped(q, "q", k.dtype, dev, k.shape)
    _shaped(v, "v", k.dtype, dev, (T, H, d_v))
    _need(gate, "gate", torch.float32, dev)
    if tuple(gate.shape) not in ((T, H), (T, H, d_k)):
        raise ValueError(f"gate must be [T, H] or [T, H, d_k], got {list(gate.shape)}")
    return bole_linear_dims_t(B, H, k.shape[1], d_k, d_v, T, fd,
                              BOLE_GATE_SCALAR if gate.dim() == 2 else BOLE_GATE_VECTOR,
                              BOLE_FLAG_FORCE_GENERIC if force_generic else 0)


def _prefill_call(H0, q, k, v, gate, seq_offsets, out, workspace, seq_status, force_generic):
    d = _dims(H0, q, k, v, gate, force_generic)
    dev = H0.device
    _shaped(seq_offsets, "seq_offsets", torch.int32, dev, (d.batch + 1,))
    out = _out(out, v)
    need = lib.bole_linear_prefill_workspace_size(ctypes.byref(d))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise ValueError(f"workspace needs {need} bytes")
    _apart([("H0", H0), ("out", out), ("workspace", workspace)] +
           _status(seq_status, "seq_status", d.batch, dev),
           [("q", q), ("k", k), ("v", v), ("gate", gate), ("seq_offsets", seq_offsets)])
    args = (_ptr(H0), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(seq_offsets), _ptr(out),
            _ptr(workspace), have, ctypes.byref(d), _ptr(seq_status))
    return out, args, (H0, q, k, v, gate, seq_offsets, out, workspace, seq_status, d)


def bole_linear_prefill_workspace_size(H0, q, k, v, gate, force_generic=False):
    """Bytes of workspace that bole_linear_prefill needs for these tensors' sizes."""
    d = _dims(H0, q, k, v, gate, force_generic)
    return int(lib.bole_linear_prefill_workspace_size(ctypes.byref(d)))


def bole_linear_prefill(H0, q, k, v, gate, seq_offsets, out=None, workspace=None, seq_status=None,
                        stream=None, force_generic=False):
    """Runs every token of the packed sequences (seq_offsets int32 [B + 1]) through
    H <- a H + k v^T, o = H^T q from the states H0, which become the states after each sequence's
    last token; returns out. Without a workspace one is allocated for the call. Calls that may
    overlap need a workspace each."""
    with _allocating_on(stream):
        out, args, _keep = _prefill_call(H0, q, k, v, gate, seq_offsets, out, workspace, seq_status,
                                         force_generic)
    _run(lib.bole_linear_prefill, "bole_linear_prefill", args, H0.device, stream)
    return out


def bind_linear_prefill(H0, q, k, v, gate, seq_offsets, out, workspace=None, seq_status=None,
                        stream=None, force_generic=False):
    """Same checks as bole_linear_prefill, done once; the bound call keeps its workspace."""
    with _allocating_on(stream):
        _, args, keep = _prefill_call(H0, q, k, v, gate, seq_offsets, out, workspace, seq_status,
                                      force_generic)
    return _BoundCall(lib.bole_linear_prefill, "bole_linear_prefill", args, H0.device, stream, keep)


def _step_call(H0, q, k, v, gate, out):
    d = _dims(H0, q, k, v, gate)
    if d.total_tokens != d.batch:
        raise ValueError("a step takes one token per sequence: T must equal B")
    out = _out(out, v)
    _apart([("H0", H0), ("out", out)], [("q", q), ("k", k), ("v", v), ("gate", gate)])
    args = (_ptr(H0), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(out), ctypes.byref(d))
    return out, args, (H0, q, k, v, gate, out, d)


def bole_linear_step(H0, q, k, v, gate, out=None, stream=None):
    """One token for each sequence (row b belongs to sequence b): H0 in place; returns out."""
    with _allocating_on(stream):
        out, args, _ = _step_call(H0, q, k, v, gate, out)
    _run(lib.bole_linear_step, "bole_linear_step", args, H0.device, stream)
    return out


def bind_linear_step(H0, q, k, v, gate, out, stream=None):
    """Same checks as bole_linear_step, done once."""
    _, args, keep = _step_call(H0, q, k, v, gate, out)
    return _BoundCall(lib.bole_linear_step, "bole_linear_step", args, H0.device, stream, keep)
