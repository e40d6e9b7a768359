"""Linear attention with a decay in fp64: token by token, no chunks.

TEST INFRASTRUCTURE ONLY: the GPU library never imports, loads or calls it.

For one head with state H [d_k][d_v], decay a (a number, or one for each of the d_k channels):
    H <- a H + k v^T,   o = H^T q   (after the token's own update);
value head h reads key head h / (H / H_k).
"""
from dataclasses import dataclass

import numpy as np


def _f64(x):
    return np.asarray(x.double().numpy() if hasattr(x, "double") else x, np.float64)


@dataclass
class Result:
    out: np.ndarray      # [T, H, d_v]; rows of no sequence are NaN
    S: np.ndarray        # [B, H, d_k, d_v] after each sequence
    S_mag: np.ndarray    # the same of every term's absolute value
    out_mag: np.ndarray  # [T, H, d_v]: sums of |q| times that
    pair: np.ndarray     # [T, H, d_v]: sums over the tokens j of i's chunk, up to i, of
    #                      D_{j->i} |q_i . k_j| |v_j| (one decay a head only)
    tokens: np.ndarray   # [T]: tokens of the row's sequence up to it


def prefill(H0, q, k, v, gate, offsets, chunk=64):
    H0, q, k, v, gate = map(_f64, (H0, q, k, v, gate))
    H = v.shape[1]
    q, k = (np.repeat(x, H // x.shape[1], axis=1) for x in (q, k))
    channel = gate.ndim == 3
    a = gate[..., None] if channel else gate[:, :, None, None]  # [T, H, d_k or 1, 1]
    r = Result(np.full(v.shape, np.nan), H0.copy(), np.abs(H0), np.zeros(v.shape), np.zeros(v.shape),
               np.zeros(len(v)))
    for b in range(H0.shape[0]):
        for t in range(offsets[b], offsets[b + 1]):
            if (t - offsets[b]) % chunk == 0:
                D, js = [], []
            kv = k[t][:, :, None] * v[t][:, None, :]
            r.S[b] = a[t] * r.S[b] + kv
            r.S_mag[b] = a[t] * r.S_mag[b] + np.abs(kv)
            r.out[t] = np.einsum("hkv,hk->hv", r.S[b], q[t])
            r.out_mag[t] = np.einsum("hkv,hk->hv", r.S_mag[b], np.abs(q[t]))
            r.tokens[t] = t - offsets[b] + 1
            if not channel:
                D = [d * gate[t] for d in D] + [np.ones(H)]
                js.append(t)
                for d, j in zip(D, js):
                    r.pair[t] += (d * np.abs((q[t] * k[j]).sum(-1)))[:, None] * np.abs(v[j])
    return r
