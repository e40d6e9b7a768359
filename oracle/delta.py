"""Gated delta rule in fp64: token by token, node by node, no closed form.

TEST INFRASTRUCTURE ONLY: the GPU library never imports, loads or calls it.

For one head with state H [d_k][d_v]:
    H' = a H,   u = b (v - H'^T k),   H <- H' + k u^T,   o = H^T q;
value head h reads key head h / (H / H_k). A tree node starts from its parent's state (the
committed state for a root); a commit walks the accepted path.
"""
import numpy as np

TREE_OK, TREE_BAD_SIZE, TREE_BAD_PARENT, TREE_BAD_PATH = 0, 1, 2, 3


def _f64(x):
    return np.asarray(x.double().numpy() if hasattr(x, "double") else x, np.float64)


def token(S, q, k, v, a, b):
    """States [H, d_k, d_v] after one token, and its outputs [H, d_v]; q may be None."""
    H = S.shape[0]
    k = np.repeat(k, H // k.shape[0], axis=0)
    S = a[:, None, None] * S
    u = b[:, None] * (v - np.einsum("hkv,hk->hv", S, k))
    S = S + k[:, :, None] * u[:, None, :]
    if q is None:
        return S, None
    return S, np.einsum("hkv,hk->hv", S, np.repeat(q, H // q.shape[0], axis=0))


def prefill(H0, q, k, v, gate, beta, offsets):
    """(out [T, H, d_v], states after each sequence); rows of no sequence are NaN."""
    H0, q, k, v, gate, beta = map(_f64, (H0, q, k, v, gate, beta))
    out, S = np.full(v.shape, np.nan), H0.copy()
    for b in range(H0.shape[0]):
        for t in range(offsets[b], offsets[b + 1]):
            S[b], out[t] = token(S[b], q[t], k[t], v[t], gate[t], beta[t])
    return out, S


def pair_terms(H0, q, k, v, gate, beta, offsets, chunk=64):
    """[T, H, d_v]: sum over the tokens j of i's chunk, up to i, of D_{j->i} |q_i . k_j| |u_j|,
    the magnitude of an output's terms that a weight per token pair stands before."""
    H0, q, k, v, gate, beta = map(_f64, (H0, q, k, v, gate, beta))
    H = v.shape[1]
    q, k = (np.repeat(x, H // x.shape[1], axis=1) for x in (q, k))
    mag = np.zeros(v.shape)
    for b in range(H0.shape[0]):
        S = H0[b].copy()
        for t in range(offsets[b], offsets[b + 1]):
            if (t - offsets[b]) % chunk == 0:
                us, ks, D = [], [], []
            S = gate[t][:, None, None] * S
            u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            D = [d * gate[t] for d in D] + [np.ones(H)]
            us.append(np.abs(u)), ks.append(k[t])
            for d, kk, uu in zip(D, ks, us):
                mag[t] += (d * np.abs((q[t] * kk).sum(-1)))[:, None] * uu
    return mag


def verify(H0, q, k, v, gate, beta, parent, offsets):
    """out [T, H, d_v] of every node of every tree."""
    H0, q, k, v, gate, beta = map(_f64, (H0, q, k, v, gate, beta))
    out = np.full(v.shape, np.nan)
    for b in range(H0.shape[0]):
        lo, states = offsets[b], []
        for i in range(offsets[b + 1] - lo):
            p, t = parent[lo + i], lo + i
            S, out[t] = token(H0[b] if p < 0 else states[p], q[t], k[t], v[t], gate[t], beta[t])
            states.append(S)
    return out


def commit(H0, k, v, gate, beta, offsets, accepted_idx, accepted_len):
    """States after each tree's accepted path."""
    H0, k, v, gate, beta = map(_f64, (H0, k, v, gate, beta))
    S = H0.copy()
    for b in range(H0.shape[0]):
        for m in range(accepted_len[b]):
            t = offsets[b] + accepted_idx[b][m]
            S[b], _ = token(S[b], None, k[t], v[t], gate[t], beta[t])
    return S
