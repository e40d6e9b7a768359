"""Sliding-window attention with visible first tokens over a paged cache, in fp64: one row,
one head, one key at a time by position.

TEST INFRASTRUCTURE ONLY: the GPU library never imports, loads or calls it.

A row at position p sees a key at position s (cached, or of a row on its own path, itself
among them) if p - s < window or s < sinks; out = softmax over the seen keys of
scale (q . k_s), times v_s.
"""
import numpy as np


def path_of(parent, lo, i):
    path = []
    while i >= 0:
        path.insert(0, i)
        i = -1 if parent is None and i == 0 else (i - 1 if parent is None else int(parent[lo + i]))
    return path


def attention(q, k, v, k_cache, v_cache, page_table, cache_len, offsets, window, sinks,
              parent=None, scale=None, rows=None):
    """(out [T, H, d], |terms| [T, H, d]: the sums of w |v|, reach [T, H]: the largest
    |scale| |q| |k| of a seen key). Rows outside `rows` (packed row numbers) are left NaN."""
    f = lambda x: np.asarray(x.double().numpy() if hasattr(x, "double") else x, np.float64)
    q, k, v, k_cache, v_cache = map(f, (q, k, v, k_cache, v_cache))
    T, H, d = q.shape
    G = H // k.shape[1]
    ps = k_cache.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, mag, reach = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.zeros((T, H))
    for b in range(len(cache_len)):
        lo, n, c = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(cache_len[b])
        for i in range(n):
            if rows is not None and lo + i not in rows:
                continue
            path = path_of(parent, lo, i)
            pos = c + len(path) - 1
            cached = [s for s in range(c) if pos - s < window or s < sinks]
            own = [lo + j for t, j in enumerate(path) if pos - (c + t) < window or c + t < sinks]
            pg = np.array([page_table[b][s // ps] for s in cached], int)
            sl = np.array([s % ps for s in cached], int)
            K = np.concatenate([k_cache[pg, :, sl].reshape(-1, *k.shape[1:]), k[own]])
            V = np.concatenate([v_cache[pg, :, sl].reshape(-1, *k.shape[1:]), v[own]])
            for h in range(H):
                z = scale * (K[:, h // G] @ q[lo + i, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                out[lo + i, h] = w @ V[:, h // G]
                mag[lo + i, h] = w @ np.abs(V[:, h // G])
                reach[lo + i, h] = abs(scale) * np.linalg.norm(q[lo + i, h]) * \
                    np.linalg.norm(K[:, h // G], axis=1).max()
    return out, mag, reach
