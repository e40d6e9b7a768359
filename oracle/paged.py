"""What surrounds attention over the paged cache, in fp64 and by position: the norm and rotation of
queries and keys, attention behind shared prefixes, new tokens into the cache.

TEST INFRASTRUCTURE ONLY: the GPU library never imports, loads or calls it.
"""
import numpy as np

from . import window

TREE_OK, TREE_BAD_SIZE, TREE_BAD_PARENT, TREE_BAD_PATH, TREE_BAD_CACHE = 0, 1, 2, 3, 6


def _f64(x):
    return np.asarray(x.double().numpy() if hasattr(x, "double") else x, np.float64)


def positions(first, offsets, parent=None):
    """{packed row: position}."""
    at = {}
    for b in range(len(first)):
        for i in range(int(offsets[b + 1] - offsets[b])):
            at[int(offsets[b]) + i] = int(first[b]) + len(window.path_of(parent, int(offsets[b]), i)) - 1
    return at


def norm_rotary(x, weight, inv_freq, at, eps, interleaved=False):
    """(y [T, h, d], bound [T, h, d]: |y_a| + |y_b| of the pair before it turns, |y| elsewhere,
    angle [T, 1, d]); rows without a position are NaN."""
    x, f = _f64(x), _f64(inv_freq)
    d, half = x.shape[2], len(f)
    y, mag, angle = np.full(x.shape, np.nan), np.full(x.shape, np.nan), np.zeros((len(x), 1, d))
    for t, p in at.items():
        z = x[t]
        if weight is not None:
            z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * _f64(weight)
        y[t], mag[t] = z, np.abs(z)
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = np.cos(p * f[j]), np.sin(p * f[j])
            y[t][:, a], y[t][:, b] = z[:, a] * c - z[:, b] * s, z[:, b] * c + z[:, a] * s
            mag[t][:, a] = mag[t][:, b] = np.abs(z[:, a]) + np.abs(z[:, b])
            angle[t, 0, a] = angle[t, 0, b] = abs(p * f[j])
    return y, mag, angle


def group_of(group_offsets, b):
    for g in range(len(group_offsets) - 1):
        if group_offsets[g] <= b < group_offsets[g + 1]:
            return g
    return None


def prefix_attention(q, k, v, k_cache, v_cache, prefix_table, prefix_len, group_offsets, page_table,
                     cache_len, offsets, parent=None, scale=None, rows=None):
    """window.attention with a window of everything over each sequence's prefix and cached tokens,
    laid out one position a page."""
    ps = k_cache.shape[2]
    K, V, lines, lens = [], [], [], []
    for b in range(len(cache_len)):
        g = group_of(group_offsets, b)
        spots = [] if g is None else [(prefix_table[g][s // ps], s % ps) for s in range(int(prefix_len[g]))]
        spots += [(page_table[b][s // ps], s % ps) for s in range(int(cache_len[b]))]
        lines.append(list(range(len(K), len(K) + len(spots))))
        lens.append(len(spots))
        for p, s in spots:
            K.append(k_cache[int(p), :, s])
            V.append(v_cache[int(p), :, s])
    table = np.zeros((len(lens), max(lens + [1])), int)
    for b, line in enumerate(lines):
        table[b, :len(line)] = line
    K, V = (np.stack([_f64(x) for x in c])[:, :, None] if c else np.zeros((1, k.shape[1], 1, k.shape[2]))
            for c in (K, V))
    return window.attention(q, k, v, K, V, table, lens, offsets, 2**40, 0, parent, scale, rows)


def append(k, v, k_cache, v_cache, page_table, cache_len, offsets, accepted_idx=None, accepted_len=None):
    """Caches and lengths after the call (all sequences valid); numpy arrays of any type."""
    k_cache, v_cache, new_len = k_cache.copy(), v_cache.copy(), np.array(cache_len)
    ps = k_cache.shape[2]
    for b in range(len(cache_len)):
        lo = int(offsets[b])
        new = (range(int(offsets[b + 1]) - lo) if accepted_idx is None
               else [int(i) for i in accepted_idx[b][:accepted_len[b]]])
        for i in new:
            page, slot = page_table[b][new_len[b] // ps], new_len[b] % ps
            k_cache[page, :, slot], v_cache[page, :, slot] = k[lo + i], v[lo + i]
            new_len[b] += 1
    return k_cache, v_cache, new_len
