"""CPU checks of windowed attention: the fp64 oracle against what its definition fixes, and
the refusals of the C ABI and the binding (nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import workloads as W
from oracle import window as O
from tree_speculative_decoding_02_amd import bole, window


def make(seed=1, **kw):
    a = dict(sizes=[4, 1, 6], cached=[9, 0, 21], heads=4, kv_heads=2, d=5, page_size=4, window=7,
             sinks=2, dtype=torch.float32)
    a.update(kw)
    return W.make_window(seed, **a)


def args(w):
    return (w.q, w.k, w.v, w.k_cache, w.v_cache, w.page_table.numpy(), w.cache_len.numpy(), w.offsets)


def test_oracle_reads_nothing_hidden():
    """Every cache slot that no row sees is NaN and its page invalid; the oracle meets none."""
    w = make()
    assert torch.isnan(w.k_cache).any() and (w.page_table < 0).any()
    for parent in (None, w.parent):
        out, _, _ = O.attention(*args(w), 7, 2, parent)
        assert np.isfinite(out).all()


def test_window_of_one_returns_the_own_value():
    w = make(window=1, sinks=0)
    out, _, _ = O.attention(*args(w), 1, 0, w.parent)
    assert np.abs(out - w.v.double().numpy().repeat(2, 1)).max() < 1e-15


def test_equal_scores_average_the_seen_values():
    w = make(window=3, sinks=1, poison=False)
    w.q.zero_()
    out, _, _ = O.attention(*args(w), 3, 1)
    k0 = w.page_table[0].tolist()
    at = lambda s: w.v_cache[k0[s // 4], :, s % 4].double().numpy()
    want = (at(0) + at(8) + w.v[0].double().numpy() + w.v[1].double().numpy()) / 4
    assert np.abs(out[1] - want.repeat(2, 0)).max() < 1e-14   # row 1 at position 10 sees 8, 9, 10 and 0


def test_a_tree_path_is_a_prompt():
    """A tree node's output is that of its path's rows as the sequence's next tokens."""
    w = make(sizes=[12], cached=[9], kind="random")
    out, _, _ = O.attention(*args(w), 7, 2, w.parent)
    for i in range(12):
        path = O.path_of(w.parent, 0, i)
        o, _, _ = O.attention(w.q[path], w.k[path], w.v[path], *args(w)[3:7],
                              np.array([0, len(path)]), 7, 2)
        assert np.abs(out[i] - o[-1]).max() < 1e-15


def test_wide_window_is_full_attention_and_sinks_then_add_nothing():
    w = make(poison=False)
    a = O.attention(*args(w), 1000, 0)[0]
    b = O.attention(*args(w), 1000, 5)[0]
    c = O.attention(*args(w), 1, 1000)[0]
    assert np.array_equal(a, b) and np.array_equal(a, c)


def dims(**kw):
    d = bole.bole_window_dims_t(4, 8, 4, 128, 100, 50, 16, 10, 64, 4, bole.BOLE_DTYPE_BF16, 0, 0.1)
    for n, x in kw.items():
        setattr(d, n, x)
    return d


@pytest.mark.parametrize("field,value,want", [
    ("batch", -1, 1), ("heads", 0, 1), ("kv_heads", 0, 1), ("kv_heads", 3, 1), ("head_dim", 0, 1),
    ("head_dim", 257, 2), ("total_rows", -1, 1), ("num_pages", -1, 1), ("page_size", 0, 1),
    ("page_size", 24, 1), ("page_size", 2048, 2), ("max_pages", -1, 1), ("max_pages", 1 << 28, 2),
    ("window", 0, 1), ("sinks", -1, 1), ("dtype", 3, 1), ("flags", 4, 1),
    ("scale", float("nan"), 1), ("scale", float("inf"), 1), ("scale", 3e38, 1), ("total_rows", 1 << 29, 2),
])
def test_check_dims_refuses(field, value, want):
    assert bole.lib.bole_window_check_dims(ctypes.byref(dims(**{field: value}))) == want


def test_check_dims_keeps_positions_and_launches_in_32_bits():
    # a key list is walked up to eight tiles of 64 keys past its end before the end stops it
    L = bole.lib
    check = lambda **kw: L.bole_window_check_dims(ctypes.byref(dims(**kw)))
    big = dict(total_rows=0, page_size=1024, window=0x7fffffff, sinks=0x7fffffff)
    assert check(max_pages=(1 << 21) - 1, **big) == bole.BOLE_OK
    assert check(max_pages=1 << 21, **big) == bole.BOLE_ERR_UNSUPPORTED
    assert check(max_pages=(1 << 21) - 1, **{**big, "total_rows": 1}) == bole.BOLE_ERR_UNSUPPORTED
    # 64 threads a row, 256 for each 64 packed rows and for three workgroups a sequence
    few = dict(max_pages=0, num_pages=0, heads=1, kv_heads=1)
    assert check(batch=1, total_rows=(1 << 26) - 1, **few) == bole.BOLE_OK
    assert check(batch=1, total_rows=1 << 26, **few) == bole.BOLE_ERR_UNSUPPORTED
    assert check(batch=(1 << 24) // 3, total_rows=0, **few) == bole.BOLE_OK
    assert check(batch=(1 << 24) // 3 + 1, total_rows=0, **few) == bole.BOLE_ERR_UNSUPPORTED


def test_check_dims_takes_valid_and_null_pointers_are_refused():
    L, bad, P = bole.lib, bole.BOLE_ERR_INVALID_VALUE, 0x1000
    assert L.bole_window_check_dims(ctypes.byref(dims())) == bole.BOLE_OK
    assert L.bole_window_check_dims(ctypes.byref(dims(flags=1))) == bole.BOLE_OK
    assert L.bole_window_check_dims(None) == bad
    d = ctypes.byref(dims())
    need = L.bole_window_workspace_size(d)
    full = [P] * 11
    for hole in (0, 1, 2, 3, 4, 5, 6, 8, 9):
        a = list(full)
        a[hole] = None
        assert L.bole_window_attention(*a, need, d, None, None) == bad, hole
    if need:
        for ws, size in ((None, need), (P + 8, need), (P, need - 1)):
            assert L.bole_window_attention(*full[:10], ws, size, d, None, None) == bad
    assert L.bole_window_attention(*[None] * 11, 0, ctypes.byref(dims(batch=0)), None, None) == bole.BOLE_OK


def test_binding_refuses():
    w = make()
    t = (w.q, w.k, w.v, w.k_cache, w.v_cache, w.page_table, w.cache_len, torch.from_numpy(w.offsets))
    with pytest.raises(ValueError, match="GPU tensor"):
        window.bole_window_attention(*t, 7, 2)
    with pytest.raises(TypeError):
        window.bole_window_attention("q", *t[1:], 7, 2)
