"""The GPU tests of the delta rule and of windowed attention leave out rows whose oracle value is
not finite, and hide NaN wherever no row may read. Here, on the CPU: on the inputs that they
compare, the oracle is finite on every row of every sequence and on no other, so nothing that a
row sees is hidden and no comparison is empty."""
import numpy as np
import pytest

import test_gpu_delta as D
import test_gpu_window as N
from oracle import delta

# sizes, cached tokens and trees of test_single_tokens, test_trees, test_prompts, test_tree_shapes
CALLS = [(11, [1] * 7, [0, 1, 63, 64, 65, 500, 16], False, 2),
         (21, [64, 33, 0, 5, 16, 1], [100, 0, 40, 3, 257, 1], True, 2),
         (31, [130, 1, 0, 77, 64], [0, 90, 10, 2, 33], False, 3)]
MORE = [((47, [1, 1], [4000, 70]), 5000, 0, False), ((47, [40, 2], [4000, 70]), 5000, 0, True),
        ((43, [20, 3], [200, 64]), 100, 4, False), ((44, [64, 20, 3], [300, 64, 1000]), 200, 4, True),
        ((22, [64, 40], [30, 5]), 20, 2, True), ((56, [64, 9], [300, 77]), 100, 4, True),
        ((53, [20, 1, 40], [100, 33, 7]), 64, 4, False)]


def one_head(w):
    """The first key head's first two dimensions: what is hidden is hidden in all of them."""
    w.q, w.k, w.v = w.q[:, :1, :2], w.k[:, :1, :2], w.v[:, :1, :2]
    w.k_cache, w.v_cache = w.k_cache[:, :1, :, :2], w.v_cache[:, :1, :, :2]
    return w


def rows_with_a_value(w, window_, sinks, tree):
    out, _, _ = N.oracle_of(one_head(w), window_, sinks, tree)
    return np.flatnonzero(np.isfinite(out).all(axis=(1, 2))).tolist()


@pytest.mark.parametrize("window_,sinks", N.VIEWS, ids=str)
@pytest.mark.parametrize("page", sorted({s[3] for s in N.SHAPES}))
def test_window_views(page, window_, sinks):
    for seed, sizes, cached, tree, spare in CALLS:
        kind = "bestfirst" if tree and window_ > 5 else "random"
        w = N.make(seed, sizes, cached, (1, 1, 2, page, N.F32), window_, sinks, kind=kind, spare_rows=spare)
        assert rows_with_a_value(w, window_, sinks, tree) == list(range(sum(sizes)))


@pytest.mark.parametrize("case", MORE, ids=lambda c: f"{c[0][1]}-{c[1]}-{c[3]}")
def test_window_calls(case):
    (seed, sizes, cached), window_, sinks, tree = case
    for kind in ("random", "chain", "star", "deep"):
        w = N.make(seed, sizes, cached, (1, 1, 2, 16, N.F32), window_, sinks, kind=kind)
        assert rows_with_a_value(w, window_, sinks, tree) == list(range(sum(sizes)))


def test_a_hidden_slot_that_a_row_sees_is_noticed():
    w = N.make(11, [1, 1], [40, 20], (1, 1, 2, 16, N.F32), 8, 2)
    w.v_cache[w.page_table[0, 2], :, 7] = float("nan")
    assert rows_with_a_value(w, 8, 2, False) == [1]


@pytest.mark.parametrize("sizes", D.PROMPTS, ids=str)
def test_prompts(sizes):
    w = D.make(21, sizes, (2, 1, 6, 3, D.F32), spare_rows=3)
    out, S = delta.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    T = sum(sizes)
    assert np.isfinite(out[:T]).all() and np.isnan(out[T:]).all() and np.isfinite(S).all()


@pytest.mark.parametrize("sizes,kind", D.TREES, ids=str)
def test_trees(sizes, kind):
    w = D.make(31, sizes, (2, 1, 6, 3, D.F32), kind=kind, spare_rows=2)
    out = delta.verify(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets)
    T = sum(sizes)
    assert np.isfinite(out[:T]).all() and np.isnan(out[T:]).all()
