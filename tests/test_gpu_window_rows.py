"""Windowed attention against the fp64 oracle, every row of every sequence compared: large scores
within limits that their arithmetic gives, scores past fp32, more sequences than a call's first
look through its offsets takes, widths and head groups beside test_gpu_window's.

Large scores: q and k are whole numbers whose products' sums stay below 2^24, so that q . k is exact
in fp32 in any order and in both types. What is left of a score's error is relative to it: the
factor scale log2 e (its constant's rounding and the product's), the product with it, the
difference to the reference and the reference's moves. Two scores of a row differ by at most twice
its largest, S: together (2 x 2 + 2 + 2 + 2) 2^-24 S in a weight, once in the numerator and once in
the sum, 20 x 2^-24 S.
"""
import numpy as np
import pytest
import torch

from oracle import window as O
from test_gpu_window import BF16, F32, SHAPES, IDS, dev, g, make, on_gpu, oracle_of
from test_gpu_window import lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def check_rows(got, ref, w, keys, weight_err, rows=None):
    """`rows` (default: all rows of sequences) and no others have a reference; weight_err [T, H]: what
    a softmax weight may be off by, relative, beside its own rounding and the sums'."""
    out, mag, _ = ref
    rows = sorted(range(int(w.offsets[-1])) if rows is None else rows)
    assert np.flatnonzero(np.isfinite(out).all(axis=(1, 2))).tolist() == rows
    bf = w.q.dtype == BF16
    half = 2.0 ** -8 if bf else 2.0 ** -24
    alg = (half if bf else 0.0) + weight_err + keys * 2.0 ** -24 + 2.0 ** -20
    lim = half * np.abs(out) + np.broadcast_to(alg, out.shape[:2])[:, :, None] * mag
    e = np.abs(got.double().cpu().numpy() - out)
    assert (e[rows] <= lim[rows]).all(), float((e[rows] / lim[rows]).max())


def whole_numbers(w, seed, q_most, k_most):
    """Replaces q, k and the cached keys by whole numbers; what nobody sees stays NaN."""
    rng = torch.Generator().manual_seed(seed)
    draw = lambda x, most: torch.randint(-most, most + 1, x.shape, generator=rng).to(x.dtype)
    w.q, w.k = draw(w.q, q_most), draw(w.k, k_most)
    w.k_cache = torch.where(w.k_cache.isnan(), w.k_cache, draw(w.k_cache, k_most))
    assert w.q.shape[2] * q_most * k_most < 2 ** 24


def largest_scores(w, window, sinks, tree, scale):
    """[T, H]: the largest |scale q . k| that a row sees."""
    q, k, kc = (x.double().numpy() for x in (w.q, w.k, w.k_cache))
    G, ps, S = q.shape[1] // k.shape[1], kc.shape[2], np.zeros(q.shape[:2])
    for b, c in enumerate(w.cache_len.tolist()):
        lo = int(w.offsets[b])
        for i in range(int(w.offsets[b + 1]) - lo):
            path = O.path_of(w.parent if tree else None, lo, i)
            pos = c + len(path) - 1
            seen = lambda s: pos - s < window or s < sinks
            K = [kc[w.page_table[b, s // ps], :, s % ps] for s in range(c) if seen(s)]
            K = np.array(K + [k[lo + j] for t, j in enumerate(path) if seen(c + t)])
            for h in range(q.shape[1]):
                S[lo + i, h] = abs(scale) * np.abs(K[:, h // G] @ q[lo + i, h]).max()
    return S


@pytest.mark.parametrize("scale", [None, -0.5, 0.0], ids=str)
@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 2, 3, 4, 5, 6, 7)],
                         ids=[IDS[i] for i in (0, 2, 3, 4, 5, 6, 7)])
def test_large_exact_scores(lib, shape, scale):
    """Scores of several hundred, and of nearly two thousand of the other sign."""
    for sizes, cached, tree in (([1, 1, 1], [400, 64, 130], False), ([30, 3], [200, 64], False),
                                ([30, 3], [200, 64], True)):
        w = make(143, sizes, cached, shape, 180, 4)
        whole_numbers(w, 144, 32, 8)
        out = lib.bole_window_attention(**on_gpu(w), window=180, sinks=4, scale=scale,
                                        parent=g(w.parent) if tree else None)
        S = largest_scores(w, 180, 4, tree, shape[2] ** -0.5 if scale is None else scale)
        assert scale is not None or S.max() > 100.0
        check_rows(out, oracle_of(w, 180, 4, tree, scale), w, 220, 20 * 2.0 ** -24 * S)


@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 2, 4, 6)], ids=[IDS[i] for i in (0, 2, 4, 6)])
def test_rows_beside_scores_past_fp32(lib, shape):
    """One node's query and key are near the type's largest value. No row is left as it was, and
    every row that does not see that key comes out as without it, in the same sequence too."""
    G = shape[0] // shape[1]
    for sizes, cached, tree in (([1, 1], [4000, 70], False), ([40, 2], [4000, 70], True),
                                ([40, 2], [100, 70], False)):
        w = make(147, sizes, cached, shape, 5000, 0)
        t = on_gpu(w)
        T = sum(sizes)
        ref = oracle_of(w, 5000, 0, tree)
        t["q"][0] = 3e38 * torch.sign(t["k"][0, :1].float()).to(t["q"].dtype)
        t["k"][0] = t["k"][0].sign() * 3e38
        out = torch.full_like(t["q"], -7.0)
        lib.bole_window_attention(**t, window=5000, sinks=0, out=out, parent=g(w.parent) if tree else None)
        assert out[0, :G].isnan().all() and not (out == -7.0).all(dim=(1, 2)).any()
        sees = lambda i: i < sizes[0] and 0 in O.path_of(w.parent if tree else None, 0, i)
        rows = [i for i in range(T) if not sees(i)]
        assert len(rows) > (sizes[1] if tree else sizes[1] - 1)
        keep = np.isin(np.arange(T), rows)
        ref = tuple(np.where(keep.reshape(-1, *[1] * (x.ndim - 1)), x, np.nan) for x in ref)
        err = 2 * (shape[2] + 2) * 2.0 ** -24 * np.nan_to_num(ref[2])
        check_rows(out, ref, w, 4100, err, rows)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[4], SHAPES[6]], ids=[IDS[0], IDS[4], IDS[6]])
@pytest.mark.parametrize("cycle", [[1], [3, 0, 1], [40, 0, 1, 0, 0]], ids=str)
def test_seven_hundred_sequences(lib, shape, cycle):
    """More sequences than four loads of offsets hold, single tokens, small and uneven trees."""
    sizes = [0] + (cycle * 700)[:698] + [0]
    cached = [(29 * b) % 41 for b in range(700)]
    w = make(146, sizes, cached, shape, 25, 2, spare_rows=2)
    t = on_gpu(w)
    T = sum(sizes)
    rows = set(range(0, T, max(1, T // 150))) | {0, T - 1}
    for parent in (None, g(w.parent)):
        out, status = torch.full_like(t["q"], -7.0), torch.full((700,), -1, dtype=torch.int32, device=dev())
        lib.bole_window_attention(**t, window=25, sinks=2, out=out, parent=parent, seq_status=status)
        ref = oracle_of(w, 25, 2, parent is not None, rows=rows)
        check_rows(out, ref, w, 70, 2 * (shape[2] + 2) * 2.0 ** -24 * ref[2], rows)
        assert status.tolist() == [0] * 700 and (out[-2:] == -7.0).all()
        assert out[:T].isfinite().all() and not (out[:T] == -7.0).all(dim=(1, 2)).any()


MORE = [(4, 2, 64, 16, F32), (6, 2, 96, 32, F32), (3, 1, 96, 8, BF16), (64, 1, 64, 16, BF16),
        (71, 1, 128, 16, BF16), (130, 1, 64, 32, BF16), (130, 2, 96, 16, F32), (200, 1, 128, 8, F32)]
MORE_IDS = ["-".join(map(str, s[:4])) + ("-bf16" if s[4] == BF16 else "-f32") for s in MORE]


@pytest.mark.parametrize("window,sinks", [(40, 3), (2**31 - 1, 0)], ids=str)
@pytest.mark.parametrize("shape", MORE, ids=MORE_IDS)
def test_more_widths_and_groups(lib, shape, window, sinks):
    """fp32 of every width with a matrix-core kernel; groups of more query heads than a tile has
    rows, whose rows lie in several tiles."""
    for seed, sizes, cached, tree in ((151, [1, 1, 1], [300, 64, 0], False),
                                      (152, [9, 0, 3, 33], [70, 10, 0, 129], True),
                                      (153, [40, 1, 0, 5], [0, 90, 10, 65], False)):
        w = make(seed, sizes, cached, shape, window, sinks, spare_rows=2)
        t = on_gpu(w)
        out, status = torch.full_like(t["q"], -7.0), torch.full((len(sizes),), -1, dtype=torch.int32, device=dev())
        lib.bole_window_attention(**t, window=window, sinks=sinks, out=out, seq_status=status,
                                  parent=g(w.parent) if tree else None)
        ref = oracle_of(w, window, sinks, tree)
        check_rows(out, ref, w, 310, 2 * (shape[2] + 2) * 2.0 ** -24 * ref[2])
        assert (out[-2:] == -7.0).all() and status.tolist() == [0] * len(sizes)


def test_refuses_heads_without_width(lib):
    """A width of 0 is refused as the other shapes are, with or without a scale."""
    w = make(148, [2, 1], [20, 5], SHAPES[0], 16, 2)
    t = {n: x[..., :0].contiguous() if n in ("q", "k", "v", "k_cache", "v_cache") else x
         for n, x in on_gpu(w).items()}
    for scale in (None, 1.0):
        with pytest.raises(ValueError, match="d at least 1"):
            lib.bole_window_attention(**t, window=16, sinks=2, scale=scale)
    t.pop("node_offsets")
    with pytest.raises(ValueError, match="d at least 1"):
        lib.bole_window_workspace_size(**t, window=16, sinks=2)
