"""Linear attention with decays above 1, whose products leave fp32's range on the way while every state
and output stays within it, against the fp64 oracle (oracle/linear.py).

Tolerances as test_gpu_linear.py derives them, but that a decay there moves what it leaves of a term
by less than 2^-24 of the term. Here products grow: an exponential's argument x is rounded to
2^-24 |x|, which moves it by ln 2 of that and so by less than |x| 2^-24, and one taken as two roots
has both roots' two steps and a rounding more, 5 2^-24. Over a prompt the arguments' sizes add up to
at most the sum A of |log2 gate|, and n tokens have at most n / 64 + 1 chunks and as many segments: A +
10 (n / 64 + 1) steps of 2^-24 of the terms' magnitudes more.
"""
from types import SimpleNamespace

import numpy as np
import pytest

from oracle import linear as O
from test_gpu_linear import BF16, F32, g, lib, make, on_gpu  # noqa: F401 (lib: the fixture)

pytestmark = pytest.mark.gpu

SHAPES = [(4, 2, 128, 64, BF16), (2, 2, 64, 128, BF16), (2, 1, 72, 40, BF16), (2, 2, 128, 64, F32), (2, 1, 40, 16, F32)]
IDS = ["-".join(map(str, s[:4])) + ("-bf16" if s[4] == BF16 else "-f32") for s in SHAPES]


def from_nothing(shape, **kw):
    """64 decays of 4 on a state of zeros: 2^128, which the last tokens see of nothing."""
    w = make(51, [70, 3], shape, **kw)
    w.H0.zero_()
    w.v *= 2.0 ** -20
    w.gate[:64], w.gate[64:] = 4.0, 0.5
    return w


def there_and_back(shape, **kw):
    """A small state grows by 1e40 and is taken back, twice; tokens before the growth are as small."""
    w = make(52, [120, 70], shape, **kw)
    w.H0 *= 1e-30
    for at in (9, 130):
        lo = 0 if at < 120 else 120
        w.v[lo:at + 2] *= 1e-30
        w.gate[lo:at] = 0.9
        w.gate[at:at + 2], w.gate[at + 2:at + 4] = 1e20, 1e-20
    return w


def a_pair_apart(shape, **kw):
    """Only the products between two tokens pass 2^128: a reset, a small token, growth."""
    w = make(53, [66], shape, **kw)
    w.gate[20] = 0.0
    w.k[20], w.v[20] = w.k[20] * 2.0 ** -60, w.v[20] * 2.0 ** -60
    w.gate[21:24], w.v[21:24] = 2.0 ** 45, w.v[21:24] * 2.0 ** -110
    w.gate[24:26] = 2.0 ** -60
    return w


def over_segments(shape, **kw):
    """300 tokens without values that grow the state by 2^175, one head's from nothing."""
    w = make(54, [600, 40], shape, **kw)
    w.H0 *= 1e-22
    w.H0[:, 0] = 0.0
    w.v[:300] = 0.0
    w.gate[:300], w.gate[300:] = 1.5, 0.9
    return w


CASES = [from_nothing, there_and_back, a_pair_apart, over_segments]


def check(out, S, w, chunked):
    r = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.offsets)
    u = 2.0 ** -24
    assert max(np.abs(r.S).max(), np.nanmax(np.abs(r.out)), r.out_mag.max()) < 1e37
    gate = w.gate.double().numpy()
    A = np.abs(np.log2(np.where(gate > 0, gate, 1.0))).reshape(len(gate), -1).max(axis=1)
    n = np.diff(w.offsets)
    more = [A[w.offsets[b]:w.offsets[b + 1]].sum() + 10 * (n[b] / 64 + 1) for b in range(len(n))]
    lim = (2 * n + 16 + more)[:, None, None, None] * u * r.S_mag + 1e-37
    e = np.abs(S.double().cpu().numpy() - r.S)
    assert (e <= lim).all(), ("state", float((e / lim).max()))
    bf = w.v.dtype == BF16
    rows = np.repeat(more, n)[:, None, None] + 2 * r.tokens[:, None, None] + 16 + w.k.shape[2]
    lim = (2.0 ** -8 if bf else u) * np.abs(r.out) + rows * u * r.out_mag
    if bf and chunked:
        lim += 2.0 ** -17 * r.out_mag + 2.0 ** -8 * r.pair
    e = np.abs(out.double().cpu().numpy() - r.out)
    assert (e <= lim + 1e-37).all(), ("out", float(np.nanmax(e / (lim + 1e-37))))


@pytest.mark.parametrize("case", CASES, ids=lambda c: c.__name__)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_chunked(lib, shape, case):  # noqa: F811
    w = case(shape)
    t = on_gpu(w)
    check(lib.bole_linear_prefill(**t, seq_offsets=g(w.offsets)), t["H0"], w, True)


@pytest.mark.parametrize("channel", [False, True], ids=["head", "channel"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: c.__name__)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_walked(lib, shape, case, channel):  # noqa: F811
    w = case(shape, channel=channel)
    t = on_gpu(w)
    check(lib.bole_linear_prefill(**t, seq_offsets=g(w.offsets), force_generic=True), t["H0"], w, False)


@pytest.mark.parametrize("shape", [(64, 32, 128, 128, BF16), (64, 32, 64, 128, BF16), (64, 16, 72, 136, BF16)], ids=str)
def test_chunked_in_128_columns(lib, shape):  # noqa: F811
    """The form with 128 columns a workgroup, where one segment of many grows; some heads against the oracle."""
    w = make(55, [2160, 90], shape, gate_value=None)
    w.gate.copy_(w.gate ** 0.02)
    for at in (700, 2200):
        lo = 0 if at < 2160 else 2160
        w.H0[int(lo > 0)] *= 1e-30
        w.v[lo:at + 2] *= 1e-30
        w.gate[at:at + 2], w.gate[at + 2:at + 4] = 1e20, 1e-20
    t = on_gpu(w)
    out = lib.bole_linear_prefill(**t, seq_offsets=g(w.offsets))
    heads = [0, 37, 63]
    keys = [h // (shape[0] // shape[1]) for h in heads]
    part = SimpleNamespace(H0=w.H0[:, heads], q=w.q[:, keys], k=w.k[:, keys], v=w.v[:, heads], gate=w.gate[:, heads],
                           offsets=w.offsets)
    check(out[:, heads], t["H0"][:, heads], part, True)
