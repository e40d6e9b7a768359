"""The gated delta rule's operators against the fp64 oracle (oracle/delta.py).

Tolerances, set from the arithmetic:
  - states: a token's products are sums of d_k terms in fp32 (error at most d_k 2^-24 of the
    terms' magnitudes), a chunk of 64 tokens adds sums of at most 64 more; what earlier tokens
    left decays with the gates (mean about a half, so their errors add up to at most twice one
    token's). 2 (d_k + 64) 2^-24 of the head's largest state value, times the tokens where
    nothing decays;
  - outputs: the same relative to |q| |H| (the largest sum a product with the state can have),
    rounded once: half a step of the output type relative to the value. bf16 factors take
    products with the state as sums of two bf16 terms, 2^-16 each of |q| |H|, four of them;
  - prompts in bf16 round each token pair's weight once to bf16 for the output (not for the
    state): half a step of each such term.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import delta as O

pytestmark = pytest.mark.gpu

BAD_SIZE, BAD_PARENT, BAD_PATH = 1, 2, 3
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tree_speculative_decoding_02_amd as t
    return t


def dev():
    return torch.device("cuda:0")


def g(x):
    return (torch.from_numpy(np.ascontiguousarray(x)) if isinstance(x, np.ndarray) else x).to(dev())


def on_gpu(w):
    return dict(H0=g(w.H0).clone(), q=g(w.q), k=g(w.k), v=g(w.v), gate=g(w.gate), beta=g(w.beta))


def state_tol(w, many=1.0):
    return 2.0 * (w.H0.shape[2] + 64) * 2.0 ** -24 * many


def check_states(got, ref, w, many=1.0):
    got = got.double().cpu().numpy()
    d = np.abs(got - ref).max(axis=(2, 3)) / np.maximum(np.abs(ref).max(axis=(2, 3)), 1e-30)
    assert np.isfinite(got).all() and d.max() <= state_tol(w, many), d.max()


def check_prompt(got, ref, w, states, many=1.0):
    extra = 0.0
    if w.q.dtype == BF16:
        extra = 2.0 ** -8 * O.pair_terms(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_out(got, ref, w, states, many, extra)


def check_out(got, ref, w, states, many=1.0, extra=0.0):
    """states: an upper bound of |H| by column, [H] (the largest over tokens)."""
    half = 2.0 ** -8 if w.q.dtype == BF16 else 2.0 ** -24
    alg = state_tol(w, many) + (4 * 2.0 ** -16 if w.q.dtype == BF16 else 0.0)
    qn = np.linalg.norm(w.q.double().numpy(), axis=-1)
    qn = np.repeat(qn, w.v.shape[1] // qn.shape[1], axis=1)          # [T, H]
    rows = np.isfinite(ref).all(axis=(1, 2))
    lim = half * np.abs(ref) + (alg * qn * states[None])[:, :, None] + extra
    e = np.abs(got.double().cpu().numpy() - ref)[rows]
    assert (e <= lim[rows]).all(), float((e / lim[rows]).max())


def column_norms(w):
    """A bound on the columns of every state met: what H0 holds and what all values can add."""
    h = np.linalg.norm(w.H0.double().numpy(), axis=2).max(axis=(0, 2))
    kmax = np.linalg.norm(w.k.double().numpy(), axis=-1).max() if w.k.numel() else 0.0
    v = np.abs(w.v.double().numpy()).max(axis=(0, 2)) if w.v.numel() else 0.0
    return h + 4.0 * v * max(kmax, 1.0)


SHAPES = [  # heads, key heads, d_k, d_v, factors
    (4, 2, 128, 128, BF16), (3, 3, 64, 64, BF16), (6, 2, 128, 96, BF16), (2, 1, 128, 64, F32),
    (2, 2, 72, 40, BF16), (3, 1, 17, 5, F32), (2, 1, 256, 256, BF16), (1, 1, 1, 1, F32),
    (2, 1, 64, 16, BF16), (2, 1, 40, 24, F32), (3, 1, 8, 8, BF16), (2, 2, 120, 200, BF16),
    (2, 1, 128, 128, F32), (2, 2, 64, 130, F32),
]
IDS = ["-".join(map(str, s[:4])) + ("-bf16" if s[4] == BF16 else "-f32") for s in SHAPES]


def make(seed, sizes, shape, **kw):
    H, HK, dk, dv, dt = shape
    return W.make_delta(seed, sizes, H, HK, dk, dv, dt, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_step(lib, shape):
    for B in (1, 5):
        w = make(11, [1] * B, shape)
        t = on_gpu(w)
        out = lib.bole_delta_step(**t)
        ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
        check_states(t["H0"], S, w)
        check_out(out, ref, w, column_norms(w))


PROMPTS = [[1], [64], [65, 0, 1, 63, 130], [7, 200], [128, 64, 0]]


@pytest.mark.parametrize("sizes", PROMPTS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_prefill(lib, shape, sizes):
    w = make(21, sizes, shape, spare_rows=3)
    t = on_gpu(w)
    out = torch.full_like(t["v"], -7.0)
    status = torch.full((len(sizes),), -1, dtype=torch.int32, device=dev())
    lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets), out=out, seq_status=status)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w)
    check_prompt(out, ref, w, column_norms(w))
    assert (out[-3:] == -7.0).all() and status.tolist() == [0] * len(sizes)
    for b, n in enumerate(sizes):  # no token: the state keeps its bits
        if n == 0:
            assert torch.equal(t["H0"][b].cpu(), w.H0[b])


@pytest.mark.parametrize("shape", [SHAPES[1], SHAPES[4], SHAPES[9], SHAPES[5]],
                         ids=[IDS[1], IDS[4], IDS[9], IDS[5]])
def test_many_sequences(lib, shape):
    """More sequences than a wavefront has lanes, empty ones among them and at both ends."""
    sizes = [0] + ([33, 1, 0, 64, 5, 0, 70] * 20)[:138] + [0]
    w = make(24, sizes, shape, spare_rows=3)
    t = on_gpu(w)
    out, status = torch.full_like(t["v"], -7.0), torch.full((140,), -1, dtype=torch.int32, device=dev())
    lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets), out=out, seq_status=status)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w)
    check_prompt(out, ref, w, column_norms(w))
    assert (out[-3:] == -7.0).all() and status.tolist() == [0] * 140


@pytest.mark.parametrize("shape", SHAPES[:4], ids=IDS[:4])
@pytest.mark.parametrize("kw", [dict(gate_value=1.0), dict(gate_value=0.0), dict(gate_value=1e-30),
                                dict(gate_value=1.02), dict(strength=0.0), dict(strength=1.0),
                                dict(strength=1.0, gate_value=1.0), dict(key_std=1e-3),
                                dict(key_std=1.3, gate_value=0.9)], ids=str)
def test_prefill_gates_and_strengths(lib, shape, kw):
    """No decay, a reset at every token, growth, no update, full updates, short and long keys."""
    w = make(22, [90, 3, 64], shape, **kw)
    t = on_gpu(w)
    out = lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets))
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    many = 90.0 if kw.get("gate_value", 0.5) >= 0.9 else 1.0
    if kw.get("gate_value") == 1.02:
        many *= 1.02 ** 90
    check_states(t["H0"], S, w, many)
    check_prompt(out, ref, w, column_norms(w) * (1.02 ** 90 if many > 100 else 1.0), many)


@pytest.mark.parametrize("shape", SHAPES[:4], ids=IDS[:4])
def test_prefill_after_strong_decays(lib, shape):
    """Forty near-resets, then tokens that hardly decay: pair weights of the later ones must
    not carry the rounding of the large sum of logarithms before them."""
    w = make(23, [128], shape)
    w.gate[:40] = 1e-20
    w.gate[40:] = 0.999
    t = on_gpu(w)
    out = lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets))
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w, 10.0)
    check_prompt(out, ref, w, column_norms(w), 10.0)


@pytest.mark.parametrize("shape", SHAPES[:4], ids=IDS[:4])
def test_prefill_with_repeated_keys(lib, shape):
    """Every token has the same key: the triangular system is as full as it can be."""
    w = make(24, [100], shape, strength=0.9)
    w.k[:] = w.k[0]
    t = on_gpu(w)
    out = lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets))
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w, 2.0)
    check_prompt(out, ref, w, column_norms(w), 2.0)


def test_prefill_is_step_by_step_and_resumable(lib):
    """A prompt in one call, in two calls, and token by token: the same states to fp32."""
    w = make(25, [75, 75], SHAPES[0])
    whole, cut, steps = on_gpu(w), on_gpu(w), on_gpu(w)
    o1 = lib.bole_delta_prefill(**whole, seq_offsets=g(w.offsets))
    rows = lambda a, b: torch.cat([torch.arange(a, b), 75 + torch.arange(a, b)]).to(dev())
    for a, b in ((0, 33), (33, 75)):
        r = rows(a, b)
        f = {n: cut[n][r].contiguous() for n in ("q", "k", "v", "gate", "beta")}
        lib.bole_delta_prefill(cut["H0"], **f, seq_offsets=g(np.array([0, b - a, 2 * (b - a)], np.int32)))
    for i in range(75):
        r = rows(i, i + 1)
        f = {n: steps[n][r].contiguous() for n in ("q", "k", "v", "gate", "beta")}
        o = lib.bole_delta_step(steps["H0"], **f)
    scale = float(whole["H0"].abs().max())
    assert float((whole["H0"] - cut["H0"]).abs().max()) <= 2 * state_tol(w) * scale
    assert float((whole["H0"] - steps["H0"]).abs().max()) <= 2 * state_tol(w) * scale
    assert float((o1[[74, 149]].float() - o.float()).abs().max()) <= 2.0 ** -7 * float(o.abs().max())


def test_prefill_bad_offsets_touch_nothing(lib):
    for bad in ([0, 5, 3, 9], [-1, 2, 3, 9], [0, 2, 3, 10]):
        w = make(26, [3, 3, 3], SHAPES[0])
        t = on_gpu(w)
        out = torch.full_like(t["v"], -7.0)
        status = torch.full((3,), -1, dtype=torch.int32, device=dev())
        lib.bole_delta_prefill(**t, seq_offsets=g(np.array(bad, np.int32)), out=out, seq_status=status)
        assert status.tolist() == [BAD_SIZE] * 3
        assert (out == -7.0).all() and torch.equal(t["H0"].cpu(), w.H0)


def test_prefill_rows_before_the_first_sequence(lib):
    """Sequences that start behind rows of nobody: those rows are not read."""
    w = make(27, [70, 0, 129], SHAPES[0])
    t = on_gpu(w)
    H = t.pop("H0")
    u = {n: torch.cat([torch.full((150, *x.shape[1:]), float("nan"), dtype=x.dtype, device=dev()), x])
         for n, x in t.items()}
    out, status = torch.full_like(u["v"], -7.0), torch.full((3,), -1, dtype=torch.int32, device=dev())
    lib.bole_delta_prefill(H, **u, seq_offsets=g(w.offsets) + 150, out=out, seq_status=status)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(H, S, w)
    check_prompt(out[150:], ref, w, column_norms(w))
    assert (out[:150] == -7.0).all() and status.tolist() == [0] * 3


TREES = [([1], "random"), ([64, 33, 0, 5, 16, 17], "random"), ([32, 31], "bestfirst"),
         ([64, 50], "chain"), ([64, 20], "star"), ([48], "deep")]


@pytest.mark.parametrize("sizes,kind", TREES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_tree_verify(lib, shape, sizes, kind):
    w = make(31, sizes, shape, kind=kind, spare_rows=2)
    t = on_gpu(w)
    out = torch.full_like(t["v"], -7.0)
    status = torch.full((len(sizes),), -1, dtype=torch.int32, device=dev())
    lib.bole_delta_tree_verify(**t, parent=g(w.parent), node_offsets=g(w.offsets), out=out,
                               tree_status=status)
    ref = O.verify(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets)
    check_out(out, ref, w, column_norms(w))
    assert (out[-2:] == -7.0).all() and status.tolist() == [0] * len(sizes)
    assert torch.equal(t["H0"].cpu(), w.H0)


@pytest.mark.parametrize("shape", SHAPES[:4], ids=IDS[:4])
def test_tree_verify_equals_generic(lib, shape):
    w = make(32, [64, 40, 7, 32], shape)
    t = on_gpu(w)
    a = dict(parent=g(w.parent), node_offsets=g(w.offsets))
    x = lib.bole_delta_tree_verify(**t, **a)
    y = lib.bole_delta_tree_verify(**t, **a, force_generic=True)
    ref = O.verify(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets)
    check_out(x, ref, w, column_norms(w))
    check_out(y, ref, w, column_norms(w))


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], SHAPES[5]], ids=[IDS[0], IDS[3], IDS[5]])
def test_tree_verify_bad_trees(lib, shape):
    """A bad-parent tree's rows become NaN, a tree of bad size is not touched, the others are."""
    w = make(33, [10, 20, 30, 5], shape)
    t = on_gpu(w)
    a = dict(parent=g(w.parent), node_offsets=g(w.offsets))
    good = lib.bole_delta_tree_verify(**t, **a)
    par = w.parent.copy()
    par[10 + 4] = 4                      # its own parent
    status = torch.full((4,), -1, dtype=torch.int32, device=dev())
    out = lib.bole_delta_tree_verify(**t, parent=g(par), node_offsets=a["node_offsets"],
                                     tree_status=status)
    assert status.tolist() == [0, BAD_PARENT, 0, 0]
    assert out[10:30].isnan().all()
    assert torch.equal(out[:10], good[:10]) and torch.equal(out[30:], good[30:])
    offs = np.array([0, 10, 8, 60, 65], np.int32)   # tree 1 runs backwards; tree 2 then has 52
    out = torch.full_like(t["v"], -7.0)
    lib.bole_delta_tree_verify(**t, parent=g(w.parent), node_offsets=g(offs), out=out,
                               tree_status=status)
    assert status.tolist()[1] == BAD_SIZE and status.tolist()[0] in (0, BAD_PARENT)
    offs = np.array([0, 10, 30, 60, 66], np.int32)  # the last tree ends outside
    out.fill_(-7.0)
    lib.bole_delta_tree_verify(**t, parent=g(w.parent), node_offsets=g(offs), out=out,
                               tree_status=status)
    assert status.tolist() == [0, 0, 0, BAD_SIZE]
    assert (out[60:] == -7.0).all() and torch.equal(out[:60], good[:60])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_commit(lib, shape):
    w = make(41, [64, 33, 0, 5, 16, 17], shape, kind="deep", spare_rows=1)
    t = on_gpu(w)
    t.pop("q")
    status = torch.full((6,), -1, dtype=torch.int32, device=dev())
    nodes = torch.full((6, 16), -9, dtype=torch.int32, device=dev())
    lib.bole_delta_commit_path(**t, parent=g(w.parent), node_offsets=g(w.offsets),
                               accepted_idx=g(w.accepted_idx), accepted_len=g(w.accepted_len),
                               path_nodes=nodes, tree_status=status)
    S = O.commit(w.H0, w.k, w.v, w.gate, w.beta, w.offsets, w.accepted_idx, w.accepted_len)
    check_states(t["H0"], S, w)
    want = np.where(w.accepted_idx >= 0, w.accepted_idx + w.offsets[:-1, None], -1)
    assert np.array_equal(nodes.cpu().numpy(), want) and status.tolist() == [0] * 6
    for b in range(6):
        if w.accepted_len[b] == 0:
            assert torch.equal(t["H0"][b].cpu(), w.H0[b])


def test_commit_long_path(lib):
    """The longest path there can be: 64 nodes of one chain."""
    w = make(42, [64, 64], SHAPES[0], kind="chain", max_path=64)
    w.accepted_idx[:] = np.arange(64)
    w.accepted_len[:] = [64, 63]
    w.accepted_idx[1, 63] = -1
    t = on_gpu(w)
    t.pop("q")
    lib.bole_delta_commit_path(**t, parent=g(w.parent), node_offsets=g(w.offsets),
                               accepted_idx=g(w.accepted_idx), accepted_len=g(w.accepted_len))
    check_states(t["H0"], O.commit(w.H0, w.k, w.v, w.gate, w.beta, w.offsets, w.accepted_idx,
                                   w.accepted_len), w)


def test_commit_bad_paths_keep_the_state(lib):
    w = make(43, [10, 20, 30, 5, 4], SHAPES[0], kind="chain")
    idx, n = w.accepted_idx.copy(), w.accepted_len.copy()
    idx[:, :3], idx[:, 3:], n[:] = [0, 1, 2], -1, 3
    idx[0, 1] = 2                       # not a chain
    n[1] = 17                           # longer than max_path
    idx[2, 0] = 1                       # does not start at a root
    par = w.parent.copy()
    par[w.offsets[3] + 1] = 3           # parent after the node
    t = on_gpu(w)
    t.pop("q")
    status = torch.full((5,), -1, dtype=torch.int32, device=dev())
    nodes = torch.full((5, 16), -9, dtype=torch.int32, device=dev())
    lib.bole_delta_commit_path(**t, parent=g(par), node_offsets=g(w.offsets), accepted_idx=g(idx),
                               accepted_len=g(n), path_nodes=nodes, tree_status=status)
    assert status.tolist() == [BAD_PATH, BAD_PATH, BAD_PATH, BAD_PARENT, 0]
    assert torch.equal(t["H0"][:4].cpu(), w.H0[:4]) and (nodes[:4] == -1).all()
    n[:4] = 0
    check_states(t["H0"], O.commit(w.H0, w.k, w.v, w.gate, w.beta, w.offsets, idx, n), w)


# ---- how a program calls them

def test_unaligned_and_sliced_buffers(lib):
    """State, factors and outputs that start off 16-byte boundaries, inside larger buffers."""
    w = make(51, [40, 70], SHAPES[0])
    t = on_gpu(w)

    def off(x, by):
        buf = torch.zeros(x.numel() + 8, dtype=x.dtype, device=dev())
        y = buf[by:by + x.numel()].view(x.shape)
        return y.copy_(x)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    for which in ("H0", "q", "k", "v", "gate", "beta"):
        u = dict(t, H0=t["H0"].clone())
        u[which] = off(u[which], 1)
        out = off(torch.zeros_like(t["v"]), 3)
        lib.bole_delta_prefill(**u, seq_offsets=g(w.offsets), out=out)
        check_states(u["H0"], S, w)
        check_prompt(out, ref, w, column_norms(w))


def test_states_past_32_bit_offsets(lib):
    """5 GB of states, the last sequences of which have rows: they come out as the oracle's, and
    the state of every sequence without a token keeps its bits."""
    H, B = 32, 2400
    shape = (H, 4, 128, 128, BF16)

    def embed(w):
        lead = B - len(w.offsets) + 1
        big = torch.empty(B, H, 128, 128, device=dev()).normal_(generator=torch.Generator(dev()).manual_seed(5))
        big[lead:] = g(w.H0)
        return big, g(np.concatenate([np.zeros(lead, np.int32), w.offsets])), lead

    w = make(55, [70, 3], shape)
    t = on_gpu(w)
    big, offs, lead = embed(w)
    before = big[:lead].clone()
    t["H0"] = big
    out = lib.bole_delta_prefill(**t, seq_offsets=offs)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(big[lead:], S, w)
    check_prompt(out, ref, w, column_norms(w))
    assert torch.equal(big[:lead], before)

    w = make(56, [20, 40], shape)
    t = on_gpu(w)
    big[lead:] = g(w.H0)
    t["H0"] = big
    a = dict(parent=g(w.parent), node_offsets=offs.clone())
    a["node_offsets"][lead:] = g(w.offsets)
    out = lib.bole_delta_tree_verify(**t, **a)
    check_out(out, O.verify(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets), w, column_norms(w))
    t.pop("q")
    idx = torch.full((B, w.accepted_idx.shape[1]), -1, dtype=torch.int32, device=dev())
    many = torch.zeros(B, dtype=torch.int32, device=dev())
    idx[lead:], many[lead:] = g(w.accepted_idx), g(w.accepted_len)
    lib.bole_delta_commit_path(**t, **a, accepted_idx=idx, accepted_len=many)
    check_states(big[lead:], O.commit(w.H0, w.k, w.v, w.gate, w.beta, w.offsets, w.accepted_idx,
                                      w.accepted_len), w)
    assert torch.equal(big[:lead], before)

    w = make(57, [1, 1], shape)
    t = on_gpu(w)
    big[lead:] = g(w.H0)
    wide = {n: torch.cat([torch.zeros(lead, *x.shape[1:], dtype=x.dtype, device=dev()), x])
            for n, x in t.items() if n != "H0"}
    wide["gate"][:lead] = 1.0            # no strength, no decay: those states stay
    out = lib.bole_delta_step(big, **wide)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(big[lead:], S, w)
    check_out(out[lead:], ref, w, column_norms(w))
    assert torch.equal(big[:lead], before)


def test_prefill_then_verify_then_commit(lib):
    """One sequence's life: a prompt, a draft tree verified on its state, the accepted path
    committed, the next tree, and a single token after it."""
    B, shape = 3, SHAPES[0]
    p = make(61, [70, 5, 129], shape)
    t = on_gpu(p)
    H = t["H0"]
    lib.bole_delta_prefill(**t, seq_offsets=g(p.offsets))
    _, S = O.prefill(p.H0, p.q, p.k, p.v, p.gate, p.beta, p.offsets)
    check_states(H, S, p)
    for step in range(3):
        w = make(70 + step, [32, 20, 64], shape, kind="bestfirst")
        w.H0 = torch.from_numpy(S).float()
        t = on_gpu(w)
        del t["H0"]
        a = dict(parent=g(w.parent), node_offsets=g(w.offsets))
        out = lib.bole_delta_tree_verify(H, **t, **a)
        check_out(out, O.verify(S, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets), w,
                  column_norms(w))
        t.pop("q")
        lib.bole_delta_commit_path(H, **t, **a, accepted_idx=g(w.accepted_idx),
                                   accepted_len=g(w.accepted_len))
        S = O.commit(S, w.k, w.v, w.gate, w.beta, w.offsets, w.accepted_idx, w.accepted_len)
        check_states(H, S, w, 2.0)
    w = make(80, [1] * B, shape)
    w.H0 = torch.from_numpy(S).float()
    t = on_gpu(w)
    del t["H0"]
    out = lib.bole_delta_step(H, **t)
    ref, S = O.prefill(S, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_out(out, ref, w, column_norms(w))
    check_states(H, S, w, 2.0)


def test_prefill_on_two_streams_at_once(lib):
    """Two prompts at the same time, each with its own workspace, and the binding's default
    stream taken from the context."""
    ws = [make(90 + i, [300, 64, 17], SHAPES[0]) for i in range(2)]
    ts = [on_gpu(w) for w in ws]
    offs = [g(w.offsets) for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ws]
    outs = []
    for t, o, s in zip(ts, offs, streams):
        with torch.cuda.stream(s):
            outs.append(lib.bole_delta_prefill(**t, seq_offsets=o))
    torch.cuda.synchronize()
    for w, t, out in zip(ws, ts, outs):
        ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
        check_states(t["H0"], S, w)
        check_prompt(out, ref, w, column_norms(w))
    # a stream given by hand: outputs and workspace belong to it
    t = on_gpu(ws[0])
    torch.cuda.synchronize()
    out = lib.bole_delta_prefill(**t, seq_offsets=offs[0], stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(out, outs[0]) and torch.equal(t["H0"], ts[0]["H0"])


def test_graph_replays_of_a_decode_step(lib):
    """Verify, commit, step and prefill captured together; every replay, with eager work in
    between, equals the eager calls bit for bit."""
    sizes = [32, 20, 64, 1]
    w, s, p = make(95, sizes, SHAPES[0]), make(96, [1] * 4, SHAPES[0]), make(97, [80, 2, 0, 64], SHAPES[0])
    a, b, c = on_gpu(w), on_gpu(s), on_gpu(p)
    H = a.pop("H0")
    b.pop("H0"), c.pop("H0")
    tree = dict(parent=g(w.parent), node_offsets=g(w.offsets))
    path = dict(accepted_idx=g(w.accepted_idx), accepted_len=g(w.accepted_len))
    ka = {n: x for n, x in a.items() if n != "q"}
    offs = g(p.offsets)
    outs = [torch.zeros_like(x["v"]) for x in (a, b, c)]
    # bound calls take the stream that is current when they are called: the capture's too
    calls = [lib.bind_delta_tree_verify(H, **a, **tree, out=outs[0]),
             lib.bind_delta_commit_path(H, **ka, **tree, **path),
             lib.bind_delta_step(H, **b, out=outs[1]),
             lib.bind_delta_prefill(H, **c, seq_offsets=offs, out=outs[2])]

    def run():
        for call in calls:
            call()
    start = H.clone()
    want = []
    for _ in range(4):
        run()
        want.append([H.clone()] + [o.clone() for o in outs])
    torch.cuda.synchronize()
    H.copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    H.copy_(start)
    for i in range(4):
        graph.replay()
        z = torch.randn(1 << 16, device=dev())
        assert float((z * 2.0).sum().item()) == float((z * 2.0).sum().item())
        torch.cuda.synchronize()
        for x, y in zip(want[i], [H] + outs):
            assert torch.equal(x, y)


def test_results_repeat_bit_for_bit(lib):
    w = make(98, [200, 64, 33], SHAPES[0])
    got = []
    for _ in range(3):
        t = on_gpu(w)
        got.append((lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets)), t["H0"]))
    for o, h in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(h, got[0][1])


def test_binding_refuses(lib):
    w = make(99, [5, 6], SHAPES[0])
    t = on_gpu(w)
    offs = g(w.offsets)
    with pytest.raises(ValueError, match="overlaps"):
        lib.bole_delta_prefill(**t, seq_offsets=offs, out=t["v"])
    with pytest.raises(ValueError, match="contiguous"):
        lib.bole_delta_prefill(**dict(t, gate=t["gate"].t().contiguous().t()), seq_offsets=offs)
    with pytest.raises(ValueError, match="divisor"):
        lib.bole_delta_prefill(**dict(t, k=t["k"].repeat(1, 2, 1)[:, :3].contiguous()), seq_offsets=offs)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        lib.bole_delta_prefill(**dict(t, k=t["k"].half(), q=t["q"].half(), v=t["v"].half()), seq_offsets=offs)
    with pytest.raises(TypeError, match="int32"):
        lib.bole_delta_prefill(**t, seq_offsets=offs.long())
    with pytest.raises(ValueError, match="T must equal B"):
        lib.bole_delta_step(**t)
    need = lib.bole_delta_prefill_workspace_size(**t)
    if need:
        with pytest.raises(ValueError, match="workspace"):
            lib.bole_delta_prefill(**t, seq_offsets=offs,
                                   workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev()))
