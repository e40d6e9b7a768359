"""The gated delta rule's launch forms that small calls do not reach, against the fp64 oracle:
the token walk with four columns a lane (batches that fill the chip), widths of the matrix-core
kernels beside test_gpu_delta's, and prompts of many chunks.

Every row of a sequence is compared: the oracle has to be finite there. Tolerances:
  - the walk is fp32 throughout. A token's sums have d_k terms, what earlier tokens left decays:
    states within 2 (d_k + 64) 2^-24 of the head's largest value, outputs within the same part of
    |q| |H| and the rounding to their type, half a step of it;
  - prompts of many chunks: states by their Frobenius norm. d_k + 64 roundings a token, of `many`
    tokens' worth that the decays keep, add up as independent ones do:
    2 sqrt((d_k + 64) many) 2^-24. A chunk's decay has an error in common of two units in its last
    place, 4 x 2^-24, for each 64 of those tokens. A column's share may be four times the mean's;
    the rest of an output's limit is test_gpu_delta's.
"""
import numpy as np
import pytest
import torch

from oracle import delta as O
from test_gpu_delta import (BF16, F32, check_out, check_prompt, check_states, column_norms, dev, g, make,
                            on_gpu, state_tol)
from test_gpu_delta import lib  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

H, HK, B = 16, 4, 65


def wide_wavefronts(d_v):
    return B * H * -(-d_v // 32)


def check_rows(got, ref, w):
    """All rows of all sequences, and no others, have a reference and are within the walk's limits."""
    T = int(w.offsets[-1])
    assert np.isfinite(ref[:T]).all() and np.isnan(ref[T:]).all()
    half = 2.0 ** -8 if w.q.dtype == BF16 else 2.0 ** -24
    qn = np.repeat(np.linalg.norm(w.q.double().numpy(), axis=-1), w.v.shape[1] // w.q.shape[1], axis=1)
    lim = half * np.abs(ref[:T]) + (state_tol(w) * qn * column_norms(w)[None])[:T, :, None]
    e = np.abs(got.double().cpu().numpy()[:T] - ref[:T])
    assert (e <= lim).all(), float((e / lim).max())


def off(x):
    """The same values one element behind a 16-byte boundary."""
    return torch.zeros(x.numel() + 8, dtype=x.dtype, device=dev())[1:1 + x.numel()].view(x.shape).copy_(x)


# key rows in whole 16-byte parts or not, of 8, 16 and 32 rows a lane, filled or not; a last block
# of columns that is partly used (40) or whole
WIDTHS = [(64, 40), (40, 64), (17, 128), (128, 40), (72, 64), (100, 128), (256, 40), (200, 64), (130, 40)]


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", WIDTHS, ids=str)
def test_wide_walk(lib, dk, dv, dt):
    assert wide_wavefronts(dv) >= 2048
    shape = (H, HK, dk, dv, dt)
    w = make(201, [1] * B, shape)
    t = on_gpu(w)
    out = lib.bole_delta_step(**t)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w)
    check_rows(out, ref, w)

    sizes = ([5, 0, 9, 1, 12] * B)[:B]
    w = make(202, sizes, shape, kind="deep", spare_rows=2)
    t = on_gpu(w)
    t.pop("q")
    status = torch.full((B,), -1, dtype=torch.int32, device=dev())
    nodes = torch.full((B, 16), -9, dtype=torch.int32, device=dev())
    lib.bole_delta_commit_path(**t, parent=g(w.parent), node_offsets=g(w.offsets),
                               accepted_idx=g(w.accepted_idx), accepted_len=g(w.accepted_len),
                               path_nodes=nodes, tree_status=status)
    assert (w.accepted_len > 1).any() and (w.accepted_len == 0).any()
    check_states(t["H0"], O.commit(w.H0, w.k, w.v, w.gate, w.beta, w.offsets, w.accepted_idx,
                                   w.accepted_len), w)
    want = np.where(w.accepted_idx >= 0, w.accepted_idx + w.offsets[:-1, None], -1)
    assert np.array_equal(nodes.cpu().numpy(), want) and status.tolist() == [0] * B
    none = g(w.accepted_len == 0)
    assert torch.equal(t["H0"][none], g(w.H0)[none])

    w = make(203, ([3, 0, 1, 6] * B)[:B], shape, spare_rows=3)
    t = on_gpu(w)
    out = torch.full_like(t["v"], -7.0)
    lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets), out=out, seq_status=status, force_generic=True)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w)
    check_rows(out, ref, w)
    assert (out[-3:] == -7.0).all() and status.tolist() == [0] * B


@pytest.mark.parametrize("which", ["H0", "k", "v", "gate"])
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_wide_walk_off_16_byte_addresses(lib, which, dt):
    """A state off 16-byte addresses is walked a column a lane, key rows off them by elements."""
    shape = (H, HK, 128, 64, dt)
    w = make(204, [1] * B, shape)
    t = on_gpu(w)
    t[which] = off(t[which])
    if which == "k":
        t["q"] = off(t["q"])
    out = lib.bole_delta_step(**t)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w)
    check_rows(out, ref, w)
    w = make(205, ([7, 1, 12] * B)[:B], shape, kind="deep")
    t = on_gpu(w)
    t.pop("q")
    t[which] = off(t[which])
    lib.bole_delta_commit_path(**t, parent=g(w.parent), node_offsets=g(w.offsets),
                               accepted_idx=g(w.accepted_idx), accepted_len=g(w.accepted_len))
    check_states(t["H0"], O.commit(w.H0, w.k, w.v, w.gate, w.beta, w.offsets, w.accepted_idx,
                                   w.accepted_len), w)


# ---- widths in pairs of columns, and fp32 ones, of the matrix-core kernels

MORE = [(4, 2, 64, 128, BF16), (2, 1, 40, 96, BF16), (2, 2, 72, 160, BF16), (4, 2, 64, 128, F32),
        (2, 1, 40, 96, F32), (2, 1, 72, 160, F32), (3, 3, 64, 64, F32), (2, 2, 72, 40, F32),
        (2, 1, 120, 200, F32)]
MORE_IDS = ["-".join(map(str, s[:4])) + ("-bf16" if s[4] == BF16 else "-f32") for s in MORE]


@pytest.mark.parametrize("shape", MORE, ids=MORE_IDS)
def test_more_widths(lib, shape):
    """Prompts and trees of widths that test_gpu_delta's shapes leave out."""
    w = make(221, [65, 0, 1, 63, 130], shape, spare_rows=3)
    t = on_gpu(w)
    out = torch.full_like(t["v"], -7.0)
    lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets), out=out)
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    check_states(t["H0"], S, w)
    assert np.isfinite(ref[:-3]).all()
    check_prompt(out, ref, w, column_norms(w))
    assert (out[-3:] == -7.0).all()
    for kind in ("random", "chain"):
        w = make(222, [64, 33, 0, 5, 16, 49], shape, kind=kind, spare_rows=2)
        t = on_gpu(w)
        out = torch.full_like(t["v"], -7.0)
        lib.bole_delta_tree_verify(**t, parent=g(w.parent), node_offsets=g(w.offsets), out=out)
        ref = O.verify(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets)
        assert np.isfinite(ref[:-2]).all()
        check_out(out, ref, w, column_norms(w))
        assert (out[-2:] == -7.0).all() and torch.equal(t["H0"].cpu(), w.H0)


@pytest.mark.parametrize("shape", [MORE[0], MORE[2], MORE[5]], ids=[MORE_IDS[0], MORE_IDS[2], MORE_IDS[5]])
def test_tree_verify_off_16_byte_addresses(lib, shape):
    w = make(223, [64, 20, 7], shape)
    t = on_gpu(w)
    a = dict(parent=g(w.parent), node_offsets=g(w.offsets))
    ref = O.verify(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.parent, w.offsets)
    for which in ("H0", "q", "k", "v", "gate", "beta", "out"):
        u = dict(t, out=torch.zeros_like(t["v"]))
        u[which] = off(u[which])
        check_out(lib.bole_delta_tree_verify(**u, **a), ref, w, column_norms(w))


# ---- prompts of many chunks

def state_norm_tol(w, many):
    return (2.0 * ((w.H0.shape[2] + 64) * many) ** 0.5 + 4.0 * many / 64) * 2.0 ** -24


def check_long(out, H0, w, many):
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    T, tol = int(w.offsets[-1]), state_norm_tol(w, many)
    d = np.linalg.norm(H0.double().cpu().numpy() - S, axis=(2, 3)) / np.linalg.norm(S, axis=(2, 3))
    print(f"states off by {d.max():.2e} of their norm, limit {tol:.2e}", flush=True)
    assert d.max() <= tol, d.max()
    assert np.isfinite(ref[:T]).all()
    bf = w.q.dtype == BF16
    lim = (2.0 ** -8 if bf else 2.0 ** -24) * np.abs(ref[:T])
    if bf:
        lim = lim + 2.0 ** -8 * O.pair_terms(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)[:T]
    qn = np.repeat(np.linalg.norm(w.q.double().numpy(), axis=-1), w.v.shape[1] // w.q.shape[1], axis=1)
    lim = lim + ((4 * tol + (4 * 2.0 ** -16 if bf else 0.0)) * qn * column_norms(w)[None])[:T, :, None]
    e = np.abs(out.double().cpu().numpy()[:T] - ref[:T])
    assert (e <= lim).all(), float((e / lim).max())


LONG = [(2, 1, 128, 128, BF16), (2, 2, 64, 16, BF16), (1, 1, 72, 40, BF16), (2, 1, 128, 64, F32),
        (1, 1, 40, 24, F32)]
LONG_IDS = ["-".join(map(str, s[:4])) + ("-bf16" if s[4] == BF16 else "-f32") for s in LONG]


@pytest.mark.parametrize("gate", [None, 0.999], ids=["drawn", "slow"])
@pytest.mark.parametrize("shape", LONG, ids=LONG_IDS)
def test_prompts_of_many_chunks(lib, shape, gate):
    """4,000 tokens, ten chunks with and without a token more, seven and a bit: lines are read
    three chunks early and dropped, buffers alternate, and states carry over all of it. With a
    decay of 0.999 a thousand tokens' worth stays."""
    w = make(211, [4000, 641, 1, 640, 0, 450], shape, spare_rows=3, gate_value=gate)
    t = on_gpu(w)
    out = torch.full_like(t["v"], -7.0)
    lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets), out=out)
    check_long(out, t["H0"], w, 1000.0 if gate else 1.0)
    assert (out[-3:] == -7.0).all() and torch.equal(t["H0"][4].cpu(), w.H0[4])


def test_walked_prompt_rounds_its_outputs_alone(lib):
    """The token walk of a prompt has bf16 outputs within their own rounding, where the chunked
    kernels also round each pair weight."""
    w = make(212, [200, 65], (4, 2, 128, 128, BF16))
    ref, S = O.prefill(w.H0, w.q, w.k, w.v, w.gate, w.beta, w.offsets)
    t = on_gpu(w)
    check_rows(lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets), force_generic=True), ref, w)
    check_states(t["H0"], S, w)
    t = on_gpu(w)
    check_prompt(lib.bole_delta_prefill(**t, seq_offsets=g(w.offsets)), ref, w, column_norms(w))
    check_states(t["H0"], S, w)
