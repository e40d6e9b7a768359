"""Launch forms and limits of linear attention and of attention behind prefixes beside those of
test_gpu_linear.py and test_gpu_paged.py, whose limits' derivations hold here: prompts that are walked
though their sizes fit the chunked form (the limits without that form's roundings), walked prompts in
segments of hundreds of tokens, a prefix against windowed attention over the same keys in one table,
calls without rows.
"""
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import paged as P
from test_gpu_linear import BF16, F32, check, dev, g, lib, make, on_gpu  # noqa: F401 (lib: the fixture)
import test_gpu_paged as paged
from test_gpu_window import check as check_attention


def off_16_bytes(x):
    buf = torch.zeros(x.numel() + 8, dtype=x.dtype, device=dev())
    return buf[1:1 + x.numel()].view(x.shape).copy_(x)


pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("channel", [False, True], ids=["head", "channel"])
@pytest.mark.parametrize("name", ["q", "k", "v", "out"])
def test_rows_off_16_bytes_are_walked_in_fp32(lib, name, channel):  # noqa: F811
    """bf16 prompts that are walked keep neither a rounded weight nor a state in two terms."""
    w = make(70, [70, 9, 300], (4, 2, 128, 64, BF16), channel=channel)
    t = dict(on_gpu(w), out=torch.zeros_like(g(w.v)))
    t[name] = off_16_bytes(t[name])
    lib.bole_linear_prefill(**t, seq_offsets=g(w.offsets))
    check(t["out"], t["H0"], w, w.offsets, chunked=False)


LONG = [(64, 32, 128, 128, BF16), (64, 32, 128, 64, F32), (64, 16, 72, 40, BF16), (64, 64, 50, 30, BF16), (40, 8, 200, 64, F32)]


@pytest.mark.parametrize("channel", [False, True], ids=["head", "channel"])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_walked_prompts_in_long_segments(lib, shape, channel):  # noqa: F811
    """Many heads, so that segments have 80 to 330 tokens; decays near one; some heads against the oracle."""
    w = make(71, [2100, 90, 0, 400], shape, channel=channel, gate_value=None)
    w.gate.copy_(w.gate ** 0.02)
    t = on_gpu(w)
    out = lib.bole_linear_prefill(**t, seq_offsets=g(w.offsets), force_generic=True)
    heads = [0, 17, shape[0] - 1]
    keys = [h // (shape[0] // shape[1]) for h in heads]
    part = SimpleNamespace(H0=w.H0[:, heads], q=w.q[:, keys], k=w.k[:, keys], v=w.v[:, heads], gate=w.gate[:, heads],
                           offsets=w.offsets)
    check(out[:, heads], t["H0"][:, heads], part, w.offsets, chunked=False)


def test_linear_prompts_without_rows(lib):  # noqa: F811
    for shape in ((4, 2, 128, 64, BF16), (2, 1, 13, 7, BF16), (2, 2, 64, 32, F32)):
        for channel in (False, True):
            w = make(72, [0, 0, 0], shape, channel=channel)
            t = on_gpu(w)
            H, status = t["H0"].clone(), torch.full((3,), -1, dtype=torch.int32, device=dev())
            out = lib.bole_linear_prefill(**dict(t, H0=H), seq_offsets=g(w.offsets), seq_status=status)
            assert out.shape[0] == 0 and torch.equal(H, t["H0"]) and status.tolist() == [0, 0, 0]


def test_rotation_without_rows(lib):  # noqa: F811
    for shape in (paged.ROTARY[0], paged.ROTARY[6]):
        for tree in (False, True):
            w = paged.make_rotary(73, [0, 0], [3, 5], shape, spare=0, tree=tree)
            status = paged.i32([-1, -1])
            q, k = paged.call_rotary(lib, w, seq_status=status)
            assert q.shape[0] == 0 and k.shape[0] == 0 and status.tolist() == [0, 0]


def one_table(w, page_size):
    """Page tables and lengths of the same sequences with their prefixes ahead of their own tokens."""
    n = lambda x: x.numpy()
    lines, lens = [], []
    for b in range(len(w.cache_len)):
        gr = P.group_of(n(w.group_offsets), b)
        head = 0 if gr is None else int(w.prefix_len[gr])
        assert head % page_size == 0
        shared = [] if gr is None else n(w.prefix_table)[gr, :head // page_size].tolist()
        lines.append(shared + n(w.page_table)[b].tolist())
        lens.append(head + int(w.cache_len[b]))
    table = np.full((len(lines), max(map(len, lines))), -1, np.int32)
    for b, line in enumerate(lines):
        table[b, :len(line)] = line
    return table, np.array(lens, np.int32)


@pytest.mark.parametrize("kind", list(paged.CALLS))
@pytest.mark.parametrize("shape", [(8, 2, 128, 16, BF16), (4, 4, 64, 64, BF16), (4, 2, 96, 16, F32), (3, 3, 33, 8, F32)], ids=str)
def test_prefix_is_windowed_attention_over_one_table(lib, shape, kind):  # noqa: F811
    """Prefixes that end with a page: the other operator, over the same pages in one table a sequence.
    Both lie within their limits of the oracle, so within twice that of each other."""
    sizes, cached = paged.CALLS[kind]
    w = paged.make(74, sizes, cached, ([320, 64, 0], [0, 2, 5, 6]), shape)
    t, tree = paged.on_gpu(w), kind == "trees"
    parent = g(w.parent) if tree else None
    got = lib.bole_prefix_attention(**t, parent=parent)
    table, lens = one_table(w, shape[3])
    own = {x: t[x] for x in ("q", "k", "v", "k_cache", "v_cache", "node_offsets")}
    whole = lib.bole_window_attention(**own, page_table=g(table), cache_len=g(lens), window=2**31 - 1, sinks=0, parent=parent)
    ref = paged.oracle_of(w, tree)
    keys = 320 + 500 + 130
    for x in (got, whole):
        check_attention(x, ref, w, keys)
    out, mag, reach = ref
    half = 2.0 ** -8 if w.q.dtype == BF16 else 2.0 ** -24
    alg = (half if w.q.dtype == BF16 else 0.0) + 2 * (w.q.shape[2] + 2) * 2.0 ** -24 * reach + keys * 2.0 ** -24 + 2.0 ** -20
    lim = 2 * (half * np.abs(out) + alg[:, :, None] * mag)
    assert (np.abs(got.double().cpu().numpy() - whole.double().cpu().numpy()) <= lim).all()
