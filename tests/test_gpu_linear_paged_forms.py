"""Launch forms and limits of linear attention and of attention behind prefixes beside those of
test_gpu_linear.py and test_gpu_paged.py, whose limits' derivations hold here: prompts that are walked
though their sizes fit the chunked form (the limits without that form's roundings), walked prompts in
segments of hundreds of tokens, a prefix against windowed attention over the same keys in one table,
calls without rows, more query heads than a tile's rows, many trees, caches filled to the end, and calls
captured once and replayed on other lengths.
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


@pytest.mark.parametrize("kind", ["tokens", "trees"])
@pytest.mark.parametrize("shape", [(32, 1, 128, 16, BF16), (40, 2, 64, 8, BF16), (24, 1, 96, 32, F32)], ids=str)
def test_prefix_of_more_query_heads_than_a_tile_has_rows(lib, shape, kind):  # noqa: F811
    sizes, cached = paged.CALLS[kind]
    w = paged.make(75, sizes, cached, ([200, 77], [0, 4, 6]), shape)
    tree = kind == "trees"
    out = lib.bole_prefix_attention(**paged.on_gpu(w), parent=g(w.parent) if tree else None)
    check_attention(out, paged.oracle_of(w, tree), w, 900)


@pytest.mark.parametrize("shape", [paged.ROTARY[0], paged.ROTARY[3], paged.ROTARY[9]], ids=str)
def test_rotation_of_many_trees(lib, shape):  # noqa: F811
    """Trees in the launch for many rows, among them ones of one node, of none, and bad ones."""
    sizes = [(17 * i) % 65 for i in range(150)]
    first = [(97 * i) % 5000 for i in range(150)]
    w = paged.make_rotary(76, sizes, first, shape, tree=True)
    assert w["offs"][-1] >= 4096
    at = {t: p for t, p in P.positions(w["first"], w["offs"], w["parent"]).items()}
    bad = [7, 90]
    for b in bad:
        w["parent"][w["offs"][b] + 1] = 1  # its own
    status = torch.full((150,), -1, dtype=torch.int32, device=dev())
    got = paged.call_rotary(lib, w, seq_status=status)
    assert status.tolist() == [paged.BAD_PARENT if b in bad else 0 for b in range(150)]
    rows = {b: range(w["offs"][b], w["offs"][b + 1]) for b in bad}
    for b in bad:
        assert all(torch.isnan(y[list(rows[b])]).all() for y in got)
    gone = {t for b in bad for t in rows[b]}
    paged.check_rotary(got, w, at={t: at[t] for t in sorted(at)[::7] if t not in gone})


def test_append_to_the_last_position_and_paths_of_none(lib):  # noqa: F811
    for path in (False, True):
        w = paged.make_append(77, [5, 3, 0, 6], [11, 0, 16, 10], 2, 64, 8, BF16, path=path)
        if path:
            w["idx"], w["len"] = w["idx"][:, :0].copy(), np.zeros(4, np.int32)
        else:
            w["table"] = w["table"][:, :2].copy()  # 16 positions: 11 + 5, 16 + 0 and 10 + 6 are the last
        status = torch.full((4,), -1, dtype=torch.int32, device=dev())
        paged.check_append(paged.call_append(lib, w, seq_status=status), w)
        assert (status == 0).all()


def replays(call, settings, results):
    """call(), captured once, replayed on each setting of its inputs (functions that write them), with
    eager work between, against the eager call on the same inputs, bit for bit."""
    settings[0]()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for setting in settings[1:] + settings[:1]:
        got = []
        for run in (call, graph.replay):
            for x in results:
                x.fill_(-3)  # (rows of no sequence keep that)
            setting()
            torch.cuda.synchronize()
            run()
            torch.randn(1 << 16, device=dev()).mul_(2.0)
            torch.cuda.synchronize()
            got.append([x.clone() for x in results])
        for a, b in zip(*got):
            assert torch.equal(a, b)


def test_captured_prompts_of_other_lengths(lib):  # noqa: F811
    """Offsets are read on the GPU: one capture serves prompts of other lengths in as many rows."""
    for shape, channel in (((4, 2, 128, 64, BF16), False), ((4, 2, 128, 64, BF16), True), ((2, 2, 64, 32, F32), False)):
        w = make(78, [700, 200, 0], shape, channel=channel)
        t = on_gpu(w)
        H, out, offs = t["H0"].clone(), torch.zeros_like(t["v"]), g(w.offsets).clone()
        call = lib.bind_linear_prefill(**dict(t, H0=H), seq_offsets=offs, out=out)

        def lengths(*ends):
            def setting():
                H.copy_(t["H0"])
                offs.copy_(torch.tensor([0, *ends], dtype=torch.int32))
            return setting
        replays(call, [lengths(700, 900, 900), lengths(1, 2, 900), lengths(900, 900, 900), lengths(300, 600, 880)], [out, H])


def test_captured_prefix_attention_of_other_lengths(lib):  # noqa: F811
    for shape in ((8, 2, 128, 16, BF16), (4, 2, 96, 16, F32)):
        w = paged.make(79, [1] * 9, [40] * 9, ([1500, 200, 64], [0, 4, 7, 9]), shape)
        t = paged.on_gpu(w)
        plen, groups, clen = t["prefix_len"].clone(), t["group_offsets"].clone(), t["cache_len"].clone()
        out = torch.zeros_like(t["q"])
        call = lib.bind_prefix_attention(**dict(t, prefix_len=plen, group_offsets=groups, cache_len=clen), out=out)

        def lengths(prefix, ends, cached):
            def setting():
                plen.copy_(torch.tensor(prefix, dtype=torch.int32))
                groups.copy_(torch.tensor(ends, dtype=torch.int32))
                clen.fill_(cached)
            return setting
        replays(call, [lengths([1500, 200, 64], [0, 4, 7, 9], 40), lengths([3, 0, 64], [0, 1, 7, 9], 7),
                       lengths([1500, 1, 1], [0, 9, 9, 9], 0), lengths([0, 200, 0], [2, 2, 5, 6], 33)], [out])
