"""Measured cases of what a hybrid-attention model's layers need before and after tree verification:

  prefill  a prompt through linear attention with a decay, whole sequences at a time (bole_linear_prefill)
  step     one token a sequence through linear attention with a decay (bole_linear_step)
  rotary   the norm of every head's query and key and its rotation by position, in one pass (bole_qk_norm_rotary)
  prefix   attention of sequences that share a long prefix, its keys read once for all of them (bole_prefix_attention)
  append   new rows, or the accepted path of each draft tree, into a paged cache (bole_cache_append)

Linear attention, for one head with state H [d_k, d_v], key k, value v, query q and decay a (one a head, or one
for each of its key channels):   H <- a H + k v^T;  o = H^T q.

A case is a dict of plain values. Its sizes and "mix" fix the ragged lengths, the trees, the paths and the
pages; the seed fixes every value. `run` computes a case with elementary torch operations in 32 bits (angles and
decays' logarithms in 64) where `own` is false, and calls the library where it is true.
"""
import math
import random

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    linear = dict(dtype="bf16", heads=32, key_heads=32, d_k=128, d_v=64, channel=False)
    heads = dict(dtype="bf16", heads=32, kv_heads=8, d=128)
    rotary = dict(heads, op="rotary", rotary=128, interleaved=False, far=16384)
    prefix = dict(heads, op="prefix", page=64)
    append = dict(heads, op="append", page=64)
    return [
        # a batch of chat prompts of uneven length, prefilled together
        dict(linear, name="linear_prompts", op="prefill", batch=8, length=2048, ragged=True, mix=1),
        # one long document, four value heads to a key head
        dict(linear, name="linear_long", op="prefill", key_heads=8, batch=1, length=32768, ragged=False, mix=2),
        # one user's next token: latency
        dict(linear, name="linear_step_one", op="step", batch=1),
        # a full serving batch's next tokens
        dict(linear, name="linear_step_batch", op="step", batch=128),
        # a serving batch's next tokens: latency
        dict(rotary, name="rotary_tokens", batch=64, rows=1, tree=False, ragged=False, mix=3),
        # the draft trees of a serving batch, a quarter of each head rotated, in neighbouring pairs
        dict(rotary, name="rotary_trees", batch=64, rows=32, tree=True, ragged=True, rotary=32, interleaved=True, mix=4),
        # two prompts
        dict(rotary, name="rotary_prompts", batch=2, rows=8192, tree=False, ragged=False, mix=5),
        # a few users of one instruction text: latency
        dict(prefix, name="prefix_few", batch=4, groups=1, prefix=1000, cached=100, rows=1, tree=False, ragged=True, mix=6),
        # a serving batch's next tokens behind one long document
        dict(prefix, name="prefix_tokens", batch=64, groups=1, prefix=16384, cached=512, rows=1, tree=False, ragged=True, mix=7),
        # draft trees of a batch with four instruction texts, and of a few sequences with none
        dict(prefix, name="prefix_trees", batch=50, groups=4, prefix=8192, cached=1000, rows=16, tree=True, ragged=True, page=16, mix=8),
        # the accepted paths of a serving batch
        dict(append, name="append_paths", batch=64, cached=16384, rows=32, tree=True, ragged=True, page=16, mix=9),
        # two prompts that continue a cached context
        dict(append, name="append_prompts", batch=2, cached=4096, rows=8192, tree=False, ragged=False, mix=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "rotary", "prefix", "prefix", "append"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), mix=rng.randrange(1 << 20), ragged=rng.random() < 0.7)
    if op in ("prefill", "step"):
        key_heads = rng.choice([1, 2, 4, 8, 16])
        case.update(key_heads=key_heads, heads=key_heads * rng.choice([1, 1, 2, 3]), d_k=rng.choice([64, 128, 128, 72, 16]), d_v=rng.choice([32, 64, 64, 128, 96, 40]),
                    channel=rng.random() < 0.25)
        if op == "step":
            case["batch"] = _log(rng, 1, 128)
        else:
            case["batch"] = _log(rng, 1, 24)
            case["length"] = _log(rng, 2, 16384 // case["batch"])
            if case["channel"]:
                case["length"] = min(case["length"], 600)
            elif case["dtype"] == "f32":
                case["length"] = min(case["length"], 2000)
        return case
    kv_heads = rng.choice([1, 2, 4, 8])
    case.update(kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), d=rng.choice([64, 128, 128, 96]))
    kind = rng.choice(["token", "tree", "prompt"])
    case.update(tree=kind == "tree", rows={"token": 1, "tree": rng.randint(1, 64), "prompt": _log(rng, 2, 2048)}[kind])
    case["batch"] = _log(rng, 1, {"token": 96, "tree": 48, "prompt": max(2, min(24, 4096 // case["rows"]))}[kind])
    if op == "rotary":
        case.update(rotary=rng.choice([case["d"], case["d"], case["d"] // 2, 10]), interleaved=rng.random() < 0.4, far=_log(rng, 1, 1 << 20))
        return case
    case.update(page=rng.choice([8, 16, 32, 64, 128]), cached=_log(rng, 1, 4096) - 1)
    if op == "prefix":
        case.update(groups=rng.choice([0, 1, 1, 2, 5]), prefix=_log(rng, 1, 8192))
        case["groups"] = min(case["groups"], case["batch"])
        if case["rows"] > 64:
            case["cached"] = min(case["cached"], 600)
        if case["dtype"] == "f32":
            case["rows"] = min(case["rows"], 300)
    return case


def _sizes(case):
    """Each sequence's tokens (prefill) or (rows, cached tokens)."""
    rng = random.Random(case.get("mix", 0))
    B = case["batch"]
    if case["op"] == "step":
        return [1] * B
    if case["op"] == "prefill":
        return [case["length"] if b == 0 or not case["ragged"] else int(case["length"] * rng.random()) for b in range(B)]
    many = case["ragged"] and case["rows"] > 1
    rows = [case["rows"] if b == 0 or not many else max(1, int(case["rows"] * rng.random())) for b in range(B)]
    most = case["far"] if case["op"] == "rotary" else case["cached"]
    cached = [most if b == 0 or not case["ragged"] else int(most * rng.random()) for b in range(B)]
    return list(zip(rows, cached))


def _groups(case):
    """Each prefix's tokens, and the sequences that share it: its first one, with the end of the last. The last few sequences have none."""
    rng = random.Random(case["mix"] + 31)
    n, B = case["groups"], case["batch"]
    sharing = B - (B // 16 if n > 1 else 0)
    lengths = [case["prefix"] if g == 0 or not case["ragged"] else max(1, int(case["prefix"] * rng.random())) for g in range(n)]
    return lengths, [sharing * g // n if n else 0 for g in range(n + 1)]


def _trees(case, sizes):
    """Parents of every tree (at most ten levels), packed, and an accepted path of each."""
    rng = random.Random(case["mix"] + 77)
    parents, paths = [], []
    for n in sizes:
        depth, tree = [], []
        for i in range(n):
            p = -1 if i == 0 or rng.random() < 0.1 else rng.randrange(max(0, i - 8), i)
            while p >= 0 and depth[p] >= 10:
                p = tree[p]
            tree.append(p)
            depth.append(1 if p < 0 else depth[p] + 1)
        path, i = [], max(range(n), key=lambda j: depth[j])
        while i >= 0:
            path.insert(0, i)
            i = tree[i]
        keep = 0
        while keep < len(path) and rng.random() < 0.8:  # geometric, as acceptance is
            keep += 1
        parents += tree
        paths.append(path[:keep])
    return parents, paths


def _offsets(lengths, dev):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=dev), at[-1]


def _tables(mix, wanted, widths):
    """Page tables [len(w), width] with a page of its own for every (row, entry) of each list in `wanted`, in shuffled order, -1 elsewhere; and the number of pages."""
    order = list(range(sum(map(len, wanted))))
    random.Random(mix + 5).shuffle(order)
    tables, taken = [], 0
    for (lines, width), pairs in zip(widths, wanted):
        t = torch.full((lines, max(1, width)), -1, dtype=torch.int32)
        if pairs:
            at = torch.tensor(pairs)
            t[at[:, 0], at[:, 1]] = torch.tensor(order[taken:taken + len(pairs)], dtype=torch.int32)
        taken += len(pairs)
        tables.append(t)
    return tables, max(1, taken)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, H = case["batch"], case["heads"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    sizes = _sizes(case)
    s = dict(case=case)
    if case["op"] in ("prefill", "step"):
        Hk, dk, dv = case["key_heads"], case["d_k"], case["d_v"]
        s["offsets"], T = _offsets(sizes, dev)
        # keys of unit length and queries of length d_k^-1/2, decays near one
        q, k = normal(T, Hk, dk), normal(T, Hk, dk)
        s["q"] = (q / q.norm(dim=-1, keepdim=True) * dk ** -0.5).to(dt)
        s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
        s["v"] = normal(T, H, dv).to(dt)
        wide = (dk,) if case["channel"] else ()
        s["gate"] = torch.exp(-torch.exp(normal(H, *wide) - 3.0) * torch.nn.functional.softplus(normal(T, H, *wide)))
        s["H0"] = 0.3 * normal(B, H, dk, dv)
        s["out"] = torch.empty(T, H, dv, dtype=dt, device=dev)
        return s
    Hk, d = case["kv_heads"], case["d"]
    rows, cached = zip(*sizes)
    s["offsets"], T = _offsets(rows, dev)
    s["cache_len"] = torch.tensor(cached, dtype=torch.int32, device=dev)
    if case["tree"]:
        parents, paths = _trees(case, rows)
        s["parent"] = torch.tensor(parents, dtype=torch.int32, device=dev)
    if case["op"] == "rotary":
        # queries, keys and values side by side, as one projection leaves them
        both = normal(T, (H + 2 * Hk) * d).to(dt)
        s["q"], s["k"] = both[:, :H * d].unflatten(1, (H, d)), both[:, H * d:(H + Hk) * d].unflatten(1, (Hk, d))
        s["q_weight"], s["k_weight"] = (1 + 0.2 * normal(d)).to(dt), (1 + 0.2 * normal(d)).to(dt)
        r = case["rotary"]
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)).float()
        s["q_out"], s["k_out"] = torch.empty(T, H, d, dtype=dt, device=dev), torch.empty(T, Hk, d, dtype=dt, device=dev)
        return s
    ps = case["page"]
    s["k"], s["v"] = normal(T, Hk, d).to(dt), normal(T, Hk, d).to(dt)
    if case["op"] == "append":
        s["new_len"] = torch.empty(B, dtype=torch.int32, device=dev)
        added = rows
        if case["tree"]:
            idx = torch.full((B, 16), -1, dtype=torch.int32)
            for b, p in enumerate(paths):
                idx[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
            s["accepted_idx"], added = idx.to(dev), [len(p) for p in paths]
            s["accepted_len"] = torch.tensor(added, dtype=torch.int32, device=dev)
        # (of each sequence, the pages that the new rows go to: what else is cached does not matter here)
        wanted = [(b, i) for b in range(B) for i in range(cached[b] // ps, -(-(cached[b] + added[b]) // ps))]
        (table,), pages = _tables(case["mix"], [wanted], [(B, (max(cached) + max(rows)) // ps + 1)])
    else:
        lengths, first = _groups(case)
        s["group_offsets"] = torch.tensor(first, dtype=torch.int32, device=dev)
        s["prefix_len"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
        own_pages = [(b, i) for b in range(B) for i in range(-(-cached[b] // ps))]
        shared = [(g, i) for g in range(len(lengths)) for i in range(-(-lengths[g] // ps))]
        (table, prefix), pages = _tables(case["mix"], [own_pages, shared], [(B, max(cached) // ps + 1), (len(lengths), -(-max(lengths, default=0) // ps))])
        s["prefix_table"] = prefix.to(dev)
        s["q"], s["out"] = normal(T, H, d).to(dt), torch.empty(T, H, d, dtype=dt, device=dev)
    s["page_table"] = table.to(dev)
    s["k_cache"], s["v_cache"] = normal(pages, Hk, ps, d).to(dt), normal(pages, Hk, ps, d).to(dt)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


# ---- the library's calls: each launch is bound once to the program's buffers, as its decode loop does

def _bound(s, make):
    if "call" not in s:
        s["call"] = make()
    s["call"]()


def _own_prefill(s):
    from tree_speculative_decoding_02_amd import bind_linear_prefill
    _bound(s, lambda: bind_linear_prefill(s["H0"], s["q"], s["k"], s["v"], s["gate"], s["offsets"], s["out"]))
    return {"out": s["out"], "H0": s["H0"]}


def _own_step(s):
    from tree_speculative_decoding_02_amd import bind_linear_step
    _bound(s, lambda: bind_linear_step(s["H0"], s["q"], s["k"], s["v"], s["gate"], s["out"]))
    return {"out": s["out"], "H0": s["H0"]}


def _own_rotary(s):
    from tree_speculative_decoding_02_amd import bind_qk_norm_rotary
    _bound(s, lambda: bind_qk_norm_rotary(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"], s["cache_len"], s["offsets"], s["q_out"], s["k_out"], eps=1e-6,
                                          parent=s.get("parent"), interleaved=s["case"]["interleaved"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _own_prefix(s):
    from tree_speculative_decoding_02_amd import bind_prefix_attention
    _bound(s, lambda: bind_prefix_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["prefix_table"], s["prefix_len"], s["group_offsets"], s["page_table"],
                                            s["cache_len"], s["offsets"], s["out"], parent=s.get("parent")))
    return {"out": s["out"]}


def _own_append(s):
    from tree_speculative_decoding_02_amd import bind_cache_append
    _bound(s, lambda: bind_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"], s["offsets"], parent=s.get("parent"),
                                        accepted_idx=s.get("accepted_idx"), accepted_len=s.get("accepted_len"), new_len=s["new_len"]))
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_len": s["new_len"]}


# ---- the plain forms

def _padded(offsets, most):
    """Packed rows of each sequence as [B, most], and which of them exist."""
    at = torch.arange(most, device=offsets.device)
    lo, n = offsets[:-1, None].long(), (offsets[1:] - offsets[:-1])[:, None]
    there = at[None] < n
    return torch.where(there, lo + at, torch.zeros_like(lo)), there


def _ancestors(parent, rows, there):
    """[B, N, N]: whether node j is on the path from the root to node i, i among them."""
    B, N = rows.shape
    p = torch.where(there, parent[rows].long(), -torch.ones_like(rows))
    m = torch.eye(N, device=rows.device) + (p[..., None] == torch.arange(N, device=rows.device)).float()
    for _ in range(max(1, math.ceil(math.log2(N + 1)))):
        m = torch.minimum(m @ m, torch.ones_like(m))
    return m > 0.5


def _plain_prefill(s):
    c = s["case"]
    C = 16 if c["channel"] else CHUNK
    N = -(-c["length"] // C) * C
    rows, there = _padded(s["offsets"], N)

    def take(x, fill):
        y = torch.where(there.reshape(there.shape + (1,) * (x.dim() - 1)), x[rows], torch.full((), fill, dtype=x.dtype, device=x.device)).transpose(1, 2)
        return y.repeat_interleave(c["heads"] // y.shape[1], 1)
    q, k, v = (take(s[n].float(), 0.0) for n in ("q", "k", "v"))
    gate = take(s["gate"], 1.0)
    S, out = s["H0"], []
    lower = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    for t in range(0, N, C):  # a chunk's tokens from the state before it, and from each other
        qc, kc, vc = (x[:, :, t:t + C] for x in (q, k, v))
        L = gate[:, :, t:t + C].double().log().cumsum(2)
        L = L if c["channel"] else L[..., None]
        between = (L[:, :, :, None] - L[:, :, None]).masked_fill(~lower[:, :, None], -math.inf).exp().float()  # [B, H, i, j, d_k or 1]
        if c["channel"]:
            pair = (qc[:, :, :, None] * kc[:, :, None] * between).sum(-1)
        else:
            pair = (qc @ kc.transpose(-1, -2)) * between[..., 0]
        start, end = L.exp().float(), (L[:, :, -1:] - L).exp().float()
        out.append((start * qc) @ S + pair @ vc)
        S = start[:, :, -1, :, None] * S + (end * kc).transpose(-1, -2) @ vc
    s["out"][rows[there]] = torch.cat(out, 2).transpose(1, 2)[there].to(s["out"].dtype)
    s["H0"].copy_(S)
    return {"out": s["out"], "H0": s["H0"]}


def _plain_step(s):
    H = s["H0"].shape[1]
    q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1) for n in ("q", "k"))
    gate = s["gate"] if s["case"]["channel"] else s["gate"][..., None]
    S = gate[..., None] * s["H0"] + k[..., None] * s["v"].float()[..., None, :]
    s["out"].copy_((S * q[..., None]).sum(-2))
    s["H0"].copy_(S)
    return {"out": s["out"], "H0": s["H0"]}


def _positions(s):
    """Of every packed row."""
    c = s["case"]
    rows, there = _padded(s["offsets"], c["rows"])
    at = _ancestors(s["parent"], rows, there).sum(-1) - 1 if c["tree"] else torch.arange(c["rows"], device=rows.device)[None].expand(rows.shape)
    return (s["cache_len"][:, None].long() + at)[there]


def _plain_rotary(s):
    angle = _positions(s).double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = s["case"]["rotary"]
    for x, w, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["case"]["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
        turned = (a * cos - b * sin, b * cos + a * sin)
        turned = torch.stack(turned, -1).flatten(-2) if s["case"]["interleaved"] else torch.cat(turned, -1)
        out.copy_(torch.cat([turned, y[..., r:]], -1))
    return {"q": s["q_out"], "k": s["k_out"]}


def _part(q, K, V, see):
    """Softmax of q K^T over the keys seen, unnormalised: the largest score, the sum, and the sum with V."""
    z = (q @ K.transpose(-1, -2).contiguous()) * q.shape[-1] ** -0.5
    if see is not None:
        z = z.masked_fill(~see, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top)
    return top, p.sum(-1, keepdim=True), p @ V


def _plain_prefix(s):
    c = s["case"]
    B, H, Hk, N, ps, d = c["batch"], c["heads"], c["kv_heads"], c["rows"], c["page"], c["d"]
    G, dev = H // Hk, s["q"].device
    rows, there = _padded(s["offsets"], N)
    # own tokens: the sequence's cached ones, then the call's rows
    at = torch.arange(s["page_table"].shape[1] * ps, device=dev)
    cached = at[None] < s["cache_len"][:, None]
    page = s["page_table"].long()[:, at // ps].clamp(min=0)
    keys = [torch.cat([cache[page, :, at % ps].float(), s[new][rows].float()], 1).transpose(1, 2) for cache, new in ((s["k_cache"], "k"), (s["v_cache"], "v"))]
    mine = _ancestors(s["parent"], rows, there) if c["tree"] else torch.ones(N, N, dtype=torch.bool, device=dev).tril()[None].expand(B, -1, -1)
    see = torch.cat([cached[:, None].expand(-1, N, -1), mine], 2)
    q = s["q"][rows].float().unflatten(2, (Hk, G)).permute(0, 2, 3, 1, 4)  # [B, Hk, G, N, d]
    top, sums, out = _part(q.reshape(B, Hk, G * N, d), *keys, see[:, None, None].expand(B, 1, G, N, -1).reshape(B, 1, G * N, -1))
    first, lengths = s["group_offsets"].tolist(), s["prefix_len"].tolist()
    for g, n in enumerate(lengths):
        b0, b1 = first[g], first[g + 1]
        at = torch.arange(n, device=dev)
        page = s["prefix_table"][g].long()[at // ps]
        K, V = (cache[page, :, at % ps].float().transpose(0, 1)[None].expand(b1 - b0, -1, -1, -1) for cache in (s["k_cache"], s["v_cache"]))
        t, l, o = _part(q[b0:b1].reshape(b1 - b0, Hk, G * N, d), K, V, None)
        both = torch.maximum(t, top[b0:b1])
        x, y = torch.exp(top[b0:b1] - both), torch.exp(t - both)
        sums[b0:b1], out[b0:b1] = x * sums[b0:b1] + y * l, x * out[b0:b1] + y * o
    out = (out / sums).unflatten(2, (G, N)).permute(0, 3, 1, 2, 4).reshape(B, N, H, d)
    s["out"][rows[there]] = out[there].to(s["out"].dtype)
    return {"out": s["out"]}


def _plain_append(s):
    c = s["case"]
    if c["tree"]:
        idx = s["accepted_idx"].long()
        there = torch.arange(idx.shape[1], device=idx.device)[None] < s["accepted_len"][:, None]
        rows, added = s["offsets"][:-1, None].long() + idx, s["accepted_len"]
    else:
        rows, there = _padded(s["offsets"], c["rows"])
        added = s["offsets"][1:] - s["offsets"][:-1]
    at = s["cache_len"][:, None].long() + torch.arange(rows.shape[1], device=rows.device)
    b = torch.arange(c["batch"], device=rows.device)[:, None].expand(rows.shape)
    page, slot, rows = s["page_table"][b[there], at[there] // c["page"]].long(), at[there] % c["page"], rows[there]
    s["k_cache"][page, :, slot] = s["k"][rows]
    s["v_cache"][page, :, slot] = s["v"][rows]
    s["new_len"].copy_(s["cache_len"] + added)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_len": s["new_len"]}


_PLAIN = {"prefill": _plain_prefill, "step": _plain_step, "rotary": _plain_rotary, "prefix": _plain_prefix, "append": _plain_append}
_OWN = {"prefill": _own_prefill, "step": _own_step, "rotary": _own_rotary, "prefix": _own_prefix, "append": _own_append}


# ---- what a pass cannot do without

def work(case):
    sizes, size = _sizes(case), 2 if case["dtype"] == "bf16" else 4
    H = case["heads"]
    if case["op"] in ("prefill", "step"):
        dk, dv, Hk = case["d_k"], case["d_v"], case["key_heads"]
        T = sum(sizes)
        gates = 4 * H * (dk if case["channel"] else 1)
        return {"bytes": float(8 * case["batch"] * H * dk * dv + T * (size * (2 * Hk * dk + 2 * H * dv) + gates)), "flops": 4.0 * T * H * dk * dv}
    Hk, d = case["kv_heads"], case["d"]
    T = sum(r for r, _ in sizes)
    if case["op"] == "rotary":
        return {"bytes": float(2 * size * T * (H + Hk) * d), "flops": 8.0 * T * (H + Hk) * d}
    if case["op"] == "append":
        if case["tree"]:
            T = sum(map(len, _trees(case, [r for r, _ in sizes])[1]))
        return {"bytes": float(4 * size * T * Hk * d), "flops": float(T * Hk * d)}
    lengths, first = _groups(case)
    depths, pairs, at = _depths(case, sizes), 0, 0
    for b, (r, c) in enumerate(sizes):
        shared = sum(n for g, n in enumerate(lengths) if first[g] <= b < first[g + 1])
        pairs += sum(shared + c + (depths[at + i] if depths else i + 1) for i in range(r))
        at += r
    keys = sum(n for g, n in enumerate(lengths) if first[g + 1] > first[g]) + sum(c for _, c in sizes)
    return {"bytes": float(size * (2 * keys * Hk * d + T * d * (2 * H + 2 * Hk))), "flops": 4.0 * pairs * H * d}


def _depths(case, sizes):
    if not case["tree"]:
        return None
    parents, depths, at = _trees(case, [r for r, _ in sizes])[0], [], 0
    for r, _ in sizes:
        for i in range(r):
            p = parents[at + i]
            depths.append(1 if p < 0 else depths[at + p] + 1)
        at += r
    return depths


# ---- the definitions, token by token and row by row, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    off = s["offsets"].tolist()
    if case["op"] in ("prefill", "step"):
        q, k = (s[n].double().repeat_interleave(case["heads"] // case["key_heads"], 1) for n in ("q", "k"))
        v, S, out = s["v"].double(), s["H0"].double(), torch.zeros(s["out"].shape, dtype=torch.float64, device=s["v"].device)
        gate = s["gate"].double().reshape(s["gate"].shape[:2] + (-1, 1))
        for t in range(max(off[b + 1] - off[b] for b in range(len(off) - 1))):
            live = [b for b in range(len(off) - 1) if off[b] + t < off[b + 1]]
            r = torch.tensor([off[b] + t for b in live], device=v.device)
            S[live] = S[live] * gate[r] + k[r][..., None] * v[r][..., None, :]
            out[r] = (S[live] * q[r][..., None]).sum(-2)
        return {"out": out, "H0": S}
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if case["op"] == "prefix":
        return {"out": _exact_prefix(case, s)}
    caches, ps = {n: s[n].double() for n in ("k_cache", "v_cache")}, case["page"]
    lengths, table = s["cache_len"].tolist(), s["page_table"].tolist()
    paths = s["accepted_idx"].tolist() if case["tree"] else None
    kept = s["accepted_len"].tolist() if case["tree"] else None
    for b in range(case["batch"]):
        for r in (paths[b][:kept[b]] if case["tree"] else range(off[b + 1] - off[b])):
            page, slot = table[b][lengths[b] // ps], lengths[b] % ps
            caches["k_cache"][page, :, slot] = s["k"][off[b] + r].double()
            caches["v_cache"][page, :, slot] = s["v"][off[b] + r].double()
            lengths[b] += 1
    return dict(caches, new_len=torch.tensor(lengths, dtype=torch.int32))


def _exact_rotary(case, s):
    sizes, r, out = _sizes(case), case["rotary"], {}
    depths = _depths(case, sizes)
    pos, at = [], 0
    for n, c in sizes:
        pos += [c + (depths[at + i] - 1 if depths else i) for i in range(n)]
        at += n
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       torch.tensor(pos, dtype=torch.float64, device=s["q"].device)[:, None, None] * s["inv_freq"].double())
    for name in ("q", "k"):
        x = s[name].double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + 1e-6) * s[name + "_weight"].double()
        pairs = x[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        x[..., :r] = (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2)
        out[name] = x
    return out


def _exact_prefix(case, s):
    ps, Hk = case["page"], case["kv_heads"]
    off, cached = s["offsets"].tolist(), s["cache_len"].tolist()
    lengths, first = _groups(case)
    dev = s["q"].device
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    parent = s["parent"].tolist() if case["tree"] else None

    def cache(table, n):
        pos = torch.arange(n, device=dev)
        page = table.long()[pos // ps]
        return (s["k_cache"][page, :, pos % ps].double(), s["v_cache"][page, :, pos % ps].double())
    for b in range(case["batch"]):
        lo, n, parts = off[b], off[b + 1] - off[b], []
        for g in range(len(lengths)):
            if first[g] <= b < first[g + 1]:
                parts.append(cache(s["prefix_table"][g], lengths[g]))
        parts += [cache(s["page_table"][b], cached[b]), (s["k"][lo:lo + n].double(), s["v"][lo:lo + n].double())]
        K, V = (torch.cat(x).transpose(0, 1) for x in zip(*parts))  # [Hk, M, d]
        lines = []
        for i in range(n):
            p = i - 1 if parent is None else parent[lo + i]
            lines.append(({i} if p < 0 else lines[p] | {i}) if parent is not None else None)
        sees = torch.ones(n, n, dtype=torch.bool, device=dev).tril() if parent is None else torch.tensor([[j in line for j in range(n)] for line in lines], device=dev)
        hidden = torch.cat([torch.zeros(n, K.shape[1] - n, dtype=torch.bool, device=dev), ~sees], 1)
        for h in range(case["heads"]):
            j = h // (case["heads"] // Hk)
            z = (s["q"][lo:lo + n, h].double() @ K[j].T) / math.sqrt(case["d"])
            out[lo:lo + n, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ V[j]
    return out
