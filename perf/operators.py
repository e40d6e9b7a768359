"""Measured cases of the operators a hybrid-attention model's layers need around tree verification:

  prefill  a prompt through the gated delta rule, whole sequences at a time (bole_delta_prefill)
  step     one token a sequence through the gated delta rule (bole_delta_step)
  verify   draft trees through the gated delta rule (bole_delta_tree_verify)
  commit   the accepted path of each tree into the state (bole_delta_commit_path)
  window   attention over a paged cache with a sliding window and visible first tokens, for single
           tokens, draft trees and prompts (bole_window_attention)

The gated delta rule, for one head with state H [d_k, d_v], key k, value v, query q, decay a and
strength b:   H' = a H;  u = b (v - H'^T k);  H <- H' + k u^T;  o = H^T q.

A case is a dict of plain values. Its sizes and "mix" fix the ragged lengths, the trees and the
paths; the seed fixes every value. `run` computes a case with elementary torch operations in 32
bits (decays' logarithms in 64) where `own` is false, and calls the library where it is true.
"""
import math
import random

import torch

own = False

CHUNK = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    delta = dict(dtype="bf16", heads=32, key_heads=16, d_k=128, d_v=128)
    window = dict(dtype="bf16", heads=32, kv_heads=8, d=128, page=64, sinks=4)
    return [
        # a batch of chat prompts of uneven length, prefilled together
        dict(delta, name="prefill_prompts", op="prefill", batch=8, length=2048, ragged=True, mix=1),
        # one long document
        dict(delta, name="prefill_long", op="prefill", batch=1, length=32768, ragged=False, mix=2),
        # one user's next token: latency
        dict(delta, name="step_one", op="step", batch=1),
        # a full serving batch's next tokens
        dict(delta, name="step_batch", op="step", batch=128),
        # a small batch with 32-node draft trees, as many key heads as value heads
        dict(delta, name="verify_small", op="verify", batch=8, key_heads=32, d_v=64, nodes=32, ragged=False, mix=3),
        # a serving batch with tree budgets from 4 to 64 nodes
        dict(delta, name="verify_batch", op="verify", batch=64, nodes=64, ragged=True, mix=4),
        # the accepted paths of a small batch in full precision
        dict(delta, name="commit_small_f32", op="commit", dtype="f32", batch=8, key_heads=32, d_v=64, nodes=32, ragged=False, mix=5),
        # the accepted paths of a serving batch
        dict(delta, name="commit_batch", op="commit", batch=64, nodes=64, ragged=True, mix=6),
        # one user's next token over a long context: latency
        dict(window, name="window_one", op="window", batch=1, cached=8191, rows=1, tree=False, ragged=False, window=4096, mix=7),
        # a serving batch's next tokens, contexts of every length, small pages
        dict(window, name="window_tokens", op="window", batch=64, cached=16384, rows=1, tree=False, ragged=True, window=4096, mix=8, page=16),
        # the draft trees of a serving batch
        dict(window, name="window_trees", op="window", batch=64, cached=16384, rows=32, tree=True, ragged=True, window=4096, mix=9),
        # two prompts that continue a cached context, wider than the window
        dict(window, name="window_prompts", op="window", batch=2, cached=4096, rows=8192, tree=False, ragged=False, window=1024, mix=10),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "step", "verify", "commit", "window", "window"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), mix=rng.randrange(1 << 20), ragged=rng.random() < 0.7)
    if op == "window":
        kv_heads = rng.choice([1, 2, 4, 8])
        case.update(kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 5, 8]), d=rng.choice([64, 128, 128, 96]), page=rng.choice([8, 16, 32, 64, 128]),
                    sinks=rng.choice([0, 1, 4, 7]), window=_log(rng, 1, 5000), cached=_log(rng, 1, 16384) - 1)
        kind = rng.choice(["token", "tree", "prompt"])
        case.update(tree=kind == "tree", rows={"token": 1, "tree": rng.randint(1, 64), "prompt": _log(rng, 2, 4096)}[kind])
        if case["dtype"] == "f32":
            case["rows"] = min(case["rows"], 600)
        case["batch"] = _log(rng, 1, {"token": 96, "tree": 48, "prompt": max(2, min(24, 8192 // case["rows"]))}[kind])
        return case
    key_heads = rng.choice([1, 2, 4, 8, 16])
    case.update(key_heads=key_heads, heads=key_heads * rng.choice([1, 2, 2, 3]), d_k=rng.choice([64, 128, 128, 128, 72]), d_v=rng.choice([32, 64, 128, 128, 96, 40]))
    if op == "prefill":
        case["batch"] = _log(rng, 1, 24)
        case["length"] = _log(rng, 2, 16384 // case["batch"])
        if case["dtype"] == "f32" or case["d_k"] == 72 or case["d_v"] == 40:
            case["length"] = min(case["length"], 700)
    else:
        case["batch"] = _log(rng, 1, 128)
    if op in ("verify", "commit"):
        case["nodes"] = rng.randint(1, 64)
    return case


def _sizes(case):
    """Each sequence's tokens (prefill), nodes (verify, commit) or (rows, cached) (window)."""
    rng = random.Random(case.get("mix", 0))
    B = case["batch"]
    if case["op"] == "step":
        return [1] * B
    if case["op"] == "prefill":
        return [case["length"] if b == 0 or not case["ragged"] else int(case["length"] * rng.random()) for b in range(B)]
    if case["op"] == "window":
        many = case["ragged"] and case["rows"] > 1
        rows = [case["rows"] if b == 0 or not many else max(1, int(case["rows"] * rng.random())) for b in range(B)]
        cached = [case["cached"] if b == 0 or not case["ragged"] else int(case["cached"] * rng.random()) for b in range(B)]
        return list(zip(rows, cached))
    return [case["nodes"] if b == 0 or not case["ragged"] else max(1, min(case["nodes"], rng.choice([4, 8, 16, 32, 64]))) for b in range(B)]


def _trees(case, sizes):
    """Parents of every tree (at most ten levels), packed, and an accepted path of each."""
    rng = random.Random(case.get("mix", 0) + 77)
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
    if case["op"] == "window":
        Hk, d, ps, W, S = case["kv_heads"], case["d"], case["page"], case["window"], case["sinks"]
        rows, cached = zip(*sizes)
        s["node_offsets"], T = _offsets(rows, dev)
        s["cache_len"] = torch.tensor(cached, dtype=torch.int32, device=dev)
        s["most_cached"] = max(cached)
        # pages that no row sees any more have been given back: their entries are -1
        table = torch.full((B, max(1, -(-(case["cached"] + 1) // ps))), -1, dtype=torch.int32)
        taken = []
        for b, c in enumerate(cached):
            first = max(0, c - W + 1) // ps
            seen = [i for i in range(-(-c // ps)) if i * ps < S or i >= first]
            taken += [(b, i) for i in seen]
        order = list(range(len(taken)))
        random.Random(case["mix"] + 5).shuffle(order)
        if taken:
            at = torch.tensor(taken)
            table[at[:, 0], at[:, 1]] = torch.tensor(order, dtype=torch.int32)
        s["page_table"] = table.to(dev)
        pages = max(1, len(taken))
        s["k_cache"], s["v_cache"] = normal(pages, Hk, ps, d).to(dt), normal(pages, Hk, ps, d).to(dt)
        s["q"], s["k"], s["v"] = normal(T, H, d).to(dt), normal(T, Hk, d).to(dt), normal(T, Hk, d).to(dt)
        if case["tree"]:
            s["parent"] = torch.tensor(_trees(case, rows)[0], dtype=torch.int32, device=dev)
        s["out"] = torch.empty(T, H, d, dtype=dt, device=dev)
        return s
    Hk, dk, dv = case["key_heads"], case["d_k"], case["d_v"]
    s["node_offsets"], T = _offsets(sizes, dev)
    # keys of unit length and queries of length d_k^-1/2, decays near one and strengths in (0, 1)
    q, k = normal(T, Hk, dk), normal(T, Hk, dk)
    s["q"] = (q / q.norm(dim=-1, keepdim=True) * dk ** -0.5).to(dt)
    s["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    s["v"] = normal(T, H, dv).to(dt)
    rate = torch.exp(normal(H) - 3.0)
    s["gate"] = torch.exp(-rate * torch.nn.functional.softplus(normal(T, H)))
    s["beta"] = torch.sigmoid(normal(T, H))
    s["H0"] = 0.3 * normal(B, H, dk, dv)
    s["out"] = torch.empty(T, H, dv, dtype=dt, device=dev)
    if case["op"] in ("verify", "commit"):
        parents, paths = _trees(case, sizes)
        s["parent"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        idx = torch.full((B, 16), -1, dtype=torch.int32)
        for b, p in enumerate(paths):
            idx[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        s["accepted_idx"] = idx.to(dev)
        s["accepted_len"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
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
    from tree_speculative_decoding_02_amd import bind_delta_prefill
    _bound(s, lambda: bind_delta_prefill(s["H0"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["node_offsets"], s["out"]))
    return {"out": s["out"], "H0": s["H0"]}


def _own_step(s):
    from tree_speculative_decoding_02_amd import bind_delta_step
    _bound(s, lambda: bind_delta_step(s["H0"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["out"]))
    return {"out": s["out"], "H0": s["H0"]}


def _own_verify(s):
    from tree_speculative_decoding_02_amd import bind_delta_tree_verify
    _bound(s, lambda: bind_delta_tree_verify(s["H0"], s["q"], s["k"], s["v"], s["gate"], s["beta"], s["parent"], s["node_offsets"], s["out"]))
    return {"out": s["out"]}


def _own_commit(s):
    from tree_speculative_decoding_02_amd import bind_delta_commit_path
    if "path_nodes" not in s:
        s["path_nodes"] = torch.empty_like(s["accepted_idx"])
    _bound(s, lambda: bind_delta_commit_path(s["H0"], s["k"], s["v"], s["gate"], s["beta"], s["parent"], s["node_offsets"], s["accepted_idx"], s["accepted_len"],
                                             path_nodes=s["path_nodes"]))
    return {"H0": s["H0"], "path_nodes": s["path_nodes"]}


def _own_window(s):
    from tree_speculative_decoding_02_amd import bind_window_attention
    c = s["case"]
    _bound(s, lambda: bind_window_attention(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_len"], s["node_offsets"], c["window"], c["sinks"],
                                            s["out"], parent=s.get("parent")))
    return {"out": s["out"]}


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


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A, row by row."""
    X = torch.eye(A.shape[-1], device=A.device).expand_as(A).contiguous()
    for i in range(1, A.shape[-1]):
        X[..., i, :] -= (A[..., i:i + 1, :i] @ X[..., :i, :])[..., 0, :]
    return X


def _factors(s, rows, there, heads):
    """q, k, v [B, H, N, d], gates [B, H, N] in 64 bits and strengths [B, H, N]; rows that do not exist change nothing."""
    def take(x, fill):
        y = torch.where(there.reshape(there.shape + (1,) * (x.dim() - 1)), x[rows], torch.full((), fill, dtype=x.dtype, device=x.device)).transpose(1, 2)
        return y.repeat_interleave(heads // y.shape[1], 1)
    return (take(s["q"].float(), 0.0), take(s["k"].float(), 0.0), take(s["v"].float(), 0.0), take(s["gate"].double(), 1.0), take(s["beta"], 0.0))


def _pairs(q, k, beta, L, seen):
    """From cumulative log decays L: the pair weights of the output, and the inverse that gives every token's update."""
    decay = torch.exp((L[..., :, None] - L[..., None, :]).masked_fill(~seen, -math.inf)).float()
    strict = seen & ~torch.eye(seen.shape[-1], dtype=torch.bool, device=seen.device)
    A = torch.where(strict, beta[..., None] * decay * (k @ k.transpose(-1, -2)), torch.zeros_like(decay))
    return decay * (q @ k.transpose(-1, -2)), _inverse(A)


def _chunks(s, rows, there, H0):
    """The tokens of each row of `rows` in order, CHUNK at a time: outputs [B, H, N, d_v] and the last state."""
    q, k, v, gate, beta = _factors(s, rows, there, H0.shape[1])
    B, H, N, dk = k.shape
    C = min(CHUNK, N)
    q, k, v = (x.reshape(B, H, N // C, C, -1) for x in (q, k, v))
    L, beta = gate.log().reshape(B, H, N // C, C).cumsum(-1), beta.reshape(B, H, N // C, C)
    seen = torch.ones(C, C, dtype=torch.bool, device=k.device).tril()
    P, X = _pairs(q, k, beta, L, seen)
    start, end = torch.exp(L).float()[..., None], torch.exp(L[..., -1:] - L).float()[..., None]
    S, out = H0, []
    for c in range(N // C):
        u = X[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - start[:, :, c] * (k[:, :, c] @ S)))
        out.append(start[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ u)
        S = start[:, :, c, -1:] * S + k[:, :, c].transpose(-1, -2) @ (end[:, :, c] * u)
    return torch.cat(out, 2), S


def _plain_prefill(s):
    most = -(-s["case"]["length"] // CHUNK) * CHUNK
    rows, there = _padded(s["node_offsets"], most)
    out, S = _chunks(s, rows, there, s["H0"])
    s["out"][rows[there]] = out.transpose(1, 2)[there].to(s["out"].dtype)
    s["H0"].copy_(S)
    return {"out": s["out"], "H0": s["H0"]}


def _plain_step(s):
    H = s["H0"].shape[1]
    q, k = (s[n].float().repeat_interleave(H // s[n].shape[1], 1) for n in ("q", "k"))
    S = s["gate"][..., None, None] * s["H0"]
    u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["out"].copy_((S * q[..., None]).sum(-2))
    s["H0"].copy_(S)
    return {"out": s["out"], "H0": s["H0"]}


def _plain_verify(s):
    rows, there = _padded(s["node_offsets"], s["case"]["nodes"])
    anc = _ancestors(s["parent"], rows, there)[:, None]
    q, k, v, gate, beta = _factors(s, rows, there, s["H0"].shape[1])
    L = (anc.double() @ gate.log()[..., None])[..., 0]
    P, X = _pairs(q, k, beta, L, anc)
    start = torch.exp(L).float()[..., None]
    u = X @ (beta[..., None] * (v - start * (k @ s["H0"])))
    out = start * (q @ s["H0"]) + P @ u
    s["out"][rows[there]] = out.transpose(1, 2)[there].to(s["out"].dtype)
    return {"out": s["out"]}


def _plain_commit(s):
    idx = s["accepted_idx"].long()
    there = torch.arange(idx.shape[1], device=idx.device)[None] < s["accepted_len"][:, None]
    rows = torch.where(there, s["node_offsets"][:-1, None].long() + idx, torch.zeros_like(idx))
    _, S = _chunks(s, rows, there, s["H0"])
    s["H0"].copy_(S)
    return {"H0": s["H0"], "path_nodes": torch.where(there, rows, -torch.ones_like(rows)).int()}


def _window_mask(s, rows, there, cached_at, cached_there):
    """[B, N, M]: which keys (cached ones, then the call's own rows) each row sees."""
    c, N = s["case"], rows.shape[1]
    if c["tree"]:
        anc = _ancestors(s["parent"], rows, there)
    else:
        anc = torch.ones(N, N, dtype=torch.bool, device=rows.device).tril()[None] & there[:, None] | torch.eye(N, dtype=torch.bool, device=rows.device)
    at = s["cache_len"][:, None].long() + (anc.sum(-1) if c["tree"] else torch.arange(1, N + 1, device=rows.device)[None]) - 1
    key_at = torch.cat([cached_at, at.expand(rows.shape)], 1)[:, None]
    near = (at[..., None] - key_at < c["window"]) | (key_at < c["sinks"])
    return near & torch.cat([cached_there[:, None].expand(-1, N, -1), anc.expand(rows.shape[0], -1, -1)], 2)


def _plain_window(s):
    c = s["case"]
    B, H, Hk, ps = c["batch"], c["heads"], c["kv_heads"], c["page"]
    rows, there = _padded(s["node_offsets"], c["rows"])
    # the cached positions that some row may see: the first tokens, and the window behind the first row
    n = s["cache_len"][:, None].long()
    first = torch.arange(c["sinks"], device=n.device)[None].expand(B, -1)
    back = n - 1 - torch.arange(min(c["window"] - 1, s["most_cached"]), device=n.device)[None]
    at = torch.cat([first, back], 1)
    real = torch.cat([first < n, back >= c["sinks"]], 1)
    page = torch.gather(s["page_table"].long(), 1, torch.where(real, at, torch.zeros_like(at)) // ps).clamp(min=0)
    spot = torch.where(real, at, torch.zeros_like(at)) % ps

    def keys(cache, new):
        return torch.cat([cache[page, :, spot].float(), new[rows].float()], 1).transpose(1, 2)
    K, V = keys(s["k_cache"], s["k"]), keys(s["v_cache"], s["v"])
    see = _window_mask(s, rows, there, at, real)
    q = s["q"][rows].float().transpose(1, 2).reshape(B, Hk, (H // Hk) * c["rows"], c["d"])
    score = ((q @ K.transpose(-1, -2).contiguous()) * c["d"] ** -0.5).reshape(B, Hk, H // Hk, c["rows"], -1)
    score = score.masked_fill(~see[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    del score
    out = (p.reshape(B, Hk, (H // Hk) * c["rows"], -1) @ V) / p.sum(-1).reshape(B, Hk, -1, 1)
    s["out"][rows[there]] = out.reshape(B, H, c["rows"], c["d"]).transpose(1, 2)[there].to(s["out"].dtype)
    return {"out": s["out"]}


_PLAIN = {"prefill": _plain_prefill, "step": _plain_step, "verify": _plain_verify, "commit": _plain_commit, "window": _plain_window}
_OWN = {"prefill": _own_prefill, "step": _own_step, "verify": _own_verify, "commit": _own_commit, "window": _own_window}


# ---- what a pass cannot do without

def work(case):
    sizes, size = _sizes(case), 2 if case["dtype"] == "bf16" else 4
    H = case["heads"]
    if case["op"] == "window":
        d, W, S = case["d"], case["window"], case["sinks"]
        rows, read, pairs = sum(r for r, _ in sizes), 0, 0
        depths = _tree_depths(case, sizes) if case["tree"] else None
        at = 0
        for r, c in sizes:
            read += min(c, min(S, c) + max(0, c - max(S, c - W + 1)))
            for i in range(r):
                n = c + (depths[at + i] if depths else i + 1)  # keys at or before this row
                pairs += min(n, W) + max(0, min(S, n - W))
            at += r
        return {"bytes": float(size * (2 * read * case["kv_heads"] * d + rows * d * (2 * H + 2 * case["kv_heads"]))), "flops": 4.0 * pairs * H * d}
    dk, dv, Hk = case["d_k"], case["d_v"], case["key_heads"]
    state = 4 * H * dk * dv
    if case["op"] == "commit":
        paths = _trees(case, sizes)[1]
        T, moved = sum(map(len, paths)), 2 * state * sum(1 for p in paths if p)
        return {"bytes": float(moved + T * (size * (Hk * dk + H * dv) + 8 * H)), "flops": 4.0 * T * H * dk * dv}
    T = sum(sizes)
    moved = case["batch"] * state * (1 if case["op"] == "verify" else 2)
    return {"bytes": float(moved + T * (size * (2 * Hk * dk + 2 * H * dv) + 8 * H)), "flops": 6.0 * T * H * dk * dv}


def _tree_depths(case, sizes):
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
    if case["op"] == "window":
        return {"out": _exact_window(case, s)}
    H = case["heads"]
    q, k = (s[n].double().repeat_interleave(H // case["key_heads"], 1) for n in ("q", "k"))
    v, gate, beta, off = s["v"].double(), s["gate"].double(), s["beta"].double(), s["node_offsets"].tolist()
    state = s["H0"].double()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=v.device)

    def token(S, r):
        """The states after, and the outputs of, the tokens at rows r [n]."""
        S = S * gate[r][..., None, None]
        u = beta[r][..., None] * (v[r] - (S * k[r][..., None]).sum(-2))
        S = S + k[r][..., None] * u[..., None, :]
        return S, (S * q[r][..., None]).sum(-2)

    if case["op"] in ("prefill", "step"):
        for t in range(max(off[b + 1] - off[b] for b in range(len(off) - 1))):
            live = [b for b in range(len(off) - 1) if off[b] + t < off[b + 1]]
            r = torch.tensor([off[b] + t for b in live], device=v.device)
            state[live], out[r] = token(state[live], r)
        return {"out": out, "H0": state}
    if case["op"] == "verify":
        parent = s["parent"].tolist()
        for b in range(len(off) - 1):
            states = []
            for r in range(off[b], off[b + 1]):
                p = parent[r]
                S, o = token(state[b:b + 1] if p < 0 else states[p], torch.tensor([r], device=v.device))
                states.append(S)
                out[r] = o[0]
        return {"out": out}
    idx, n = s["accepted_idx"].tolist(), s["accepted_len"].tolist()
    nodes = torch.full(s["accepted_idx"].shape, -1, dtype=torch.int32, device=v.device)
    for b in range(len(n)):
        for m in range(n[b]):
            r = off[b] + idx[b][m]
            nodes[b, m] = r
            state[b:b + 1], _ = token(state[b:b + 1], torch.tensor([r], device=v.device))
    return {"H0": state, "path_nodes": nodes}


def _exact_window(case, s):
    W, S, ps, G = case["window"], case["sinks"], case["page"], case["heads"] // case["kv_heads"]
    off, cached, table = s["node_offsets"].tolist(), s["cache_len"].tolist(), s["page_table"].long()
    parent = s["parent"].tolist() if case["tree"] else None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    dev = out.device
    for b in range(len(cached)):
        lo, hi, c = off[b], off[b + 1], cached[b]
        keep = [p for p in range(c) if p < S or p > c - W]
        pos = torch.tensor(keep, dtype=torch.long, device=dev)
        page, spot = table[b, pos // ps], pos % ps
        own_at = torch.arange(c, c + hi - lo, device=dev)
        sees = torch.ones(hi - lo, hi - lo, dtype=torch.bool, device=dev).tril()
        if parent is not None:
            lines = []
            for i in range(hi - lo):
                p = parent[lo + i]
                lines.append({i} if p < 0 else lines[p] | {i})
            sees = torch.tensor([[j in line for j in range(hi - lo)] for line in lines], device=dev)
            own_at = torch.tensor([c + len(line) - 1 for line in lines], device=dev)
        key_at = torch.cat([pos, own_at])
        for h in range(case["kv_heads"]):
            K = torch.cat([s["k_cache"][page, h, spot], s["k"][lo:hi, h]]).double()
            V = torch.cat([s["v_cache"][page, h, spot], s["v"][lo:hi, h]]).double()
            for i in range(0, hi - lo, 1024):  # a few rows at a time
                at = own_at[i:i + 1024, None]
                ok = (at - key_at < W) | (key_at < S)
                ok[:, len(keep):] &= sees[i:i + 1024]
                for g in range(h * G, h * G + G):
                    z = (s["q"][lo + i:min(hi, lo + i + 1024), g].double() @ K.T) / math.sqrt(case["d"])
                    w = torch.exp(torch.where(ok, z - torch.where(ok, z, -math.inf).amax(1, keepdim=True), -math.inf))
                    out[lo + i:lo + i + 1024, g][:len(w)] = (w @ V) / w.sum(1, keepdim=True)
    return out
