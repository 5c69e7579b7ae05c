"""Cases of a serving step with drafted trees: what is timed, and the operators' plain forms.

Five operators take such a step from the projections to the verified tokens, over a paged key/value cache:

* ``tree``: parents of every request's nodes -> positions and ancestor masks (``attn_paged_tree``);
* ``rope``: norms of queries and keys for each head and their rotation, to the cache with the values beside them
  (``attn_paged_rope``) or to buffers (``attn_rope``);
* ``attend``: the nodes attend over the cache and over their ancestors (``attn_fwd_paged_tree``), prompts' chunks beside them;
* ``accept``: the walk along the nodes that the model's own choices confirm (``attn_paged_accept``);
* ``move``: accepted rows go to where a chain would have them, in every layer's cache (``attn_paged_move``).

``run`` computes the plain forms out of elementary torch operations, or, with ``own`` true, calls the library.  Request
lengths come from a case's own ``mix`` number, trees, tokens and values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# (query heads, key/value heads): the repository's benchmark workloads and small ones
HEADS = ((32, 8), (32, 4), (16, 16), (16, 2), (8, 8), (6, 2), (4, 1))
PAGES = (16, 32, 48, 64, 128, 256)


def _tree(name, B, nodes, words, chunks=0, chunk=(1, 1), idle=0, pad=0, spread=8, mix=1):
    return {"name": name, "op": "tree", "B": B, "ctx_lo": 1, "ctx_hi": 9000, "n_lo": nodes[0], "n_hi": nodes[1], "words": words,
            "chunks": chunks, "chunk_lo": chunk[0], "chunk_hi": chunk[1], "idle": idle, "pad": pad, "spread": spread, "mix": mix}


def _rope(name, rows, heads, d, dtype, page=0, pad=0, norm="type", rot=None, axes=1, pairs="halves", layout="tokens", far=40000, mix=1):
    return {"name": name, "op": "rope", "rows": rows, "pad": pad, "Hq": heads[0], "Hkv": heads[1], "d": d, "dtype": dtype, "page": page,
            "norm": norm, "rot": d if rot is None else rot, "axes": axes, "pairs": pairs, "layout": layout, "far": far, "mix": mix}


def _attend(name, B, ctx, nodes, words, heads, d, dtype, page, window=-1, chunks=0, chunk=(1, 1), idle=0, pad=0, spread=8, rows="tokens",
            cache="heads", mix=1):
    return {"name": name, "op": "attend", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "n_lo": nodes[0], "n_hi": nodes[1], "words": words,
            "chunks": chunks, "chunk_lo": chunk[0], "chunk_hi": chunk[1], "idle": idle, "pad": pad, "spread": spread, "Hq": heads[0],
            "Hkv": heads[1], "d": d, "dtype": dtype, "page": page, "window": window, "rows": rows, "cache": cache, "mix": mix}


def _accept(name, B, ctx, nodes, page, steps, chunks=0, chunk=(1, 1), idle=0, pad=0, spread=8, likely=0.7, mix=1):
    return {"name": name, "op": "accept", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "n_lo": nodes[0], "n_hi": nodes[1], "chunks": chunks,
            "chunk_lo": chunk[0], "chunk_hi": chunk[1], "idle": idle, "pad": pad, "spread": spread, "page": page, "steps": steps,
            "likely": likely, "mix": mix}


def _move(name, B, layers, nodes, steps, Hkv, d, dtype, page, cache="heads", mix=1):
    return {"name": name, "op": "move", "B": B, "layers": layers, "n_lo": nodes[0], "n_hi": nodes[1], "steps": steps, "Hkv": Hkv, "d": d,
            "dtype": dtype, "page": page, "cache": cache, "mix": mix}


def listed():
    return [
        # the masks of one user's drafted tree: latency
        _tree("tree_b1_n26", 1, (26, 26), 1, mix=11),
        # a large server's step: hundreds of trees of up to 64 nodes, prompts' chunks and idle entries among them
        _tree("tree_b301_n64", 301, (20, 64), 2, chunks=7, chunk=(200, 2000), idle=20, pad=100, mix=12),
        # one layer's queries, keys and values of a decoding step, in a batch padded to a captured size
        _rope("rope_decode_b64", 61, (32, 8), 128, "bf16", page=16, pad=3, mix=21),
        # one layer's rows of admitted prompts
        _rope("rope_prompts_16k", 16900, (32, 8), 128, "bf16", page=64, mix=22),
        # patches of a video: time, height and width, to buffers of their own; weights of the norms in 32 bits
        _rope("rope_video_8k", 8190, (16, 2), 128, "fp16", norm="f32", axes=3, layout="heads", far=9000, mix=23),
        # checking one user's drafted tree: latency
        _attend("attend_b1_n26_2k", 1, (2001, 2001), (26, 26), 1, (32, 8), 128, "bf16", 16, mix=31),
        # checking trees of up to 64 nodes for an ordinary ragged batch
        _attend("attend_b24_n64_8k", 24, (3000, 8000), (40, 64), 2, (32, 4), 128, "bf16", 64, mix=32),
        # small trees with a sliding window, two prompts' chunks and an idle entry beside them
        _attend("attend_mixed_b30", 30, (300, 8000), (5, 17), 1, (32, 8), 64, "fp16", 32, window=4095, chunks=2, chunk=(300, 450), idle=1,
                pad=5, cache="tokens", mix=33),
        # the walk along one small batch's trees
        _accept("accept_b8_n26", 8, (100, 4000), (26, 26), 16, 8, mix=41),
        # a large server's step
        _accept("accept_b301_n64", 301, (1, 9000), (20, 64), 16, 12, chunks=7, chunk=(200, 2000), idle=20, pad=100, mix=42),
        # one layer's accepted rows
        _move("move_b8_l1", 8, 1, (26, 26), 8, 8, 128, "bf16", 16, mix=51),
        # accepted rows of a batch in all layers at once
        _move("move_b61_l32", 61, 32, (20, 64), 8, 8, 128, "bf16", 16, mix=52),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    op = rng.choice(("tree", "rope", "rope", "attend", "attend", "attend", "accept", "move"))
    words = rng.choice((1, 1, 2, 2, 4, 8))
    n_hi = rng.randint(1, 32 * words)
    nodes = (rng.choice((1, n_hi // 2 or 1, n_hi)), n_hi)
    spread = rng.choice((1, 2, 8, 32))
    pad = rng.choice((0, 0, 5, 100))
    if op in ("tree", "accept"):
        B = _log(rng, 1, max(1, min(300, 12000 // n_hi)))
        chunks = rng.choice((0, 0, min(B, 3)))
        chunk = (32 * words + 1, 32 * words + _log(rng, 8, 1000))
        idle = rng.randrange(B // 4 + 1)
        if op == "tree":
            return {k: v for k, v in _tree("", B, nodes, words, chunks, chunk, idle, pad, spread, mix).items() if k != "name"}
        c = _accept("", B, (rng.choice((0, 1, 500)), _log(rng, 600, 9000)), nodes, rng.choice(PAGES), rng.randint(1, 16), chunks, chunk, idle, pad,
                    spread, rng.choice((0.3, 0.7, 0.95)), mix)
        return {k: v for k, v in c.items() if k != "name"}
    heads, d, dtype, page = rng.choice(HEADS), rng.choice((64, 128)), rng.choice(("bf16", "fp16")), rng.choice(PAGES)
    if op == "rope":
        rows = _log(rng, 1, 16000)
        c = _rope("", rows, heads, d, dtype, rng.choice((0, page)), pad, rng.choice(("none", "type", "f32")), rng.choice((d, d, d // 2, 16)),
                  rng.choice((1, 1, 2, 3, 4)), rng.choice(("halves", "alternate")), rng.choice(("tokens", "heads")), _log(rng, 100, 1000000), mix)
        return {k: v for k, v in c.items() if k != "name"}
    if op == "move":
        B, layers = _log(rng, 1, 60), rng.choice((1, 1, 2, 7, 24))
        c = _move("", B, layers, nodes, rng.randint(1, 8), heads[1], d, dtype, page, rng.choice(("heads", "tokens")), mix)
        return {k: v for k, v in c.items() if k != "name"}
    B = _log(rng, 1, 64)
    chunks, top = 0, n_hi
    chunk = (1, 1)
    if rng.random() < 0.25 and B > 2:
        chunks = rng.randint(1, 2)
        chunk = (32 * words + 1, 32 * words + _log(rng, 8, 200))
        top = chunk[1]
    ctx = _log(rng, 16, max(17, min(100000, 60000000000 // (B * top * heads[0] * d * 4), 300000000 // (B * heads[1] * d * 4))))
    c = _attend("", B, (rng.choice((0, max(1, ctx // 3), ctx)), ctx), nodes, words, heads, d, dtype, page, rng.choice((-1, -1, -1, _log(rng, 1, 4000))),
                chunks, chunk, rng.randrange(B // 8 + 1), rng.choice((0, 0, 5)), spread, rng.choice(("tokens", "heads")),
                rng.choice(("heads", "tokens")), mix)
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(case):
    """Cached tokens, nodes (or a chunk's tokens) and whether it is a chunk, of every request, from the case alone."""
    r = random.Random(case["mix"])
    B = case["B"]
    ctx, new, chunk = [], [], []
    for b in range(B):
        lo, hi = case["ctx_lo"], case["ctx_hi"]
        ctx.append(lo if lo == hi else max(lo, _log(r, max(1, lo), hi)))
        chunk.append(b < case["chunks"])
        new.append(r.randint(case["chunk_lo"], case["chunk_hi"]) if chunk[-1] else r.randint(case["n_lo"], case["n_hi"]))
    order = list(range(B))
    r.shuffle(order)
    ctx, new, chunk = ([x[i] for i in order] for x in (ctx, new, chunk))
    small = [b for b in range(B) if not chunk[b]]
    for b in small[:min(case["idle"], len(small) - 1 if len(small) == B else len(small))]:
        new[b] = 0
    return ctx, new, chunk


def _pages(n, page):
    return -(-n // page)


def _depths(case, g, dev):
    """Parents of every node, request by request [rows]: node 0 has none, a chunk is a chain."""
    ctx, new, chunk = _lengths(case)
    first = np.repeat(np.concatenate([[0], np.cumsum(new)])[:-1], new)
    i = torch.from_numpy(np.arange(sum(new)) - first).to(dev)
    chain = torch.from_numpy(np.repeat(np.array(chunk), new)).to(dev)
    back = (torch.rand(i.numel(), device=dev, generator=g) * torch.minimum(i, torch.full_like(i, case["spread"]))).long()
    return torch.where(chain, i - 1, i - 1 - back.clamp(max=i)).int()


def _rows(case):
    return sum(_lengths(case)[1]) + case["pad"]


def _moves(case):
    """Nodes of every request and accepted ones, in order: sources lie behind the destinations, so that a pass can be repeated."""
    r = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        n = r.randint(case["n_lo"], case["n_hi"]) + case["steps"]
        out.append((n, sorted(r.sample(range(case["steps"] + 1, n + 1), min(r.randint(0, case["steps"]), n - case["steps"])))))
    return out


def work(case):
    op = case["op"]
    if op == "rope":
        rows, row = case["rows"], case["d"] * 2
        heads = case["Hq"] + case["Hkv"] * (2 if case["page"] else 1)
        return {"bytes": 2 * rows * heads * row + 4 * rows * (case["axes"] + (1 if case["page"] else 0)),
                "flops": 8 * rows * (case["Hq"] + case["Hkv"]) * case["d"]}
    if op == "move":
        n = sum(len(path) for _, path in _moves(case))
        return {"bytes": 4 * case["layers"] * n * case["Hkv"] * case["d"] * 2 + 8 * case["B"] * case["steps"], "flops": 0}
    ctx, new, chunk = _lengths(case)
    B, total = case["B"], sum(new)
    if op == "tree":
        trees = sum(n for n, c in zip(new, chunk) if not c)
        return {"bytes": 8 * B + 4 * total + trees * (4 + 4 * case["words"]), "flops": 0}
    if op == "accept":
        trees = sum(n for n, c in zip(new, chunk) if not c)
        return {"bytes": 12 * trees + 8 * B + 12 * B + 12 * B * case["steps"], "flops": 0}
    pairs = keys = 0
    for c, n, ch in zip(ctx, new, chunk):
        if n:
            seen = c if case["window"] < 0 else min(c, case["window"])
            # a row sees its context and, of the new rows, itself and those above it
            pairs += n * seen + (n * (n + 1) // 2 if ch else n * min(n, 5))
            keys += seen + n
    q = total * case["Hq"] * case["d"] * 2
    return {"bytes": 2 * q + 4 * total * case["Hq"] + 2 * keys * case["Hkv"] * case["d"] * 2, "flops": 4 * pairs * case["Hq"] * case["d"]}


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _gen(seed, dev):
    return torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)


def _block_tables(case, ctx, new, g, dev):
    """Pages of every request, ids in the order of a pool that has been in use for long; the free ids behind them."""
    held = [_pages(c + n, case["page"]) for c, n in zip(ctx, new)]
    W = max(1, max(held)) + 3
    num_pages = sum(held) + 11
    perm = torch.randperm(num_pages, device=dev, generator=g).to(torch.int32)
    starts = np.concatenate([[0], np.cumsum(held)])
    at = np.arange(W)[None] + starts[:-1, None]
    at = torch.from_numpy(np.where(np.arange(W)[None] < np.array(held)[:, None], at, -1)).to(dev)
    table = torch.where(at >= 0, perm[at.clamp(min=0)], torch.full_like(perm[:1], -1)).contiguous()
    return table, num_pages, perm, int(starts[-1])


def _prepare_rope(case, seed, dev):
    g = _gen(seed, dev)
    n, Hq, Hkv, d, dt, page = case["rows"] + case["pad"], case["Hq"], case["Hkv"], case["d"], DTYPES[case["dtype"]], case["page"]
    heads = Hq + 2 * Hkv
    # the projections' output: a row per token with all heads side by side, or head by head; sizes differ from head to head
    size = torch.exp(torch.randn((heads, 1, 1), generator=g, device=dev))
    if case["layout"] == "tokens":
        qkv = (torch.randn((n, heads, d), generator=g, device=dev) * size.transpose(0, 1)).to(dt).transpose(0, 1)
    else:
        qkv = (torch.randn((heads, n, d), generator=g, device=dev) * size).to(dt)
    A, rot = case["axes"], case["rot"]
    # each pair belongs to one axis: the first pairs to the first, ...; frequencies fall from 1 to 1 / base
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    axis = torch.arange(rot // 2) * A // (rot // 2)
    inv = torch.where(axis[None] == torch.arange(A)[:, None], freq[None], 0.0).float().to(dev)
    pos = torch.randint(0, case["far"], (A, n), generator=g, device=dev, dtype=torch.int32)
    s = {"op": "rope", "q": qkv[:Hq], "k": qkv[Hq:Hq + Hkv], "v": qkv[Hq + Hkv:], "inv": inv, "pos": pos if A > 1 else pos[0], "axes": A,
         "rot": rot, "alternate": case["pairs"] == "alternate", "page": page, "eps": 1e-6, "wq": None, "wk": None,
         "qo": torch.zeros((n, Hq, d), dtype=dt, device=dev).transpose(0, 1) if case["layout"] == "tokens" else
         torch.zeros((Hq, n, d), dtype=dt, device=dev)}
    if case["norm"] != "none":
        w = 1.0 + 0.2 * torch.randn((2, d), generator=g, device=dev)
        s["wq"], s["wk"] = w if case["norm"] == "f32" else w.to(dt)
    if page:
        num_pages = _pages(n, page) + 5
        slots = torch.randperm(num_pages * page, generator=g, device=dev)[:n].int()
        if case["pad"]:
            slots[case["rows"]:] = -1
        s.update(slots=slots, k_cache=torch.zeros((num_pages, Hkv, page, d), dtype=dt, device=dev),
                 v_cache=torch.zeros((num_pages, Hkv, page, d), dtype=dt, device=dev))
    else:
        s["ko"] = torch.zeros((Hkv, n, d), dtype=dt, device=dev)
    return s


def _prepare_move(case, seed, dev):
    g = _gen(seed, dev)
    moves, page, P = _moves(case), case["page"], case["steps"]
    rows = [n + 1 for n, _ in moves]
    table, num_pages, _, _ = _block_tables(case, [0] * case["B"], rows, g, dev)
    host = table.cpu().numpy().astype(np.int64)
    src, dst = np.full((case["B"], P), -1), np.full((case["B"], P), -1)
    for b, (_, path) in enumerate(moves):
        for j, a in enumerate(path):
            src[b, j] = host[b, a // page] * page + a % page
            dst[b, j] = host[b, (j + 1) // page] * page + (j + 1) % page
    shape = (case["layers"], num_pages, case["Hkv"], page, case["d"])
    if case["cache"] == "tokens":
        shape = (case["layers"], num_pages, page, case["Hkv"], case["d"])
    k, v = (torch.randn(shape, generator=g, device=dev, dtype=DTYPES[case["dtype"]]) for _ in range(2))
    if case["cache"] == "tokens":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    return {"op": "move", "k_cache": k, "v_cache": v, "src": _ints(src.tolist(), dev), "dst": _ints(dst.tolist(), dev), "page": page}


def prepare(case, seed):
    dev, op = "cuda", case["op"]
    if op in ("rope", "move"):
        return _prepare_rope(case, seed, dev) if op == "rope" else _prepare_move(case, seed, dev)
    g = _gen(seed, dev)
    ctx, new, chunk = _lengths(case)
    B, n = case["B"], _rows(case)
    total = sum(new)
    parents = torch.full((n,), -1, dtype=torch.int32, device=dev)
    parents[:total] = _depths(case, g, dev)
    lens = [c + m for c, m in zip(ctx, new)]
    s = {"op": op, "B": B, "rows": n, "max_n": max(new), "cu": _ints(np.concatenate([[0], np.cumsum(new)]).tolist(), dev),
         "lens": _ints(lens, dev), "parents": parents, "max_k": max(lens)}
    if op == "accept":
        page = case["page"]
        table, num_pages, perm, used = _block_tables(case, ctx, new, g, dev)
        free = torch.full((num_pages,), -1, dtype=torch.int32, device=dev)
        free[:num_pages - used] = perm[used:]
        tokens = torch.randint(0, 32000, (n,), generator=g, device=dev, dtype=torch.int32)
        # where the model agrees with the draft, its choice behind a node is the token of one of the node's children
        first = torch.from_numpy(np.repeat(np.concatenate([[0], np.cumsum(new)])[:-1], new)).to(dev)
        up = (parents[:total].long() + first)[parents[:total] >= 0]
        kids = torch.arange(total, device=dev)[parents[:total] >= 0]
        child = torch.full((n,), n, device=dev).scatter_reduce(0, up, kids, "amax", include_self=False)
        targets = torch.randint(0, 32000, (n,), generator=g, device=dev, dtype=torch.int32)
        agrees = (torch.rand(n, generator=g, device=dev) < case["likely"]) & (child < n)
        targets = torch.where(agrees, tokens[child.clamp(max=n - 1)], targets)
        confirmed = [m if c else min(m, 1) for m, c in zip(new, chunk)]
        out = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)  # noqa: E731
        P = case["steps"]
        s.update(page=page, num_pages=num_pages, table=table, free=free, free_count=_ints([num_pages - used], dev), free_left=out(1),
                 tokens=tokens, targets=targets.int(), confirmed=_ints(confirmed, dev), steps=P, accepted=out(B), ctx=out(B), next=out(B),
                 path=out(B, P), src=out(B, P), dst=out(B, P))
        return s
    s.update(words=case["words"], mask=torch.zeros((n, case["words"]), dtype=torch.int32, device=dev),
             positions=torch.full((n,), -1, dtype=torch.int32, device=dev))
    if op == "tree":
        return s
    _tree_plain(s)
    Hq, Hkv, d, dt, page = case["Hq"], case["Hkv"], case["d"], DTYPES[case["dtype"]], case["page"]
    table, num_pages, _, _ = _block_tables(case, ctx, new, g, dev)
    shape = (num_pages, Hkv, page, d) if case["cache"] == "heads" else (num_pages, page, Hkv, d)
    # a used cache: every row holds something, those that no request owns any longer too
    k, v = (torch.randn(shape, generator=g, device=dev, dtype=dt) for _ in range(2))
    if case["cache"] == "tokens":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    if case["rows"] == "tokens":
        q = torch.randn((n, Hq, d), generator=g, device=dev, dtype=dt).transpose(0, 1)
        o = torch.zeros((n, Hq, d), dtype=dt, device=dev).transpose(0, 1)
    else:
        q, o = torch.randn((Hq, n, d), generator=g, device=dev, dtype=dt), torch.zeros((Hq, n, d), dtype=dt, device=dev)
    s.update(q=q, k_cache=k, v_cache=v, o=o, lse=torch.zeros((Hq, n), dtype=torch.float32, device=dev), table=table, page=page,
             window=case["window"], scale=1.0 / math.sqrt(d))
    return s


# ------------------------------------------------------------------------------ plain forms
def _spans(s):
    """Request of every packed row, its number in it, whether it has one; the requests' rows."""
    cu = s["cu"].long()
    t = torch.arange(s["rows"], device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=s["B"] - 1)
    return b, t - cu[b], t < cu[-1], cu[1:] - cu[:-1]


def _tree_plain(s):
    b, i, live, count = _spans(s)
    most = 32 * s["words"]
    tree = live & (count[b] <= most)
    ctx = (s["lens"].long() - count)[b]
    # the nodes above each node: the relation "is it or its parent", multiplied with itself until it reaches the root
    n = min(most, s["max_n"])
    up = torch.zeros((s["B"], n, n), device=b.device)
    at = i.clamp(max=n - 1)
    up.index_put_((b, at, at), torch.where(tree, 1.0, 0.0), accumulate=True)
    par = s["parents"].long()
    up.index_put_((b, at, par.clamp(0, n - 1)), torch.where(tree & (par >= 0), 1.0, 0.0), accumulate=True)
    up = (up > 0).float()
    for _ in range(max(1, (n - 1).bit_length())):
        up = ((up @ up) > 0).float()
    depth = up.sum(-1).long() - 1
    pos = ctx + torch.where(tree, depth[b, at], i)
    bits = torch.zeros((s["B"], n, most), dtype=torch.long, device=b.device)
    bits[:, :, :n] = up.long()
    word = (bits.view(s["B"], n, s["words"], 32) << torch.arange(32, device=b.device)).sum(-1)
    word = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
    s["positions"].copy_(torch.where(live, pos, s["positions"]))
    s["mask"].copy_(torch.where(tree[:, None], word[b, at], s["mask"]))
    return {"positions": s["positions"], "mask": s["mask"]}


def _turned(x, w, cos, sin, s):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
    rot = s["rot"]
    y = x.clone()
    if s["alternate"]:
        a, c = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - c * sin, c * cos + a * sin
    else:
        a, c = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - c * sin, c * cos + a * sin
    return y


def _rope_plain(s):
    angle = s["pos"].view(s["axes"], -1).double().T @ s["inv"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k = _turned(s["q"], s["wq"], cos, sin, s), _turned(s["k"], s["wk"], cos, sin, s)
    if not s["page"]:
        s["qo"].copy_(q)
        s["ko"].copy_(k)
        return {"q": s["qo"], "k": s["ko"]}
    live = s["slots"] >= 0
    s["qo"].copy_(torch.where(live[None, :, None], q.to(s["qo"].dtype), s["qo"]))
    slot = s["slots"][live].long()
    page, off = slot // s["page"], slot % s["page"]
    s["k_cache"][page, :, off] = k.to(s["k_cache"].dtype).transpose(0, 1)[live]
    s["v_cache"][page, :, off] = s["v"].transpose(0, 1)[live]
    return {"q": s["qo"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, table):
    """The pages of every request one behind the other: [B, Hkv, keys, d] in 32 bits."""
    x = cache[table.long().clamp(min=0)].float()
    B, n, H, page, d = x.shape
    return x.transpose(1, 2).reshape(B, H, n * page, d)


def _attend_plain(s):
    q, dev = s["q"], s["q"].device
    Hq, n, d = q.shape
    Hkv, B, mq, mk = s["k_cache"].shape[1], s["B"], s["max_n"], s["max_k"]
    table = s["table"][:, :-(-mk // s["page"])]
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    ctx = lens - count
    i = torch.arange(mq, device=dev)
    row = (cu[:-1, None] + i[None]).clamp(max=n - 1)                                          # [B, mq]
    qp = q.transpose(0, 1)[row].float().transpose(1, 2).reshape(B, Hkv, Hq // Hkv * mq, d)    # heads of a group side by side
    sc = (qp * s["scale"]) @ _gathered(s["k_cache"], table).transpose(2, 3)
    j = torch.arange(sc.shape[-1], device=dev)
    pos = s["positions"].long()[row][..., None]
    most = 32 * s["words"]
    bits = ((s["mask"].long()[..., None] >> torch.arange(32, device=dev)) & 1).bool().view(n, most)
    rel = j[None] - ctx[:, None]                                                               # [B, keys]: number of the new row
    among = torch.gather(bits[row], 2, rel.clamp(0, most - 1)[:, None].expand(B, mq, -1)) & (rel < most)[:, None]
    among = torch.where((count <= most)[:, None, None], among, j <= pos)
    if s["window"] >= 0:
        near = j >= pos - s["window"]
        among = torch.where((count <= most)[:, None, None], among, among & near)
    else:
        near = torch.ones_like(among)
    keep = torch.where((rel >= 0)[:, None], among, near) & (j < lens[:, None])[:, None]
    keep = keep[:, None, None]                                                                # [B, 1, 1, mq, keys]
    sc = sc.view(B, Hkv, Hq // Hkv, mq, -1).masked_fill_(~keep, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, -1, p.shape[-1]) @ _gathered(s["v_cache"], table)
    o = o.view(B, Hq, mq, d) / l.view(B, Hq, mq, 1).clamp(min=1e-38)
    lse = (m + l.log()).view(B, Hq, mq)
    # back to packed rows; those behind the last request stay as they were
    b, at, live, _ = _spans(s)
    at = at.clamp(0, mq - 1)
    s["o"].copy_(torch.where(live[None, :, None], o[b, :, at].transpose(0, 1).to(q.dtype), s["o"]))
    s["lse"].copy_(torch.where(live[None], lse[b, :, at].transpose(0, 1), s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def _accept_plain(s):
    dev, B, P, page = s["cu"].device, s["B"], s["steps"], s["page"]
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    ctx = lens - count
    i = torch.arange(s["max_n"], device=dev)
    row = (cu[:-1, None] + i[None]).clamp(max=s["rows"] - 1)
    mine = i[None] < count[:, None]
    tokens, targets, parents = (s[k].long()[row] for k in ("tokens", "targets", "parents"))
    sure = torch.minimum(s["confirmed"].long(), count)
    cur, taken, alive = sure - 1, torch.zeros_like(sure), count > 0
    path = torch.full((B, P), -1, device=dev)
    for step in range(P):
        want = torch.gather(targets, 1, cur.clamp(min=0)[:, None])
        ok = mine & (parents == cur[:, None]) & (tokens == want) & (i[None] > cur[:, None])
        child = torch.where(ok, i[None], s["max_n"]).amin(1)
        alive = alive & (child < s["max_n"])
        path[:, step] = torch.where(alive, child, -1)
        cur = torch.where(alive, child, cur)
        taken = taken + alive
    accepted = sure + taken
    after = ctx + accepted
    slot_of = lambda p: torch.gather(s["table"].long(), 1, p // page) * page + p % page  # noqa: E731
    to = sure[:, None] + torch.arange(P, device=dev)[None]
    moves = (path >= 0) & (path != to)
    src = torch.where(moves, slot_of(ctx[:, None] + path.clamp(min=0)), -1)
    dst = torch.where(moves, slot_of(torch.where(moves, ctx[:, None] + to, 0)), -1)
    nxt = torch.where(count > 0, torch.gather(targets, 1, cur.clamp(min=0)[:, None])[:, 0], -1)
    # pages that hold no token any longer go back, request by request
    keep, held = (after + page - 1) // page, (lens + page - 1) // page
    col = torch.arange(s["table"].shape[1], device=dev)
    back = (col[None] >= keep[:, None]) & (col[None] < held[:, None])
    back = s["table"][back]
    have = s["free_count"].long()
    free = s["free"]
    f = torch.arange(free.numel(), device=dev)
    came = (f >= have) & (f < have + back.numel())
    if back.numel():
        free.copy_(torch.where(came, back[(f - have).clamp(0, back.numel() - 1)], free))
    return {"accepted": accepted.int(), "ctx": after.int(), "next": nxt.int(), "path": path.int(), "src": src.int(), "dst": dst.int(),
            "free": free, "free_left": (have + back.numel()).int()}


def _move_plain(s):
    live = s["src"] >= 0
    src, dst, page = s["src"][live].long(), s["dst"][live].long(), s["page"]
    for c in (s["k_cache"], s["v_cache"]):
        c[:, dst // page, :, dst % page] = c[:, src // page, :, src % page]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    s = state
    if not own:
        return {"tree": _tree_plain, "rope": _rope_plain, "attend": _attend_plain, "accept": _accept_plain, "move": _move_plain}[s["op"]](s)
    import attention_forward_07_gb300 as af
    if s["op"] == "tree":
        af.attn_paged_tree(s["parents"], s["cu"], s["lens"], s["positions"], s["mask"])
        return {"positions": s["positions"], "mask": s["mask"]}
    if s["op"] == "rope":
        if s["page"]:
            af.attn_paged_rope(s["q"], s["k"], s["v"], s["qo"], s["k_cache"], s["v_cache"], s["slots"], s["pos"], s["inv"], s["wq"], s["wk"],
                               eps=s["eps"], interleaved=s["alternate"])
            return {"q": s["qo"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        af.attn_rope(s["q"], s["k"], s["qo"], s["ko"], s["pos"], s["inv"], s["wq"], s["wk"], eps=s["eps"], interleaved=s["alternate"])
        return {"q": s["qo"], "k": s["ko"]}
    if s["op"] == "attend":
        af.attn_fwd_paged_tree(s["q"], s["k_cache"], s["v_cache"], s["o"], s["table"], s["cu"], s["lens"], s["max_n"], s["mask"],
                               positions=s["positions"], lse=s["lse"], window_left=s["window"], scale=s["scale"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "accept":
        af.attn_paged_accept(s["tokens"], s["targets"], s["parents"], s["cu"], s["lens"], s["table"], s["free"], s["free_count"], s["page"],
                             s["num_pages"], s["accepted"], s["ctx"], s["next"], s["path"], s["src"], s["dst"], confirmed=s["confirmed"],
                             free_count_out=s["free_left"])
        return {"accepted": s["accepted"], "ctx": s["ctx"], "next": s["next"], "path": s["path"], "src": s["src"], "dst": s["dst"],
                "free": s["free"], "free_left": s["free_left"]}
    af.attn_paged_move(s["k_cache"], s["v_cache"], s["src"], s["dst"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ------------------------------------------------------------------------------ definitions in 64 bits
def _exact_rope(case, s):
    rot, rows, d = case["rot"], case["rows"], case["d"]
    pos = s["pos"].double().reshape(case["axes"], -1)
    angle = sum(pos[a][:, None] * s["inv"][a].double()[None] for a in range(case["axes"]))
    turn = torch.polar(torch.ones_like(angle), angle)
    first = torch.arange(0, rot, 2) if s["alternate"] else torch.arange(rot // 2)
    second = first + (1 if s["alternate"] else rot // 2)

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + s["eps"]) * w.double()
        z = torch.complex(x[:, first], x[:, second]) * turn
        out = x.clone()
        out[:, first], out[:, second] = z.real, z.imag
        return out

    q = torch.stack([one(h, s["wq"]) for h in s["q"]])
    k = torch.stack([one(h, s["wk"]) for h in s["k"]])
    if not case["page"]:
        return {"q": q, "k": k}
    q[:, rows:] = s["qo"][:, rows:].double()
    out = {"q": q}
    slots = s["slots"][:rows].long()
    for name, new in (("k_cache", k), ("v_cache", s["v"].double())):
        c = s[name].double()
        for h in range(case["Hkv"]):
            flat = c[:, h].reshape(-1, d)
            flat[slots] = new[h, :rows]
            c[:, h] = flat.view(-1, case["page"], d)
        out[name] = c
    return out


def exact(case, seed):
    """The definitions, request by request in 64 bits; trees and walks are whole numbers."""
    if case["op"] in ("tree", "accept"):
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "move":
        out = {}
        src, dst = s["src"].flatten().tolist(), s["dst"].flatten().tolist()
        for name in ("k_cache", "v_cache"):
            c = s[name].double()
            for a, b in zip(src, dst):
                if a >= 0:
                    c[:, b // s["page"], :, b % s["page"]] = s[name][:, a // s["page"], :, a % s["page"]].double()
            out[name] = c
        return out
    ctx, new, chunk = _lengths(case)
    o, lse = s["o"].double(), s["lse"].double()
    parents = s["parents"].tolist()
    g, first = case["Hq"] // case["Hkv"], 0
    for b in range(case["B"]):
        n, keys = new[b], ctx[b] + new[b]
        if n == 0:
            continue
        keep = np.zeros((n, keys), bool)
        for i in range(n):
            if chunk[b]:
                keep[i, :ctx[b] + i + 1] = True
                if case["window"] >= 0:
                    keep[i, :max(0, ctx[b] + i - case["window"])] = False
                continue
            above, a = [], i
            while a >= 0:
                above.append(ctx[b] + a)
                a = parents[first + a]
            keep[i, :ctx[b]] = True
            if case["window"] >= 0:
                keep[i, :min(ctx[b], max(0, ctx[b] + len(above) - 1 - case["window"]))] = False
            keep[i, above] = True
        out = ~torch.from_numpy(keep).to(o.device)
        ids = s["table"][b, :_pages(keys, case["page"])].long()
        for h in range(case["Hkv"]):
            k = torch.cat(list(s["k_cache"][ids, h]))[:keys].double()
            v = torch.cat(list(s["v_cache"][ids, h]))[:keys].double()
            for hq in range(h * g, (h + 1) * g):
                x = ((s["q"][hq, first:first + n].double() @ k.T) / math.sqrt(case["d"])).masked_fill(out, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[hq, first:first + n] = z
                o[hq, first:first + n] = torch.exp(x - z[:, None]) @ v
        first += n
    return {"o": o, "lse": lse}
