"""Cases of the paged key/value-cache operators: what is timed, and their plain forms.

Three operators make one serving step of a model whose keys and values live in pages:

* ``tables``: request lengths -> block tables, slot map, positions and row offsets
  (``attn_paged_tables``);
* ``append``: the step's new key / value rows go to their slots in the paged cache
  (``attn_paged_append``);
* ``attend``: the step's query rows attend over the paged cache (``attn_fwd_paged``), from one
  token per request (decoding) to chunks of thousands.

``run`` computes the plain forms out of elementary torch operations in 32 bits, or, with
``own`` true, calls the library.  The cache layout is ``[num_pages, Hkv, page_size, d]``; query,
key and value rows are packed, ``[H, rows, d]``, request after request.  A case's request
lengths come from its own ``mix`` number, its values from the seed.
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


def _attend(name, B, ctx, new, heads, d, dtype, page, window=-1, chunks=0, chunk=(1, 1), idle=0, pad=0, rows="tokens",
            cache="heads", mix=1):
    return {"name": name, "op": "attend", "B": B, "ctx_lo": ctx[0], "ctx_hi": ctx[1], "new_lo": new[0], "new_hi": new[1],
            "chunks": chunks, "chunk_lo": chunk[0], "chunk_hi": chunk[1], "idle": idle, "pad": pad, "Hq": heads[0],
            "Hkv": heads[1], "d": d, "dtype": dtype, "page": page, "window": window, "rows": rows, "cache": cache, "mix": mix}


def listed():
    return [
        # the tables of an ordinary decoding step: every request grows by one token
        {"name": "tables_decode_b64", "op": "tables", "B": 64, "ctx_lo": 200, "ctx_hi": 8000, "new_lo": 1, "new_hi": 1,
         "chunks": 0, "chunk_lo": 1, "chunk_hi": 1, "idle": 0, "pad": 0, "page": 16, "mix": 11},
        # a large step of a busy server: hundreds of decoding requests, long prompts admitted beside them, idle
        # entries of a fixed batch size, and room behind the last token
        {"name": "tables_admit_b509", "op": "tables", "B": 509, "ctx_lo": 1, "ctx_hi": 16000, "new_lo": 1, "new_hi": 1,
         "chunks": 12, "chunk_lo": 500, "chunk_hi": 8000, "idle": 40, "pad": 1000, "page": 16, "mix": 12},
        # one layer's new rows of a decoding step, in a batch padded to a captured size
        {"name": "append_decode_b64", "op": "append", "B": 61, "ctx_lo": 200, "ctx_hi": 4000, "new_lo": 1, "new_hi": 1,
         "chunks": 0, "chunk_lo": 1, "chunk_hi": 1, "idle": 0, "pad": 3, "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16",
         "page": 16, "rows": "tokens", "cache": "heads", "mix": 21},
        # one layer's new rows of admitted prompts
        {"name": "append_chunks_16k", "op": "append", "B": 9, "ctx_lo": 0, "ctx_hi": 9000, "new_lo": 1500, "new_hi": 2300,
         "chunks": 0, "chunk_lo": 1, "chunk_hi": 1, "idle": 0, "pad": 0, "Hq": 32, "Hkv": 8, "d": 128, "dtype": "fp16",
         "page": 64, "rows": "tokens", "cache": "tokens", "mix": 22},
        # decoding, one request alone: latency
        _attend("decode_b1_1k", 1, (1001, 1001), (1, 1), (32, 8), 128, "bf16", 16, mix=31),
        # decoding, an ordinary ragged batch, padded to a captured size
        _attend("decode_b64_8k", 61, (500, 8192), (1, 1), (32, 8), 128, "bf16", 16, pad=3, mix=32),
        # decoding against long caches, few requests
        _attend("decode_b3_100k", 3, (60000, 120000), (1, 1), (32, 4), 128, "fp16", 64, mix=33),
        # decoding with a sliding window, a head of its own for every query head
        _attend("decode_window_b32", 32, (700, 16000), (1, 1), (16, 16), 64, "fp16", 32, window=1023, cache="tokens", mix=34),
        # checking a few proposed tokens of every request at once
        _attend("verify_b24_6k", 24, (300, 6000), (3, 6), (32, 4), 128, "bf16", 128, mix=35),
        # a decoding batch with two prompts' chunks beside it
        _attend("mixed_b14_5k", 14, (300, 5000), (1, 1), (32, 8), 128, "bf16", 16, chunks=2, chunk=(300, 450), idle=1, mix=36),
        # one chunk of a long prompt against what is cached of it
        _attend("chunk_2k_30k", 1, (30011, 30011), (2037, 2037), (32, 8), 128, "bf16", 16, mix=37),
        # whole prompts admitted at once
        _attend("prefill_b4_4k", 4, (0, 0), (3500, 4500), (32, 8), 128, "bf16", 64, rows="heads", mix=38),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    op = rng.choice(("tables", "append", "attend", "attend", "attend", "attend"))
    page = rng.choice(PAGES)
    if op == "tables":
        B = _log(rng, 1, 700)
        hi = _log(rng, 16, 16000)
        return {"op": op, "B": B, "ctx_lo": rng.choice((0, 1, hi // 2)), "ctx_hi": hi, "new_lo": 1, "new_hi": rng.choice((1, 1, 4, 64)),
                "chunks": rng.choice((0, 0, min(B, 3), min(B, 8))), "chunk_lo": 1, "chunk_hi": _log(rng, 64, 8000),
                "idle": rng.randrange(B // 4 + 1), "pad": rng.choice((0, 7, 500)), "page": page, "mix": mix}
    heads = rng.choice(HEADS)
    base = {"op": op, "idle": 0, "pad": rng.choice((0, 0, 5)), "Hq": heads[0], "Hkv": heads[1], "d": rng.choice((64, 128)),
            "dtype": rng.choice(("bf16", "fp16")), "page": page, "rows": rng.choice(("tokens", "heads")),
            "cache": rng.choice(("heads", "tokens")), "mix": mix}
    if op == "append":
        B = _log(rng, 1, 128)
        top = _log(rng, 1, max(1, 16000 // B))
        return dict(base, B=B, ctx_lo=0, ctx_hi=_log(rng, 1, 8000), new_lo=rng.choice((1, max(1, top // 2))), new_hi=top, chunks=0, chunk_lo=1,
                    chunk_hi=1, idle=rng.randrange(B // 4 + 1))
    window = rng.choice((-1, -1, -1, _log(rng, 1, 4000)))
    kind = rng.choice(("decode", "decode", "verify", "mixed", "chunk"))
    if kind in ("decode", "verify"):
        B = _log(rng, 1, 128)
        hi = _log(rng, 16, min(100000, 600000 // B))
        new = (1, 1) if kind == "decode" else (1, rng.randint(2, 9))
        return dict(base, B=B, ctx_lo=rng.choice((1, max(1, hi // 3), hi)), ctx_hi=hi, new_lo=new[0], new_hi=new[1], chunks=0, chunk_lo=1,
                    chunk_hi=1, window=window, idle=rng.randrange(B // 8 + 1))
    if kind == "mixed":
        B = _log(rng, 3, 20)
        return dict(base, B=B, ctx_lo=1, ctx_hi=_log(rng, 64, 5000), new_lo=1, new_hi=1, chunks=rng.randint(1, 2), chunk_lo=17,
                    chunk_hi=_log(rng, 20, 450), window=window)
    new = _log(rng, 20, 2500)
    return dict(base, B=rng.randint(1, 3), ctx_lo=0, ctx_hi=_log(rng, 16, 16000), new_lo=max(1, new // 2), new_hi=new, chunks=0, chunk_lo=1,
                chunk_hi=1, window=window)


def _lengths(case):
    """Cached and new tokens of every request, from the case alone."""
    r = random.Random(case["mix"])
    ctx, new = [], []
    for b in range(case["B"]):
        lo, hi = case["ctx_lo"], case["ctx_hi"]
        ctx.append(0 if hi == 0 else lo if lo == hi else max(lo, _log(r, max(1, lo), hi)))
        new.append(r.randint(case["chunk_lo"], case["chunk_hi"]) if b < case["chunks"] else r.randint(case["new_lo"], case["new_hi"]))
    order = list(range(case["B"]))
    r.shuffle(order)
    new = [new[i] for i in order]
    idle = [i for i in order[::-1] if new[i] <= case["new_hi"]][:min(case["idle"], case["B"] - 1)]
    for i in idle:
        new[i] = 0
    if not any(new):
        new[0] = 1
    return ctx, new


def _pages(n, page):
    return -(-n // page)


def _kept(ctx, new, window):
    """Kept (query, key) pairs and read keys of a causal chunk."""
    pos = np.arange(ctx, ctx + new, dtype=np.int64)
    lo = np.maximum(pos - window, 0) if window >= 0 else np.zeros_like(pos)
    return int((pos + 1 - lo).sum()), int(ctx + new - lo[0]) if new else 0


def work(case):
    ctx, new = _lengths(case)
    total, B, page = sum(new), case["B"], case["page"]
    if case["op"] == "tables":
        grown = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(ctx, new))
        # lengths in, offsets and lengths out, the open page's entry; the new pages' ids in and out; a slot and a position per token
        return {"bytes": 4 * (5 * B + 1) + 8 * grown + 8 * (total + case["pad"]), "flops": 0}
    row = case["Hkv"] * case["d"] * 2
    if case["op"] == "append":
        return {"bytes": 4 * total * row + 4 * (total + case["pad"]), "flops": 0}
    pairs = keys = 0
    for c, n in zip(ctx, new):
        p, k = _kept(c, n, case["window"])
        pairs, keys = pairs + p, keys + k
    q = total * case["Hq"] * case["d"] * 2
    return {"bytes": 2 * q + 4 * total * case["Hq"] + 2 * keys * row, "flops": 4 * pairs * case["Hq"] * case["d"]}


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 13)
    ctx, new = _lengths(case)
    page, B = case["page"], case["B"]
    tables = case["op"] == "tables"
    # pages the requests hold when the call comes: for `tables` those of the cached tokens, else the new ones' too
    held = [_pages(c + (0 if tables else n), page) for c, n in zip(ctx, new)]
    want = [_pages(c + n, page) for c, n in zip(ctx, new)]
    W = max(1, max(want)) + 3
    num_pages = sum(want) + 11
    # ids in the order of a pool that has been in use for long
    perm = torch.randperm(num_pages, device=dev, generator=g).to(torch.int32)
    starts = np.concatenate([[0], np.cumsum(held)])
    at = np.full((B, W), -1, np.int64)
    for b in range(B):
        at[b, :held[b]] = np.arange(starts[b], starts[b + 1])
    at = torch.from_numpy(at).to(dev)
    table = torch.where(at >= 0, perm[at.clamp(min=0)], torch.full_like(perm[:1], -1))
    s = {"op": case["op"], "page": page, "num_pages": num_pages, "B": B, "table": table.contiguous(),
         "rows": sum(new) + case["pad"]}
    n = s["rows"]
    if tables:
        free = perm[int(starts[-1]):].contiguous()
        s.update(ctx=_ints(ctx, dev), new=_ints(new, dev), free=free, free_count=_ints([free.numel()], dev),
                 free_left=_ints([0], dev), cu=_ints([0] * (B + 1), dev), lens=_ints([0] * B, dev),
                 slots=torch.zeros(n, dtype=torch.int32, device=dev), positions=torch.zeros(n, dtype=torch.int32, device=dev))
        return s
    Hq, Hkv, d, dt = case["Hq"], case["Hkv"], case["d"], DTYPES[case["dtype"]]
    cu = np.concatenate([[0], np.cumsum(new)])
    # a used cache: every row holds something, those that no request owns any longer too
    shape = (num_pages, Hkv, page, d) if case["cache"] == "heads" else (num_pages, page, Hkv, d)
    caches = []
    for _ in range(2):
        c = torch.randn(shape, generator=g, device=dev, dtype=dt)
        caches.append(c if case["cache"] == "heads" else c.transpose(1, 2))
    s.update(k_cache=caches[0], v_cache=caches[1])
    # the projections' output: a row per token with all heads side by side, or head by head
    if case["rows"] == "tokens":
        qkv = torch.randn((n, Hq + 2 * Hkv, d), generator=g, device=dev, dtype=dt).transpose(0, 1)
    else:
        qkv = torch.randn((Hq + 2 * Hkv, n, d), generator=g, device=dev, dtype=dt)
    if case["op"] == "append":
        b = np.repeat(np.arange(B), new)
        pos = np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, new)])
        host = table.cpu().numpy().astype(np.int64)
        slots = np.concatenate([host[b, pos // page] * page + pos % page, np.full(case["pad"], -1)])
        s.update(k=qkv[Hq:Hq + Hkv], v=qkv[Hq + Hkv:], slots=_ints(slots.tolist(), dev))
        return s
    q = qkv[:Hq]
    o = torch.zeros((n, Hq, d), dtype=dt, device=dev).transpose(0, 1) if case["rows"] == "tokens" else torch.zeros((Hq, n, d), dtype=dt, device=dev)
    s.update(q=q, o=o, lse=torch.zeros((Hq, n), dtype=torch.float32, device=dev), cu=_ints(cu.tolist(), dev),
             lens=_ints([c + m for c, m in zip(ctx, new)], dev), max_q=max(new), max_k=max(c + m for c, m in zip(ctx, new)),
             window=case["window"], scale=1.0 / math.sqrt(d))
    return s


# ------------------------------------------------------------------------------ plain forms
def _tables(s):
    ctx, new, page = s["ctx"].long(), s["new"].long(), s["page"]
    lens = ctx + new
    cu = torch.cat([torch.zeros_like(lens[:1]), torch.cumsum(new, 0)])
    held, want = (ctx + page - 1) // page, (lens + page - 1) // page
    need = want - held
    before = torch.cumsum(need, 0) - need
    col = torch.arange(s["table"].shape[1], device=ctx.device)
    take = s["free_count"] - 1 - (before - held)[:, None] - col[None]  # the last free page goes first
    grown = (col[None] >= held[:, None]) & (col[None] < want[:, None])
    table = torch.where(grown, s["free"][take.clamp(0, s["free"].numel() - 1)], s["table"])
    t = torch.arange(s["rows"], device=ctx.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=s["B"] - 1)
    pos = ctx[b] + t - cu[b]
    live = t < cu[-1]
    slots = table[b, torch.where(live, pos // page, 0)].long() * page + pos % page
    return {"table": table, "slots": torch.where(live, slots, -1).int(), "positions": torch.where(live, pos, -1).int(),
            "cu": cu.int(), "lens": lens.int(), "free_left": (s["free_count"] - need.sum()).int()}


def _append(s):
    keep = s["slots"] >= 0
    slot = s["slots"][keep].long()
    page, off = slot // s["page"], slot % s["page"]
    s["k_cache"][page, :, off] = s["k"].transpose(0, 1)[keep]
    s["v_cache"][page, :, off] = s["v"].transpose(0, 1)[keep]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, table):
    """The pages of every request one behind the other: [B, Hkv, keys, d] in 32 bits."""
    x = cache[table.long().clamp(min=0)].float()
    B, n, H, page, d = x.shape
    return x.transpose(1, 2).reshape(B, H, n * page, d)


def _attention(s):
    q, dev = s["q"], s["q"].device
    Hq, n, d = q.shape
    Hkv, B, mq, mk = s["k_cache"].shape[1], s["B"], s["max_q"], s["max_k"]
    table = s["table"][:, :-(-mk // s["page"])]
    cu, lens = s["cu"].long(), s["lens"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(mq, device=dev)
    row = (cu[:-1, None] + i[None]).clamp(max=n - 1)                                          # [B, mq]
    qp = q.transpose(0, 1)[row].float().transpose(1, 2).reshape(B, Hkv, Hq // Hkv * mq, d)    # heads of a group side by side
    sc = (qp * s["scale"]) @ _gathered(s["k_cache"], table).transpose(2, 3)
    pos = (lens - count)[:, None] + i[None]
    j = torch.arange(sc.shape[-1], device=dev)
    keep = (j <= pos[..., None]) & (j < lens[:, None, None])
    if s["window"] >= 0:
        keep &= j >= pos[..., None] - s["window"]
    keep = keep[:, None, None]                                                                # [B, 1, 1, mq, keys]
    sc = sc.view(B, Hkv, Hq // Hkv, mq, -1).masked_fill_(~keep, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    l = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, -1, p.shape[-1]) @ _gathered(s["v_cache"], table)
    o = o.view(B, Hq, mq, d) / l.view(B, Hq, mq, 1).clamp(min=1e-38)
    lse = (m + l.log()).view(B, Hq, mq)
    # back to packed rows; those behind the last request stay as they were
    t = torch.arange(n, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    live = t < cu[-1]
    at = (t - cu[b]).clamp(0, mq - 1)
    s["o"].copy_(torch.where(live[None, :, None], o[b, :, at].transpose(0, 1).to(q.dtype), s["o"]))
    s["lse"].copy_(torch.where(live[None], lse[b, :, at].transpose(0, 1), s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    s = state
    if own:
        import attention_forward_07_gb300 as af
        if s["op"] == "tables":
            af.attn_paged_tables(s["ctx"], s["new"], s["table"], s["free"], s["free_count"], s["page"], s["num_pages"], s["cu"],
                                 s["lens"], s["slots"], positions=s["positions"], free_count_out=s["free_left"])
            return {"table": s["table"], "slots": s["slots"], "positions": s["positions"], "cu": s["cu"], "lens": s["lens"],
                    "free_left": s["free_left"]}
        if s["op"] == "append":
            af.attn_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        af.attn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["o"], s["table"], s["cu"], s["lens"], s["max_q"], lse=s["lse"],
                          causal=True, window_left=s["window"], scale=s["scale"])
        return {"o": s["o"], "lse": s["lse"]}
    return {"tables": _tables, "append": _append, "attend": _attention}[s["op"]](s)


def exact(case, seed):
    """The definitions, request by request: attention in 64 bits, the cache with its new rows moved in; tables are whole numbers."""
    if case["op"] == "tables":
        return None
    if case["op"] == "append":
        s = prepare(case, seed)
        ctx, new = _lengths(case)
        out, first = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}, 0
        for b in range(case["B"]):
            for i in range(new[b]):
                page, off = divmod(ctx[b] + i, case["page"])
                for name in ("k", "v"):
                    out[name + "_cache"][s["table"][b, page], :, off] = s[name][:, first + i].double()
            first += new[b]
        return out
    if work(case)["flops"] > 4e12:
        return None
    ctx, new = _lengths(case)
    s = prepare(case, seed)
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    o = s["o"].double()
    lse = s["lse"].double()
    first = 0
    for b in range(case["B"]):
        n, keys = new[b], ctx[b] + new[b]
        if n == 0:
            continue
        ids = s["table"][b, :_pages(keys, page)].long()
        pos = torch.arange(ctx[b], keys, device=o.device)[:, None]
        j = torch.arange(keys, device=o.device)[None]
        out = (j > pos) if case["window"] < 0 else (j > pos) | (j < pos - case["window"])
        for h in range(Hkv):
            k = torch.cat(list(s["k_cache"][ids, h]))[:keys].double()
            v = torch.cat(list(s["v_cache"][ids, h]))[:keys].double()
            for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = (s["q"][hq, first:first + n].double() @ k.T) / math.sqrt(d)
                x = x.masked_fill(out, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[hq, first:first + n] = z
                o[hq, first:first + n] = torch.exp(x - z[:, None]) @ v
        first += n
    return {"o": o, "lse": lse}
