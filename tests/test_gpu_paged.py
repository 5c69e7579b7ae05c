"""The paged-cache operators on the GPU against their plain 64-bit forms (paged_ref.py): tables
and slot maps, the append, attention over pages, and the three together as a serving loop runs them."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

from paged_ref import DTYPES, Batch, attention, pages, tables, tolerances

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ tables
def _run_tables(ctx, new, table, free, count, page, num_pages, max_rows, in_place=True, positions=True):
    t, f, c = _i32(table), _i32(free), _i32([count])
    out = c if in_place else _i32([-7])
    B = len(ctx)
    cu, lens, slots, pos = _i32([-5] * (B + 1)), _i32([-5] * B), _i32([-5] * max_rows), _i32([-5] * max_rows)
    af.attn_paged_tables(_i32(ctx), _i32(new), t, f, c, page, num_pages, cu, lens, slots, pos if positions else None,
                         None if in_place else out)
    bad = False
    try:
        af.attn_check()
    except af.AttnError as e:
        assert e.status == -6
        bad = True
    got = dict(table=t, cu=cu, lens=lens, slots=slots, positions=pos)
    return {k: v.cpu().numpy() for k, v in got.items()} | {"left": int(out), "bad": bad}


def _check_tables(ctx, new, table, free, count, page, num_pages, max_rows, **kw):
    got = _run_tables(ctx, new, table, free, count, page, num_pages, max_rows, **kw)
    ref = tables(ctx, new, table, free, count, page, num_pages, max_rows)
    for k in ("table", "cu", "lens", "slots", "left", "bad") + (("positions",) if kw.get("positions", True) else ()):
        assert np.array_equal(got[k], ref[k]), k
    return got


def _held(ctx, page, W, num_pages, rng):
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((len(ctx), W), -1, np.int32)
    at = 0
    for b, c in enumerate(ctx):
        m = pages(max(c, 0), page)
        table[b, :m] = perm[at:at + m]
        at += m
    return table, perm[at:]


@pytest.mark.parametrize("B,page,top_ctx,top_new,pad", [
    (1, 16, 1, 1, 0), (1, 16, 40, 0, 3), (3, 48, 100, 70, 5), (64, 16, 900, 1, 0), (33, 256, 3000, 700, 9),
    (1025, 32, 300, 5, 100), (2500, 16, 60, 30, 1), (16384, 16, 20, 2, 0), (16384, 16, 20, 9, 2)])
def test_tables(B, page, top_ctx, top_new, pad):
    rng = np.random.default_rng(B + page)
    ctx = rng.integers(0, top_ctx + 1, B)
    new = rng.integers(0, top_new + 1, B)
    if B > 2:
        ctx[:3], new[:3] = (0, page, -4), (0, 1, 3)
        new[-1] = -2
    W = pages(top_ctx + top_new + 3, page) + 1
    need = sum(pages(max(c, 0) + max(n, 0), page) for c, n in zip(ctx, new))
    num_pages = need + 5
    table, free = _held(ctx, page, W, num_pages, rng)
    rows = max(1, int(np.maximum(new, 0).sum()) + pad)
    got = _check_tables(ctx, new, table, free, len(free), page, num_pages, rows, in_place=bool(B % 2))
    assert not got["bad"]


@pytest.mark.parametrize("what", ["short", "empty list", "count too large", "count negative", "narrow", "bad free id", "bad held id",
                                  "few rows"])
def test_tables_bad_pages(what):
    """What is missing or out of range is left out, reported, and nothing else suffers."""
    rng = np.random.default_rng(5)
    page, num_pages = 16, 60
    ctx, new = np.array([5, 16, 0, 33, 40]), np.array([3, 40, 20, 1, 30])
    W, rows = 6, int(new.sum()) + 4
    table, free = _held(ctx, page, W, num_pages, rng)
    count = len(free)
    if what == "short":
        count = 4
    elif what == "empty list":
        count = 0
    elif what == "count too large":
        count += 3
    elif what == "count negative":
        count = -2
    elif what == "narrow":
        W = 4
        table = np.ascontiguousarray(table[:, :W])
    elif what == "bad free id":
        free[-2], free[-3] = num_pages, -9
    elif what == "bad held id":
        table[0, 0], table[3, 2] = num_pages + 7, -1
    elif what == "few rows":
        rows = 50
    got = _check_tables(ctx, new, table, free, count, page, num_pages, rows)
    assert got["bad"]
    af.attn_check()  # reading the status cleared it


def test_tables_strided_table_and_no_positions():
    rng = np.random.default_rng(9)
    ctx, new = np.array([7, 100, 31]), np.array([1, 1, 1])
    table, free = _held(ctx, 16, 9, 40, rng)
    wide = torch.full((3, 20), 77, dtype=torch.int32, device="cuda")
    wide[:, 4:13] = _i32(table)
    cu, lens, slots = _i32([0] * 4), _i32([0] * 3), _i32([0] * 3)
    c = _i32([len(free)])
    af.attn_paged_tables(_i32(ctx), _i32(new), wide[:, 4:13], _i32(free), c, 16, 40, cu, lens, slots)
    af.attn_check()
    ref = tables(ctx, new, table, free, len(free), 16, 40, 3)
    assert np.array_equal(wide[:, 4:13].cpu().numpy(), ref["table"]) and np.array_equal(slots.cpu().numpy(), ref["slots"])
    assert torch.all(wide[:, :4] == 77) and torch.all(wide[:, 13:] == 77) and int(c) == ref["left"]


# ------------------------------------------------------------------------------ append
@pytest.mark.parametrize("rows,Hkv,d,page,dtype,new_layout,cache_layout", [
    (1, 1, 64, 16, "f16", "tokens", "heads"), (5, 8, 128, 16, "bf16", "tokens", "heads"), (333, 3, 64, 48, "bf16", "heads", "tokens"),
    (1000, 8, 128, 64, "f16", "tokens", "tokens"), (4097, 2, 128, 256, "f16", "heads", "heads"), (50, 20, 128, 32, "bf16", "tokens", "heads")])
def test_append(rows, Hkv, d, page, dtype, new_layout, cache_layout):
    g = torch.Generator().manual_seed(rows)
    dt = DTYPES[dtype]
    num_pages = pages(rows, page) + 3
    slots = torch.randperm(num_pages * page, generator=g)[:rows].int()
    slots[torch.rand(rows, generator=g) < 0.2] = -1
    if rows > 4:
        slots[-3:] = torch.tensor([-1, -2 ** 31, -7])
    new = torch.randn((Hkv + 2, rows, 2 * d), generator=g).to(dt)   # inside a larger buffer
    shape = (num_pages, Hkv, page, d)
    caches = [torch.randn(shape, generator=g).to(dt) for _ in range(2)]
    ref = [c.clone() for c in caches]
    live = slots >= 0
    s = slots[live].long()
    for c, x in zip(ref, (new[1:-1, :, :d], new[1:-1, :, d:])):
        c[s // page, :, s % page] = x.transpose(0, 1)[live]
    dev = new.cuda()
    if new_layout == "tokens":
        dev = dev.transpose(0, 1).contiguous().transpose(0, 1)
    got = [c.cuda() for c in caches]
    if cache_layout == "tokens":
        got = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in got]
    af.attn_paged_append(dev[1:-1, :, :d], dev[1:-1, :, d:], *got, slots.cuda())
    af.attn_check()
    for a, b in zip(got, ref):
        assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))


def test_append_slots_past_the_cache_are_left_out_and_reported():
    k = torch.randn((2, 4, 64), device="cuda").half()
    kc, vc = (torch.zeros((3, 2, 16, 64), dtype=torch.float16, device="cuda") for _ in range(2))
    af.attn_paged_append(k, k, kc, vc, _i32([48, 2 ** 31 - 1, 47, -1]))
    with pytest.raises(af.AttnError) as e:
        af.attn_check()
    assert e.value.status == -6
    want = torch.zeros_like(kc)
    want[2, :, 15] = k[:, 2]
    assert torch.equal(kc, want) and torch.equal(vc, want)


# ------------------------------------------------------------------------------ attention
CASES = [
    # lens_q, lens_k, Hq, Hkv, d, dtype, page, causal, wl, wr, kwargs
    # one token per request
    ([1], [1], 1, 1, 128, "bf16", 16, True, -1, -1, {}),
    ([1], [2000], 8, 1, 128, "bf16", 16, True, -1, -1, {}),
    ([1, 1, 1, 1, 1], [1, 63, 64, 65, 300], 8, 2, 128, "f16", 16, True, -1, -1, dict(rows="heads")),
    ([1, 1, 0, 1], [500, 129, 40, 17], 4, 4, 64, "f16", 32, True, -1, -1, dict(cache="tokens")),
    ([1, 1, 1], [700, 90, 1000], 6, 2, 64, "bf16", 48, True, -1, -1, {}),
    ([1, 1, 1], [700, 90, 1000], 16, 1, 128, "bf16", 80, True, 100, -1, {}),
    ([1] * 40, list(range(1, 400, 10)), 2, 2, 128, "f16", 64, False, -1, -1, {}),
    ([1, 1], [0, 70], 4, 2, 128, "bf16", 16, True, -1, -1, {}),                       # no key at all
    ([1, 1], [300, 257], 32, 1, 128, "bf16", 256, True, -1, -1, {}),                  # 32 heads of one K/V head
    ([1], [150], 128, 1, 64, "f16", 16, True, -1, -1, {}),                            # 128 of them
    ([1, 1], [600, 33], 4, 1, 64, "bf16", 16, True, 0, -1, {}),                       # a window of one key
    ([1], [3000], 1, 1, 64, "bf16", 16, True, -1, -1, {}),                            # one item over many runs
    # a few tokens per request
    ([3, 5, 2, 4], [200, 5, 66, 1000], 8, 2, 128, "bf16", 16, True, -1, -1, {}),
    ([4, 1, 6], [300, 64, 100], 8, 1, 64, "f16", 128, True, 50, -1, {}),
    ([2, 7], [128, 129], 4, 4, 128, "f16", 16, False, 40, 2, {}),
    ([4, 1, 3, 2], [500, 64, 100, 2], 8, 1, 128, "f16", 16, True, -1, -1, {}),        # up to 32 rows of a head
    ([4, 4, 0], [700, 63, 10], 8, 1, 64, "bf16", 48, True, 90, -1, dict(cache="tokens")),
    ([2, 9], [2, 300], 3, 1, 128, "bf16", 32, False, -1, 4, dict(rows="heads")),
    ([5, 2], [150, 400], 128, 1, 64, "f16", 16, True, -1, -1, {}),                    # more heads than a tile's half
    ([3], [77], 100, 1, 128, "bf16", 16, True, -1, -1, {}),
    ([16, 7, 1], [900, 300, 40], 8, 1, 128, "f16", 64, True, -1, -1, {}),             # one tile of rows, many key tiles
    ([20, 1], [64, 1000], 6, 1, 64, "bf16", 16, True, 200, -1, {}),
    # chunks
    ([100, 33], [100, 500], 4, 2, 128, "bf16", 16, True, -1, -1, {}),
    ([129], [129], 2, 1, 64, "f16", 16, True, -1, -1, {}),
    ([300, 1, 0, 257], [700, 400, 16, 257], 4, 2, 128, "f16", 64, True, -1, -1, dict(spare_rows=9)),
    ([260], [900], 3, 3, 64, "bf16", 32, False, -1, -1, dict(rows="heads", cache="tokens")),
    ([150, 200], [600, 200], 6, 2, 128, "bf16", 48, True, 120, -1, {}),
    ([90], [400], 4, 2, 64, "f16", 16, False, 30, 20, {}),
    ([200, 70], [90, 70], 8, 2, 128, "bf16", 16, True, -1, -1, {}),                   # fewer keys than queries
    ([200], [90], 4, 1, 64, "f16", 16, False, 20, 10, {}),
    ([40, 1, 60], [0, 0, 60], 4, 2, 128, "f16", 16, True, -1, -1, {}),
    ([513], [1300], 1, 1, 128, "bf16", 256, True, -1, -1, {}),
    ([70, 1], [300, 300], 7, 1, 128, "f16", 16, True, -1, -1, {}),                    # a group of 7
]


def _attend(bt, causal, wl, wr, scale, max_q=None, dev=None, **kw):
    q, k, v, o, lse = dev or bt.device()
    af.attn_fwd_paged(q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), max_q or bt.max_q, lse=lse, causal=causal,
                      window_left=wl, window_right=wr, scale=scale, **kw)
    return o, lse


@pytest.mark.parametrize("case", CASES, ids=lambda c: "q{}_k{}_{}x{}_d{}_{}_p{}_c{}_w{}_{}".format(
    "-".join(map(str, c[0][:4])), "-".join(map(str, c[1][:4])), *c[2:7], int(c[7]), c[8], c[9]))
def test_attention(case):
    lq, lk, Hq, Hkv, d, dtype, page, causal, wl, wr, kw = case
    bt = Batch(lq, lk, Hq, Hkv, d, dtype, page, seed=sum(lk) + d, **kw)
    scale = float(np.float32(d ** -0.5))
    o, lse = _attend(bt, causal, wl, wr, scale)
    af.attn_check()
    bt.check(o.cpu(), lse.cpu(), causal, wl, wr, scale, what=str(case))


@pytest.mark.parametrize("d,Hkv,lq,lk", [
    (64, 4, [1] * 8 + [90, 2, 4] + [1] * 8, [4200] * 8 + [300, 900, 77] + [4100, 1, 4000, 3000, 4500, 3900, 4400, 4300]),
    (128, 8, [1] * 24 + [200] + [1] * 16, [4600] * 24 + [900] + [4500] * 16)])
def test_many_decoding_requests_beside_a_chunk(d, Hkv, lq, lk):
    """Enough keys of few-row requests that they take a path of their own beside the chunk; checked on some requests."""
    g = torch.Generator(device="cuda").manual_seed(d)
    page, Hq, B = 16, 2 * Hkv, len(lq)
    need = [pages(n, page) for n in lk]
    num = sum(need)
    k, v = (torch.randn((num, Hkv, page, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn((Hq, sum(lq), d), generator=g, device="cuda", dtype=torch.bfloat16)
    perm = torch.randperm(num, generator=g, device="cuda").int().cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = np.concatenate([[0], np.cumsum(need)])
    for b in range(B):
        table[b, :need[b]] = perm[at[b]:at[b + 1]]
    cu = np.concatenate([[0], np.cumsum(lq)])
    o, lse = torch.full_like(q, float("nan")), torch.full((Hq, q.shape[1]), float("nan"), device="cuda")
    af.attn_fwd_paged(q, k, v, o, table.cuda(), _i32(cu), _i32(lk), max(lq), lse=lse, causal=True, scale=0.1)
    af.attn_check()
    assert torch.all(torch.isfinite(o.float())) and torch.all(torch.isfinite(lse))
    for b in (0, 7, 8, 9, 10, 12, B - 8, B - 1) if d == 64 else (0, 23, 24, B - 1):
        rows, ids = slice(cu[b], cu[b + 1]), table[b, :need[b]].long()
        own = torch.arange(need[b], dtype=torch.int32)[None]
        kb, vb, qb = (x.cpu() for x in (k[ids.cuda()], v[ids.cuda()], q[:, rows]))
        ro, rl, A, S = attention(qb, kb, vb, own, [0, lq[b]], [lk[b]], lq[b], True, -1, -1, float(np.float32(0.1)))
        to, tl = tolerances(torch.bfloat16, d, lk[b], ro, rl, A, S)
        assert torch.all((o[:, rows].cpu().double() - ro).abs() <= to), f"request {b}"
        assert torch.all((lse[:, rows].cpu().double() - rl).abs() <= tl), f"request {b}"


def test_one_long_request_among_many_short_ones():
    """A unit longer than an SM's share: everything is cut into runs."""
    lq = [40] + [21] * 30
    lk = [9000] + [30 + 3 * i for i in range(30)]
    for d, Hq, Hkv in ((128, 2, 1), (64, 8, 2)):
        bt = Batch(lq, lk, Hq, Hkv, d, "bf16", 32, seed=33)
        o, lse = _attend(bt, True, -1, -1, 0.1)
        af.attn_check()
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1)


@pytest.mark.parametrize("wl", [-1, 50])
@pytest.mark.parametrize("B,new,Hkv,d", [(1, [7], 2, 128), (33, [3, 0, 5, 7], 1, 64), (70, [3, 0, 5, 7], 2, 128), (512, [0, 5, 3], 1, 128),
                                         (513, [3, 0, 5, 7], 1, 64), (60, [5, 1, 1, 1], 2, 64), (61, [1, 6, 1, 1, 0], 1, 128)])
def test_a_few_tokens_of_many_requests(B, new, Hkv, d, wl):
    """Requests of one tile of rows at most, with a plan and without (up to 512 of more than 16 rows on the average)."""
    lq = [new[b % len(new)] for b in range(B)]
    lk = [(977 * b) % (3000 if B < 40 else 400 if B < 100 else 150) + lq[b] * (b % 5 != 0) for b in range(B)]
    bt = Batch(lq, lk, 8 * Hkv, Hkv, d, "bf16", 16, seed=B + d)
    o, lse = _attend(bt, True, wl, -1, 0.1)
    af.attn_check()
    bt.check(o.cpu(), lse.cpu(), True, wl, -1, 0.1)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,d,dtype,page", [
    ([30, 1, 887, 5, 276, 29, 13, 308, 21, 558, 51, 110, 23, 512, 7, 855, 10, 18, 229, 2, 10, 7, 1],
     [49, 2503, 1, 626, 20, 1, 64, 4, 513, 4, 3773, 11, 5, 73, 184, 1006, 8, 13, 1472, 37, 475, 22, 2], 9, 3, 64, "f16", 16),
    ([129, 248, 9, 164, 1, 4, 5, 111, 240, 3], [481, 14, 1, 58, 617, 619, 28, 965, 27, 11], 96, 3, 64, "bf16", 256),
    ([2, 283], [6378, 2072], 128, 8, 64, "bf16", 256),
    ([40, 130, 40, 130] * 6, [700, 900, 650, 130] * 6, 4, 2, 128, "bf16", 32)])
def test_units_of_one_tile_before_units_of_two(lq, lk, Hq, Hkv, d, dtype, page):
    """A Q tile that has no key tiles for a whole unit does not take the other one's scores for its own in the
    next: the softmax of the idle tile is ahead of the products by the whole ring of descriptors."""
    bt = Batch(lq, lk, Hq, Hkv, d, dtype, page, seed=sum(lq))
    q, k, v, o, lse = bt.device()
    args = (k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.max_q)
    first = None
    for _ in range(30):
        o.fill_(float("nan"))
        af.attn_fwd_paged(q, *args, lse=lse, causal=True, scale=0.125)
        af.attn_check()
        if first is None:
            first = o.clone(), lse.clone()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    if Hq <= 32:
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.125)
    assert torch.all(torch.isfinite(o[:, :sum(lq)].float()))


@pytest.mark.parametrize("lq,lk,d,page,wl", [([1, 1, 1], [65, 17, 300], 128, 16, -1), ([1, 1], [333, 90], 64, 64, 40),
                                             ([70, 3], [200, 39], 128, 32, -1), ([150, 90], [400, 90], 64, 48, 33),
                                             ([200], [517], 128, 256, 64)])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_what_no_query_sees_may_hold_anything(lq, lk, d, page, wl, fill):
    """NaN and infinities in rows behind the last key and ahead of the window, and pages that the table
    no longer lists there, do not reach the result."""
    bt = Batch(lq, lk, 4, 2, d, "bf16", page, seed=3, fill=fill)
    if wl >= 0:
        for b, (n, sk) in enumerate(zip(lq, lk)):
            first = max(0, sk - n - wl)           # the first key that any row of the request sees
            for key in range(first):
                for c in (bt.k, bt.v):
                    c[int(bt.table[b, key // page]), :, key % page] = fill
        gone = bt.table.clone()
        for b, (n, sk) in enumerate(zip(lq, lk)):
            gone[b, :max(0, sk - n - wl) // page] = -1
        dev = bt.device()
        keep, bt.table = bt.table, gone
        o, lse = _attend(bt, True, wl, -1, 0.1, dev=dev)
        bt.table = keep
    else:
        o, lse = _attend(bt, True, wl, -1, 0.1)
    af.attn_check()
    bt.check(o.cpu(), lse.cpu(), True, wl, -1, 0.1)


def test_scores_of_every_size():
    """Scores of hundreds, rising along the keys, so the running maximum moves at every tile."""
    for lq in ([1, 1, 2], [140, 1, 20]):
        bt = Batch(lq, [300, 600, 100], 4, 2, 128, "f16", 16, seed=8)
        bt.q[..., 0] = 24.0
        for b in range(3):
            for key in range(bt.lens_k[b]):
                bt.k[int(bt.table[b, key // 16]), :, key % 16, 0] = 0.5 * key - 60
        o, lse = _attend(bt, True, -1, -1, 0.0625)
        af.attn_check()
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.0625, what=str(lq))


def test_requests_longer_than_max_seqlen_q_are_cut():
    bt = Batch([3, 40, 1], [50, 200, 30], 4, 2, 64, "bf16", 16, seed=4)
    o, lse = _attend(bt, True, -1, -1, 0.125, max_q=25)
    af.attn_check()
    bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.125, max_q=25)


@pytest.mark.parametrize("lq", [[1, 1, 1], [200, 1, 60]])
def test_bad_page_ids_are_reported_and_stay_in_their_request(lq):
    bt = Batch(lq, [400, 100, 300], 4, 2, 128, "bf16", 16, seed=6)
    dev = bt.device()
    good = bt.table
    bt.table = good.clone()
    bt.table[0, 3], bt.table[0, 5], bt.table[2, 0], bt.table[2, 1] = -1, bt.num_pages, 2 ** 31 - 1, -2 ** 31
    o, lse = _attend(bt, True, -1, -1, 0.1, dev=dev)
    with pytest.raises(af.AttnError) as e:
        af.attn_check()
    assert e.value.status == -6
    bt.table = good
    assert torch.all(torch.isfinite(o[:, int(bt.cu[0]):].float()))
    bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1, skip=(0, 2))
    af.attn_check()


def test_lengths_past_the_table_are_cut():
    bt = Batch([1, 30], [64, 100], 4, 2, 64, "f16", 16, seed=7, spare_width=0)
    bt.lens = torch.tensor([2 ** 31 - 1, 100], dtype=torch.int32)
    bt.table = bt.table[:, :7].contiguous()
    bt.table[0, 4:] = bt.table[1, :3]
    o, lse = _attend(bt, True, -1, -1, 0.1)
    af.attn_check()
    bt.lens = torch.tensor([112, 100], dtype=torch.int32)
    bt.lens_k = [112, 100]
    bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, the pages used at its end."""
    page, Hkv, d = 256, 8, 128
    num = (1 << 32) // (page * Hkv * d) + 200
    bt = Batch([1, 90], [700, 300], 16, Hkv, d, "bf16", page, seed=12)
    q, _, _, o, lse = bt.device()
    big = [torch.empty((num, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    first = num - bt.num_pages
    for x, c in zip(big, (bt.k, bt.v)):
        x[first:] = c.cuda()
    table = torch.where(bt.table >= 0, bt.table + first, -1).cuda()
    af.attn_fwd_paged(q, *big, o, table, bt.cu.cuda(), bt.lens.cuda(), bt.max_q, lse=lse, causal=True, scale=0.1)
    af.attn_check()
    bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1)
    # and the append at its last slot
    new = torch.randn((Hkv, 1, d), device="cuda").bfloat16()
    af.attn_paged_append(new, -new, *big, _i32([num * page - 1]))
    af.attn_check()
    assert torch.equal(big[0][-1, :, -1], new[:, 0]) and torch.equal(big[1][-1, :, -1], -new[:, 0])


@pytest.mark.parametrize("lq", [[1] * 9, [5, 1, 200, 1, 1, 33, 1, 1, 1]])
def test_repeated_calls_are_bit_identical(lq):
    bt = Batch(lq, [900, 30, 700, 1, 64, 800, 333, 128, 2000], 8, 2, 128, "bf16", 16, seed=14)
    first = None
    for _ in range(4):
        o, lse = _attend(bt, True, -1, -1, 0.1)
        af.attn_check()
        got = (o.cpu()[:, :int(bt.cu[-1])], lse.cpu()[:, :int(bt.cu[-1])])
        if first is None:
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_other_streams_and_own_workspace():
    bt = Batch([1, 70, 1], [500, 300, 90], 8, 2, 128, "f16", 16, seed=15)
    ws = torch.full((af.attn_paged_workspace(3, 8, 2, 128, 71 + 1, bt.max_q) + 64,), 255, dtype=torch.uint8, device="cuda")
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    dev = bt.device()
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        o, lse = torch.full_like(dev[3], float("nan")), torch.full_like(dev[4], float("nan"))
        tables_dev = bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda()
        torch.cuda.synchronize()
        af.attn_fwd_paged(*dev[:3], o, *tables_dev, bt.max_q, lse=lse, causal=True, scale=0.1, stream=s,
                          workspace=ws if i == 1 else None)
        outs.append((o, lse))
    for s in streams:
        af.attn_check(s)
    for o, lse in outs:
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1)


# ------------------------------------------------------------------------------ together
class Server:
    """A small serving loop: requests grow by their own steps; the history is kept to check against."""

    def __init__(self, B, Hq, Hkv, d, dtype, page, W, num_pages, max_rows, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.d, self.page, self.num_pages, self.max_rows = B, Hq, Hkv, d, page, num_pages, max_rows
        self.dt = DTYPES[dtype]
        self.hist = [[torch.zeros((Hkv, 0, d)).to(self.dt) for _ in range(2)] for _ in range(B)]
        dev = "cuda"
        self.ctx, self.new = _i32([0] * B), _i32([0] * B)
        self.table = torch.full((B, W), -1, dtype=torch.int32, device=dev)
        self.free = torch.randperm(num_pages, generator=self.g).int().cuda()
        self.count = _i32([num_pages])
        self.cu, self.lens = _i32([0] * (B + 1)), _i32([0] * B)
        self.slots, self.pos = _i32([0] * max_rows), _i32([0] * max_rows)
        self.k, self.v = (torch.full((num_pages, Hkv, page, d), float("nan"), dtype=self.dt, device=dev) for _ in range(2))
        self.qkv = torch.zeros((max_rows, Hq + 2 * Hkv, d), dtype=self.dt, device=dev)
        self.o = torch.zeros((max_rows, Hq, d), dtype=self.dt, device=dev)
        self.lse = torch.zeros((Hq, max_rows), device=dev)

    def enqueue(self, max_q):
        af.attn_paged_tables(self.ctx, self.new, self.table, self.free, self.count, self.page, self.num_pages, self.cu, self.lens,
                             self.slots, self.pos)
        heads = self.qkv.transpose(0, 1)
        af.attn_paged_append(heads[self.Hq:self.Hq + self.Hkv], heads[self.Hq + self.Hkv:], self.k, self.v, self.slots)
        af.attn_fwd_paged(heads[:self.Hq], self.k, self.v, self.o.transpose(0, 1), self.table, self.cu, self.lens, max_q, lse=self.lse,
                          causal=True)
        self.ctx.copy_(self.lens)

    def feed(self, new):
        """Host side of a step: this step's rows."""
        n = sum(new)
        self.rows = torch.randn((self.max_rows, self.Hq + 2 * self.Hkv, self.d), generator=self.g).to(self.dt)
        self.qkv.copy_(self.rows)
        self.new.copy_(_i32(new))
        self.o.fill_(float("nan"))
        self.lse.fill_(float("nan"))
        at = 0
        for b, m in enumerate(new):
            x = self.rows[at:at + m].transpose(0, 1)
            self.hist[b] = [torch.cat([self.hist[b][0], x[self.Hq:self.Hq + self.Hkv]], 1), torch.cat([self.hist[b][1], x[self.Hq + self.Hkv:]], 1)]
            at += m
        assert at == n

    def verify(self, new):
        at, o, lse = 0, self.o.transpose(0, 1).cpu(), self.lse.cpu()
        for b, m in enumerate(new):
            if m == 0:
                continue
            k, v = self.hist[b]
            sk = k.shape[1]
            q = self.rows[at:at + m, :self.Hq].transpose(0, 1)
            # the request's history as one page
            ro, rl, A, S = attention(q, k[None], v[None], torch.zeros((1, 1), dtype=torch.int32), [0, m], [sk], m, True, -1, -1, float(np.float32(self.d ** -0.5)))
            to, tl = tolerances(self.dt, self.d, sk, ro, rl, A, S)
            assert torch.all((o[:, at:at + m].double() - ro).abs() <= to), f"request {b}"
            assert torch.all((lse[:, at:at + m].double() - rl).abs() <= tl), f"request {b}"
            at += m
        assert torch.all(torch.isnan(o[:, at:])) and torch.all(torch.isnan(lse[:, at:]))


def test_a_serving_loop():
    """Prompts admitted in chunks beside decoding requests, idle ones, pages taken as lengths grow."""
    steps = [[40, 0, 7, 0], [1, 100, 1, 0], [1, 55, 1, 16], [1, 1, 1, 1], [0, 1, 3, 1], [1, 1, 0, 33], [1, 1, 1, 1]]
    sv = Server(4, 8, 2, 128, "bf16", 16, W=20, num_pages=64, max_rows=170, seed=31)
    for new in steps:
        sv.feed(new)
        sv.enqueue(max(new))
        af.attn_check()
        sv.verify(new)
    assert int(sv.count) == 64 - sum(pages(h[0].shape[1], 16) for h in sv.hist)


def test_a_captured_step_replayed():
    """One captured decoding step (tables, append, attention) replayed while the lengths grow, beside an eager
    loop's calls and beside another captured loop's replays on another stream."""
    a = Server(3, 4, 2, 64, "f16", 16, W=12, num_pages=40, max_rows=8, seed=41)
    b = Server(5, 6, 2, 128, "bf16", 32, W=8, num_pages=40, max_rows=6, seed=42)
    for sv, new in ((a, [3, 1, 2]), (b, [1, 1, 1, 1, 2])):
        sv.feed(new)
        sv.enqueue(8)       # warm up, and a first step
        af.attn_check()
        sv.verify(new)
    graphs = []
    for sv in (a, b):
        sv.new.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.enqueue(8)
        graphs.append(g)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for step in range(12):
        na, nb = [1, step % 2, 4 if step == 3 else 1], [1, 1, 0, 1, 1 + step % 2]
        a.feed(na)
        b.feed(nb)
        torch.cuda.synchronize()
        with torch.cuda.stream(sa):
            graphs[0].replay()
        with torch.cuda.stream(sb):
            graphs[1].replay()
        torch.cuda.synchronize()
        a.verify(na)
        b.verify(nb)
    af.attn_check()


def test_a_wait_that_runs_out_is_reported():
    """The chunk path's waits are bounded, as attn_fwd's are: a Q tile that never comes ends the launch with a status."""
    lib = af.library()
    bt = Batch([70, 1], [90, 50], 4, 2, 128, "bf16", 16, seed=16)
    assert lib.attn_set_wait_timeout_ns(50_000_000) == 0
    try:
        assert lib.attn_debug_inject(1) == 0
        _attend(bt, True, -1, -1, 0.1)
        with pytest.raises(af.AttnError) as e:
            af.attn_check()
        assert e.value.status == -4
    finally:
        lib.attn_debug_inject(0)
        lib.attn_set_wait_timeout_ns(0)
    o, lse = _attend(bt, True, -1, -1, 0.1)
    af.attn_check()
    bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1)


@pytest.mark.parametrize("lq", [[1, 1, 2], [3, 1, 8], [150, 1, 40]])
def test_nan_in_a_query_row_stays_in_it(lq):
    """A NaN that a row does see comes out as NaN, in O and LSE, and in no other row."""
    bt = Batch(lq, [900, 70, 300], 4, 2, 128, "bf16", 16, seed=21)
    clean, _ = _attend(bt, True, -1, -1, 0.1)
    bt.q[1, 0, 5] = float("nan")
    o, lse = _attend(bt, True, -1, -1, 0.1)
    af.attn_check()
    assert torch.all(torch.isnan(o[1, 0])) and torch.isnan(lse[1, 0])
    o[1, 0] = clean[1, 0]
    assert torch.equal(o[:, :int(bt.cu[-1])], clean[:, :int(bt.cu[-1])])


def test_the_streams_workspace_and_maps_are_reused():
    """Without a workspace of the caller's, repeated calls allocate nothing and encode nothing after the first of a
    shape; a released workspace comes back; a captured call gets none of it."""
    s = torch.cuda.Stream()
    small, big = Batch([1, 1], [300, 90], 8, 2, 128, "f16", 16, seed=22), Batch([1, 200], [300, 900], 8, 2, 128, "f16", 16, seed=23)
    af.attn_release_workspace(s)
    with torch.cuda.stream(s):
        devs = [b.device() for b in (small, big)]
        tabs = [(b.table.cuda(), b.cu.cuda(), b.lens.cuda()) for b in (small, big)]
        seen = []
        for which in (0, 0, 1, 1, 0, 1):
            b, d, t = (small, big)[which], devs[which], tabs[which]
            af.attn_fwd_paged(*d[:4], *t, b.max_q, lse=d[4], causal=True, scale=0.1)
            seen.append(af.debug_counters())
        af.attn_check(s)
        assert [c["workspace_allocs"] - seen[0]["workspace_allocs"] for c in seen] == [0, 0, 1, 1, 1, 1]
        assert seen[3]["map_encodes"] == seen[2]["map_encodes"] == seen[-1]["map_encodes"]
        af.attn_release_workspace(s)
        af.attn_fwd_paged(*devs[1][:4], *tabs[1], big.max_q, lse=devs[1][4], causal=True, scale=0.1)
        af.attn_check(s)
    for b, d in zip((small, big), devs):
        b.check(d[3].cpu(), d[4].cpu(), True, -1, -1, 0.1)
    af.attn_release_workspace(s)
    g = torch.cuda.CUDAGraph()
    n = af.debug_counters()["workspace_allocs"]
    with torch.cuda.graph(g, stream=s):
        af.attn_fwd_paged(*devs[0][:4], *tabs[0], small.max_q, lse=devs[0][4], causal=True, scale=0.1)
    assert af.debug_counters()["workspace_allocs"] == n
    g.replay()
    torch.cuda.synchronize()
    small.check(devs[0][3].cpu(), devs[0][4].cpu(), True, -1, -1, 0.1)


def test_a_workspace_that_is_too_small_is_refused():
    bt = Batch([1, 60], [300, 90], 8, 2, 128, "f16", 16, seed=24)
    n = af.attn_paged_workspace(2, 8, 2, 128, 61, 60)
    with pytest.raises(af.AttnError) as e:
        _attend(bt, True, -1, -1, 0.1, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -1
    with pytest.raises(ValueError):
        _attend(bt, True, -1, -1, 0.1, workspace=torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError):
        _attend(bt, True, -1, -1, 0.1, workspace=torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])


def test_threads_on_one_stream_and_on_their_own():
    """Host threads that call at the same time, sharing a stream (and its workspace) or not."""
    import threading
    bts = [Batch([1, 1, 1], [900, 30, 400], 8, 2, 128, "bf16", 16, seed=25), Batch([130, 1], [400, 600], 8, 2, 128, "bf16", 16, seed=26),
           Batch([2, 4], [64, 1000], 8, 2, 64, "f16", 32, seed=27), Batch([9, 3], [300, 500], 8, 2, 64, "bf16", 16, seed=28)]
    devs = [b.device() for b in bts]
    tabs = [(b.table.cuda(), b.cu.cuda(), b.lens.cuda()) for b in bts]
    torch.cuda.synchronize()
    for streams in ([torch.cuda.Stream()] * 4, [torch.cuda.Stream() for _ in range(4)]):
        def work(i):
            for _ in range(20):
                af.attn_fwd_paged(*devs[i][:4], *tabs[i], bts[i].max_q, lse=devs[i][4], causal=True, scale=0.1, stream=streams[i])
        threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        for s in streams:
            af.attn_check(s)
        for b, d in zip(bts, devs):
            b.check(d[3].cpu(), d[4].cpu(), True, -1, -1, 0.1)
            d[3].fill_(float("nan"))
            d[4].fill_(float("nan"))
        torch.cuda.synchronize()


def test_a_process_whose_first_calls_are_captured():
    """Nothing that the library sets up on its first call stands in the way of a capture."""
    code = (
        "import torch, attention_forward_07_gb300 as af\n"
        "i = lambda *s: torch.zeros(s, dtype=torch.int32, device='cuda')\n"
        "q, kc = (torch.randn(s, device='cuda', dtype=torch.bfloat16) for s in ((8, 40, 64), (9, 2, 16, 64)))\n"
        "vc, o, new = kc.flip(0).contiguous(), torch.empty_like(q), torch.randn((2, 40, 64), device='cuda', dtype=torch.bfloat16)\n"
        "ctx, n, table, free, cnt = i(2), torch.tensor([1, 39], dtype=torch.int32, device='cuda'), i(2, 4), torch.arange(9, dtype=torch.int32, device='cuda'), i(1) + 9\n"
        "left, cu, lens, slots = i(1), i(3), i(2), i(40)\n"
        "ws = torch.empty(af.attn_paged_workspace(2, 8, 2, 64, 40, 39), dtype=torch.uint8, device='cuda')\n"
        "def step():\n"
        "    af.attn_paged_tables(ctx, n, table, free, cnt, 16, 9, cu, lens, slots, free_count_out=left)\n"
        "    af.attn_paged_append(new, new, kc, vc, slots)\n"
        "    af.attn_fwd_paged(q, kc, vc, o, table, cu, lens, 39, causal=True, scale=0.125, workspace=ws)\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    step()\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "first = o.clone()\n"
        "step()\n"
        "torch.cuda.synchronize()\n"
        "assert torch.equal(first, o) and left.item() == 5 and first.float().abs().sum() > 0\n"
        "print('captured')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]


@pytest.mark.parametrize("d", [64, 128])
def test_calls_on_three_streams_at_once(d):
    """Kernels that share the machine lose time anywhere; what each waits for is still told apart."""
    shapes = [([693, 210, 40], [1311, 700, 900], 8, 1), ([1] * 30, [1000 + 90 * b for b in range(30)], 32, 8), ([6, 3, 5, 2], [3000, 200, 900, 1], 8, 1),
              ([300, 1, 1, 1, 120], [900, 3000, 10, 700, 120], 8, 2), ([90] * 9, [700] * 9, 4, 4)]
    calls = []
    for lq, lk, Hq, Hkv in shapes:
        bt = Batch(lq, lk, Hq, Hkv, d, "bf16", 64, seed=sum(lk))
        q, k, v, o, lse = bt.device()
        args = (q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.max_q)
        af.attn_fwd_paged(*args, lse=lse, causal=True, scale=0.125)
        af.attn_check()
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.125)
        calls.append((args, o, lse, o.clone(), lse.clone()))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for rep in range(60):
        for _, o, lse, _, _ in calls:
            o.fill_(float("nan"))
            lse.zero_()
        torch.cuda.synchronize()
        for i in range(len(calls)):
            args, _, lse, _, _ = calls[(i + rep) % len(calls)]
            with torch.cuda.stream(streams[(i * 7 + rep) % 3]):
                af.attn_fwd_paged(*args, lse=lse, causal=True, scale=0.125)
        for st in streams:
            af.attn_check(st)
        for args, o, lse, o0, lse0 in calls:
            rows = int(args[5][-1])
            assert torch.equal(o[:, :rows], o0[:, :rows]) and torch.equal(lse[:, :rows], lse0[:, :rows])
    for st in streams:
        af.attn_release_workspace(st)
