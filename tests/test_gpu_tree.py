"""The operators of drafted trees on the GPU against their plain forms (tree_ref.py): masks and positions, norms and rotation,
attention under masks, acceptance, moves, and all of them together as a serving loop runs them."""
import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

import tree_ref
from paged_ref import DTYPES, Batch, pages, tolerances

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _reported():
    try:
        af.attn_check()
    except af.AttnError as e:
        assert e.status == -6
        return True
    return False


# ------------------------------------------------------------------------------ masks and positions
@pytest.mark.parametrize("sizes,ctx,words,window,kw", [
    ([1], [0], 1, -1, {}), ([26], [500], 1, -1, {}), ([32, 1, 0, 33, 31], [5, 0, 9, 100, 7], 1, -1, {}), ([64, 65, 40], [10, 0, 3], 2, 3, {}),
    ([256, 255, 257, 1000], [1, 2, 3, 4], 8, -1, dict(spread=300)), ([1024, 1000], [70000, 0], 32, 5, dict(spread=2)), ([200], [9], 8, -1, dict(chain=True)),
    ([7] * 300, list(range(300)), 1, 0, {})])
def test_tree(sizes, ctx, words, window, kw):
    rng = np.random.default_rng(sum(sizes))
    parents = np.concatenate([tree_ref.random_parents(n, rng, **kw) for n in sizes] + [[-1, -1, 5]])
    cu, lens = np.concatenate([[0], np.cumsum(sizes)]), np.array(ctx) + sizes
    rows = len(parents)
    pos, wide = _i32(np.full(rows, -7)), torch.full((rows, words + 2), -7, dtype=torch.int32, device="cuda")
    af.attn_paged_tree(_i32(parents), _i32(cu), _i32(lens), pos, wide[:, 1:-1], window_left=window)
    assert not _reported()
    pos_ref, mask_ref, _ = tree_ref.tree(parents[:cu[-1]], cu, lens, words, window)
    assert np.array_equal(pos.cpu().numpy()[:cu[-1]], pos_ref)
    written = mask_ref[:, 0] >= 0
    got = wide[:cu[-1], 1:-1].cpu()
    assert np.array_equal(tree_ref.from_words(got)[written], mask_ref[written])
    assert (got[~torch.from_numpy(written)] == -7).all() and (wide[:, 0] == -7).all() and (wide[:, -1] == -7).all()
    assert (wide[cu[-1]:] == -7).all() and (pos[cu[-1]:] == -7).all()


def test_tree_parents_out_of_range_count_as_none_and_are_reported():
    parents, cu, lens = np.array([0, 0, 9, 1, -5, 2 ** 31 - 1]), [0, 6], [6]
    pos, mask = _i32([-7] * 6), _i32([[-7]] * 6)
    af.attn_paged_tree(_i32(parents), _i32(cu), _i32(lens), pos, mask)
    assert _reported() and not _reported()
    pos_ref, mask_ref, bad = tree_ref.tree(parents, cu, lens, 1)
    assert bad and np.array_equal(pos.cpu().numpy(), pos_ref) and np.array_equal(tree_ref.from_words(mask), mask_ref)


# ------------------------------------------------------------------------------ norms and rotation
ROPE = [
    # rows, Hq, Hkv, d, dtype, rot, axes, interleaved, norm, layout
    (1, 1, 1, 64, "f16", 64, 1, False, None, "heads"), (5, 32, 8, 128, "bf16", 128, 1, False, "type", "tokens"), (305, 6, 2, 128, "bf16", 64, 3, False, "f32", "tokens"),
    (306, 16, 16, 64, "f16", 32, 2, True, "type", "heads"), (1003, 3, 1, 64, "bf16", 16, 4, False, None, "heads"), (700, 5, 3, 128, "f16", 128, 3, True, "f32", "tokens"),
    (64, 8, 8, 64, "bf16", 0, 1, False, "type", "tokens"), (3, 40, 9, 128, "f16", 96, 1, False, "q only", "heads"), (311, 4, 2, 128, "bf16", 112, 2, False, "k only", "tokens")]


def _rope_inputs(rows, Hq, Hkv, d, dtype, rot, axes, norm, layout, seed):
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    x = torch.randn((Hq + 2 * Hkv + 1, rows, d), generator=g) * torch.exp(2 * torch.randn((Hq + 2 * Hkv + 1, rows, 1), generator=g))
    x = x.to(dt)
    w = [None, None]
    if norm:
        w = [1 + 0.3 * torch.randn(d, generator=g) for _ in range(2)]
        w = [v if norm == "f32" else v.to(dt) for v in w]
        if norm in ("q only", "k only"):
            w[norm == "q only"] = None
    pos = torch.randint(-50, 10 ** 6, (axes, rows), generator=g).int()
    pos[:, 0] = 0
    inv = None
    if rot:
        inv = (10000.0 ** (-torch.arange(rot // 2) / (rot / 2.0)))[None] * (torch.arange(rot // 2)[None] % axes == torch.arange(axes)[:, None])
    dev = x.cuda()
    if layout == "tokens":
        dev = dev.transpose(0, 1).contiguous().transpose(0, 1)
    return x, dev, w, pos, inv


def _dev(x):
    return None if x is None else x.cuda()


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_rope(case, in_place):
    rows, Hq, Hkv, d, dtype, rot, axes, interleaved, norm, layout = case
    x, dev, w, pos, inv = _rope_inputs(rows, Hq, Hkv, d, dtype, rot, axes, norm, layout, rows)
    q, k = dev[:Hq], dev[Hq:Hq + Hkv]
    qo, ko = (q, k) if in_place else (torch.full((Hq, rows, d), 7.0, dtype=q.dtype, device="cuda"), torch.full((rows, Hkv, d), 7.0, dtype=q.dtype, device="cuda").transpose(0, 1))
    p, f = _dev(pos), _dev(inv)
    if axes == 1 and rows % 2:
        p, f = p[0], None if f is None else f[0]
    af.attn_rope(q, k, qo, ko, p, f, _dev(w[0]), _dev(w[1]), eps=1e-5, interleaved=interleaved)
    af.attn_check()
    for got, src, weight in ((qo, x[:Hq], w[0]), (ko, x[Hq:Hq + Hkv], w[1])):
        want, tol = tree_ref.rope(src, weight, pos, inv, 1e-5, interleaved, x.dtype)
        err = (got.cpu().double() - want).abs() - tol
        assert err.max() <= 0, f"off by {err.max()} over the bound, {int((err > 0).sum())} of {err.numel()}"
    assert torch.equal(dev[Hq + Hkv:].cpu().view(torch.int16), x[Hq + Hkv:].view(torch.int16))


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("cache", ["heads", "tokens"])
def test_paged_rope(case, cache):
    rows, Hq, Hkv, d, dtype, rot, axes, interleaved, norm, layout = case
    x, dev, w, pos, inv = _rope_inputs(rows, Hq, Hkv, d, dtype, rot, axes, norm, layout, rows + 1)
    page = 48
    num_pages = pages(rows, page) + 2
    g = torch.Generator().manual_seed(rows)
    slots = torch.randperm(num_pages * page, generator=g)[:rows].int()
    if rows > 2:
        slots[torch.rand(rows, generator=g) < 0.2] = -1
        slots[1], slots[-1] = num_pages * page, -2 ** 31
    caches = [torch.randn((num_pages, Hkv, page, d), generator=g).to(x.dtype) for _ in range(2)]
    got = [c.cuda() for c in caches]
    if cache == "tokens":
        got = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in got]
    qo = torch.full((rows, Hq, d), 7.0, dtype=x.dtype, device="cuda").transpose(0, 1)
    af.attn_paged_rope(dev[:Hq], dev[Hq:Hq + Hkv], dev[Hq + Hkv:-1], qo, *got, slots.cuda(), _dev(pos), _dev(inv), _dev(w[0]), _dev(w[1]), interleaved=interleaved)
    assert _reported() == (rows > 2)
    live = (slots >= 0) & (slots < num_pages * page)
    s = slots[live].long()
    want, tol = tree_ref.rope(x[:Hq], w[0], pos, inv, 1e-6, interleaved, x.dtype)
    want[:, ~live], tol[:, ~live] = 7.0, 0.0
    assert ((qo.cpu().double() - want).abs() <= tol).all()
    k, tol_k = tree_ref.rope(x[Hq:Hq + Hkv], w[1], pos, inv, 1e-6, interleaved, x.dtype)
    want, tol = caches[0].double(), torch.zeros(caches[0].shape, dtype=torch.float64)
    want[s // page, :, s % page], tol[s // page, :, s % page] = k[:, live].transpose(0, 1), tol_k[:, live].transpose(0, 1)
    assert ((got[0].cpu().double() - want).abs() <= tol).all()
    caches[1][s // page, :, s % page] = x[Hq + Hkv:-1][:, live].transpose(0, 1)
    assert torch.equal(got[1].cpu().view(torch.int16), caches[1].view(torch.int16))


def test_rope_far_positions_and_rows_of_one_value():
    """Positions up to 2^31 - 1 keep the documented 2^-21 of a turn (and the function's 2^-22); rows of zeros stay zeros."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1, 0], dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(32) / 32.0)
    x = torch.zeros((1, 5, 64))
    x[..., :32] = 1.0
    x = x.half()
    out, kz = torch.empty((1, 5, 64), dtype=torch.float16, device="cuda"), torch.zeros((1, 5, 64), dtype=torch.float16, device="cuda")
    ko = torch.full_like(kz, 3.0)
    af.attn_rope(x.cuda(), kz, out, ko, pos.cuda(), inv.cuda(), None, torch.ones(64, dtype=torch.float16, device="cuda"))
    af.attn_check()
    phi = pos.double()[:, None] * inv.double()[None]
    want = torch.cat([phi.cos(), phi.sin()], -1)
    tol = want.abs() * 2.0 ** -11 + 2 * np.pi * 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -25
    assert ((out[0].cpu().double() - want).abs() <= tol).all()
    assert torch.all(ko == 0)


# ------------------------------------------------------------------------------ attention
ATTEND = [
    # nodes, keys, Hq, Hkv, d, dtype, page, words, window, Batch's keywords
    # few rows
    ([1], [1], 1, 1, 128, "bf16", 16, 1, -1, {}), ([2], [700], 8, 1, 128, "bf16", 16, 1, -1, {}), ([5, 1, 3, 0, 4], [5, 64, 200, 9, 1003], 4, 2, 64, "f16", 48, 2, -1, {}),
    ([4, 4, 2], [66, 130, 3], 8, 2, 128, "f16", 16, 1, 40, dict(rows="heads")), ([16, 9], [300, 9], 1, 1, 64, "bf16", 32, 1, -1, {}),
    ([8, 3, 8], [129, 600, 8], 4, 1, 128, "bf16", 64, 1, -1, dict(cache="tokens")), ([31, 32], [900, 33], 1, 1, 128, "f16", 16, 1, 70, {}),
    ([6, 2], [5, 400], 3, 1, 64, "bf16", 16, 1, -1, {}),                                   # fewer keys than nodes
    # one tile of rows: key tiles by turns
    ([26], [500], 4, 1, 128, "bf16", 16, 1, -1, {}), ([12, 16, 5], [140, 127, 260], 8, 1, 64, "f16", 16, 1, -1, dict(spare_rows=3)),
    ([30, 17, 32, 1], [30, 144, 1029, 500], 4, 1, 128, "f16", 128, 1, 100, {}), ([20, 20], [15, 400], 6, 1, 64, "bf16", 16, 1, -1, dict(cache="tokens")),
    ([1, 1], [300, 2], 100, 1, 128, "bf16", 16, 1, -1, {}), ([18] * 9, [60 * i + 18 for i in range(9)], 7, 1, 128, "bf16", 16, 1, -1, {}),
    # more
    ([64, 33, 50], [200, 161, 1000], 8, 2, 128, "bf16", 64, 2, -1, {}), ([64, 60], [64, 700], 16, 2, 64, "f16", 16, 3, -1, dict(rows="heads", cache="tokens")),
    ([200, 256, 130], [300, 256, 2000], 2, 1, 128, "f16", 16, 8, -1, {}), ([150, 100], [90, 400], 4, 2, 64, "bf16", 32, 5, 60, {}),
    ([256], [640], 1, 1, 64, "f16", 256, 8, 200, {}), ([40, 1, 64], [400, 64, 127], 32, 1, 128, "bf16", 16, 2, -1, {}),
    # chunks beside trees
    ([20, 300, 1, 33, 0, 32], [700, 500, 64, 33, 5, 90], 4, 2, 128, "bf16", 16, 1, -1, dict(spare_rows=5)),
    ([10, 200, 3], [300, 260, 1500], 8, 1, 64, "f16", 32, 1, 90, {}), ([20, 1100, 3], [300, 1200, 50], 8, 1, 64, "bf16", 16, 1, -1, {}),
    ([31, 1, 530], [70, 20, 600], 16, 1, 128, "f16", 64, 1, 300, {}), ([65, 64, 2, 400], [200, 70, 300, 410], 2, 2, 128, "f16", 48, 2, 130, {})]


def _run_attend(bt, words, wl, scale, mask, pos, stride=0, max_q=None, dev=None, **kw):
    q, k, v, o, lse = dev or bt.device()
    n = mask.shape[0]
    wide = torch.full((n, words + stride), -1, dtype=torch.int32, device="cuda")
    wide[:, :words] = tree_ref.to_words(mask).cuda()
    af.attn_fwd_paged_tree(q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), max_q or bt.max_q, wide[:, :words],
                           positions=None if pos is None else _i32(pos), lse=lse, window_left=wl, scale=scale, **kw)
    return o, lse


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "n{}_k{}_{}x{}_d{}_{}_p{}_m{}_w{}".format("-".join(map(str, c[0][:4])), "-".join(map(str, c[1][:4])), *c[2:9]))
def test_attention(case, kind):
    """Trees, and masks of any bits (rows without a key among them, bits past the request's rows set)."""
    nodes, keys, Hq, Hkv, d, dtype, page, words, wl, kw = case
    bt = Batch(nodes, keys, Hq, Hkv, d, dtype, page, seed=sum(keys) + d, fill=float("nan"), **kw)
    n = bt.q.shape[1]
    rng = np.random.default_rng(n)
    if kind == "tree":
        parents = np.concatenate([tree_ref.random_parents(m, rng) for m in nodes] + [np.full(n - sum(nodes), -1)])
        pos, mask, _ = tree_ref.tree(parents, bt.cu.tolist(), keys, words)
        mask = np.maximum(mask, 0)
    else:
        mask = (rng.random((n, 32 * words)) < rng.choice([0.0, 0.05, 0.5, 1.0], (n, 1))).astype(np.int64)
        at = np.concatenate([np.arange(m) + k - m for m, k in zip(nodes, keys)] + [np.zeros(n - sum(nodes))]).astype(np.int64)
        pos = at + rng.integers(-30, 30, n)
    scale = float(np.float32(d ** -0.5))
    o, lse = _run_attend(bt, words, wl, scale, mask, None if wl < 0 and kind == "any" else pos, stride=sum(nodes) % 3)
    af.attn_check()
    tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask, words, pos, wl, scale, what=str(case))


@pytest.mark.parametrize("d,Hq,Hkv,n,ctx", [(128, 8, 2, 40, 3000), (64, 4, 1, 8, 5000), (128, 4, 4, 4, 900)])
def test_a_chain_is_what_the_causal_call_computes(d, Hq, Hkv, n, ctx):
    """The same rows as a chain under a mask and in attn_fwd_paged's causal order: both within the bounds of one reference."""
    bt = Batch([n, n - 3, 1], [ctx + n, ctx // 2, n], Hq, Hkv, d, "bf16", 32, seed=n)
    mask = np.zeros((bt.q.shape[1], 64), np.int64)
    for b in range(3):
        for i in range(bt.lens_q[b]):
            mask[int(bt.cu[b]) + i, :i + 1] = 1
    o, lse = _run_attend(bt, 2, -1, d ** -0.5, mask, None)
    q, k, v, o2, lse2 = bt.device()
    af.attn_fwd_paged(q, k, v, o2, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.max_q, lse=lse2, causal=True, scale=d ** -0.5)
    af.attn_check()
    for got in ((o, lse), (o2, lse2)):
        tree_ref.check_attention(bt, got[0].cpu(), got[1].cpu(), mask, 2, np.zeros(len(mask)), -1, d ** -0.5)


@pytest.mark.parametrize("B,n,top,Hq,Hkv,d,words", [(40, 24, 2600, 4, 1, 64, 1), (600, 3, 300, 4, 1, 64, 1), (1, 20, 9000, 8, 2, 128, 1), (3, 70, 7000, 8, 2, 64, 3),
                                                   (25, 64, 1500, 8, 1, 128, 2), (70, 40, 900, 16, 2, 64, 2), (160, 20, 400, 7, 1, 128, 1)])
def test_attention_of_many_requests(B, n, top, Hq, Hkv, d, words):
    """Few requests whose keys are spread over all SMs, many whose units are cut into equal runs, chunks (B > 3: one) among them."""
    rng = np.random.default_rng(B + d)
    nodes = rng.integers(0 if B > 1 else n, n + 1, B).tolist()
    if B > 3 and n > 10:
        nodes[B // 2] = 32 * words + 100
    keys = [m + int(rng.integers(top // 2 if B < 4 else 0, top)) for m in nodes]
    bt = Batch(nodes, keys, Hq, Hkv, d, "bf16", 16, seed=B)
    parents = np.concatenate([tree_ref.random_parents(m, rng) for m in nodes])
    pos, mask, _ = tree_ref.tree(parents, bt.cu.tolist(), keys, words)
    mask = np.maximum(mask, 0)
    for wl in (-1, 500):
        o, lse = _run_attend(bt, words, wl, 0.125, mask, pos)
        af.attn_check()
        tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask, words, pos, wl, 0.125, what=str((B, wl)))


def test_infinite_keys_in_masked_places():
    """A masked new row's key may hold infinities (its value is finite): its score counts for nothing."""
    bt = Batch([40, 3], [200, 30], 4, 1, 128, "bf16", 16, seed=4)
    mask = np.zeros((43, 64), np.int64)
    for i in range(43):
        mask[i, i if i < 40 else i - 40] = 1
    mask[:, 1] = 0
    for b, at in ((0, 161), (1, 28)):  # node 1 of each request
        bt.k[int(bt.table[b, at // 16]), :, at % 16] = float("inf") if b else -float("inf")
    o, lse = _run_attend(bt, 2, -1, 0.1, mask, None)
    af.attn_check()
    live = [r for r in range(43) if r not in (1, 41)]
    ref = tree_ref.attention(bt, mask, 2, np.zeros(43), -1, 0.1)
    assert torch.isfinite(o.cpu()[:, live].float()).all() and (lse.cpu().double()[:, live] - ref[1][:, live]).abs().max() < 1e-3


def test_longer_requests_than_max_seqlen_q_are_cut_before_the_mask_counts():
    bt = Batch([40, 10], [140, 90], 4, 1, 128, "bf16", 16, seed=8)
    mask = np.tril(np.ones((50, 32), np.int64))
    mask[40:] = np.tril(np.ones((10, 32), np.int64))
    o, lse = _run_attend(bt, 1, -1, 0.1, mask, None, max_q=32)
    af.attn_check()
    tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask, 1, np.zeros(50), -1, 0.1, max_q=32)


# ------------------------------------------------------------------------------ acceptance
def _accept_case(sizes, ctx, confirmed, seed, page=16, likely=0.8, spread=6, W=None, vocabulary=50):
    rng = np.random.default_rng(seed)
    B = len(sizes)
    parents = np.concatenate([tree_ref.random_parents(n, rng, spread) for n in sizes] + [[0, 1]]).astype(np.int64)
    cu, lens = np.concatenate([[0], np.cumsum(sizes)]), np.array(ctx) + sizes
    rows = len(parents)
    tokens, targets = rng.integers(0, vocabulary, rows), rng.integers(0, vocabulary, rows)
    for b in range(B):
        for i in range(int(cu[b]) + 1, int(cu[b + 1])):
            if rng.random() < likely:
                targets[cu[b] + parents[i]] = tokens[i]
    held = [pages(int(n), page) for n in lens]
    W = W or max(held) + 2
    num_pages = sum(held) + 9
    perm = rng.permutation(num_pages)
    table, at = np.full((B, W), -1, np.int64), 0
    for b in range(B):
        m = min(held[b], W)
        table[b, :m] = perm[at:at + m]
        at += held[b]
    free = np.full(num_pages, -3, np.int64)
    free[:num_pages - at] = perm[at:]
    return dict(tokens=tokens, targets=targets, parents=parents, confirmed=confirmed, cu=cu, lens=lens, table=table, free=free, count=num_pages - at,
                page=page, num_pages=num_pages)


def _check_accept(c, P, in_place=True):
    B = len(c["lens"])
    out = {k: _i32(np.full(B, -9)) for k in ("accepted", "ctx", "next")} | {k: _i32(np.full((B, P), -9)) for k in ("path", "src", "dst")}
    free, count = (None, None) if c["free"] is None else (_i32(c["free"]), _i32([c["count"]]))
    left = count if in_place or count is None else _i32([-9])
    table = _i32(c["table"])
    af.attn_paged_accept(_i32(c["tokens"]), _i32(c["targets"]), _i32(c["parents"]), _i32(c["cu"]), _i32(c["lens"]), table, free, count, c["page"],
                         c["num_pages"], out["accepted"], out["ctx"], out["next"], out["path"], out["src"], out["dst"],
                         confirmed=None if c["confirmed"] is None else _i32(c["confirmed"]), free_count_out=None if in_place else left)
    bad = _reported()
    ref = tree_ref.accept(P=P, **c)
    for k, v in out.items():
        assert np.array_equal(v.cpu().numpy(), ref[k]), k
    if free is not None:
        assert np.array_equal(free.cpu().numpy(), ref["free"]) and int(left) == ref["left"]
        if not in_place:
            assert int(count) == c["count"]
    assert bad == ref["bad"] and np.array_equal(table.cpu().numpy(), c["table"])
    return ref


@pytest.mark.parametrize("sizes,ctx,confirmed,P,kw", [
    ([1], [0], None, 1, {}), ([26], [100], None, 8, {}), ([26, 0, 1, 64, 33], [3, 40, 15, 16, 1000], None, 5, {}),
    ([200, 128, 129, 300], [0, 1, 2, 3], None, 40, dict(spread=3)), ([200, 300, 5], [7, 50, 11], [200, 1, 3], 40, dict(spread=3)),
    ([40, 500], [5, 5], [0, 600], 100, dict(spread=1)), ([20] * 700, list(range(700)), None, 12, {}), ([3] * 6000, [17] * 6000, None, 2, {}),
    ([60, 60], [100, 0], None, 64, dict(spread=1, likely=1.0)), ([90] * 5, [33] * 5, None, 9, dict(vocabulary=2)), ([300], [0], None, 3, dict(likely=0.0))])
@pytest.mark.parametrize("in_place", [True, False])
def test_accept(sizes, ctx, confirmed, P, kw, in_place):
    c = _accept_case(sizes, ctx, confirmed, seed=sum(sizes), **kw)
    assert not _check_accept(c, P, in_place)["bad"]


def test_accept_without_a_free_list_and_without_rows():
    c = _accept_case([26, 9], [5, 60], None, seed=3)
    c["free"] = None
    _check_accept(c, 6)
    c = _accept_case([0, 0], [5, 60], None, seed=4)
    for k in ("tokens", "targets", "parents"):
        c[k] = c[k][:0]
    ref = _check_accept(c, 6)
    assert ref["ctx"].tolist() == [5, 60] and ref["next"].tolist() == [-1, -1]


@pytest.mark.parametrize("what", ["no room", "bad id", "narrow table", "count too large", "count negative", "fewer keys than rows"])
def test_accept_bad_values(what):
    c = _accept_case([60] * 6, [90, 4, 31, 7, 64, 200], None, seed=11, likely=0.9, spread=3)
    if what == "no room":
        c["free"] = c["free"][:c["count"] + 3]
    elif what == "bad id":
        c["table"][:, 1::2] = np.where(np.arange(c["table"][:, 1::2].size).reshape(6, -1) % 2, c["num_pages"], -4)
    elif what == "narrow table":
        c["table"] = np.ascontiguousarray(c["table"][:, :4])
    elif what == "count too large":
        c["count"] = len(c["free"]) + 5
    elif what == "count negative":
        c["count"] = -1
    else:
        c["lens"] = np.array([30, 0, 59, 60, 61, -4])
    ref = _check_accept(c, 20)
    assert ref["bad"] or what == "fewer keys than rows"


# ------------------------------------------------------------------------------ moves
@pytest.mark.parametrize("layers,lists,length,Hkv,d,page,cache", [(None, 1, 1, 1, 64, 16, "heads"), (None, 9, 5, 8, 128, 16, "tokens"), (3, 5, 20, 3, 64, 48, "tokens"),
                                                              (2, 2, 150, 20, 128, 32, "heads"), (1, 40, 3, 2, 128, 64, "heads")])
def test_move(layers, lists, length, Hkv, d, page, cache):
    rng = np.random.default_rng(lists * length)
    per = 3 * length + 4  # slots of a list
    num_pages = pages(lists * per, page) + 1
    slots = rng.permutation(num_pages * page)[:lists * per].reshape(lists, per)
    src, dst = np.full((lists, length), -1), np.full((lists, length), -1)
    for i in range(lists):  # ascending paths, whose later sources lie where earlier moves do not write
        path = np.sort(rng.choice(np.arange(1, per), length, replace=False))
        for j, a in enumerate(path):
            if a != j and rng.random() < 0.9:
                src[i, j], dst[i, j] = slots[i, a], slots[i, j]
    shape = (num_pages, Hkv, page, d)
    caches = [torch.randn((layers or 1,) + shape, generator=torch.Generator().manual_seed(x)).bfloat16() for x in (1, 2)]
    got = [c.cuda() for c in caches]
    if cache == "tokens":
        got = [c.transpose(2, 3).contiguous().transpose(2, 3) for c in got]
    af.attn_paged_move(*(c if layers else c[0] for c in got), _i32(src), _i32(dst))
    assert not _reported()
    for g, c in zip(got, caches):
        for i in range(lists):
            for s, t in zip(src[i], dst[i]):
                if s >= 0:
                    c[:, t // page, :, t % page] = c[:, s // page, :, s % page].clone()
        assert torch.equal(g.cpu(), c)


def test_move_slots_past_the_cache_are_left_out_and_reported():
    k = torch.randn((3, 2, 16, 64), device="cuda").half()
    want = k.clone()
    want[0, :, 1] = k[2, :, 15]
    v = k.clone()
    af.attn_paged_move(k, v, _i32([[48, 3, 2 ** 31 - 1], [47, -1, 5]]), _i32([[2, 48, 4], [1, 6, -1]]))
    assert _reported() and not _reported()
    assert torch.equal(k, want) and torch.equal(v, want)


# ------------------------------------------------------------------------------ all together
class Server:
    """A small serving loop: B requests whose tokens' queries, keys and values are looked up in fixed tables, `layers` caches, drafted
    trees of random tokens, and a model whose choice behind a node is a function of the node's token that the drafts guess at times."""

    def __init__(self, B, layers, Hq, Hkv, d, dtype, page, words, seed, stream=None):
        self.B, self.layers, self.Hq, self.Hkv, self.d, self.page, self.words = B, layers, Hq, Hkv, d, page, words
        self.rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.V = 40
        dt = DTYPES[dtype]
        self.raw = torch.randn((layers, self.V, Hq + 2 * Hkv, d), generator=g).to(dt)
        self.w = [(1 + 0.2 * torch.randn(d, generator=g)).to(dt) for _ in range(2)]
        self.inv = 10000.0 ** (-torch.arange(d // 2) / (d / 2.0))
        self.num_pages, self.W, self.rows = 40 * B, 30, 60 * B
        self.kc, self.vc = (torch.full((layers, self.num_pages, Hkv, page, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
        self.table, self.free = _i32(np.full((B, self.W), -1)), _i32(self.rng.permutation(self.num_pages))
        self.count, self.ctx, self.new = _i32([self.num_pages]), _i32([0] * B), _i32([0] * B)
        self.cu, self.lens, self.slots = _i32([0] * (B + 1)), _i32([0] * B), _i32([-1] * self.rows)
        self.pos, self.mask, self.parents = _i32([-1] * self.rows), _i32(np.zeros((self.rows, words))), _i32([-1] * self.rows)
        self.tokens, self.targets, self.confirmed = _i32([0] * self.rows), _i32([0] * self.rows), _i32([1] * B)
        self.accepted, self.next = _i32([0] * B), _i32([0] * B)
        self.path, self.src, self.dst = (_i32(np.zeros((B, 6))) for _ in range(3))
        self.q = torch.zeros((layers, self.rows, Hq, d), dtype=dt, device="cuda")
        self.o = torch.zeros((layers, self.rows, Hq, d), dtype=dt, device="cuda")
        self.qkv = torch.zeros((layers, self.rows, Hq + 2 * Hkv, d), dtype=dt, device="cuda")
        self.raw_dev, self.w_dev, self.inv_dev = self.raw.cuda(), [x.cuda() for x in self.w], self.inv.cuda()
        self.ws = torch.empty(af.attn_paged_workspace(B, Hq, Hkv, d, self.rows, 60), dtype=torch.uint8, device="cuda")
        self.texts = [[] for _ in range(B)]   # tokens in the cache
        self.known = [[int(t) for t in self.rng.integers(0, self.V, n)] for n in self.rng.integers(1, 50, B)]  # tokens known, not yet in the cache

    def choice(self, token):
        return (token * 7 + 3) % self.V

    def draft(self):
        """Known tokens as a chain (a prompt at first), a tree below the last one (none beside a long prompt)."""
        self.trees = []
        for b in range(self.B):
            tokens, parents = list(self.known[b]), list(range(-1, len(self.known[b]) - 1))
            extra = 0 if len(tokens) > 10 else int(self.rng.integers(0, 20))
            for _ in range(extra):
                p = int(self.rng.integers(len(self.known[b]) - 1, len(tokens)))
                parents.append(p)
                tokens.append(self.choice(tokens[p]) if self.rng.random() < 0.6 else int(self.rng.integers(0, self.V)))
            self.trees.append((tokens, parents))
        flat = lambda k: [x for t in self.trees for x in t[k]]  # noqa: E731
        n = len(flat(0))
        self.n = n
        for dst, x in ((self.tokens, flat(0)), (self.parents, flat(1)), (self.targets, [self.choice(t) for t in flat(0)])):
            dst.copy_(_i32(x + [7] * (self.rows - n)))
        self.new.copy_(_i32([len(t[0]) for t in self.trees]))
        self.confirmed.copy_(_i32([len(k) for k in self.known]))

    def step(self):
        """The step's calls, as they may be captured."""
        af.attn_paged_tables(self.ctx, self.new, self.table, self.free, self.count, self.page, self.num_pages, self.cu, self.lens, self.slots)
        af.attn_paged_tree(self.parents, self.cu, self.lens, self.pos, self.mask)
        for i in range(self.layers):
            torch.index_select(self.raw_dev[i], 0, self.tokens, out=self.qkv[i])
            x = self.qkv[i].transpose(0, 1)
            q, o = self.q[i].transpose(0, 1), self.o[i].transpose(0, 1)
            af.attn_paged_rope(x[:self.Hq], x[self.Hq:self.Hq + self.Hkv], x[self.Hq + self.Hkv:], q, self.kc[i], self.vc[i], self.slots, self.pos,
                               self.inv_dev, *self.w_dev)
            af.attn_fwd_paged_tree(q, self.kc[i], self.vc[i], o, self.table, self.cu, self.lens, 60, self.mask, workspace=self.ws)
        af.attn_paged_accept(self.tokens, self.targets, self.parents, self.cu, self.lens, self.table, self.free, self.count, self.page, self.num_pages,
                             self.accepted, self.ctx, self.next, self.path, self.src, self.dst, confirmed=self.confirmed)
        af.attn_paged_move(self.kc, self.vc, self.src, self.dst)

    def check(self):
        """O of every node against the formulas, and the caches' rows against the accepted texts."""
        af.attn_check()
        first = 0
        for b in range(self.B):
            tokens, parents = self.trees[b]
            n, ctx = len(tokens), len(self.texts[b])
            chunk = n > 32 * self.words
            above = []
            for i in range(n):
                above.append([i] if parents[i] < 0 else above[parents[i]] + [i])
            pos = [ctx + (i if chunk else len(above[i]) - 1) for i in range(n)]
            all_tokens, all_pos = self.texts[b] + tokens, list(range(ctx)) + pos
            walk, cur = [], len(self.known[b]) - 1
            while len(walk) < 6:
                kids = [i for i in range(cur + 1, n) if parents[i] == cur and tokens[i] == self.choice(tokens[cur])]
                if not kids:
                    break
                cur = kids[0]
                walk.append(cur)
            for i in range(self.layers):
                raw = self.raw[i][all_tokens].transpose(0, 1)
                p = torch.tensor(all_pos)[None]
                k, dk = tree_ref.rounded_rope(raw[self.Hq:self.Hq + self.Hkv], self.w[1], p, self.inv[None], 1e-6, False, raw.dtype)
                q, dq = tree_ref.rounded_rope(raw[:self.Hq, ctx:], self.w[0], p[:, ctx:], self.inv[None], 1e-6, False, raw.dtype)
                v = raw[self.Hq + self.Hkv:].double()
                keep = torch.zeros((n, ctx + n), dtype=torch.bool)
                keep[:, :ctx] = True
                for x in range(n):
                    keep[x, [ctx + y for y in (range(x + 1) if chunk else above[x])]] = True
                got = self.o[i, first:first + n].transpose(0, 1).cpu().double()
                for h in range(self.Hq):
                    hk, scale = h // (self.Hq // self.Hkv), self.d ** -0.5
                    s = (q[h] @ k[hk].T * scale).masked_fill(~keep, -float("inf"))
                    w = torch.softmax(s, -1)
                    want, A = w @ v[hk], w @ v[hk].abs()
                    size = (q[h].abs() @ k[hk].abs().T * scale * keep).amax(-1)
                    tol, _ = tolerances(raw.dtype, self.d, ctx + n, want, torch.logsumexp(s, -1), A, size)
                    # elements of q and k a step apart move a score by this much, and a weight by twice that
                    moved = ((dq[h] @ (k[hk] + dk[hk]).abs().T + q[h].abs() @ dk[hk].T) * scale * keep).amax(-1)
                    assert ((got[h] - want).abs() <= tol + 2.1 * moved[:, None] * A).all()
                # the caches hold the accepted text, row by row as attn_rope rounds it
                text = self.texts[b] + self.known[b] + [tokens[a] for a in walk]
                at = torch.arange(len(text))
                pg = self.table[b].cpu()[at // self.page].long()
                raw = self.raw[i][text].transpose(0, 1)
                want, tol = tree_ref.rope(raw[self.Hq:self.Hq + self.Hkv], self.w[1], at[None], self.inv[None], 1e-6, False, raw.dtype)
                rows = self.kc[i].cpu()[pg, :, at % self.page].transpose(0, 1).double()
                assert ((rows - want).abs() <= tol).all()
                assert torch.equal(self.vc[i].cpu()[pg, :, at % self.page].transpose(0, 1), raw[self.Hq + self.Hkv:])
            assert int(self.ctx[b]) == len(text) and int(self.next[b]) == self.choice(tokens[cur])
            self.texts[b], self.known[b] = text, [int(self.next[b])]
            first += n
        # no page is lost, none is twice in use
        held = [int(x) for b in range(self.B) for x in self.table[b, :pages(int(self.ctx[b]), self.page)]]
        free = self.free[:int(self.count)].tolist()
        assert sorted(held + free) == list(range(self.num_pages))


@pytest.mark.parametrize("Hq,Hkv,d,dtype,words,captured", [(4, 2, 64, "f16", 1, False), (8, 1, 128, "bf16", 1, True), (2, 2, 128, "bf16", 2, True)])
def test_serving_loop(Hq, Hkv, d, dtype, words, captured):
    """Prompts, then several steps of drafted trees, each checked whole; captured, one graph is replayed for all of them."""
    s = Server(5, 2, Hq, Hkv, d, dtype, 16, words, seed=Hq + d)
    graph = None
    for step in range(6):
        s.draft()
        if not captured or step == 0:
            s.step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    s.step()
            graph.replay()
        torch.cuda.synchronize()
        s.check()


def test_all_on_another_stream_and_in_a_graph_without_a_workspace():
    """The calls go to the stream they are given; a captured attention without a workspace brings its own."""
    bt = Batch([26, 7], [300, 90], 8, 2, 128, "bf16", 16, seed=1)
    rng = np.random.default_rng(0)
    parents = np.concatenate([tree_ref.random_parents(m, rng) for m in (26, 7)])
    pos_ref, mask_ref, _ = tree_ref.tree(parents, bt.cu.tolist(), bt.lens_k, 1)
    q, k, v, o, lse = bt.device()
    pos, mask = _i32([-1] * 33), _i32(np.zeros((33, 1)))
    args = [_i32(parents), bt.cu.cuda(), bt.lens.cuda()]
    table = bt.table.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def go(**kw):
        af.attn_paged_tree(*args, pos, mask, **kw)
        af.attn_fwd_paged_tree(q, k, v, o, table, args[1], args[2], 26, mask, lse=lse, **kw)

    go(stream=stream)
    af.attn_check(stream)
    tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask_ref, 1, pos_ref, -1, 128 ** -0.5)
    o.fill_(float("nan")), lse.fill_(float("nan")), mask.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    graph.replay()
    torch.cuda.synchronize()
    tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask_ref, 1, pos_ref, -1, 128 ** -0.5)
