"""Plain forms (CPU, whole numbers or 64 bits) of the operators of drafted trees, and bounds on their roundings."""
import math

import numpy as np
import torch

from paged_ref import tolerances


def random_parents(n, rng, spread=8, chain=False):
    """Parents of a tree of n nodes: node 0 has none, node i one of the `spread` nodes ahead of it."""
    return np.array([-1] + [i - 1 if chain else int(rng.integers(max(0, i - spread), i)) for i in range(1, n)][:max(0, n - 1)][:n], np.int64)[:n]


def tree(parents, cu, lens, words, window=-1):
    """attn_paged_tree: positions and masks (0 / 1, [rows, 32 words]) with -7 / -7 where nothing is written, and whether it reports."""
    rows = len(parents)
    pos, mask, bad = np.full(rows, -7, np.int64), np.full((rows, 32 * words), -7, np.int64), False
    for b in range(len(lens)):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        n, ctx = r1 - r0, max(int(lens[b]) - (r1 - r0), 0)
        if n > 32 * words:
            pos[r0:r1] = ctx + np.arange(n)
            continue
        depth = []
        for i in range(n):
            x = int(parents[r0 + i])
            if x >= i or x < -1:
                bad, x = True, -1
            above = [] if x < 0 else [x] + depth[x]
            depth.append(above)
            pos[r0 + i] = ctx + len(above)
            mask[r0 + i] = 0
            mask[r0 + i, [i] + (above if window < 0 else above[:window])] = 1
    return pos, mask, bad


def to_words(bits):
    """[rows, 32 words] of 0 / 1 -> int32 [rows, words]."""
    b = np.asarray(bits).astype(np.uint64).reshape(len(bits), -1, 32)
    return torch.from_numpy((b << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32).copy())


def from_words(words):
    w = words.cpu().numpy().view(np.uint32)
    return ((w[..., None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(len(w), -1).astype(np.int64)


def rope(x, weight, pos, inv, eps, interleaved, dtype):
    """Norm and rotation of x [H, n, d] in 64 bits; pos [axes, n], inv float32 [axes, pairs] or None.  Also a bound on the error of the
    kernel's 32-bit arithmetic and one rounding to dtype.

    A product of weight, cosine and element: cosine and sine are off by 2^-21 at most (the angle's rounding to 24 bits of a
    half turn, pi 2^-24; its 64-bit product, 2 pi 2^-23.6 at positions below 2^31, so 2^-30 here, where they stay below 2^20; the
    function itself, 2^-22), the product's and sum's roundings are 4 2^-24: (2^-21 + 2^-22) (|x_a w_a| + |x_b w_b|) r.  r: a sum of
    d squares, each addition off by 2^-24 of the sum, halved by the root, and 4 2^-24 for the division by d, eps and the
    function (2 ulp): (d / 2 + 8) 2^-24 of the result.  The rounding: half a step, of the smallest numbers at least."""
    x = x.double()
    d = x.shape[-1]
    r = torch.ones(x.shape[:-1] + (1,), dtype=torch.float64)
    y = x.clone()
    if weight is not None:
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + float(np.float32(eps)))
        y = x * r * weight.double()
    out, size = y.clone(), y.abs()
    if inv is not None and inv.shape[-1]:
        half = inv.shape[-1]
        a = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
        b = a + (1 if interleaved else half)
        phi = (pos.double()[:, :, None] * inv.double()[:, None]).sum(0)
        c, s = phi.cos(), phi.sin()
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    info = torch.finfo(dtype)
    e = size * (2.0 ** -21 + 2.0 ** -22 + (0 if weight is None else (d / 2 + 8) * 2.0 ** -24))
    return out, info.eps / 2 * out.abs() + (1 + info.eps) * e + info.smallest_normal * info.eps / 2


def rounded_rope(x, weight, pos, inv, eps, interleaved, dtype):
    """rope's result rounded to dtype, in 64 bits, and by how much the kernel's may differ: a step where its 32-bit error may cross a tie."""
    y, tol = rope(x, weight, pos, inv, eps, interleaved, dtype)
    info = torch.finfo(dtype)
    e = tol - info.eps / 2 * y.abs()
    lo, hi = (y - e).to(dtype).double(), (y + e).to(dtype).double()
    return y.to(dtype).double(), hi - lo


def attention(bt, mask, words, pos, wl, scale, max_q=None):
    """attn_fwd_paged_tree over a paged_ref.Batch: mask 0 / 1 [rows, 32 words], pos [rows].  O, LSE (NaN in rows of no request), A, S as
    paged_ref.attention gives them."""
    q, (Hq, n, d), Hkv, page = bt.q, bt.q.shape, bt.Hkv, bt.page
    g, max_q = Hq // Hkv, max_q or bt.max_q
    o, lse = torch.full((Hq, n, d), float("nan"), dtype=torch.float64), torch.full((Hq, n), float("nan"), dtype=torch.float64)
    A, S = torch.zeros((Hq, n, d), dtype=torch.float64), torch.zeros((Hq, n), dtype=torch.float64)
    for b in range(bt.B):
        r0 = int(bt.cu[b])
        sq, sk = min(int(bt.cu[b + 1]) - r0, max_q), int(bt.lens[b])
        if sq <= 0:
            continue
        rows, off = slice(r0, r0 + sq), sk - sq
        keep = torch.zeros((sq, sk), dtype=torch.bool)
        for i in range(sq):
            if sq > 32 * words:
                lo = 0 if wl < 0 else max(0, i + off - wl)
                keep[i, lo:max(0, i + off + 1)] = True
                continue
            lo = 0 if wl < 0 else max(0, max(int(pos[r0 + i]), off) - wl)
            keep[i, lo:max(off, 0)] = True
            for j in range(sq):
                if mask[r0 + i][j] and off + j >= 0:
                    keep[i, off + j] = True
        seen = torch.nonzero(keep.any(0)).flatten()
        kb, vb = (torch.zeros((Hkv, sk, d), dtype=torch.float64) for _ in range(2))
        pg = bt.table[b, seen // page].long()
        kb[:, seen] = bt.k[pg, :, seen % page].double().transpose(0, 1)
        vb[:, seen] = bt.v[pg, :, seen % page].double().transpose(0, 1)
        for hq in range(Hq):
            qq = q[hq, rows].double()
            s = ((qq @ kb[hq // g].T) * scale).masked_fill(~keep, -math.inf)
            z = torch.logsumexp(s, -1) if sk else torch.full((sq,), -math.inf, dtype=torch.float64)
            w = torch.where(keep, torch.exp(s - torch.where(z > -math.inf, z, 0.0)[:, None]), 0.0)
            o[hq, rows], A[hq, rows], lse[hq, rows] = w @ vb[hq // g], w @ vb[hq // g].abs(), z
            if sk:
                S[hq, rows] = ((qq.abs() @ kb[hq // g].abs().T) * scale * keep).amax(-1)
    return o, lse, A, S


def check_attention(bt, o, lse, mask, words, pos, wl, scale, max_q=None, what=""):
    o_ref, lse_ref, A, S = attention(bt, mask, words, pos, wl, scale, max_q)
    to, tl = tolerances(bt.dtype, bt.d, max(bt.lens_k + [1]), o_ref, lse_ref, A, S)
    live = ~torch.isnan(lse_ref)
    assert torch.all(torch.isnan(lse[~live])) and torch.all(torch.isnan(o[~live])), f"{what}: rows of no request were written"
    o, lse = o.double()[live], lse.double()[live]
    assert torch.all(torch.isfinite(o)), f"{what}: O not finite"
    err = (o - o_ref[live]).abs() - to[live]
    assert err.numel() == 0 or err.max() <= 0, f"{what}: O off by {err.max()} over its bound, {int((err > 0).sum())} of {err.numel()}"
    empty = torch.isinf(lse_ref[live])
    assert torch.equal(torch.isinf(lse), empty) and torch.all(lse[empty] < 0), f"{what}: LSE of empty rows"
    assert torch.all(o[empty] == 0), f"{what}: O of empty rows"
    err = ((lse - lse_ref[live]).abs() - tl[live])[~empty]
    assert err.numel() == 0 or err.max() <= 0, f"{what}: LSE off by {err.max()} over its bound"


def accept(tokens, targets, parents, confirmed, cu, lens, table, free, count, page, num_pages, P):
    """attn_paged_accept by its documentation."""
    B, W = table.shape
    out = dict(accepted=np.zeros(B, np.int64), ctx=np.zeros(B, np.int64), next=np.full(B, -1, np.int64),
               path=np.full((B, P), -1, np.int64), src=np.full((B, P), -1, np.int64), dst=np.full((B, P), -1, np.int64))
    bad, free = False, None if free is None else free.copy()
    have = 0
    if free is not None:
        have = min(max(count, 0), len(free))
        bad |= have != count

    def slot(b, p):
        i = p // page
        if p < 0 or i >= W or not 0 <= table[b, i] < num_pages:
            return -1
        return int(table[b, i]) * page + p % page

    for b in range(B):
        r0, keys = int(cu[b]), max(int(lens[b]), 0)
        n = int(cu[b + 1]) - r0
        ctx = keys - n
        sure = min(max(1 if confirmed is None else int(confirmed[b]), 1), n)
        cur, walk = sure - 1, []
        while n and len(walk) < P:
            kids = [i for i in range(cur + 1, n) if parents[r0 + i] == cur and tokens[r0 + i] == targets[r0 + cur]]
            if not kids:
                break
            cur = kids[0]
            walk.append(cur)
        out["accepted"][b] = sure + len(walk)
        after = max(ctx + sure + len(walk), 0)
        out["ctx"][b] = after
        if n:
            out["next"][b] = targets[r0 + cur]
        for j, a in enumerate(walk):
            out["path"][b, j] = a
            if a != sure + j:
                s, d = slot(b, ctx + a), slot(b, ctx + sure + j)
                if s < 0 or d < 0:
                    bad = True
                else:
                    out["src"][b, j], out["dst"][b, j] = s, d
        if free is not None:
            for i in range(-(-after // page), -(-keys // page)):
                pid = int(table[b, i]) if i < W else -1
                if not 0 <= pid < num_pages or have == len(free):
                    bad = True
                    continue
                free[have] = pid
                have += 1
    return out | dict(free=free, left=have, bad=bad)
