"""Plain 64-bit forms of the paged-cache operators and helpers that build their inputs (CPU)."""
import numpy as np
import torch

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def pages(n, page):
    return -(-n // page)


def tables(ctx, new, table, free, count, page, num_pages, max_rows):
    """attn_paged_tables by its documentation: returns what it writes, and whether it reports a bad page."""
    table = table.copy()
    B, W = table.shape
    count_in, count = count, min(max(count, 0), len(free))
    bad = count_in != count
    cu, lens, slots, positions = [0], [], [], []
    taken = 0
    for b in range(B):
        c, n = max(int(ctx[b]), 0), max(int(new[b]), 0)
        held, want = pages(c, page), pages(c + n, page)
        got = {}
        for i in range(held, want):
            at = count - 1 - taken
            taken += 1
            pid = int(free[at]) if at >= 0 else -1
            if not 0 <= pid < num_pages:
                pid = -1
            got[i] = pid
            bad |= pid < 0 or i >= W
            if i < W:
                table[b, i] = pid
        for p in range(c, c + n):
            i = p // page
            pid = -1
            if i < W:
                pid = got[i] if i in got else int(table[b, i])
            ok = 0 <= pid < num_pages
            slots.append(pid * page + p % page if ok else -1)
            positions.append(p)
            if len(slots) <= max_rows:
                bad |= not ok
        cu.append(cu[-1] + n)
        lens.append(c + n)
    bad |= len(slots) > max_rows
    pad = [-1] * max(0, max_rows - len(slots))
    return dict(table=table, cu=np.array(cu), lens=np.array(lens), slots=np.array((slots + pad)[:max_rows]),
                positions=np.array((positions + pad)[:max_rows]), left=max(count - taken, 0), bad=bad)


def attention(q, k_cache, v_cache, table, cu, lens, max_q, causal, wl, wr, scale):
    """O, LSE (float64; NaN in rows of no request) of q [Hq, rows, d] over caches [pages, Hkv, page, d], and for the
    tolerances A = sum_j w_j |v_j| and S = max_j sum_x |q_x k_jx| * scale of every row."""
    Hq, n, d = q.shape
    _, Hkv, page, _ = k_cache.shape
    g = Hq // Hkv
    o = torch.full((Hq, n, d), float("nan"), dtype=torch.float64)
    A = torch.zeros((Hq, n, d), dtype=torch.float64)
    lse = torch.full((Hq, n), float("nan"), dtype=torch.float64)
    S = torch.zeros((Hq, n), dtype=torch.float64)
    er = 0 if causal else wr
    for b in range(len(lens)):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        sq, sk = min(r1 - r0, max_q), int(lens[b])
        if sq == 0:
            continue
        rows = slice(r0, r0 + sq)
        pos = torch.arange(sq)[:, None] + sk - sq
        j = torch.arange(sk)[None]
        keep = torch.ones((sq, sk), dtype=torch.bool)
        if wl >= 0:
            keep &= j >= pos - wl
        if er >= 0:
            keep &= j <= pos + er
        seen = keep.any(0)
        kb = torch.zeros((Hkv, sk, d), dtype=torch.float64)
        vb = torch.zeros((Hkv, sk, d), dtype=torch.float64)
        key = torch.nonzero(seen).flatten()
        pg = torch.as_tensor(table)[b, key // page].long()
        kb[:, key] = k_cache[pg, :, key % page].double().transpose(0, 1)
        vb[:, key] = v_cache[pg, :, key % page].double().transpose(0, 1)
        for hq in range(Hq):
            qq = q[hq, rows].double()
            s = (qq @ kb[hq // g].T) * scale
            s = s.masked_fill(~keep, -float("inf"))
            z = torch.logsumexp(s, -1) if sk else torch.full((sq,), -float("inf"), dtype=torch.float64)
            w = torch.where(keep, torch.exp(s - torch.where(z > -float("inf"), z, 0.0)[:, None]), 0.0)
            o[hq, rows] = w @ vb[hq // g]
            A[hq, rows] = w @ vb[hq // g].abs()
            lse[hq, rows] = z
            if sk:
                S[hq, rows] = ((qq.abs() @ kb[hq // g].abs().T) * scale * keep).amax(-1)
    return o, lse, A, S


def tolerances(dtype, d, keys, o, lse, A, S):
    """Bounds on |O - O_ref| and |LSE - LSE_ref|.

    A score is a sum of d exact products, each addition off by at most 2^-23 of the running sum of
    magnitudes (a matrix instruction may truncate), so off by d 2^-23 S; scaled and turned into an exponent it is off by a few
    2^-24 of itself more: e = (d + 8) 2^-23 S + 2^-20.  A weight is then off by 2 e relative to the
    normalised one (itself and the sum it is divided by), plus the sum's own additions, keys 2^-24, plus
    its rounding to the values' type, u = eps / 2.  The product with V adds keys 2^-23 in 32 bits, and O is rounded once to its type.
    LSE is off by e, by the sum's additions and by a few 2^-24 of itself."""
    u = torch.finfo(dtype).eps / 2
    e = (d + 8) * 2.0 ** -23 * S + 2.0 ** -20
    w = 2 * e + keys * (2.0 ** -24 + 2.0 ** -23) + u
    smallest = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    to = u * o.abs() + (1 + u) * w[..., None] * A + smallest
    tl = e + keys * 2.0 ** -24 + 2.0 ** -21 * lse.abs().clamp(max=1e30)
    return to, tl


class Batch:
    """Random requests over a paged cache, on the CPU."""

    def __init__(self, lens_q, lens_k, Hq, Hkv, d, dtype, page, seed, spare_rows=0, spare_width=2, fill="randn", rows="tokens",
                 cache="heads", spare_pages=3):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.page, self.B = DTYPES[dtype], page, len(lens_q)
        self.lens_q, self.lens_k = list(lens_q), list(lens_k)
        self.Hq, self.Hkv, self.d = Hq, Hkv, d
        need = [pages(n, page) for n in lens_k]
        self.num_pages = sum(need) + spare_pages
        W = max(max(need), 1) + spare_width
        perm = torch.randperm(self.num_pages, generator=g)
        self.table = torch.full((self.B, W), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = perm[at:at + m].int()
            at += m
        self.cu = torch.tensor([0] + list(np.cumsum(lens_q)), dtype=torch.int32)
        self.lens = torch.tensor(lens_k, dtype=torch.int32)
        n = int(self.cu[-1]) + spare_rows
        self.q = torch.randn((Hq, n, d), generator=g).to(self.dtype)
        shape = (self.num_pages, Hkv, page, d)
        if fill == "randn":
            self.k, self.v = (torch.randn(shape, generator=g).to(self.dtype) for _ in range(2))
        else:  # rows that no request owns hold `fill`
            self.k, self.v = (torch.full(shape, fill, dtype=self.dtype) for _ in range(2))
            for b in range(self.B):
                for key in range(lens_k[b]):
                    pg = int(self.table[b, key // page])
                    for c in (self.k, self.v):
                        c[pg, :, key % page] = torch.randn((Hkv, d), generator=g).to(self.dtype)
        self.rows, self.cache = rows, cache
        self.max_q = max(max(lens_q), 1)

    def device(self, dev="cuda"):
        """q, k_cache, v_cache, o, lse on the device in this batch's layouts, o and lse full of NaN."""
        def laid(x, tokens, a, b):
            x = x.to(dev)
            return x.transpose(a, b).contiguous().transpose(a, b) if tokens else x
        q = laid(self.q, self.rows == "tokens", 0, 1)
        k, v = (laid(c, self.cache == "tokens", 1, 2) for c in (self.k, self.v))
        o = laid(torch.full_like(self.q, float("nan")), self.rows == "tokens", 0, 1)
        lse = torch.full(self.q.shape[:2], float("nan"), dtype=torch.float32, device=dev)
        return q, k, v, o, lse

    def check(self, o, lse, causal, wl, wr, scale, max_q=None, what="", skip=()):
        """o, lse (CPU) against the plain form; rows of no request are untouched NaN; requests in `skip` are not looked at."""
        max_q = max_q or self.max_q
        o_ref, lse_ref, A, S = attention(self.q, self.k, self.v, self.table, self.cu, self.lens, max_q, causal, wl, wr, scale)
        to, tl = tolerances(self.dtype, self.d, max(self.lens_k + [1]), o_ref, lse_ref, A, S)
        live = ~torch.isnan(lse_ref)
        for b in skip:
            r = slice(int(self.cu[b]), int(self.cu[b + 1]))
            live[:, r] = False
            o, lse = o.clone(), lse.clone()
            o[:, r], lse[:, r] = float("nan"), float("nan")
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
