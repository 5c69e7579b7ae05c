"""Bounds for requests of few rows whose weights go into the product with V in two parts, so that O's own rounding is
all that a type of fewer than 32 bits leaves."""
import torch

from paged_ref import Batch

# lens_q, lens_k, Hq, Hkv, d: at most 16 packed rows, or 32 at d = 64
CASES = [([1] * 6, [64, 50, 33, 64, 17, 48], 16, 2, 128), ([1] * 6, [64, 50, 33, 64, 17, 48], 16, 1, 64), ([2, 4, 3], [64, 40, 57], 8, 2, 128),
         ([4, 1, 3, 2], [64, 60, 64, 39], 16, 2, 64), ([7, 2], [64, 50], 8, 2, 64)]
SCALE = 2.0 ** -9  # scores of some hundredths: their own errors stay below the weights' rounding, which is looked for


def batch(case, dtype, seed):
    lq, lk, Hq, Hkv, d = case
    return Batch(lq, lk, Hq, Hkv, d, dtype, 16, seed=seed)


def exact(bt):
    """Per request: rows, O in 64 bits, the bound on it, and scores, weights relative to the row's largest, kept values."""
    u = torch.finfo(bt.dtype).eps / 2
    half_step = torch.finfo(bt.dtype).smallest_normal * torch.finfo(bt.dtype).eps / 2  # of the smallest numbers
    out = []
    g = bt.Hq // bt.Hkv
    for b in range(bt.B):
        sq, sk = bt.lens_q[b], bt.lens_k[b]
        rows = slice(int(bt.cu[b]), int(bt.cu[b]) + sq)
        key = torch.arange(sk)
        pg = bt.table[b, key // bt.page].long()
        k, v = (c[pg, :, key % bt.page].double().transpose(0, 1).repeat_interleave(g, 0) for c in (bt.k, bt.v))
        q = bt.q[:, rows].double()
        keep = key[None] <= torch.arange(sk - sq, sk)[:, None]
        s = (q @ k.transpose(1, 2) * SCALE).masked_fill(~keep, -float("inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        total = p.sum(-1, keepdim=True)
        o, A = p @ v / total, p @ v.abs() / total
        S = ((q.abs() @ k.abs().transpose(1, 2)) * SCALE * keep).amax(-1, keepdim=True)
        # As in paged_ref.tolerances, but a weight p is held as h + r, h = p and r = p - h rounded: off by u^2 p, or by
        # half a step of the smallest numbers of the type (relative to a base of at most the row's maximum: p may
        # stand 2^8 higher than here, and then its sum does too).
        e = (bt.d + 8) * 2.0 ** -23 * S + 2.0 ** -20
        w = 2 * e + sk * (2.0 ** -24 + 2.0 ** -23) + u * u
        bound = u * o.abs() + (1 + u) * (w * A + half_step * (keep.double() @ v.abs()) / total) + 2 * half_step
        out.append((rows, o, bound, p, v, total))
    return out


def emulated(bt, parts):
    """O of each request with the weights in `parts` parts, all else exact: [(rows, o rounded)]."""
    out = []
    for rows, _, _, p, v, total in exact(bt):
        h = p.to(bt.dtype).double()
        r = (p - h).to(bt.dtype).double() if parts == 2 else 0.0
        out.append((rows, ((h + r) @ v / total).to(bt.dtype).double()))
    return out
