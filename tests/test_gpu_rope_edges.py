"""attn_rope where its arithmetic could go wrong: elements that are not turned beside infinities and NaN, axes that share their positions, positions
at both ends of their type."""
import math

import pytest
import torch

import attention_forward_07_gb300 as af

import tree_ref
from paged_ref import DTYPES

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def _rotated(x, weight, pos, inv, interleaved, cache=False):
    """x [H, rows, d] as queries and as keys of one call; with `cache` the keys go to slots 0, 1, ... of a cache."""
    H, rows, d = x.shape
    xd, p, f = x.cuda(), pos.cuda(), None if inv is None else inv.cuda()
    w = None if weight is None else weight.cuda()
    q = torch.full_like(xd, 7.0)
    if not cache:
        k = torch.full_like(xd, 7.0)
        af.attn_rope(xd, xd, q, k, None if f is None else p, f, w, w, eps=1e-5, interleaved=interleaved)
    else:
        kc = torch.full((-(-rows // 16), H, 16, d), 7.0, dtype=x.dtype, device="cuda")
        vc = torch.full_like(kc, 7.0)
        af.attn_paged_rope(xd, xd, xd, q, kc, vc, torch.arange(rows, dtype=torch.int32, device="cuda"), p, f, w, w, eps=1e-5, interleaved=interleaved)
        k, v = (c.transpose(0, 1).reshape(H, -1, d)[:, :rows] for c in (kc, vc))
        assert torch.equal(v.view(torch.int16), xd.view(torch.int16))
    af.attn_check()
    assert torch.equal(q.view(torch.int16), k.contiguous().view(torch.int16))
    return q.cpu()


NOT_TURNED = [(64, 0, False), (64, 16, False), (64, 32, True), (128, 0, False), (128, 0, True), (128, 64, False), (128, 96, True), (128, 112, False)]


@pytest.mark.parametrize("d,rot,interleaved", NOT_TURNED)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cache", [False, True])
def test_elements_that_are_not_turned_keep_their_bits_beside_infinities(d, rot, interleaved, dtype, cache):
    """Without a weight an element past the pairs that are turned is copied, whatever its neighbours hold, zeros' signs included (a NaN stays one)."""
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn((5, 37, d), generator=g).to(DTYPES[dtype])
    odd = torch.tensor([INF, -INF, NAN, 0.0, -0.0]).to(x.dtype)
    x[..., rot:] = torch.where(torch.rand((5, 37, d - rot), generator=g) < 0.15, odd[torch.randint(0, 5, (5, 37, d - rot), generator=g)], x[..., rot:])
    x[0, 0, rot:] = x[1, 0, rot:].abs() + 1  # one of each alone in its row
    x[0, 0, rot + 3] = -INF
    pos = torch.arange(37, dtype=torch.int32)
    inv = 100.0 ** (-torch.arange(rot // 2) / (rot / 2)) if rot else None
    got = _rotated(x, None, pos, inv, interleaved, cache)
    nan = torch.isnan(x[..., rot:])
    assert torch.equal(torch.isnan(got[..., rot:]), nan)
    assert torch.equal(got[..., rot:].view(torch.int16)[~nan], x[..., rot:].view(torch.int16)[~nan])
    if rot:
        want, tol = tree_ref.rope(x[..., :rot], None, pos[None], inv[None], 1e-5, interleaved, x.dtype)
        assert ((got[..., :rot].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("d,rot,interleaved", NOT_TURNED)
@pytest.mark.parametrize("weight", ["f32", "type"])
def test_infinities_under_a_norm_are_what_the_formula_makes_of_them(d, rot, interleaved, weight):
    """An infinite element makes the mean infinite and the row's others zeros (itself, and what it is turned with, NaN); a NaN makes all NaN."""
    g = torch.Generator().manual_seed(d + rot + 1)
    x = torch.randn((3, 40, d), generator=g).bfloat16()
    x[0, 5, d - 1] = INF
    x[1, 6, 0] = -INF
    x[2, 7, d - 3] = NAN
    w = 1 + 0.3 * torch.randn(d, generator=g)
    w[d - 2] = 0.0
    w = w if weight == "f32" else w.bfloat16()
    pos = torch.arange(1, 41, dtype=torch.int32)
    inv = 100.0 ** (-torch.arange(rot // 2) / (rot / 2)) if rot else None
    got = _rotated(x, w, pos, inv, interleaved)
    want, tol = tree_ref.rope(x, w, pos[None], None if inv is None else inv[None], 1e-5, interleaved, x.dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    odd = [(0, 5), (1, 6), (2, 7)]
    for h, t in odd:
        live = ~torch.isnan(want[h, t])
        assert (got[h, t][live] == 0).all()
    keep = torch.ones((3, 40), dtype=torch.bool)
    keep[tuple(zip(*odd))] = False
    assert ((got.double() - want).abs() <= tol)[keep].all()


@pytest.mark.parametrize("axes", [2, 3])
def test_axes_that_share_their_positions(axes):
    """An expanded row of positions (its axes' stride is 0) is what a copy of it for every axis is."""
    g = torch.Generator().manual_seed(axes)
    x = torch.randn((6, 50, 128), generator=g).bfloat16().cuda()
    pos = torch.randint(0, 1000, (1, 50), generator=g).int().cuda().expand(axes, 50)
    inv = (1000.0 ** (-torch.arange(64) / 64.0))[None] * (torch.arange(64)[None] % axes == torch.arange(axes)[:, None])
    assert pos.stride(0) == 0
    outs = []
    for p in (pos, pos.contiguous()):
        q, k = torch.empty_like(x[:4]), torch.empty_like(x[4:])
        af.attn_rope(x[:4], x[4:], q, k, p, inv.cuda())
        outs.append((q, k))
    af.attn_check()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    want, tol = tree_ref.rope(x[:4].cpu(), None, pos.cpu(), inv, 1e-6, False, torch.bfloat16)
    assert ((outs[0][0].cpu().double() - want).abs() <= tol).all()


def _turns(pos, inv):
    """Angles sum_a pos[a, t] inv[a, i] as parts of a turn in [0, 1), in whole numbers of 2^-200 (inv's floats are exact; 2 pi from Machin's formula)."""
    bits = 400
    arctan = lambda n: sum((-1) ** i * (1 << bits) // ((2 * i + 1) * n ** (2 * i + 1)) for i in range(200))  # noqa: E731
    two_pi = 2 * (16 * arctan(5) - 4 * arctan(239))
    out = torch.empty((pos.shape[1], inv.shape[1]), dtype=torch.float64)
    ratios = [[float(f).as_integer_ratio() for f in row] for row in inv]
    for i in range(inv.shape[1]):
        turns = [((n << (200 + bits)) // (den * two_pi)) for n, den in (row[i] for row in ratios)]
        for t in range(pos.shape[1]):
            out[t, i] = (sum(int(pos[a, t]) * turns[a] for a in range(len(turns))) % (1 << 200)) / (1 << 200)
    return out


@pytest.mark.parametrize("axes,d,interleaved,top", [(1, 128, False, 1.0), (1, 64, True, 1.0), (3, 128, False, 1.0), (4, 128, True, 1.0), (2, 64, True, 2.0 ** 60)])
def test_angles_at_both_ends_of_the_positions(axes, d, interleaved, top):
    """Angles keep 2^-25 of a turn at any position: a frequency's part of a turn is cut at 2^-64, so 2^-33 of a turn for each axis's position, the
    sum at 2^-32 and then rounded to a float, half a step of which is 2^-26 of a turn.  The function: 2 ulp of a value of at most 1, 2^-23.  Ones and zeros are
    turned, so the rounding to fp16, small next to 0, is all else: products by 0 and 1 and sums with 0 are exact."""
    g = torch.Generator().manual_seed(axes * d)
    half = d // 2
    rows = 400
    pos = torch.cat([torch.randint(2 ** 31 - 1000, 2 ** 31, (axes, rows // 2), generator=g), torch.randint(-2 ** 31, -2 ** 31 + 1000, (axes, rows // 2), generator=g)], 1)
    pos[:, 0], pos[:, -1] = 2 ** 31 - 1, -2 ** 31
    pos = torch.stack([p[torch.randperm(rows, generator=g)] for p in pos])
    inv = (top * 10000.0 ** (-torch.arange(half) / half)).float()
    inv = inv[None].repeat(axes, 1) * (0.5 + 0.5 * torch.rand((axes, half), generator=g))  # (every axis turns every pair)
    first = torch.arange(0, d, 2) if interleaved else torch.arange(half)
    second = first + (1 if interleaved else half)
    x = torch.zeros((1, rows, d), dtype=torch.float16)
    x[..., first] = 1.0
    q, k = torch.empty((1, rows, d), dtype=torch.float16, device="cuda"), torch.empty((1, rows, d), dtype=torch.float16, device="cuda")
    af.attn_rope(x.cuda(), x.cuda(), q, k, pos.int().cuda(), inv.cuda(), interleaved=interleaved)
    af.attn_check()
    phi = 2 * math.pi * _turns(pos, inv)
    err = 2 * math.pi * (axes * 2.0 ** -33 + 2.0 ** -32 + 2.0 ** -26) + 2.0 ** -23
    for got, want in ((q[0].cpu().double()[:, first], phi.cos()), (q[0].cpu().double()[:, second], phi.sin())):
        assert ((got - want).abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -25 + (1 + 2.0 ** -10) * err).all()
    assert torch.equal(q, k)
