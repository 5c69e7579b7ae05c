"""attn_rope where its arithmetic could go wrong: elements that are not turned beside infinities and NaN, axes that share their positions."""
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
