"""attn_fwd_packed where entries of one Q tile of rows and of two take turns on an SM."""
import pytest
import torch

import attention_forward_07_gb300 as af

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("lens", [[(100, 900), (250, 900)], [(60, 700), (128, 1100), (200, 640), (256, 1000)], [(1, 1500), (300, 1500), (30, 400)]])
def test_entries_of_one_tile_among_others(lens, d, dtype):
    """A Q tile without rows has its softmax ahead of the products; the scores it takes in the next unit are its own.
    Against 64 bits; each call the same bits.  Tolerance: half a step for every weight and half for the output."""
    g = torch.Generator(device="cuda").manual_seed(d + len(lens))
    lens = lens * (48 // len(lens))
    Hq, Hkv = 8, 4
    tq, tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q = torch.randn((Hq, tq, d), generator=g, device="cuda", dtype=dtype)
    k, v = (torch.randn((Hkv, tk, d), generator=g, device="cuda", dtype=dtype) for _ in range(2))
    cu = [torch.tensor([0] + [x[i] for x in lens], device="cuda").cumsum(0).int() for i in range(2)]
    o, lse = torch.empty_like(q), torch.empty((Hq, tq), device="cuda")
    first = None
    for _ in range(30):
        o.fill_(float("nan"))
        af.attn_fwd_packed(q, k, v, o, cu[0], cu[1], max(a for a, _ in lens), max(b for _, b in lens), lse=lse, causal=True, scale=0.1)
        af.attn_check()
        if first is None:
            first = o.clone(), lse.clone()
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    u = torch.finfo(dtype).eps / 2
    a = b = 0
    for sq, sk in lens:
        kb, vb = (x[:, b:b + sk].double().repeat_interleave(Hq // Hkv, 0) for x in (k, v))
        s = q[:, a:a + sq].double() @ kb.transpose(1, 2) * 0.1
        s = s.masked_fill(torch.arange(sk, device="cuda")[None] > torch.arange(sk - sq, sk, device="cuda")[:, None], -float("inf"))
        w = torch.softmax(s, -1)
        want, size = w @ vb, w @ vb.abs()
        # 2^-12: the scores' and sums' 32-bit errors, of a thousand terms at most, times the weights' sizes
        assert torch.all((o[:, a:a + sq].double() - want).abs() <= u * want.abs() + (u + 2.0 ** -12) * (1 + u) * size + 1e-7)
        assert torch.all((lse[:, a:a + sq].double() - torch.logsumexp(s, -1)).abs() <= 1e-3)
        a, b = a + sq, b + sk
