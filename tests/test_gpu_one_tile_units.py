"""attn_fwd_packed where entries of one Q tile of rows and of two take turns on an SM, and calls on several streams."""
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


@pytest.mark.parametrize("d", [64, 128])
def test_calls_on_three_streams_at_once(d):
    """Kernels that share the machine lose time anywhere; what each waits for is still told apart."""
    g = torch.Generator(device="cuda").manual_seed(d)
    calls = []
    for B, H, S in ((3, 8, 384), (2, 4, 1500), (16, 16, 200)):
        q, k, v = (torch.randn((B, H, S, d), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
        o, lse = torch.empty_like(q), torch.empty((B, H, S), device="cuda")
        af.attn_fwd(q, k, v, o, lse, causal=True, scale=0.1)
        af.attn_check()
        calls.append((q, k, v, o, lse, o.clone(), lse.clone()))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for rep in range(60):
        torch.cuda.synchronize()
        for i, (q, k, v, o, lse, _, _) in enumerate(calls):
            with torch.cuda.stream(streams[(i + rep) % 3]):
                o.zero_()
                af.attn_fwd(q, k, v, o, lse, causal=True, scale=0.1)
        for st in streams:
            af.attn_check(st)
        for _, _, _, o, lse, o0, lse0 in calls:
            assert torch.equal(o, o0) and torch.equal(lse, lse0)

