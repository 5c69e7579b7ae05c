"""Edges of the paged-cache operators on the GPU: captures that fork."""
import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

from paged_ref import Batch

pytestmark = pytest.mark.gpu


def _device(bt):
    q, k, v, o, lse = bt.device()
    return (q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.max_q), dict(lse=lse, causal=True, scale=0.125)


@pytest.mark.parametrize("d", [64, 128])
def test_calls_on_streams_forked_in_one_capture(d):
    """Calls on two side streams of one graph, through `stream=`, and buffers that the main branch takes meanwhile: each
    call's workspace is its own, so every replay gives the bits of the calls alone."""
    shapes = [([150, 1, 40], [900, 2500, 300]), ([1] * 9, [700 + 200 * b for b in range(9)]), ([300, 20], [300, 1500]), ([5, 3, 4], [2000, 90, 800])]
    calls = []
    for lq, lk in shapes:
        bt = Batch(lq, lk, 8, 2, d, "bf16", 16, seed=sum(lk) + d)
        args, kw = _device(bt)
        af.attn_fwd_paged(*args, **kw)
        af.attn_check()
        bt.check(args[3].cpu(), kw["lse"].cpu(), True, -1, -1, 0.125)
        calls.append((args, kw, args[3].clone(), kw["lse"].clone()))
    room = max(af.attn_paged_workspace(a[6].numel(), 8, 2, d, a[0].shape[1], a[7]) for a, *_ in calls)
    sides = [torch.cuda.Stream() for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        for s in sides:
            s.wait_stream(main)
        for i, (args, kw, _, _) in enumerate(calls):
            af.attn_fwd_paged(*args, **kw, stream=sides[i % 2])
            junk = torch.full((room,), 255, dtype=torch.uint8, device="cuda")
            del junk
        for s in sides:
            main.wait_stream(s)
    for _ in range(20):
        for args, kw, _, _ in calls:
            args[3].fill_(float("nan"))
            kw["lse"].zero_()
        g.replay()
        torch.cuda.synchronize()
        for args, kw, o, lse in calls:
            n = int(args[5][-1])
            assert torch.equal(args[3][:, :n], o[:, :n]) and torch.equal(kw["lse"][:, :n], lse[:, :n])
    for s in (main, *sides):
        af.attn_check(s)
