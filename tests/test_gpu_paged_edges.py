"""Edges of the paged-cache operators on the GPU: captures that fork, waits that run out, the
tensor maps of many layers, empty lists and maps, the longest lengths, weights in two parts."""
import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

import paged_bounds
from paged_ref import Batch
from test_gpu_paged import _check_tables

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


@pytest.mark.parametrize("lq,lk", [([70, 1], [90, 50]), ([300, 20, 1], [2000, 90, 700]), ([5, 3, 4], [2000, 90, 800])])
@pytest.mark.parametrize("d", [64, 128])
def test_a_q_tile_that_never_comes_ends_the_launch_at_either_head_dim(d, lq, lk):
    """(8 heads to a K/V head: no case has 32 rows at most, which another kernel takes.)  Every wait of the chunk path's roles has a limit, with units of two Q tiles and with key tiles by turns; the
    call after it is right."""
    lib = af.library()
    bt = Batch(lq, lk, 16, 2, d, "bf16", 16, seed=16)
    args, kw = _device(bt)
    assert lib.attn_set_wait_timeout_ns(50_000_000) == 0
    try:
        assert lib.attn_debug_inject(1) == 0
        af.attn_fwd_paged(*args, **kw)
        with pytest.raises(af.AttnError) as e:
            af.attn_check()
        assert e.value.status == -4
    finally:
        lib.attn_debug_inject(0)
        lib.attn_set_wait_timeout_ns(0)
    args[3].fill_(float("nan"))
    kw["lse"].fill_(float("nan"))
    af.attn_fwd_paged(*args, **kw)
    af.attn_check()
    bt.check(args[3].cpu(), kw["lse"].cpu(), True, -1, -1, 0.125)


def test_the_tensor_maps_of_a_models_layers_are_kept():
    """A step that goes over the caches of 96 layers makes no tensor map that the step before has made; a flood of other
    buffers may drop them, and then they are made again."""
    B, Hq, Hkv, d, page, n = 2, 4, 2, 64, 16, 96
    bt = Batch([33, 20], [70, 20], Hq, Hkv, d, "f16", page, seed=5)
    q, k, v, o, lse = bt.device()
    tabs = bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda()
    layers = [(torch.empty_like(k).copy_(k), torch.empty_like(v).copy_(v), torch.empty_like(q).copy_(q)) for _ in range(n)]

    def step():
        before = af.debug_counters()["map_encodes"]
        for kc, vc, x in layers:
            o.fill_(float("nan"))
            af.attn_fwd_paged(x, kc, vc, o, *tabs, bt.max_q, lse=lse, causal=True, scale=0.125)
        af.attn_check()
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.125)
        return af.debug_counters()["map_encodes"] - before

    assert step() <= 3 * n
    assert step() == 0
    pool = torch.zeros(k.numel() + 8 * 5000, dtype=k.dtype, device="cuda")
    before = af.debug_counters()["map_encodes"]
    for i in range(5000):
        x = pool[8 * i:8 * i + k.numel()].view(k.shape)
        af.attn_fwd_paged(q, x, x, o, *tabs, bt.max_q, lse=lse, causal=True, scale=0.125)
    af.attn_check()
    assert af.debug_counters()["map_encodes"] - before >= 5000
    assert 0 < step() <= 3 * n
    assert step() == 0


@pytest.mark.parametrize("ctx,new,free,rows,bad", [
    ([5, 16, 0], [3, 0, 0], 0, 3, False),     # room in the pages held: no free page needed
    ([5, 16, 0], [0, 0, 0], 4, 0, False),     # no new row at all
    ([5, 16, 0], [0, 0, 0], 0, 0, False),
    ([5, 16, 0], [1, 1, 1], 0, 3, True),      # pages wanted, none there
    ([5, 16, 0], [1, 1, 0], 4, 0, True)])     # rows without a place in the map
def test_tables_with_an_empty_free_list_or_no_rows(ctx, new, free, rows, bad):
    table = np.array([[3, -1, -1], [1, -1, -1], [-1, -1, -1]], np.int32)
    got = _check_tables(np.array(ctx), np.array(new), table, np.array([0, 2, 4, 5][:free], np.int32), free, 16, 6, rows)
    assert got["bad"] == bad


@pytest.mark.parametrize("ctx,new", [([2 ** 31 - 20, 7], [15, 12]), ([3, 2 ** 31 - 10], [2, 9]), ([0, 2 ** 31 - 1], [17, 0]),
                                     ([2 ** 31 - 300], [299])])
@pytest.mark.parametrize("page", [16, 256])
def test_tables_of_lengths_up_to_31_bits(ctx, new, page):
    """Lengths whose pages no table holds: reported, counted as all others, and the other requests unharmed."""
    num_pages = 40
    table = np.full((len(ctx), 3), -1, np.int32)
    table[:, 0] = 7
    got = _check_tables(np.array(ctx), np.array(new), table, np.arange(10, 30, dtype=np.int32), 20, page, num_pages, sum(new) + 2)
    assert got["bad"] == any(n for c, n in zip(ctx, new) if c > 2 ** 30)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(paged_bounds.CASES)))
def test_weights_of_few_rows_keep_twice_the_bits(case, dtype):
    """O within a bound that has no room for weights rounded to the values' type (paged_bounds.py)."""
    bt = paged_bounds.batch(paged_bounds.CASES[case], dtype, seed=case)
    q, k, v, o, lse = bt.device()
    af.attn_fwd_paged(q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.max_q, lse=lse, causal=True, scale=paged_bounds.SCALE)
    af.attn_check()
    for rows, want, bound, *_ in paged_bounds.exact(bt):
        err = (o[:, rows].cpu().double() - want).abs() - bound
        assert err.max() <= 0, f"{int((err > 0).sum())} of {err.numel()} over the bound, by {err.max()}"
