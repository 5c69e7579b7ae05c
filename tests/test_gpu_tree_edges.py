"""Drafted trees on the GPU where calls meet: waits that run out, several streams and graphs at once, a process whose first calls are
captured, places past 32 bits, lengths up to 31."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

import tree_ref
from paged_ref import Batch

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Call:
    """attn_fwd_paged_tree on a batch of random trees (or chunks, where a request has more nodes than the masks bits)."""

    def __init__(self, nodes, keys, Hq, Hkv, d, words=2, wl=-1, page=16, seed=0):
        self.bt, self.words, self.wl = Batch(nodes, keys, Hq, Hkv, d, "bf16", page, seed=seed), words, wl
        rng = np.random.default_rng(seed)
        parents = np.concatenate([tree_ref.random_parents(m, rng) for m in nodes])
        self.pos, mask, _ = tree_ref.tree(parents, self.bt.cu.tolist(), keys, words)
        self.mask = np.maximum(mask, 0)
        q, k, v, self.o, self.lse = self.bt.device()
        self.args = (q, k, v, self.o, self.bt.table.cuda(), self.bt.cu.cuda(), self.bt.lens.cuda(), self.bt.max_q, tree_ref.to_words(self.mask).cuda())
        self.positions = _i32(self.pos)

    def __call__(self, **kw):
        af.attn_fwd_paged_tree(*self.args, positions=self.positions, lse=self.lse, window_left=self.wl, scale=0.125, **kw)

    def clear(self):
        self.o.fill_(float("nan"))
        self.lse.fill_(float("nan"))

    def check(self):
        tree_ref.check_attention(self.bt, self.o.cpu(), self.lse.cpu(), self.mask, self.words, self.pos, self.wl, 0.125)


# one tile, units of several tiles and a chunk, many requests (with a plan)
SHAPES = [([26, 5], [300, 700], 8, 1), ([64, 40, 200, 1], [900, 2000, 500, 77], 16, 2), ([40] + [2] * 600, [700] + [30 + i % 50 for i in range(600)], 4, 1)]


@pytest.mark.parametrize("shape", range(3))
@pytest.mark.parametrize("d", [64, 128])
def test_a_q_tile_that_never_comes_ends_the_launch(d, shape):
    """Every wait has a limit; what the kernels behind read of the workspace has been written all the same; the next call is right."""
    lib = af.library()
    call = Call(*SHAPES[shape], d, seed=shape)
    q = call.args[0]
    ws = torch.full((af.attn_paged_workspace(call.bt.B, q.shape[0], call.bt.Hkv, d, q.shape[1], call.bt.max_q),), 255, dtype=torch.uint8, device="cuda")
    assert lib.attn_set_wait_timeout_ns(50_000_000) == 0
    try:
        assert lib.attn_debug_inject(1) == 0
        call(workspace=ws)
        with pytest.raises(af.AttnError) as e:
            af.attn_check()
        assert e.value.status == -4
    finally:
        lib.attn_debug_inject(0)
        lib.attn_set_wait_timeout_ns(0)
    ws.fill_(255)
    call.clear()
    call(workspace=ws)
    af.attn_check()
    call.check()


@pytest.mark.parametrize("nodes,g,d", [([32, 30], 7, 128), ([2, 2, 1], 100, 64), ([80, 75], 3, 64), ([42], 6, 128), ([4, 3], 60, 128)])
def test_groups_that_do_not_fill_a_q_tile(nodes, g, d):
    """Cut units of two Q tiles of fewer than 128 rows each: all rows of the second one are joined."""
    call = Call(nodes, [6000 + 500 * i + m for i, m in enumerate(nodes)], 2 * g, 2, d, words=3, seed=g)
    call()
    af.attn_check()
    call.check()


def test_a_workspace_that_is_too_small_is_refused():
    call = Call(*SHAPES[0], 128)
    n = af.attn_paged_workspace(2, 8, 1, 128, 31, 26)
    with pytest.raises(af.AttnError) as e:
        call(workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -1


@pytest.mark.parametrize("d", [64, 128])
def test_calls_on_three_streams_at_once(d):
    """Attention of trees beside its like and beside rotations, walks and moves: outputs equal those of each call alone."""
    calls = [Call(*s, d, seed=i) for i, s in enumerate(SHAPES)] + [Call([5, 3, 8], [3000, 200, 900], 2, 1, d, seed=9), Call([60] * 9, [700] * 9, 4, 4, d, wl=300, seed=8)]
    want = []
    for c in calls:
        c()
        af.attn_check()
        c.check()
        want.append((c.o.clone(), c.lse.clone()))
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn((12, 900, d), generator=g, device="cuda", dtype=torch.float16)
    inv, pos = (10000.0 ** (-torch.arange(d // 2, device="cuda") / (d / 2.0))).float(), torch.arange(900, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty_like(x[:8]), torch.empty_like(x[8:])
    af.attn_rope(x[:8], x[8:], qo, ko, pos, inv)
    af.attn_check()
    q0, k0 = qo.clone(), ko.clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for rep in range(40):
        for c in calls:
            c.clear()
        qo.zero_(), ko.zero_()
        torch.cuda.synchronize()
        for i in range(len(calls) + 1):
            n = (i + rep) % (len(calls) + 1)
            with torch.cuda.stream(streams[(i * 7 + rep) % 3]):
                if n < len(calls):
                    calls[n]()
                else:
                    af.attn_rope(x[:8], x[8:], qo, ko, pos, inv)
        for st in streams:
            af.attn_check(st)
        for c, (o, lse) in zip(calls, want):
            assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
        assert torch.equal(qo, q0) and torch.equal(ko, k0)
    for st in streams:
        af.attn_release_workspace(st)


def test_two_graphs_at_once():
    """Captured calls without a workspace bring one each: their replays may run side by side."""
    calls = [Call(*SHAPES[0], 128, seed=3), Call(*SHAPES[1], 128, seed=4)]
    want = []
    for c in calls:
        c()
        af.attn_check()
        c.check()
        want.append((c.o.clone(), c.lse.clone()))
    graphs, streams = [], [torch.cuda.Stream() for _ in calls]
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
            c()
        graphs.append(g)
    for _ in range(30):
        for c in calls:
            c.clear()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c, (o, lse) in zip(calls, want):
            assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


def test_a_process_whose_first_calls_are_captured():
    """Nothing that the library sets up on its first call stands in the way of a capture."""
    code = (
        "import torch, attention_forward_07_gb300 as af\n"
        "i = lambda *s: torch.zeros(s, dtype=torch.int32, device='cuda')\n"
        "n = lambda *x: torch.tensor(x, dtype=torch.int32, device='cuda')\n"
        "x = torch.randn((12, 40, 64), device='cuda', dtype=torch.bfloat16)\n"
        "kc = torch.randn((9, 2, 16, 64), device='cuda', dtype=torch.bfloat16)\n"
        "vc, q, o = kc.flip(0).contiguous(), torch.empty_like(x[:8]), torch.empty_like(x[:8])\n"
        "w, inv = torch.ones(64, device='cuda'), torch.ones(32, device='cuda')\n"
        "ctx, new, table, free, cnt = i(2), n(1, 39), i(2, 4), torch.arange(9, dtype=torch.int32, device='cuda'), n(9)\n"
        "left, cu, lens, slots, pos, mask = i(1), i(3), i(2), i(40), i(40), i(40, 2)\n"
        "parents = n(-1, *range(-1, 38))\n"
        "tok, tgt, sure = n(*range(40)), n(*range(1, 41)), n(1, 3)\n"
        "acc, after, nxt, path, src, dst, last = i(2), i(2), i(2), i(2, 5), i(2, 5), i(2, 5), i(1)\n"
        "ws = torch.empty(af.attn_paged_workspace(2, 8, 2, 64, 40, 39), dtype=torch.uint8, device='cuda')\n"
        "def step():\n"
        "    af.attn_paged_tables(ctx, new, table, free, cnt, 16, 9, cu, lens, slots, free_count_out=left)\n"
        "    af.attn_paged_tree(parents, cu, lens, pos, mask)\n"
        "    af.attn_paged_rope(x[:8], x[8:10], x[10:], q, kc, vc, slots, pos, inv, w, w)\n"
        "    af.attn_fwd_paged_tree(q, kc, vc, o, table, cu, lens, 39, mask, scale=0.125, workspace=ws)\n"
        "    af.attn_paged_accept(tok, tgt, parents, cu, lens, table, free, left, 16, 9, acc, after, nxt, path, src, dst, confirmed=sure, free_count_out=last)\n"
        "    af.attn_paged_move(kc, vc, src, dst)\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    step()\n"
        "g.replay()\n"
        "torch.cuda.synchronize()\n"
        "first = o.clone()\n"
        "step()\n"
        "torch.cuda.synchronize()\n"
        "af.attn_check()\n"
        "assert torch.equal(first, o) and first.float().abs().sum() > 0 and torch.isfinite(first.float()).all()\n"
        "assert acc.tolist() == [1, 8] and after.tolist() == [1, 8] and nxt.tolist() == [1, 9] and left.item() == 5 and last.item() == 7\n"
        "print('captured')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]


def test_places_past_32_bits():
    """Pages whose rows begin past 2^31 elements: rotated rows reach them, moves and attention find them."""
    page, Hkv, d, num_pages = 16, 2, 128, 560_000  # 2.3e9 elements a cache
    kc, vc = (torch.empty((num_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = [num_pages - 1, num_pages - 2, 3, num_pages - 5]
    n, ctx = 20, 40
    g = torch.Generator().manual_seed(5)
    x = torch.randn((8 + 2 * Hkv, ctx + n, d), generator=g).bfloat16()
    slots = np.array([ids[p // page] * page + p % page for p in range(ctx + n)])
    assert slots.max() * Hkv * d > 2 ** 31
    qo = torch.empty((8, ctx + n, d), dtype=torch.bfloat16, device="cuda")
    xd = x.cuda()
    af.attn_paged_rope(xd[:8], xd[8:10], xd[10:], qo, kc, vc, _i32(slots), None, None)
    parents = tree_ref.random_parents(n, np.random.default_rng(1))
    pos, mask, _ = tree_ref.tree(parents, [0, n], [ctx + n], 1)
    q, o = qo[:, ctx:], torch.empty((8, n, d), dtype=torch.bfloat16, device="cuda")
    af.attn_fwd_paged_tree(q, kc, vc, o, _i32([ids]), _i32([0, n]), _i32([ctx + n]), n, tree_ref.to_words(mask).cuda(), scale=0.1)
    af.attn_check()
    keep = torch.cat([torch.ones((n, ctx), dtype=torch.bool), torch.from_numpy(mask[:, :n] > 0)], 1)
    for h in range(8):
        k, v = x[8 + h // 4].double(), x[10 + h // 4].double()
        w = torch.softmax((x[h, ctx:].double() @ k.T * 0.1).masked_fill(~keep, -float("inf")), -1)
        # weights and O each rounded to bf16 (half a step, 2^-8), scores and sums in 32 bits (below 2^-10 here)
        assert ((o[h].cpu().double() - w @ v).abs() <= 2.0 ** -8 * (w @ v).abs() + 1.3 * 2.0 ** -8 * (w @ v.abs())).all()
    af.attn_paged_move(kc, vc, _i32([[slots[50], slots[59]]]), _i32([[slots[41], slots[42]]]))
    assert af.attn_check() == 0
    for c, at in ((kc, 8), (vc, 10)):
        for s, p in ((50, 41), (59, 42)):
            assert torch.equal(c[slots[p] // page, :, slots[p] % page].cpu(), x[at:at + Hkv, s])


@pytest.mark.parametrize("lens", [[2 ** 31 - 1, 40], [2 ** 31 - 1, 2 ** 31 - 2], [2 ** 30, 30]])
def test_lengths_up_to_31_bits(lens):
    """Contexts that no table holds: positions and walks as ever, their slots reported, other requests unharmed."""
    rng = np.random.default_rng(3)
    sizes = [20, 25]
    cu = [0, 20, 45]
    parents = np.concatenate([tree_ref.random_parents(m, rng, spread=2) for m in sizes])
    pos, mask = _i32([0] * 45), _i32(np.zeros((45, 1)))
    af.attn_paged_tree(_i32(parents), _i32(cu), _i32(lens), pos, mask)
    af.attn_check()
    pos_ref, mask_ref, _ = tree_ref.tree(parents, cu, lens, 1)
    assert np.array_equal(pos.cpu().numpy(), pos_ref) and np.array_equal(tree_ref.from_words(mask), mask_ref)
    tokens, targets = rng.integers(0, 2, 45), rng.integers(0, 2, 45)
    table = np.array([[5, 3, 1], [0, 2, 4]])
    free = np.array([7, -1, -1, -1, -1, -1, -1, -1])
    ref = tree_ref.accept(tokens, targets, parents, None, cu, lens, table, free, 1, 16, 8, 6)
    out = {k: _i32([-9] * 2) for k in ("accepted", "ctx", "next")} | {k: _i32(np.full((2, 6), -9)) for k in ("path", "src", "dst")}
    f, count = _i32(free), _i32([1])
    af.attn_paged_accept(_i32(tokens), _i32(targets), _i32(parents), _i32(cu), _i32(lens), _i32(table), f, count, 16, 8, out["accepted"], out["ctx"],
                         out["next"], out["path"], out["src"], out["dst"])
    if ref["bad"]:
        with pytest.raises(af.AttnError):
            af.attn_check()
    else:
        af.attn_check()
    for k, v in out.items():
        assert np.array_equal(v.cpu().numpy(), ref[k]), k
    assert np.array_equal(f.cpu().numpy(), ref["free"]) and int(count) == ref["left"]
