"""attn_fwd and attn_fwd_packed captured into graphs: the scratch they work in stays theirs."""
import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af
from attention_forward_07_gb300 import inputs as inp

from paged_ref import Batch

pytestmark = pytest.mark.gpu


class Calls:
    """A masked call and a packed one, with what they give outside a graph."""

    def __init__(self, d, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        S, lens = 400, [300, 70, 513]
        self.q, self.k, self.v = rnd(2, 4, S, d), rnd(2, 4, S, d), rnd(2, 4, S, d)
        self.mask = torch.from_numpy(inp.pack_bits(inp.bernoulli_mask(2, S, seed)).view(np.int32)).cuda()
        n = sum(lens)
        self.pq, self.pk, self.pv = rnd(4, n, d), rnd(2, n, d), rnd(2, n, d)
        self.cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
        self.longest = max(lens)
        self.o, self.po = torch.empty_like(self.q), torch.empty_like(self.pq)
        self.run()
        af.attn_check()
        self.want = self.o.clone(), self.po.clone()

    def run(self):
        af.attn_fwd(self.q, self.k, self.v, self.o, None, self.mask, causal=True, scale=0.1)
        af.attn_fwd_packed(self.pq, self.pk, self.pv, self.po, self.cu, self.cu, self.longest, self.longest, causal=True, scale=0.1)

    def clear(self):
        self.o.fill_(float("nan"))
        self.po.fill_(float("nan"))

    def check(self):
        assert torch.equal(self.o, self.want[0]) and torch.equal(self.po, self.want[1])


def _churn():
    for n in (1 << 20, 1 << 27, 3 << 20):
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("warm", [True, False])
def test_a_graph_keeps_its_scratch_while_the_stream_goes_on(d, warm):
    """Captured after a call on the stream (which has made its workspace) or as the first one, then replayed between calls
    on the stream that need more, paged ones among them, and beside a second graph's replays in turn."""
    a, b = Calls(d, 5), Calls(d, 6)
    bt = Batch([200, 1, 40], [900, 700, 300], 8, 2, d, "bf16", 16, seed=3)
    q, k, v, o, lse = bt.device()
    tabs = bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda()
    s = torch.cuda.Stream()
    af.attn_release_workspace(s)
    torch.cuda.synchronize()
    if warm:
        with torch.cuda.stream(s):
            a.run()
        af.attn_check(s)
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run()
        graphs.append(g)

    def replay():
        for c, g in zip((a, b), graphs):
            c.clear()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                g.replay()
            af.attn_check(s)
            c.check()

    replay()
    for _ in range(3):
        with torch.cuda.stream(s):  # needs more than the forward's calls do
            af.attn_fwd_paged(q, k, v, o, *tabs, bt.max_q, lse=lse, causal=True, scale=0.1)
        af.attn_check(s)
        bt.check(o.cpu(), lse.cpu(), True, -1, -1, 0.1)
        _churn()
        replay()
        a.clear()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            a.run()
        af.attn_check(s)
        a.check()
    del graphs
    af.attn_release_workspace(s)
    torch.cuda.synchronize()
