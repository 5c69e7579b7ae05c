"""attn_fwd_paged_tree at random: groups that do and do not fill a Q tile, masks of trees and of any bits, windows, chunks, idle requests, fewer
keys than nodes, pages of any size, workspaces full of rubbish."""
import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

import tree_ref
from paged_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(48))
def test_random_batch(seed):
    rng = np.random.default_rng(seed + 100)
    pick = lambda *x: x[int(rng.integers(len(x)))]  # noqa: E731
    while True:
        g = pick(1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 25, 32, 64, 100, 128)
        Hkv, d, words, B = pick(1, 2, 4) if g < 16 else 1, pick(64, 128), pick(1, 1, 2, 3, 8), pick(1, 1, 2, 3, 5, 9, 30)
        top = int(rng.integers(1, 32 * words + 1))
        nodes = rng.integers(min(pick(0, 1, top), top), top + 1, B).tolist()
        if rng.random() < 0.25:
            nodes[int(rng.integers(B))] = 32 * words + int(rng.integers(1, 200))
        most = int(np.exp(rng.uniform(0, np.log(5000 if B < 6 else 800))))
        keys = [max(0, m + int(rng.integers(-m - 1 if rng.random() < 0.05 else 0, most + 1))) for m in nodes]
        if sum(nodes) and sum(nodes) * g * Hkv * max(keys) < 2e7:
            break
    page, wl = pick(16, 32, 48, 64, 112, 128, 256), pick(-1, -1, -1, 0, 1, 17, 100, 1000)
    bt = Batch(nodes, keys, g * Hkv, Hkv, d, pick("bf16", "f16"), page, seed=seed, fill=float("nan") if sum(keys) < 2000 else "randn",
               rows=pick("tokens", "heads"), cache=pick("tokens", "heads"), spare_rows=pick(0, 0, 3, 40))
    n = bt.q.shape[1]
    if rng.random() < 0.5:
        parents = np.concatenate([tree_ref.random_parents(m, rng) for m in nodes] + [np.full(n - sum(nodes), -1)])
        pos, mask, _ = tree_ref.tree(parents, bt.cu.tolist(), keys, words)
        mask = np.maximum(mask, 0)
    else:
        mask = (rng.random((n, 32 * words)) < rng.choice([0.0, 0.05, 0.5, 1.0], (n, 1))).astype(np.int64)
        at = np.concatenate([np.arange(m) + k - m for m, k in zip(nodes, keys)] + [np.zeros(n - sum(nodes))]).astype(np.int64)
        pos = at + rng.integers(-30, 30, n)
    scale, max_q = float(np.float32(d ** -0.5)), max(1, max(nodes) + pick(0, 0, 5, 100))
    q, k, v, o, lse = bt.device()
    wide = torch.full((n, words + pick(0, 1, 2)), -1, dtype=torch.int32, device="cuda")
    wide[:, :words] = tree_ref.to_words(mask).cuda()
    ws = torch.full((af.attn_paged_workspace(B, g * Hkv, Hkv, d, n, max_q),), 255, dtype=torch.uint8, device="cuda") if rng.random() < 0.5 else None
    af.attn_fwd_paged_tree(q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), max_q, wide[:, :words], lse=lse, window_left=wl, scale=scale,
                           positions=torch.tensor(pos, dtype=torch.int32, device="cuda"), workspace=ws)
    af.attn_check()
    tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask, words, pos, wl, scale, max_q, what=str((nodes[:6], keys[:6], g, Hkv, d, words, page, wl)))
