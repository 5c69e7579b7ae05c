"""attn_fwd_paged_tree with infinite keys in places that no row's mask keeps, on the paths of few rows and of many: O whole, not only finite."""
import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af

import tree_ref
from paged_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes,g,words", [([4, 3], 4, 1), ([1, 4, 2], 4, 1), ([16, 9], 1, 1), ([30, 32], 1, 1), ([40, 3], 4, 2), ([64, 50, 7], 8, 2)])
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16"), (128, "f16"), (64, "bf16")])
@pytest.mark.parametrize("wl", [-1, 30])
def test_infinite_keys_that_no_mask_keeps(nodes, g, words, d, dtype, wl):
    """At most 16 packed rows, 32 of one head, more than either; nodes 1 and the last are kept by no row.  The bound's score sizes go by kept keys."""
    keys = [200 + 37 * i + m for i, m in enumerate(nodes)]
    bt = Batch(nodes, keys, 2 * g, 2, d, dtype, 16, seed=g + d)
    n = sum(nodes)
    parents = np.concatenate([tree_ref.random_parents(m, np.random.default_rng(m)) for m in nodes])
    pos, mask, _ = tree_ref.tree(parents, bt.cu.tolist(), keys, words)
    mask = np.maximum(mask, 0)
    for b, m in enumerate(nodes):
        for j in {1, m - 1} - {0, m}:
            mask[int(bt.cu[b]):int(bt.cu[b + 1]), j] = 0
            at = keys[b] - m + j
            bt.k[int(bt.table[b, at // 16]), :, at % 16] = float("inf") if (b + j) % 2 else -float("inf")
    assert not torch.isfinite(bt.k.float()).all()
    q, k, v, o, lse = bt.device()
    scale = float(np.float32(d ** -0.5))
    af.attn_fwd_paged_tree(q, k, v, o, bt.table.cuda(), bt.cu.cuda(), bt.lens.cuda(), bt.max_q, tree_ref.to_words(mask).cuda(),
                           positions=torch.tensor(pos[:n], dtype=torch.int32, device="cuda"), lse=lse, window_left=wl, scale=scale)
    af.attn_check()
    tree_ref.check_attention(bt, o.cpu(), lse.cpu(), mask, words, pos, wl, scale, what=str((nodes, g, d)))
