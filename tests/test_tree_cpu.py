"""The operators of drafted trees without a GPU: their refusals, their parameter blocks, and the plain forms the GPU tests go by."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af
from attention_forward_07_gb300 import _binding as bd

import tree_ref
from test_paged_cpu import ATTEND, INT_MAX, P, lib  # noqa: F401

ROPE = dict(q=P, k=P, v=P, q_out=P, k_out=0, k_cache=P, v_cache=P, q_weight=P, k_weight=P, positions=P, slots=P, inv_freq=P, q_row_stride=128,
            q_head_stride=64, k_row_stride=128, k_head_stride=64, v_row_stride=128, v_head_stride=64, q_out_row_stride=128, q_out_head_stride=64,
            k_out_row_stride=0, k_out_head_stride=0, cache_page_stride=2048, cache_head_stride=1024, cache_row_stride=64, position_stride=3, rows=3,
            Hq=2, Hkv=2, d=64, rot_dim=64, axes=2, interleaved=0, weight_f32=0, num_pages=8, page_size=16, eps=1e-6, dtype=1)
BUFFERS = dict(slots=0, v=0, k_cache=0, v_cache=0, k_out=P, k_out_row_stride=128, k_out_head_stride=64, num_pages=0, page_size=0, cache_row_stride=0)
TREE = dict(parents=P, cu_seqlens_q=P, seqlens_k=P, positions=P, tree_mask=P, B=2, rows=5, mask_words=2, mask_stride=2, window_left=-1)
ACCEPT = dict(tokens=P, targets=P, parents=P, confirmed=P, cu_seqlens_q=P, seqlens_k=P, block_table=P, free_pages=P, free_count=P, free_count_out=P,
              accepted=P, ctx_lens=P, next_tokens=P, path=P, src_slots=P, dst_slots=P, B=2, rows=5, max_path=4, table_width=4, table_stride=4,
              max_free=8, page_size=16, num_pages=8)
MOVE = dict(k_cache=P, v_cache=P, src_slots=P, dst_slots=P, cache_layer_stride=16384, cache_page_stride=2048, cache_head_stride=1024,
            cache_row_stride=64, layers=2, lists=2, length=4, Hkv=2, d=64, num_pages=8, page_size=16, dtype=0)
MASKED = dict(tree_mask=P, positions=P, mask_words=2, mask_stride=2)

REFUSALS = (
    [("rope", {k: 0}, -1) for k in ("q", "k", "v", "q_out", "k_cache", "v_cache", "positions", "inv_freq")] +
    [("rope", {k: P + 8}, -1) for k in ("q", "k", "v", "q_out", "k_cache", "v_cache")] +
    [("rope", {k: P + 2}, -1) for k in ("positions", "inv_freq", "slots")] +
    [("rope", {k: P + 1}, -1) for k in ("q_weight", "k_weight")] + [("rope", dict(q_weight=P + 2, weight_f32=1), -1)] +
    [("rope", {k: v}, -1) for k in ROPE if k.endswith("stride") and k != "position_stride" and not k.startswith("k_out") for v in (60, -64, (1 << 38) + 8)] +
    [("rope", {k: 0}, -1) for k in ("q_out_row_stride", "q_out_head_stride", "cache_page_stride", "cache_head_stride", "cache_row_stride")] +
    [("rope", kw, st) for kw, st in (
        (dict(d=96), -2), (dict(dtype=2), -2), (dict(rows=0), -1), (dict(rows=(1 << 30) + 1), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1),
        (dict(Hq=(1 << 16) + 1), -1), (dict(rot_dim=8), -1), (dict(rot_dim=80), -1), (dict(rot_dim=-16), -1), (dict(axes=0), -1), (dict(axes=5), -1),
        (dict(position_stride=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(num_pages=0), -1),
        (dict(page_size=24), -1), (dict(num_pages=INT_MAX), -1))] +
    [("rope", dict(BUFFERS, **kw), -1) for kw in (dict(k_out=0), dict(k_out=P + 8), dict(k_out_row_stride=0), dict(k_out_head_stride=0),
                                                  dict(k_out_row_stride=60), dict(k_out_head_stride=-8))] +
    [("tree", {k: v}, -1) for k in TREE if TREE[k] == P for v in (0, P + 2)] +
    [("tree", kw, -1) for kw in (dict(B=0), dict(B=16385), dict(rows=0), dict(rows=(1 << 30) + 1), dict(mask_words=0), dict(mask_words=33, mask_stride=33),
                                 dict(mask_stride=1), dict(window_left=-2))] +
    [("accept", {k: 0}, -1) for k in ACCEPT if ACCEPT[k] == P and k not in ("confirmed", "free_pages")] +
    [("accept", {k: P + 2}, -1) for k in ACCEPT if ACCEPT[k] == P] + [("accept", dict(free_pages=0), -1)] +
    [("accept", kw, -1) for kw in (dict(B=0), dict(B=16385), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(max_path=0), dict(max_path=1025),
                                   dict(table_width=0), dict(table_stride=3), dict(max_free=0), dict(page_size=8), dict(num_pages=0),
                                   dict(num_pages=INT_MAX), dict(table_width=1 << 27, table_stride=1 << 27))] +
    [("move", {k: v}, -1) for k in ("k_cache", "v_cache") for v in (0, P + 8)] + [("move", {k: v}, -1) for k in ("src_slots", "dst_slots") for v in (0, P + 2)] +
    [("move", {k: v}, -1) for k in MOVE if k.endswith("stride") for v in (0, 60, -64, (1 << 38) + 8)] +
    [("move", kw, st) for kw, st in ((dict(d=32), -2), (dict(dtype=5), -2), (dict(layers=0), -1), (dict(lists=0), -1), (dict(length=0), -1), (dict(Hkv=0), -1),
                                     (dict(layers=(1 << 16) + 1), -1), (dict(lists=(1 << 20) + 1), -1), (dict(length=(1 << 20) + 1), -1),
                                     (dict(num_pages=0), -1), (dict(page_size=20), -1), (dict(num_pages=INT_MAX), -1))] +
    [("attend", kw, -1) for kw in (dict(tree_mask=0), dict(tree_mask=P + 2), dict(positions=P + 2), dict(mask_words=0), dict(mask_words=(1 << 20) + 1, mask_stride=1 << 21),
                                   dict(mask_stride=1), dict(call=dict(causal=0)), dict(call=dict(window_left=5), positions=0), dict(call=dict(q=0)),
                                   dict(call=dict(scale=0.0)), dict(call=dict(workspace=0, stream=2)))] +
    [("attend", dict(call=dict(d=80)), -2)])


def _block(op, kw):
    if op == "attend":
        kw = dict(kw)
        call = bd.FwdPagedParams(**dict(ATTEND, **kw.pop("call", {})))
        return bd.FwdPagedTreeParams(call=call, **dict(MASKED, **kw))
    cls, base = {"rope": (bd.RopeParams, ROPE), "tree": (bd.PagedTreeParams, TREE), "accept": (bd.PagedAcceptParams, ACCEPT),
                 "move": (bd.PagedMoveParams, MOVE)}[op]
    return cls(**dict(base, **kw))


def _call(lib, op, kw):  # noqa: F811
    fn = {"rope": lib.attn_rope, "tree": lib.attn_paged_tree, "accept": lib.attn_paged_accept, "move": lib.attn_paged_move,
          "attend": lib.attn_fwd_paged_tree}[op]
    return fn(ctypes.byref(_block(op, kw)))


@pytest.mark.parametrize("op,kw,status", REFUSALS, ids=lambda x: str(x).replace(" ", ""))
def test_refusals(lib, op, kw, status):  # noqa: F811
    assert _call(lib, op, kw) == status


def test_null_parameters(lib):  # noqa: F811
    assert lib.attn_rope(None) == lib.attn_paged_tree(None) == lib.attn_fwd_paged_tree(None) == lib.attn_paged_accept(None) == lib.attn_paged_move(None) == -1


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device(lib):  # noqa: F811
    for op, kw in (("rope", {}), ("rope", BUFFERS), ("rope", dict(rot_dim=0, positions=0, inv_freq=0, axes=0)), ("rope", dict(q_weight=0, k_weight=0)),
                   ("tree", {}), ("accept", {}), ("accept", dict(confirmed=0)), ("accept", dict(free_pages=0, max_free=0, free_count=0, free_count_out=0)),
                   ("accept", dict(rows=0, tokens=0, targets=0, parents=0)), ("move", {}), ("move", dict(layers=1, cache_layer_stride=0)), ("attend", {}),
                   ("attend", dict(positions=0)), ("attend", dict(call=dict(window_left=5)))):
        assert _call(lib, op, kw) == -5, (op, kw)


def test_packed_blocks_have_the_structures_layout():
    def flat(cls):
        return [x for name, kind in cls._fields_ for x in (flat(kind) if isinstance(kind, type) and issubclass(kind, ctypes.Structure) else [kind])]

    def values(s):
        return [x for name, kind in s._fields_ for x in (values(getattr(s, name)) if issubclass(kind, ctypes.Structure) else [getattr(s, name)])]

    for fmts, cls in (((bd._ROPE,), bd.RopeParams), ((bd._TREE,), bd.PagedTreeParams), ((bd._ACCEPT,), bd.PagedAcceptParams), ((bd._MOVE,), bd.PagedMoveParams),
                      ((bd._ATTEND, bd._MASK), bd.FwdPagedTreeParams)):
        assert sum(f.size for f in fmts) == ctypes.sizeof(cls)
        want = [float(i) if kind is ctypes.c_float else i + 1 for i, kind in enumerate(flat(cls))]
        first = len(flat(bd.FwdPagedParams))
        raw = fmts[0].pack(*want) if len(fmts) == 1 else fmts[0].pack(*want[:first]) + fmts[1].pack(*want[first:])
        assert values(cls.from_buffer_copy(raw)) == want


def test_the_binding_refuses_what_it_can_see():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    f = lambda *s: torch.zeros(s)  # noqa: E731
    kc, q, k = h(4, 2, 16, 64), h(4, 3, 64), h(2, 3, 64)
    ok = dict(positions=i(3), inv=f(32))
    for kw in ({}, dict(positions=i(4)), dict(positions=i(3).long()), dict(inv=f(32).double()), dict(positions=i(2, 3)), dict(inv=f(2, 32)),
               dict(wq=h(32)), dict(wq=f(64), wk=h(64)), dict(ko=h(2, 4, 64)), dict(qo=h(4, 3, 128)), dict(qo=q.bfloat16())):
        a = dict(ok, qo=q.clone(), ko=k.clone(), wq=None, wk=None) | kw
        with pytest.raises(ValueError):
            af.attn_rope(q, k, a["qo"], a["ko"], a["positions"], a["inv"], a["wq"], a["wk"])
    for kw in ({}, dict(v=h(2, 4, 64)), dict(slots=i(4)), dict(kc=h(4, 3, 16, 64)), dict(vc=h(4, 16, 2, 64).transpose(1, 2))):
        a = dict(v=k, slots=i(3), kc=kc, vc=kc) | kw
        with pytest.raises(ValueError):
            af.attn_paged_rope(q, k, a["v"], q.clone(), a["kc"], a["vc"], a["slots"], i(3), f(32))
    with pytest.raises(TypeError):
        af.attn_rope(q.float(), k.float(), q.float(), k.float(), i(3), f(32))
    for kw in ({}, dict(mask=i(4, 2)), dict(mask=i(5, 2).long()), dict(mask=i(5, 4)[:, ::2]), dict(cu=i(2)), dict(pos=i(4))):
        a = dict(mask=i(5, 2), cu=i(3), pos=i(5)) | kw
        with pytest.raises(ValueError):
            af.attn_paged_tree(i(5), a["cu"], i(2), a["pos"], a["mask"])
    for kw in ({}, dict(path=i(2, 5)), dict(path=i(3, 4)), dict(free=i(0)), dict(targets=i(4)), dict(table=i(2, 8)[:, ::2]), dict(confirmed=i(3))):
        a = dict(path=i(2, 4), free=i(9), targets=i(5), table=i(2, 4), confirmed=None) | kw
        with pytest.raises(ValueError):
            af.attn_paged_accept(i(5), a["targets"], i(5), i(3), i(2), a["table"], a["free"], i(1), 16, 9, i(2), i(2), i(2), a["path"], i(2, 4), i(2, 4),
                                 confirmed=a["confirmed"])
    for kw in ({}, dict(src=i(2, 5)), dict(src=i(8)), dict(vc=h(4, 2, 16, 128)), dict(src=i(2, 4).long())):
        a = dict(src=i(2, 4), vc=kc) | kw
        with pytest.raises(ValueError):
            af.attn_paged_move(kc, a["vc"], a["src"], i(2, 4))
    for kw in ({}, dict(mask=i(4, 2)), dict(mask=i(3, 2).long()), dict(pos=i(4)), dict(mask=i(3, 4)[:, ::2])):
        a = dict(mask=i(3, 2), pos=i(3)) | kw
        with pytest.raises(ValueError):
            af.attn_fwd_paged_tree(q, kc, kc, q.clone(), i(2, 4), i(3), i(2), 2, a["mask"], positions=a["pos"])


# ------------------------------------------------------------------------------ plain forms
def test_plain_tree_and_words():
    #        0
    #     1     2
    #    3 4    5     (and a second request of two nodes, the second without a parent)
    parents = np.array([-1, 0, 0, 1, 1, 2, -1, -1])
    pos, mask, bad = tree_ref.tree(parents, [0, 6, 8], [106, 2], 1)
    assert pos.tolist() == [100, 101, 101, 102, 102, 102, 0, 0] and not bad
    assert tree_ref.to_words(mask)[:, 0].tolist() == [1, 3, 5, 11, 19, 37, 1, 2]
    assert np.array_equal(tree_ref.from_words(tree_ref.to_words(mask)), mask)
    _, near, _ = tree_ref.tree(parents, [0, 6, 8], [106, 2], 1, window=1)
    assert tree_ref.to_words(near)[:, 0].tolist() == [1, 3, 5, 10, 18, 36, 1, 2]
    assert tree_ref.tree(np.array([0, 0]), [0, 2], [2], 1)[2]


def test_plain_walk():
    parents, tokens = np.array([-1, 0, 0, 1, 2, 2, 4]), np.array([5, 7, 8, 9, 9, 9, 3])
    targets = np.array([8, 0, 9, 0, 3, 0, 77])
    out = tree_ref.accept(tokens, targets, parents, None, [0, 7], [40], np.array([[3, 1, 2]]), np.array([9, -1, -1]), 1, 16, 10, 4)
    assert out["path"].tolist() == [[2, 4, 6, -1]] and out["next"].tolist() == [77] and out["accepted"].tolist() == [4] and out["ctx"].tolist() == [37]
    # context 33: node 2 lies at 35, in page 2 (its id is 2) row 3, and goes to 34
    assert out["src"].tolist() == [[35, 37, 39, -1]] and out["dst"].tolist() == [[34, 35, 36, -1]] and out["left"] == 1 and not out["bad"]
    out = tree_ref.accept(tokens, targets * 0 - 1, parents, [7], [0, 7], [40], np.array([[3, 1, 2]]), None, 0, 16, 10, 4)
    assert out["accepted"].tolist() == [7] and out["next"].tolist() == [-1] and out["ctx"].tolist() == [40]


def test_plain_rotation_keeps_lengths_and_the_bound_tells_a_wrong_pairing():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((2, 5, 64), generator=g).half()
    pos, inv = torch.randint(0, 10 ** 6, (1, 5), generator=g), 10000.0 ** (-torch.arange(16) / 16.0)[None]
    y, tol = tree_ref.rope(x, None, pos, inv, 0.0, False, torch.float16)
    assert torch.allclose(y.square().sum(-1), x.double().square().sum(-1)) and torch.equal(y[..., 32:], x[..., 32:].double())
    z, _ = tree_ref.rope(x, None, pos, inv, 0.0, True, torch.float16)
    assert ((y - z).abs() > tol)[..., :32].float().mean() > 0.9
    assert ((y.half().double() - y).abs() <= tol).all()
