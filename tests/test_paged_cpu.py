"""The paged-cache operators without a GPU: their refusals, and the plain forms the GPU tests go by."""
import ctypes

import numpy as np
import pytest
import torch

import attention_forward_07_gb300 as af
from attention_forward_07_gb300 import _binding as bd

import paged_ref

P = 0x100000  # never dereferenced: validation comes before any access
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from attention_forward_07_gb300 import build
    build.build()
    return af.library()


TABLES = dict(ctx_lens=P, new_lens=P, block_table=P, free_pages=P, free_count=P, free_count_out=P, cu_seqlens_q=P, seqlens_k=P, slots=P,
              B=2, table_width=4, table_stride=4, max_free=8, max_rows=3, page_size=16, num_pages=8)
APPEND = dict(k_new=P, v_new=P, k_cache=P, v_cache=P, slots=P, k_row_stride=64, k_head_stride=64, v_row_stride=64, v_head_stride=64,
              cache_page_stride=2048, cache_head_stride=1024, cache_row_stride=64, rows=3, Hkv=2, d=64, num_pages=8, page_size=16, dtype=0)
ATTEND = dict(q=P, k_cache=P, v_cache=P, o=P, block_table=P, cu_seqlens_q=P, seqlens_k=P, workspace=P, workspace_bytes=1 << 40,
              q_row_stride=128, q_head_stride=64, o_row_stride=128, o_head_stride=64, cache_page_stride=2048, cache_head_stride=1024,
              cache_row_stride=64, B=2, Hq=2, Hkv=2, d=64, total_q=3, max_seqlen_q=2, num_pages=8, page_size=16, table_width=4,
              table_stride=4, causal=1, window_left=-1, window_right=-1, scale=0.125, dtype=0)

REFUSALS = (
    [("tables", {k: 0}, -1) for k in TABLES if TABLES[k] == P] +
    [("tables", {k: P + 2}, -1) for k in TABLES if TABLES[k] == P] +
    [("tables", kw, -1) for kw in (dict(B=0), dict(B=16385), dict(table_width=0), dict(table_stride=3), dict(max_free=-1), dict(max_rows=0), dict(max_rows=(1 << 30) + 1),
                                   dict(page_size=8), dict(page_size=24), dict(num_pages=0), dict(num_pages=INT_MAX), dict(positions=P + 1))] +
    [("append", {k: 0}, -1) for k in ("k_new", "v_new", "k_cache", "v_cache", "slots")] +
    [("append", {k: P + 8}, -1) for k in ("k_new", "v_new", "k_cache", "v_cache")] +
    [("append", {k: v}, -1) for k in APPEND if k.endswith("stride") for v in (60, -64)] +
    [("append", kw, st) for kw, st in ((dict(cache_row_stride=0), -1), (dict(cache_page_stride=0), -1), (dict(cache_head_stride=0), -1), (dict(d=96), -2), (dict(dtype=2), -2), (dict(rows=0), -1), (dict(Hkv=0), -1), (dict(slots=P + 1), -1),
                                       (dict(page_size=20), -1), (dict(num_pages=INT_MAX), -1))] +
    [("attend", {k: 0}, -1) for k in ATTEND if ATTEND[k] == P and k != "workspace"] +
    [("attend", {k: P + 8}, -1) for k in ("q", "k_cache", "v_cache", "o", "workspace")] +
    [("attend", {k: P + 2}, -1) for k in ("lse", "block_table", "cu_seqlens_q", "seqlens_k")] +
    [("attend", {k: v}, -1) for k in ATTEND if k.endswith("_stride") and k != "table_stride" for v in (60, -64)] +
    [("attend", kw, st) for kw, st in (
        (dict(B=0), -1), (dict(B=16385), -1), (dict(cache_row_stride=0), -1), (dict(cache_page_stride=0), -1), (dict(cache_head_stride=0), -1),
        (dict(cache_page_stride=1536), -2), (dict(num_pages=1 << 27, cache_head_stride=64), -2), (dict(q_head_stride=0), -1), (dict(q_row_stride=0), -1), (dict(o_head_stride=0), -1), (dict(o_row_stride=0), -1), (dict(Hq=3), -1), (dict(Hkv=0), -1), (dict(d=80), -2), (dict(dtype=7), -2), (dict(total_q=0), -1),
        (dict(max_seqlen_q=0), -1), (dict(num_pages=0), -1), (dict(page_size=0), -1), (dict(page_size=8), -1), (dict(page_size=40), -1),
        (dict(table_width=0), -1), (dict(table_stride=3), -1), (dict(window_left=-2), -1), (dict(window_right=-2), -1),
        (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(Hq=258, Hkv=2), -2),
        (dict(table_width=1 << 27, table_stride=1 << 27), -1), (dict(Hq=128, Hkv=1, total_q=1 << 25), -1))] +
    # a scale whose exponent-of-two form is infinite, strides that no memory spans, a row count past the row counter,
    # the library's workspace for a handle (2: the calling thread's default stream) that is a stream per thread
    [("attend", dict(scale=3e38), -1), ("append", dict(rows=(1 << 30) + 1), -1), ("attend", dict(workspace=0, stream=2), -1)] +
    [(op, {k: (1 << 38) + 8}, -1) for op, base in (("append", APPEND), ("attend", ATTEND)) for k in base
     if k.endswith("_stride") and k != "table_stride"])


def _call(lib, op, kw):
    cls, base, fn = {"tables": (bd.PagedTablesParams, TABLES, lib.attn_paged_tables),
                     "append": (bd.PagedAppendParams, APPEND, lib.attn_paged_append),
                     "attend": (bd.FwdPagedParams, ATTEND, lib.attn_fwd_paged)}[op]
    return fn(ctypes.byref(cls(**dict(base, **kw))))


@pytest.mark.parametrize("op,kw,status", REFUSALS, ids=lambda x: str(x).replace(" ", ""))
def test_refusals(lib, op, kw, status):
    assert _call(lib, op, kw) == status


def test_packed_blocks_have_the_structures_layout():
    for fmt, cls in ((bd._TABLES, bd.PagedTablesParams), (bd._APPEND, bd.PagedAppendParams), (bd._ATTEND, bd.FwdPagedParams)):
        assert fmt.size == ctypes.sizeof(cls)
        values = [float(i) if kind is ctypes.c_float else i + 1 for i, (_, kind) in enumerate(cls._fields_)]
        got = cls.from_buffer_copy(fmt.pack(*values))
        assert [getattr(got, name) for name, _ in cls._fields_] == values


def test_null_parameters(lib):
    n = ctypes.c_ulonglong(0)
    assert lib.attn_paged_tables(None) == lib.attn_paged_append(None) == lib.attn_fwd_paged(None) == -1
    assert lib.attn_paged_workspace(None, ctypes.byref(n)) == -1
    assert lib.attn_paged_workspace(ctypes.byref(bd.FwdPagedParams(**ATTEND)), None) == -1
    assert lib.attn_paged_workspace(ctypes.byref(bd.FwdPagedParams(**dict(ATTEND, d=32))), ctypes.byref(n)) == -2


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_valid_calls_without_a_device(lib):
    for op in ("tables", "append", "attend"):
        assert _call(lib, op, {}) == -5
    with pytest.raises(af.AttnError):
        af.attn_paged_workspace(1, 8, 2, 128, 1, 1)


def test_status_has_a_text(lib):
    assert af.attn_strerror(-6) == "page id, slot or page count out of range"


def test_the_binding_refuses_what_it_can_see():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    kc, q = h(4, 2, 16, 64), h(4, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        af.attn_paged_append(h(2, 3, 64), h(2, 3, 64), kc, kc, i(3))
    with pytest.raises(ValueError, match="CUDA"):
        af.attn_paged_tables(i(2), i(2), i(2, 4), i(9), i(1), 16, 9, i(3), i(2), i(5))
    with pytest.raises(ValueError, match="CUDA"):
        af.attn_fwd_paged(q, kc, kc, q.clone(), i(2, 4), i(3), i(2), 2)
    with pytest.raises(TypeError):
        af.attn_paged_append(h(2, 3, 64).float(), h(2, 3, 64), kc, kc, i(3))
    for bad in (dict(k=h(2, 4, 64)), dict(k=h(2, 3, 128)), dict(kc=h(4, 2, 16, 128)[..., ::2]), dict(vc=h(5, 2, 16, 64)),
                dict(vc=h(4, 16, 2, 64).transpose(1, 2)), dict(slots=i(3).long()), dict(slots=i(3, 1))):
        a = dict(k=h(2, 3, 64), kc=kc, vc=kc, slots=i(3), **{}) | bad
        with pytest.raises(ValueError):
            af.attn_paged_append(a["k"], h(2, 3, 64), a["kc"], a["vc"], a["slots"])
    for bad in (dict(cu=i(2)), dict(table=i(3, 4)), dict(table=i(2, 8)[:, ::2]), dict(o=h(4, 2, 64)), dict(o=q.bfloat16()),
                dict(lse=torch.zeros(4, 2)), dict(lse=torch.zeros(4, 3, dtype=torch.float64)), dict(q=h(4, 3, 128))):
        a = dict(q=q, o=q.clone(), table=i(2, 4), cu=i(3), lse=None) | bad
        with pytest.raises(ValueError):
            af.attn_fwd_paged(a["q"], kc, kc, a["o"], a["table"], a["cu"], i(2), 2, lse=a["lse"])
    with pytest.raises(ValueError):
        af.attn_paged_tables(i(2), i(2), i(2, 4), i(9), i(1), 16, 9, i(2), i(2), i(5))
    with pytest.raises(ValueError):
        af.attn_paged_tables(i(2), i(3), i(2, 4), i(9), i(1), 16, 9, i(3), i(2), i(5))


def test_every_tensor_of_the_tables_is_looked_at(monkeypatch):
    """Each wrong type, length, stride or rank of each argument is refused (the launch itself is replaced)."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = dict(ctx_lens=i(2), new_lens=i(2), block_table=i(2, 4), free_pages=i(9), free_count=i(1), cu_seqlens_q=i(3), seqlens_k=i(2),
                slots=i(5), positions=i(5), free_count_out=i(1))
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    bd._with_torch()
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    launched = []
    monkeypatch.setattr(bd, "_launch", lambda index, fn, block: launched.append(block))
    af.attn_paged_tables(**good, page_size=16, num_pages=9)
    assert len(launched) == 1
    for name, t in good.items():
        longer = i(*[n + 1 for n in t.shape])
        wrong = [t.long(), t[None], i(*[2 * n + 2 for n in t.shape])[tuple(slice(0, 2 * n, 2) for n in t.shape)]]
        if name not in ("free_pages", "slots"):  # (whose own length is what they hold)
            wrong.append(longer if name != "block_table" else i(3, 4))
        for bad in wrong:
            if name in ("free_count", "free_count_out") and bad.shape == (1,) and bad.dtype is torch.int32:
                continue  # one entry has no stride
            if name == "slots" and bad.dtype is torch.int32 and bad.is_contiguous() and bad.dim() == 1:
                continue
            with pytest.raises(ValueError):
                af.attn_paged_tables(**dict(good, **{name: bad}), page_size=16, num_pages=9)
    assert len(launched) == 1


# ---- the plain forms themselves, against the oracle and by hand
def test_plain_attention_against_the_oracle():
    import oracle
    from attention_forward_07_gb300 import inputs as inp
    Hq, Hkv, d, page = 4, 2, 64, 16
    for sq, sk, causal, wl, wr in ((1, 70, True, -1, -1), (37, 90, True, 20, -1), (20, 50, False, 7, 3)):
        bt = paged_ref.Batch([sq], [sk], Hq, Hkv, d, "f16", page, seed=sk)
        o, lse, _, _ = paged_ref.attention(bt.q, bt.k, bt.v, bt.table, bt.cu, bt.lens, sq, causal, wl, wr, 0.125)
        ids = bt.table[0, :paged_ref.pages(sk, page)].long()
        k, v = (c[ids].transpose(0, 1).reshape(Hkv, -1, d)[:, :sk][None].contiguous() for c in (bt.k, bt.v))
        ro, rl = oracle.attn_rows_ex(inp.as_u16(bt.q[None]), inp.as_u16(k), inp.as_u16(v), inp.F16, None, None, False, causal, wl, wr, 0.125)
        assert np.allclose(o.numpy(), ro[0], rtol=0, atol=1e-12) and np.allclose(lse.numpy(), rl[0], rtol=0, atol=1e-12)


def test_plain_tables_by_hand():
    t = np.array([[7, -1, -1], [3, 4, -1]], np.int32)
    r = paged_ref.tables([10, 32], [8, 2], t, np.array([0, 1, 2, 5]), 4, 16, 9, 12)
    assert r["table"].tolist() == [[7, 5, -1], [3, 4, 2]] and r["left"] == 2 and not r["bad"]
    assert r["cu"].tolist() == [0, 8, 10] and r["lens"].tolist() == [18, 34]
    assert r["slots"].tolist() == [122, 123, 124, 125, 126, 127, 80, 81, 32, 33, -1, -1]
    assert r["positions"].tolist() == [10, 11, 12, 13, 14, 15, 16, 17, 32, 33, -1, -1]
