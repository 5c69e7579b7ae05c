"""Edges of the paged-cache operators that need no GPU: whose workspace a captured call takes, how kernels that start early
read, empty lists and maps, sizes past what is counted, what tells weights in two parts from weights in one, and
that no C entry lets an exception out."""
import contextlib
import ctypes
import os
import re
import types

import pytest
import torch

import attention_forward_07_gb300 as af
from attention_forward_07_gb300 import _binding as bd

import paged_bounds
from test_paged_cpu import ATTEND, P, TABLES, lib  # noqa: F401


# ---- the workspace of a call that is being captured
class _Streams:
    """Stands in for torch's streams: a current one, some that are being captured, and what was allocated on which."""

    def __init__(self, monkeypatch, captured, status=-1):
        self.status = status
        self.current, self.taken, self.blocks = self.make(1), [], []
        self.captured = captured
        empty = torch.empty

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before

        def taking(*a, **kw):
            if kw.get("dtype") is torch.uint8:
                self.taken.append((self.current.cuda_stream, a[0]))
            return empty(*a, **kw)

        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "device", lambda i: contextlib.nullcontext())
        monkeypatch.setattr(torch.cuda, "current_stream", lambda i=None: self.current)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.current.cuda_stream in self.captured)
        monkeypatch.setattr(torch, "empty", taking)
        bd._with_torch()
        monkeypatch.setattr(bd, "_raw_stream", lambda i: self.current.cuda_stream)
        monkeypatch.setattr(bd, "_device", lambda: 0)
        monkeypatch.setattr(bd, "_workspace_bytes", lambda shape: 512)
        monkeypatch.setattr(bd, "_lib", types.SimpleNamespace(attn_fwd_paged=None, attn_strerror=lambda status: b"refused"))
        monkeypatch.setattr(bd, "_launch", self.launch)

    def launch(self, index, fn, block):
        """As the library: no launch on a captured stream without a workspace."""
        prm = bd.FwdPagedParams.from_buffer_copy(block)
        if prm.workspace is None and prm.stream in self.captured:
            raise bd.AttnError(self.status, "attn_fwd_paged")
        self.blocks.append(prm)

    @staticmethod
    def make(handle):
        return types.SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", 0))


@pytest.mark.parametrize("captured,on,taken_on", [
    ((), None, None), ((), 2, None),
    ((1,), None, 1), ((1, 2, 3), 2, 2), ((1, 2, 3), 3, 3),   # streams forked from the one that is captured
    ((2,), 2, 2),                                            # captured, and not the current one
    ((1,), 2, None)])                                        # the current one is captured, the launch goes elsewhere
@pytest.mark.parametrize("own", [False, True])
def test_a_captured_call_takes_its_workspace_on_the_stream_it_runs_on(monkeypatch, captured, on, taken_on, own):
    st = _Streams(monkeypatch, captured)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kc = torch.zeros((4, 3, 64)).half(), torch.zeros((4, 2, 16, 64)).half()
    ws = torch.zeros(768, dtype=torch.uint8) if own else None
    af.attn_fwd_paged(q, kc, kc, q.clone(), i(2, 4), i(3), i(2), 2, stream=on and st.make(on), workspace=ws)
    (block,) = st.blocks
    assert (block.stream or 0) == (on or 1)
    if own:  # the caller's, whatever is captured
        assert not st.taken and (block.workspace, block.workspace_bytes) == (ws.data_ptr(), 768)
        return
    assert st.taken == ([] if taken_on is None else [(taken_on, 512)])
    assert block.workspace_bytes == (0 if taken_on is None else 512) and (block.workspace is None) == (taken_on is None)
    assert st.current.cuda_stream == 1


@pytest.mark.parametrize("captured,status", [((), -1), ((1,), -3)])
def test_other_refusals_come_through(monkeypatch, captured, status):
    """What is refused outside a capture, or for another reason, is not tried again."""
    st = _Streams(monkeypatch, captured, status)
    tried = []

    def launch(index, fn, block):
        tried.append(block)
        raise bd.AttnError(status, "attn_fwd_paged")

    monkeypatch.setattr(bd, "_launch", launch)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, kc = torch.zeros((4, 3, 64)).half(), torch.zeros((4, 2, 16, 64)).half()
    with pytest.raises(af.AttnError) as e:
        af.attn_fwd_paged(q, kc, kc, q.clone(), i(2, 4), i(3), i(2), 2)
    assert e.value.status == status and len(tried) == 1 and not st.taken


# ---- kernels that start before the one ahead has ended
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_07_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//.*", "", f.read())


@pytest.mark.parametrize("name", ["paged.cuh", "paged_attn.cu", "paged_tile.cu", "paged_cache.cu"])
def test_the_paged_kernels_read_nothing_as_constant_for_their_life(name):
    """Any input may be what the kernel ahead on the stream writes, after this one has started."""
    text = _code(name)
    assert "__ldg" not in text and ".nc" not in text and "__restrict__" not in text


def test_the_forward_reads_its_own_lists_with_plain_loads():
    """Work order, slot list, liveness and flags come from the dependent kernels ahead."""
    text = _code("attn_fwd.cu")
    assert not re.search(r"__ldg\((p\.order|p\.rowmap|rm\b|p\.live|p\.tflags|flags16)", text)
    assert not re.search(r"const \w+\* __restrict__ (flags16|live|rowmap|tflags|order)\b", text)


# ---- empty lists and maps
@pytest.mark.parametrize("kw,status", [
    (dict(free_pages=0, max_free=0), -5), (dict(slots=0, max_rows=0), -5), (dict(free_pages=0, max_free=0, slots=0, max_rows=0), -5),
    (dict(free_pages=0, max_free=1), -1), (dict(slots=0, max_rows=1), -1), (dict(slots=0, max_rows=0, positions=P), -1),
    (dict(slots=0, max_rows=-1), -1), (dict(slots=P, max_rows=0), -1)], ids=str)
@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are none: what is accepted must find no device")
def test_tables_without_free_pages_or_rows(lib, kw, status):  # noqa: F811
    assert lib.attn_paged_tables(ctypes.byref(bd.PagedTablesParams(**dict(TABLES, **kw)))) == status


@pytest.mark.parametrize("free,rows", [(0, 5), (9, 0), (0, 0)])
@pytest.mark.parametrize("positions", [False, True])
def test_empty_tensors_become_null(monkeypatch, free, rows, positions):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    bd._with_torch()
    monkeypatch.setattr(bd, "_raw_stream", lambda index: 0)
    got = []
    monkeypatch.setattr(bd, "_launch", lambda index, fn, block: got.append(bd.PagedTablesParams.from_buffer_copy(block)))
    # (slices of longer tensors: an empty slice may have an address)
    af.attn_paged_tables(i(2), i(2), i(2, 4), i(9)[:free], i(1), 16, 9, i(3), i(2), i(5)[:rows], i(5)[:rows] if positions else None)
    assert (got[0].max_free, got[0].max_rows) == (free, rows)
    assert (got[0].free_pages is None) == (free == 0) and (got[0].slots is None) == (rows == 0)
    assert (got[0].positions is None) == (rows == 0 or not positions)


# ---- sizes past what is counted
@pytest.mark.parametrize("kw", [dict(total_q=2 ** 31 - 1, max_seqlen_q=2 ** 31 - 1), dict(total_q=2 ** 30, max_seqlen_q=1),
                                dict(Hq=128, Hkv=1, total_q=1 << 25, max_seqlen_q=64)], ids=str)
def test_no_workspace_size_for_what_the_attention_refuses(lib, kw):  # noqa: F811
    n = ctypes.c_ulonglong(77)
    prm = bd.FwdPagedParams(**dict(ATTEND, **kw))
    assert lib.attn_paged_workspace(ctypes.byref(prm), ctypes.byref(n)) == -1 and n.value == 77
    assert lib.attn_fwd_paged(ctypes.byref(prm)) == -1


# ---- weights in two parts
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", range(len(paged_bounds.CASES)))
def test_the_bound_for_two_parts_tells_them_from_one(case, dtype):
    """Emulated in 64 bits: with the remainder's product O is within the bound, without it far from it."""
    bt = paged_bounds.batch(paged_bounds.CASES[case], dtype, seed=case)
    over = {1: 0, 2: 0}
    n = 0
    for parts in over:
        for (rows, o, bound, *_), (_, got) in zip(paged_bounds.exact(bt), paged_bounds.emulated(bt, parts)):
            over[parts] += int(((got - o).abs() > bound).sum())
            n += o.numel() if parts == 2 else 0
    assert over[2] == 0 and over[1] > n // 50


# ---- C entries
def test_c_entries_turn_exceptions_into_a_status():
    """Whatever allocates on the host or takes a lock runs inside entry(), in all of the library's C functions."""
    seen = set()
    for name in ("attn_fwd.cu", "paged_attn.cu", "paged_cache.cu"):
        text = _code(name)
        for fn, body in re.findall(r"\nint (attn_\w+)\([^)]*\) {\n(.*?)\n}\n", text[text.index('extern "C"'):], flags=re.S):
            if re.search(r"fwd_impl|stream_state|host_|Plan\b", body):
                seen.add(fn)
                assert re.search(r"return attn::entry\(", body), fn
    assert seen == {"attn_fwd", "attn_fwd_ex", "attn_fwd_visited", "attn_fwd_noalloc", "attn_check", "attn_release_workspace",
                    "attn_paged_tables", "attn_paged_append", "attn_fwd_paged", "attn_paged_workspace"}
