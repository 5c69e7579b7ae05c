"""ctypes binding over libattn.so (the C-ABI in include/attn.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the launch stream, and non-zero status codes become
``AttnError``.  Every step of the computation runs in the library's kernels.
The library is loaded on first use; if it is missing or cannot be loaded the
call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

ATTN_F16 = 0
ATTN_BF16 = 1
ATTN_ERR_INVALID = -1

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libattn.so"
_lock = threading.Lock()
_lib = None

# The symbols include/attn.h declares (checked by the CPU test-suite).
EXPORTS = (
    "attn_fwd",
    "attn_fwd_visited",
    "attn_fwd_noalloc",
    "attn_fwd_ex",
    "attn_paged_tables",
    "attn_paged_append",
    "attn_fwd_paged",
    "attn_paged_workspace",
    "attn_rope",
    "attn_paged_tree",
    "attn_fwd_paged_tree",
    "attn_paged_accept",
    "attn_paged_move",
    "attn_check",
    "attn_release_workspace",
    "attn_debug_counters",
    "attn_strerror",
    "attn_tile_shape",
    "attn_set_wait_timeout_ns",
    "attn_debug_inject",
    "attn_version",
)


class FwdParams(ctypes.Structure):
    """attn_fwd_params_t of include/attn.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("o", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("mask_bits", ctypes.c_void_p), ("mask_per_head", ctypes.c_int),
                ("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("Sq", ctypes.c_int),
                ("Sk", ctypes.c_int), ("d", ctypes.c_int), ("causal", ctypes.c_int), ("window_left", ctypes.c_int),
                ("window_right", ctypes.c_int), ("scale", ctypes.c_float), ("dtype", ctypes.c_int),
                ("stream", ctypes.c_void_p), ("visited", ctypes.c_void_p), ("seqlens_q", ctypes.c_void_p),
                ("seqlens_k", ctypes.c_void_p), ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
                ("max_seqlen_q", ctypes.c_int), ("max_seqlen_k", ctypes.c_int)]


def _fields(text):
    """A struct's fields from 'type: names' lines; p = pointer, i = int, l = long long, u = unsigned long long, f = float."""
    kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int, "l": ctypes.c_longlong, "u": ctypes.c_ulonglong, "f": ctypes.c_float}
    return [(name, kinds[kind]) for kind, names in (line.split(":") for line in text.strip().splitlines()) for name in names.split()]


class PagedTablesParams(ctypes.Structure):
    """attn_paged_tables_params_t of include/attn.h."""
    _fields_ = _fields("""p: ctx_lens new_lens block_table free_pages free_count free_count_out cu_seqlens_q seqlens_k slots positions
i: B table_width table_stride max_free max_rows page_size num_pages
p: stream""")


class PagedAppendParams(ctypes.Structure):
    """attn_paged_append_params_t of include/attn.h."""
    _fields_ = _fields("""p: k_new v_new k_cache v_cache slots
l: k_row_stride k_head_stride v_row_stride v_head_stride cache_page_stride cache_head_stride cache_row_stride
i: rows Hkv d num_pages page_size dtype
p: stream""")


class FwdPagedParams(ctypes.Structure):
    """attn_fwd_paged_params_t of include/attn.h."""
    _fields_ = _fields("""p: q k_cache v_cache o lse block_table cu_seqlens_q seqlens_k workspace
u: workspace_bytes
l: q_row_stride q_head_stride o_row_stride o_head_stride cache_page_stride cache_head_stride cache_row_stride
i: B Hq Hkv d total_q max_seqlen_q num_pages page_size table_width table_stride causal window_left window_right
f: scale
i: dtype
p: stream""")


class RopeParams(ctypes.Structure):
    """attn_rope_params_t of include/attn.h."""
    _fields_ = _fields("""p: q k v q_out k_out k_cache v_cache q_weight k_weight positions slots inv_freq
l: q_row_stride q_head_stride k_row_stride k_head_stride v_row_stride v_head_stride q_out_row_stride q_out_head_stride
l: k_out_row_stride k_out_head_stride cache_page_stride cache_head_stride cache_row_stride position_stride
i: rows Hq Hkv d rot_dim axes interleaved weight_f32 num_pages page_size
f: eps
i: dtype
p: stream""")


class PagedTreeParams(ctypes.Structure):
    """attn_paged_tree_params_t of include/attn.h."""
    _fields_ = _fields("""p: parents cu_seqlens_q seqlens_k positions tree_mask
i: B rows mask_words mask_stride window_left
p: stream""")


class FwdPagedTreeParams(ctypes.Structure):
    """attn_fwd_paged_tree_params_t of include/attn.h."""
    _fields_ = [("call", FwdPagedParams)] + _fields("""p: tree_mask positions
i: mask_words mask_stride""")


class PagedAcceptParams(ctypes.Structure):
    """attn_paged_accept_params_t of include/attn.h."""
    _fields_ = _fields("""p: tokens targets parents confirmed cu_seqlens_q seqlens_k block_table free_pages free_count free_count_out
p: accepted ctx_lens next_tokens path src_slots dst_slots
i: B rows max_path table_width table_stride max_free page_size num_pages
p: stream""")


class PagedMoveParams(ctypes.Structure):
    """attn_paged_move_params_t of include/attn.h."""
    _fields_ = _fields("""p: k_cache v_cache src_slots dst_slots
l: cache_layer_stride cache_page_stride cache_head_stride cache_row_stride
i: layers lists length Hkv d num_pages page_size dtype
p: stream""")


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {attn_strerror(status)} ({status})")


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def library():
    """Load libattn.so (built in-tree by __graft_entry__.build()); raise if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        p, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        fwd_args = [p, p, p, p, p, p, i, i, i, i, i, i, f, i, p]
        lib.attn_fwd.argtypes = fwd_args
        lib.attn_fwd.restype = i
        lib.attn_fwd_visited.argtypes = fwd_args + [p]
        lib.attn_fwd_visited.restype = i
        lib.attn_fwd_noalloc.argtypes = fwd_args
        lib.attn_fwd_noalloc.restype = i
        lib.attn_fwd_ex.argtypes = [ctypes.POINTER(FwdParams)]
        lib.attn_fwd_ex.restype = i
        # (parameter blocks as bytes or by reference)
        lib.attn_paged_tables.argtypes = [p]
        lib.attn_paged_tables.restype = i
        lib.attn_paged_append.argtypes = [p]
        lib.attn_paged_append.restype = i
        lib.attn_fwd_paged.argtypes = [p]
        lib.attn_fwd_paged.restype = i
        for fn in (lib.attn_rope, lib.attn_paged_tree, lib.attn_fwd_paged_tree, lib.attn_paged_accept, lib.attn_paged_move):
            fn.argtypes = [p]
            fn.restype = i
        lib.attn_paged_workspace.argtypes = [p, ctypes.POINTER(ctypes.c_ulonglong)]
        lib.attn_paged_workspace.restype = i
        lib.attn_check.argtypes = [p]
        lib.attn_check.restype = i
        lib.attn_release_workspace.argtypes = [p]
        lib.attn_release_workspace.restype = i
        lib.attn_debug_counters.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), i]
        lib.attn_debug_counters.restype = i
        lib.attn_strerror.argtypes = [i]
        lib.attn_strerror.restype = ctypes.c_char_p
        lib.attn_tile_shape.argtypes = [i, ctypes.POINTER(i), ctypes.POINTER(i)]
        lib.attn_tile_shape.restype = i
        lib.attn_set_wait_timeout_ns.argtypes = [ctypes.c_ulonglong]
        lib.attn_set_wait_timeout_ns.restype = i
        lib.attn_debug_inject.argtypes = [i]
        lib.attn_debug_inject.restype = i
        lib.attn_version.argtypes = []
        lib.attn_version.restype = i
        _lib = lib
        return lib


def attn_strerror(status: int) -> str:
    return library().attn_strerror(int(status)).decode()


def _dtype_code(t) -> int:
    torch = _torch or _with_torch()
    if t.dtype == torch.float16:
        return ATTN_F16
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; fp16 or bf16 expected")


def _lens_ptr(t, B):
    import torch
    if t.dtype != torch.int32 or t.numel() != B or not t.is_contiguous():
        raise ValueError("sequence lengths must be a contiguous int32 tensor of B entries")
    return t.data_ptr()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _call(fn, q, k, v, o, lse, mask_bits, causal, scale, stream, extra=()):
    """q/o: [B,Hq,S,d]; k/v: [B,Hkv,S,d]; lse: fp32 [B,Hq,S] or None;
    mask_bits: int32/uint32 [B,S,ceil(S/32)] or None.  Shapes are taken from q and k."""
    B, Hq, S, d = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = 1.0 / (d ** 0.5)
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(mask_bits), int(B), int(Hq), int(Hkv),
            int(S), int(d), int(bool(causal)), ctypes.c_float(scale), _dtype_code(q), _stream_handle(stream),
            *extra)
    if rc != 0:
        raise AttnError(rc, fn.__name__)


def attn_fwd(q, k, v, o, lse=None, mask_bits=None, causal=False, scale=None, stream=None):
    """Launch the fused forward on `stream` (default: torch's current stream).

    The caller owns every tensor (device memory, contiguous, [B,H,S,d]); the
    call is asynchronous; use attn_check() to collect in-kernel errors."""
    lib = library()
    _call(lib.attn_fwd, q, k, v, o, lse, mask_bits, causal, scale, stream)


def attn_fwd_visited(q, k, v, o, lse, mask_bits, causal, scale, visited, stream=None):
    """attn_fwd that also sets visited[b, hq, qtile, ktile] = 1 (uint8) for every
    (query tile, key tile) block the kernel computed; the caller zeroes it first."""
    lib = library()
    _call(lib.attn_fwd_visited, q, k, v, o, lse, mask_bits, causal, scale, stream, extra=(_ptr(visited),))


def attn_fwd_noalloc(q, k, v, o, lse=None, mask_bits=None, causal=False, scale=None, stream=None):
    """attn_fwd for callers that may not allocate device memory: a custom mask's
    pre-pass output goes into a fixed array the library reserves per GPU (see
    include/attn.h for the size limit and the rules on sharing it)."""
    lib = library()
    _call(lib.attn_fwd_noalloc, q, k, v, o, lse, mask_bits, causal, scale, stream)


def attn_fwd_ex(q, k, v, o, lse=None, mask_bits=None, mask_per_head=False, causal=False, window_left=-1,
                window_right=-1, scale=None, visited=None, stream=None, seqlens_q=None, seqlens_k=None):
    """Generalised forward: q/o [B,Hq,Sq,d], k/v [B,Hkv,Sk,d] with Sk >= Sq (bottom-right
    aligned), a band of kept keys (window_left / window_right, -1 = unbounded), custom masks
    [B,Sq,ceil(Sk/32)] or per head [B,Hq,Sq,ceil(Sk/32)], per-entry lengths seqlens_q /
    seqlens_k (int32 device tensors [B]); see include/attn.h."""
    B, Hq, Sq, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / (d ** 0.5)
    prm = FwdParams(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), o=o.data_ptr(),
                    lse=None if lse is None else lse.data_ptr(),
                    mask_bits=None if mask_bits is None else mask_bits.data_ptr(),
                    mask_per_head=int(bool(mask_per_head)), B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, d=d,
                    causal=int(bool(causal)), window_left=int(window_left), window_right=int(window_right),
                    scale=float(scale), dtype=_dtype_code(q), stream=_stream_handle(stream).value,
                    visited=None if visited is None else visited.data_ptr(),
                    seqlens_q=None if seqlens_q is None else _lens_ptr(seqlens_q, B),
                    seqlens_k=None if seqlens_k is None else _lens_ptr(seqlens_k, B))
    rc = library().attn_fwd_ex(ctypes.byref(prm))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_ex")


def attn_fwd_packed(q, k, v, o, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, lse=None, causal=False,
                    window_left=-1, window_right=-1, scale=None, visited=None, stream=None):
    """attn_fwd_ex over packed variable-length batches: q/o [Hq, total_q, d], k/v [Hkv, total_k, d],
    lse [Hq, total_q]; cu_seqlens_q / cu_seqlens_k int32 device tensors [B+1] of row offsets;
    max_seqlen_q / max_seqlen_k bound the entries' lengths.  See include/attn.h."""
    Hq, Sq, d = q.shape
    Hkv, Sk = k.shape[0], k.shape[1]
    B = cu_seqlens_q.numel() - 1
    if scale is None:
        scale = 1.0 / (d ** 0.5)
    prm = FwdParams(q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), o=o.data_ptr(),
                    lse=None if lse is None else lse.data_ptr(), mask_bits=None, mask_per_head=0,
                    B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, d=d, causal=int(bool(causal)),
                    window_left=int(window_left), window_right=int(window_right), scale=float(scale),
                    dtype=_dtype_code(q), stream=_stream_handle(stream).value,
                    visited=None if visited is None else visited.data_ptr(),
                    cu_seqlens_q=_lens_ptr(cu_seqlens_q, B + 1), cu_seqlens_k=_lens_ptr(cu_seqlens_k, B + 1),
                    max_seqlen_q=int(max_seqlen_q), max_seqlen_k=int(max_seqlen_k))
    rc = library().attn_fwd_ex(ctypes.byref(prm))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_ex")


# The paged operators are called once or more per layer and decoding step, where a microsecond counts: their parameter blocks
# are packed as bytes (in the layout of the structures above), each tensor is asked only for what is checked, all checks of a
# call stand in one condition, and what is wrong is worked out only once that has failed.
_TABLES = struct.Struct("@10P7iP")
_APPEND = struct.Struct("@5P7q6iP")
_ATTEND = struct.Struct("@9PQ7q13ifiP")
_MASK = struct.Struct("@2P2i")  # what follows _ATTEND in attn_fwd_paged_tree's
_ROPE = struct.Struct("@12P14q10ifiP")
_TREE = struct.Struct("@5P5iP")
_ACCEPT = struct.Struct("@16P8iP")
_MOVE = struct.Struct("@4P4q8iP")
_torch = None
_raw_stream = None
_device = None


def _with_torch():
    """torch, imported on first use (with it the cheapest ways it has to name a device's current stream and the current
    device, once there are CUDA tensors)."""
    global _torch, _raw_stream, _device
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
        _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch = torch
    return _torch


def _stream_on(index, stream):
    """Handle of `stream`, checked to be on CUDA device `index`."""
    if stream.device.index != index:
        raise ValueError(f"the tensors are on CUDA device {index}, the stream is on {stream.device}")
    return stream.cuda_stream


def _launch(index, fn, block):
    """Calls fn(block) with CUDA device `index` current; raises on a status other than 0."""
    if _device() == index:
        rc = fn(block)
    else:
        with _torch.cuda.device(index):
            rc = fn(block)
    if rc != 0:
        raise AttnError(rc, fn.__name__)


def _refuse(index, vectors=(), table=None, rows=(), caches=None, others=()):
    """Raises for the first of the tensors that is not as its caller wants it.  vectors: (tensor, entries, name); table:
    (tensor, B); rows: (tensor, shape, dtype, name); caches: (k, v, dtype, d); others: (wrong, what is wanted)."""
    i32 = _torch.int32
    if index < 0:
        raise ValueError("the paged operators take CUDA tensors")
    for t, n, name in vectors:
        if t.dtype is not i32 or t.get_device() != index or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 vector of {n} entries on CUDA device {index}")
    if table is not None:
        raise_if = table[0].dtype is not i32 or table[0].get_device() != index or table[0].dim() != 2 or table[0].shape[0] != table[1]
        if raise_if or (table[0].shape[1] > 1 and table[0].stride(1) != 1):
            raise ValueError(f"block_table must be int32 [{table[1]}, pages] on CUDA device {index}, each row contiguous")
    for t, shape, dtype, name in rows:
        if t.dtype is not dtype or t.get_device() != index or t.shape != shape or t.stride(-1) != 1:
            raise ValueError(f"{name} must be {dtype} {tuple(shape)} on CUDA device {index}, its last dimension contiguous")
    if caches is not None:
        k, v, dtype, d = caches
        raise ValueError(f"k_cache and v_cache must be {dtype} [num_pages, Hkv, page_size, {d}] on CUDA device {index}, of the same "
                         f"strides, their last dimension contiguous; got {tuple(k.shape)} and {tuple(v.shape)}")
    for wrong, wanted in others:
        if wrong:
            raise ValueError(wanted)


def attn_paged_tables(ctx_lens, new_lens, block_table, free_pages, free_count, page_size, num_pages, cu_seqlens_q, seqlens_k,
                      slots, positions=None, free_count_out=None, stream=None):
    """Block tables, slot map, positions and row offsets of a serving step from its requests' lengths.

    int32 device tensors: ctx_lens, new_lens [B] (tokens cached, tokens to come), block_table [B, W] (in / out: the
    pages added are filled in), free_pages [F] with free_count [1] (taken from the end) -> cu_seqlens_q [B+1],
    seqlens_k [B], slots and positions [max rows] (-1 behind the last new row), free_count_out [1] (default: free_count
    itself).  free_pages and slots may be empty.  See include/attn.h."""
    torch = _torch or _with_torch()
    i32, index = torch.int32, ctx_lens.get_device()
    one, many, after = ctx_lens.shape, slots.shape, cu_seqlens_q.shape
    (B,), (rows,), (free,) = one, many, free_pages.shape
    left = free_count if free_count_out is None else free_count_out
    width = block_table.shape[-1]
    if (index < 0 or not ctx_lens.dtype is new_lens.dtype is free_pages.dtype is free_count.dtype is left.dtype is cu_seqlens_q.dtype is
            seqlens_k.dtype is slots.dtype is block_table.dtype is i32 or
            not index == new_lens.get_device() == free_pages.get_device() == free_count.get_device() == left.get_device() ==
            cu_seqlens_q.get_device() == seqlens_k.get_device() == slots.get_device() == block_table.get_device() or
            not (ctx_lens.is_contiguous() and new_lens.is_contiguous() and free_pages.is_contiguous() and cu_seqlens_q.is_contiguous() and
                 seqlens_k.is_contiguous() and slots.is_contiguous()) or
            new_lens.shape != one or seqlens_k.shape != one or free_count.shape != (1,) or left.shape != (1,) or after != (B + 1,) or
            block_table.dim() != 2 or block_table.shape[0] != B or (block_table.stride(1) != 1 and width > 1) or
            (positions is not None and (positions.dtype is not i32 or positions.get_device() != index or positions.shape != many or
                                        not positions.is_contiguous()))):
        _refuse(index, ((ctx_lens, B, "ctx_lens"), (new_lens, B, "new_lens"), (free_pages, free, "free_pages"),
                        (free_count, 1, "free_count"), (left, 1, "free_count_out"), (cu_seqlens_q, B + 1, "cu_seqlens_q"),
                        (seqlens_k, B, "seqlens_k"), (slots, rows, "slots")) +
                (() if positions is None else ((positions, rows, "positions"),)), (block_table, B))
    _launch(index, (_lib or library()).attn_paged_tables,
            _TABLES.pack(ctx_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr() if free else 0,
                         free_count.data_ptr(), left.data_ptr(), cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(),
                         slots.data_ptr() if rows else 0, 0 if positions is None or not rows else positions.data_ptr(), B, width,
                         block_table.stride(0) if B > 1 else width, free, rows, page_size, num_pages, _raw_stream(index) if stream is None else _stream_on(index, stream)))


def attn_paged_append(k_new, v_new, k_cache, v_cache, slots, stream=None):
    """Write new rows k_new, v_new [Hkv, rows, d] to their slots (int32 [rows]; negative: left out) of the caches
    [num_pages, Hkv, page_size, d].  Any strides whose last dimension is contiguous; see include/attn.h."""
    torch = _torch or _with_torch()
    dtype, index = k_new.dtype, k_new.get_device()
    code = _dtype_code(k_new)
    cs, ks, vs = k_cache.stride(), k_new.stride(), v_new.stride()
    (rows,) = slots.shape
    if (index < 0 or len(cs) != 4 or k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.get_device() != index or
            v_cache.get_device() != index or v_cache.shape != k_cache.shape or v_cache.stride() != cs or cs[3] != 1):
        _refuse(index, caches=(k_cache, v_cache, dtype, "d"))
    num_pages, Hkv, page_size, d = k_cache.shape
    shape = (Hkv, rows, d)
    if (v_new.dtype is not dtype or v_new.get_device() != index or k_new.shape != shape or v_new.shape != shape or ks[2] != 1 or
            vs[2] != 1 or slots.dtype is not torch.int32 or slots.get_device() != index or not slots.is_contiguous()):
        _refuse(index, ((slots, rows, "slots"),), rows=((k_new, shape, dtype, "k_new"), (v_new, shape, dtype, "v_new")))
    handle = _raw_stream(index) if stream is None else _stream_on(index, stream)
    if rows == 0:
        return
    _launch(index, (_lib or library()).attn_paged_append,
            _APPEND.pack(k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), slots.data_ptr(), ks[1], ks[0], vs[1],
                         vs[0], cs[0], cs[1], cs[2], rows, Hkv, d, num_pages, page_size, code, handle))


def attn_fwd_paged(q, k_cache, v_cache, o, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q, lse=None, causal=False,
                   window_left=-1, window_right=-1, scale=None, workspace=None, stream=None):
    """Attention of packed query rows over a paged cache: q/o [Hq, total_q, d], caches [num_pages, Hkv, page_size, d] (any
    strides whose last dimension is contiguous), lse fp32 [Hq, total_q] or None; block_table int32 [B, W], cu_seqlens_q
    int32 [B+1], seqlens_k int32 [B] (keys per request, the new rows' own included).  One token per request, a few or whole
    chunks, mixed freely.  workspace: a uint8 tensor of attn_paged_workspace() bytes for calls that do not run at the same
    time; None uses the stream's own, or, while the stream is being captured, one of the call's own from the graph's memory
    pool.  See include/attn.h."""
    _fwd_paged(None, q, k_cache, v_cache, o, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q, lse, causal, window_left, window_right, scale,
               workspace, stream)


def attn_fwd_paged_tree(q, k_cache, v_cache, o, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q, tree_mask, positions=None, lse=None,
                        window_left=-1, scale=None, workspace=None, stream=None):
    """attn_fwd_paged with a mask among each request's new rows, as for drafted trees: a row sees its context (within
    window_left of its position) and new row j of its request iff bit j of its row of tree_mask is set (int32 [total_q, words], rows
    contiguous).  positions: int32 [total_q], wanted with a window.  Requests of more than 32 * words rows are chunks, causal.
    See include/attn.h."""
    if (tree_mask.dtype is not (_torch or _with_torch()).int32 or tree_mask.get_device() != q.get_device() or tree_mask.dim() != 2 or
            tree_mask.shape[0] != q.shape[1] or (tree_mask.stride(1) != 1 and tree_mask.shape[1] > 1)):
        raise ValueError(f"tree_mask must be int32 [{q.shape[1]}, words] on q's device, each row contiguous")
    if positions is not None:
        if (positions.dtype is not _torch.int32 or positions.get_device() != q.get_device() or positions.shape != (q.shape[1],) or
                not positions.is_contiguous()):
            raise ValueError(f"positions must be a contiguous int32 vector of {q.shape[1]} entries on q's device")
    words = tree_mask.shape[1]
    mask = _MASK.pack(tree_mask.data_ptr(), 0 if positions is None else positions.data_ptr(), words,
                      tree_mask.stride(0) if tree_mask.shape[0] > 1 else words)
    _fwd_paged(mask, q, k_cache, v_cache, o, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q, lse, True, window_left, -1, scale, workspace,
               stream)


def _fwd_paged(mask, q, k_cache, v_cache, o, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q, lse, causal, window_left, window_right, scale,
               workspace, stream):
    """attn_fwd_paged, or, with the packed fields of a mask, attn_fwd_paged_tree."""
    torch = _torch or _with_torch()
    dtype, index, i32 = q.dtype, q.get_device(), torch.int32
    code = _dtype_code(q)
    shape, qs, ost, cs = q.shape, q.stride(), o.stride(), k_cache.stride()
    Hq, total_q, d = shape
    (B,) = seqlens_k.shape
    if (index < 0 or len(cs) != 4 or k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.get_device() != index or
            v_cache.get_device() != index or v_cache.shape != k_cache.shape or v_cache.stride() != cs or cs[3] != 1 or
            k_cache.shape[3] != d):
        _refuse(index, caches=(k_cache, v_cache, dtype, d))
    num_pages, Hkv, page_size, _ = k_cache.shape
    if (o.dtype is not dtype or o.get_device() != index or o.shape != shape or qs[2] != 1 or ost[2] != 1 or
            cu_seqlens_q.dtype is not i32 or cu_seqlens_q.get_device() != index or cu_seqlens_q.shape != (B + 1,) or
            not cu_seqlens_q.is_contiguous() or seqlens_k.dtype is not i32 or seqlens_k.get_device() != index or
            not seqlens_k.is_contiguous() or block_table.dtype is not i32 or block_table.get_device() != index or
            block_table.dim() != 2 or block_table.shape[0] != B or (block_table.stride(1) != 1 and block_table.shape[1] > 1) or
            (lse is not None and (lse.dtype is not torch.float32 or lse.get_device() != index or lse.shape != (Hq, total_q) or
                                  not lse.is_contiguous()))):
        _refuse(index, ((cu_seqlens_q, B + 1, "cu_seqlens_q"), (seqlens_k, B, "seqlens_k")), (block_table, B),
                ((q, shape, dtype, "q"), (o, shape, dtype, "o")),
                others=((True, f"lse must be contiguous fp32 {(Hq, total_q)} on CUDA device {index}"),))
    handle = _raw_stream(index) if stream is None else _stream_on(index, stream)
    if total_q == 0:
        return
    width = block_table.shape[1]
    lib = _lib or library()
    fn = lib.attn_fwd_paged if mask is None else lib.attn_fwd_paged_tree

    def block(at, n):
        call = _ATTEND.pack(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), o.data_ptr(), 0 if lse is None else lse.data_ptr(),
                            block_table.data_ptr(), cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), at, n, qs[1], qs[0],
                            ost[1], ost[0], cs[0], cs[1], cs[2], B, Hq, Hkv, d, total_q, max_seqlen_q, num_pages, page_size, width,
                            block_table.stride(0) if B > 1 else width, 1 if causal else 0, window_left, window_right,
                            d ** -0.5 if scale is None else scale, code, handle)
        return call if mask is None else call + mask

    if workspace is None:
        try:
            return _launch(index, fn, block(0, 0))  # in the library's own of the stream
        except AttnError as e:
            if e.status != ATTN_ERR_INVALID:
                raise
            # Captured, a call needs one that nothing beside it uses, and the library refuses it without: it gets one from
            # the graph's memory pool, taken with the launch stream current.  A block that is given back is handed out again
            # in the order of the stream it was taken on, and is this call's alone only if that is the stream that runs it.
            with torch.cuda.stream(torch.cuda.current_stream(index) if stream is None else stream):
                if not torch.cuda.is_current_stream_capturing():
                    raise
                workspace = torch.empty(_workspace_bytes((B, Hq, Hkv, d, total_q, max_seqlen_q)), dtype=torch.uint8, device=q.device)
    _refuse(index, others=((workspace.get_device() != index or not workspace.is_contiguous(),
                            f"workspace must be contiguous and on CUDA device {index}"),))
    _launch(index, fn, block(workspace.data_ptr(), workspace.numel() * workspace.element_size()))


def _workspace_bytes(shape) -> int:
    B, Hq, Hkv, d, total_q, max_seqlen_q = shape
    n = ctypes.c_ulonglong(0)
    prm = FwdPagedParams(B=B, Hq=Hq, Hkv=Hkv, d=d, total_q=total_q, max_seqlen_q=max_seqlen_q)
    rc = library().attn_paged_workspace(ctypes.byref(prm), ctypes.byref(n))
    if rc != 0:
        raise AttnError(rc, "attn_paged_workspace")
    return n.value


def attn_paged_workspace(B, Hq, Hkv, d, total_q, max_seqlen_q) -> int:
    """Bytes of workspace attn_fwd_paged wants on the current device."""
    return _workspace_bytes((B, Hq, Hkv, d, total_q, max_seqlen_q))


def _one(t, n):
    """Whether t is anything but a contiguous vector of n entries."""
    return t.shape != (n,) or not t.is_contiguous()


def _refuse_rope(index, dtype, q, k, v, outs, slots, positions, inv_freq, weights):
    """Raises for what attn_rope and attn_paged_rope cannot take (outs: (tensor, heads, name))."""
    Hq, rows, d = q.shape
    Hkv = k.shape[0]
    kv = (Hkv, rows, d)
    if inv_freq is not None:
        axes = 1 if inv_freq.dim() == 1 else inv_freq.shape[0]
        wanted = (rows,) if axes == 1 and (positions is None or positions.dim() == 1) else (axes, rows)
        _refuse(index, others=((positions is None or positions.dtype is not _torch.int32 or positions.get_device() != index or positions.shape != wanted or
                                (rows > 1 and positions.stride(-1) != 1), f"positions must be int32 {wanted} on CUDA device {index}, each axis contiguous"),
                               (inv_freq.dtype is not _torch.float32 or inv_freq.get_device() != index or not inv_freq.is_contiguous() or inv_freq.dim() > 2,
                                f"inv_freq must be contiguous fp32 [pairs] or [axes, pairs] on CUDA device {index}")))
    f32 = any(w is not None and w.dtype is _torch.float32 for w, _ in weights)
    for w, name in weights:
        if w is not None and (w.dtype is not (_torch.float32 if f32 else dtype) or w.get_device() != index or _one(w, d)):
            raise ValueError(f"{name} must be a contiguous vector of {d} entries of {dtype} or (both weights) fp32 on CUDA device {index}")
    _refuse(index, () if slots is None else ((slots, rows, "slots"),),
            rows=((q, (Hq, rows, d), dtype, "q"), (k, kv, dtype, "k")) + (() if v is None else ((v, kv, dtype, "v"),)) +
            tuple((t, (heads, rows, d), dtype, name) for t, heads, name in outs))


def _rope_shared(q, k, positions, inv_freq, q_weight, k_weight, dtype, index, rows, d):
    """What both calls check and pack alike: (wrong, pairs turned, axes, from an axis to the next, addresses, whether weights are fp32)."""
    f32 = _torch.float32
    wrong = k.dtype is not dtype or k.get_device() != index
    rot = axes = step = at_pos = at_inv = at_q = at_k = 0
    if inv_freq is not None:
        shape = inv_freq.shape
        axes, pairs = (1, shape[0]) if len(shape) == 1 else shape if len(shape) == 2 else (0, 0)
        rot = 2 * pairs
        if positions is None:
            return True, 0, 0, 0, 0, 0, 0, 0, False
        ps = positions.shape
        wrong = (wrong or inv_freq.dtype is not f32 or inv_freq.get_device() != index or not inv_freq.is_contiguous() or axes == 0 or
                 positions.dtype is not _torch.int32 or positions.get_device() != index or
                 (ps != (axes, rows) if len(ps) != 1 else axes != 1 or ps[0] != rows) or (rows > 1 and positions.stride(-1) != 1))
        step = positions.stride(0) if axes > 1 and not wrong else rows
        at_pos, at_inv = positions.data_ptr(), inv_freq.data_ptr()
    fp32 = False
    if q_weight is not None:
        fp32 = q_weight.dtype is f32
        wrong = (wrong or (not fp32 and q_weight.dtype is not dtype) or q_weight.get_device() != index or q_weight.shape != (d,) or
                 not q_weight.is_contiguous())
        at_q = q_weight.data_ptr()
    if k_weight is not None:
        mine = k_weight.dtype
        wrong = (wrong or (mine is not q_weight.dtype if q_weight is not None else mine is not f32 and mine is not dtype) or
                 k_weight.get_device() != index or k_weight.shape != (d,) or not k_weight.is_contiguous())
        fp32 = fp32 or mine is f32
        at_k = k_weight.data_ptr()
    return wrong, rot, axes, step, at_pos, at_inv, at_q, at_k, fp32


def attn_rope(q, k, q_out, k_out, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, stream=None):
    """Norms of queries and keys for each head (where there are weights, [d] of q's type or fp32) and their rotation by position,
    in one pass: q, q_out [Hq, rows, d], k, k_out [Hkv, rows, d], any strides whose last dimension is contiguous; an output may be
    its input.  positions int32 [rows] with inv_freq fp32 [pairs], or [axes, rows] (each axis contiguous, or one row expanded) with [axes, pairs],
    whose columns hold a pair's frequency in its axis and 0 elsewhere; pairs are halves' or, interleaved, neighbours', and elements past 2 * pairs are not
    turned.  inv_freq None: norms alone.  A contiguous [B, H, S, d] of shared positions goes in as view(B * H, S, d).  See include/attn.h."""
    _torch or _with_torch()
    dtype, index, shape = q.dtype, q.get_device(), q.shape
    code = _dtype_code(q)
    Hq, rows, d = shape
    kv = k.shape
    Hkv = kv[0]
    qs, ks, qo, ko = q.stride(), k.stride(), q_out.stride(), k_out.stride()
    wrong, rot, axes, step, at_pos, at_inv, at_q, at_k, fp32 = _rope_shared(q, k, positions, inv_freq, q_weight, k_weight, dtype, index, rows, d)
    if (wrong or index < 0 or kv != (Hkv, rows, d) or q_out.shape != shape or k_out.shape != kv or not qs[2] == ks[2] == qo[2] == ko[2] == 1 or
            not q_out.dtype is k_out.dtype is dtype or not index == q_out.get_device() == k_out.get_device()):
        _refuse_rope(index, dtype, q, k, None, ((q_out, Hq, "q_out"), (k_out, Hkv, "k_out")), None, positions, inv_freq,
                     ((q_weight, "q_weight"), (k_weight, "k_weight")))
    handle = _raw_stream(index) if stream is None else _stream_on(index, stream)
    if rows == 0:
        return
    _launch(index, (_lib or library()).attn_rope,
            _ROPE.pack(q.data_ptr(), k.data_ptr(), 0, q_out.data_ptr(), k_out.data_ptr(), 0, 0, at_q, at_k, at_pos, 0, at_inv, qs[1], qs[0], ks[1], ks[0], 0,
                       0, qo[1], qo[0], ko[1], ko[0], 0, 0, 0, step, rows, Hq, Hkv, d, rot, axes, 1 if interleaved else 0, fp32, 0, 0, eps, code, handle))


def attn_paged_rope(q, k, v, q_out, k_cache, v_cache, slots, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                    stream=None):
    """attn_rope whose keys go, with the values v [Hkv, rows, d], to their slots (int32 [rows]) of the caches [num_pages, Hkv, page_size, d];
    rows of negative slots are left out, of q_out too.  See include/attn.h."""
    i32 = (_torch or _with_torch()).int32
    dtype, index, shape = q.dtype, q.get_device(), q.shape
    code = _dtype_code(q)
    Hq, rows, d = shape
    kv = k.shape
    Hkv = kv[0]
    cache, cs = k_cache.shape, k_cache.stride()
    if (index < 0 or len(cs) != 4 or k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.get_device() != index or
            v_cache.get_device() != index or v_cache.shape != cache or v_cache.stride() != cs or cs[3] != 1 or cache[1] != Hkv or cache[3] != d):
        _refuse(index, caches=(k_cache, v_cache, dtype, d))
    qs, ks, vs, qo = q.stride(), k.stride(), v.stride(), q_out.stride()
    wrong, rot, axes, step, at_pos, at_inv, at_q, at_k, fp32 = _rope_shared(q, k, positions, inv_freq, q_weight, k_weight, dtype, index, rows, d)
    if (wrong or kv != (Hkv, rows, d) or q_out.shape != shape or v.shape != kv or not qs[2] == ks[2] == qo[2] == vs[2] == 1 or
            not q_out.dtype is v.dtype is dtype or not index == q_out.get_device() == v.get_device() == slots.get_device() or slots.dtype is not i32 or
            slots.shape != (rows,) or not slots.is_contiguous()):
        _refuse_rope(index, dtype, q, k, v, ((q_out, Hq, "q_out"),), slots, positions, inv_freq, ((q_weight, "q_weight"), (k_weight, "k_weight")))
    handle = _raw_stream(index) if stream is None else _stream_on(index, stream)
    if rows == 0:
        return
    _launch(index, (_lib or library()).attn_rope,
            _ROPE.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), 0, k_cache.data_ptr(), v_cache.data_ptr(), at_q, at_k, at_pos,
                       slots.data_ptr(), at_inv, qs[1], qs[0], ks[1], ks[0], vs[1], vs[0], qo[1], qo[0], 0, 0, cs[0], cs[1], cs[2], step, rows, Hq, Hkv, d,
                       rot, axes, 1 if interleaved else 0, fp32, cache[0], cache[2], eps, code, handle))


def attn_paged_tree(parents, cu_seqlens_q, seqlens_k, positions, tree_mask, window_left=-1, stream=None):
    """Positions (context + depth) and ancestor masks of drafted trees.  int32 device tensors: parents [rows] (number of the node above
    among the request's nodes, -1: none), cu_seqlens_q [B+1], seqlens_k [B] -> positions [rows], tree_mask [rows, words].  Requests of
    more than 32 * words nodes are chunks: chains without a mask.  See include/attn.h."""
    i32, index = (_torch or _with_torch()).int32, parents.get_device()
    many, one, mask = parents.shape, seqlens_k.shape, tree_mask.shape
    (rows,), (B,) = many, one
    if (index < 0 or not parents.dtype is cu_seqlens_q.dtype is seqlens_k.dtype is positions.dtype is tree_mask.dtype is i32 or
            not index == cu_seqlens_q.get_device() == seqlens_k.get_device() == positions.get_device() == tree_mask.get_device() or
            not (parents.is_contiguous() and cu_seqlens_q.is_contiguous() and seqlens_k.is_contiguous() and positions.is_contiguous()) or
            cu_seqlens_q.shape != (B + 1,) or positions.shape != many or len(mask) != 2 or mask[0] != rows or
            (mask[1] > 1 and tree_mask.stride(1) != 1)):
        _refuse(index, ((parents, rows, "parents"), (cu_seqlens_q, B + 1, "cu_seqlens_q"), (seqlens_k, B, "seqlens_k"),
                        (positions, rows, "positions")),
                others=((True, f"tree_mask must be int32 [{rows}, words] on CUDA device {index}, each row contiguous"),))
    handle = _raw_stream(index) if stream is None else _stream_on(index, stream)
    if rows == 0:
        return
    _launch(index, (_lib or library()).attn_paged_tree,
            _TREE.pack(parents.data_ptr(), cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), positions.data_ptr(), tree_mask.data_ptr(), B, rows,
                       mask[1], tree_mask.stride(0) if rows > 1 else mask[1], window_left, handle))


def attn_paged_accept(tokens, targets, parents, cu_seqlens_q, seqlens_k, block_table, free_pages, free_count, page_size, num_pages, accepted,
                      ctx_lens, next_tokens, path, src_slots, dst_slots, confirmed=None, free_count_out=None, stream=None):
    """Which nodes of every request's tree the model confirms: from the last known node to the first child whose token is the
    model's choice behind it, and on from there.

    int32 device tensors: tokens, targets (the model's choice behind each node), parents [rows], cu_seqlens_q [B+1], seqlens_k [B],
    block_table [B, W], confirmed [B] (leading nodes that are known; None: 1 each) -> accepted, ctx_lens, next_tokens [B], path, src_slots,
    dst_slots [B, max path] (-1 behind the last; the slots are attn_paged_move's).  Pages without a token go back to free_pages [F] behind
    its free_count [1] ids, free_count_out [1] (default: free_count itself) counts them; free_pages None: they do not.  Such pages may hold rows
    that are still to be moved: order every layer's attn_paged_move ahead of the next write to the caches behind an attn_paged_tables on this
    free list (on one stream it is).  See include/attn.h."""
    i32, index = (_torch or _with_torch()).int32, tokens.get_device()
    many, one, lists, width = tokens.shape, seqlens_k.shape, path.shape, block_table.shape[-1]
    (rows,), (B,) = many, one
    if (index < 0 or not tokens.dtype is targets.dtype is parents.dtype is cu_seqlens_q.dtype is seqlens_k.dtype is block_table.dtype is
            accepted.dtype is ctx_lens.dtype is next_tokens.dtype is path.dtype is src_slots.dtype is dst_slots.dtype is i32 or
            not index == targets.get_device() == parents.get_device() == cu_seqlens_q.get_device() == seqlens_k.get_device() ==
            block_table.get_device() == accepted.get_device() == ctx_lens.get_device() == next_tokens.get_device() == path.get_device() ==
            src_slots.get_device() == dst_slots.get_device() or
            not many == targets.shape == parents.shape or not one == accepted.shape == ctx_lens.shape == next_tokens.shape or
            cu_seqlens_q.shape != (B + 1,) or len(lists) != 2 or lists[0] != B or not lists == src_slots.shape == dst_slots.shape or
            not (tokens.is_contiguous() and targets.is_contiguous() and parents.is_contiguous() and cu_seqlens_q.is_contiguous() and
                 seqlens_k.is_contiguous() and accepted.is_contiguous() and ctx_lens.is_contiguous() and next_tokens.is_contiguous() and
                 path.is_contiguous() and src_slots.is_contiguous() and dst_slots.is_contiguous()) or
            block_table.dim() != 2 or block_table.shape[0] != B or (block_table.stride(1) != 1 and width > 1)):
        _refuse(index, ((tokens, rows, "tokens"), (targets, rows, "targets"), (parents, rows, "parents"), (cu_seqlens_q, B + 1, "cu_seqlens_q"),
                        (seqlens_k, B, "seqlens_k"), (accepted, B, "accepted"), (ctx_lens, B, "ctx_lens"), (next_tokens, B, "next_tokens")),
                (block_table, B), others=((True, f"path, src_slots and dst_slots must be contiguous int32 [{B}, max path] on CUDA device {index}"),))
    free = at_free = at_count = at_left = at_sure = 0
    if free_pages is not None:
        (free,) = free_pages.shape
        left = free_count if free_count_out is None else free_count_out
        if free == 0:
            raise ValueError("free_pages must have room for one page at least (None: no page goes back)")
        if (not free_pages.dtype is free_count.dtype is left.dtype is i32 or
                not index == free_pages.get_device() == free_count.get_device() == left.get_device() or not free_pages.is_contiguous() or
                free_count.shape != (1,) or left.shape != (1,)):
            _refuse(index, ((free_pages, free, "free_pages"), (free_count, 1, "free_count"), (left, 1, "free_count_out")))
        at_free, at_count, at_left = free_pages.data_ptr(), free_count.data_ptr(), left.data_ptr()
    if confirmed is not None:
        if confirmed.dtype is not i32 or confirmed.get_device() != index or confirmed.shape != one or not confirmed.is_contiguous():
            _refuse(index, ((confirmed, B, "confirmed"),))
        at_sure = confirmed.data_ptr()
    _launch(index, (_lib or library()).attn_paged_accept,
            _ACCEPT.pack(tokens.data_ptr() if rows else 0, targets.data_ptr() if rows else 0, parents.data_ptr() if rows else 0, at_sure,
                         cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), block_table.data_ptr(), at_free, at_count, at_left, accepted.data_ptr(),
                         ctx_lens.data_ptr(), next_tokens.data_ptr(), path.data_ptr(), src_slots.data_ptr(), dst_slots.data_ptr(), B, rows,
                         lists[1], width, block_table.stride(0) if B > 1 else width, free, page_size, num_pages,
                         _raw_stream(index) if stream is None else _stream_on(index, stream)))


def attn_paged_move(k_cache, v_cache, src_slots, dst_slots, stream=None):
    """Rows of the caches ([num_pages, Hkv, page_size, d], or of all layers at once, [layers, num_pages, Hkv, page_size, d]) go from src_slots
    to dst_slots (int32 [lists, length]; pairs with a negative slot are left out).  Within a list no source is an earlier pair's
    destination; lists share no slot that either writes.  Lists of attn_paged_accept: to be moved before the caches are written with slots of a
    later attn_paged_tables, which may hand out the sources' pages.  See include/attn.h."""
    torch = _torch or _with_torch()
    dtype, index, i32 = k_cache.dtype, k_cache.get_device(), torch.int32
    code = _dtype_code(k_cache)
    shape, cs, lists = k_cache.shape, k_cache.stride(), src_slots.shape
    if (index < 0 or len(cs) not in (4, 5) or v_cache.dtype is not dtype or v_cache.get_device() != index or v_cache.shape != shape or
            v_cache.stride() != cs or cs[-1] != 1):
        _refuse(index, caches=(k_cache, v_cache, dtype, "d"))
    if (len(lists) != 2 or dst_slots.shape != lists or not src_slots.dtype is dst_slots.dtype is i32 or
            not index == src_slots.get_device() == dst_slots.get_device() or not (src_slots.is_contiguous() and dst_slots.is_contiguous())):
        raise ValueError(f"src_slots and dst_slots must be contiguous int32 [lists, length] on CUDA device {index}")
    handle = _raw_stream(index) if stream is None else _stream_on(index, stream)
    if lists[0] == 0 or lists[1] == 0 or shape[0] == 0:
        return
    layers, layer = (shape[0], cs[0]) if len(cs) == 5 else (1, 0)
    num_pages, Hkv, page_size, d = shape[-4:]
    _launch(index, (_lib or library()).attn_paged_move,
            _MOVE.pack(k_cache.data_ptr(), v_cache.data_ptr(), src_slots.data_ptr(), dst_slots.data_ptr(), layer, cs[-4], cs[-3], cs[-2], layers,
                       lists[0], lists[1], Hkv, d, num_pages, page_size, code, handle))


def attn_check(stream=None) -> int:
    """Synchronise `stream` and return the library status (0 = OK); raises on error."""
    rc = library().attn_check(_stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_check")
    return rc


def attn_release_workspace(stream=None) -> None:
    """Free the workspace the library holds for `stream` (stream-ordered)."""
    rc = library().attn_release_workspace(_stream_handle(stream))
    if rc != 0:
        raise AttnError(rc, "attn_release_workspace")


def debug_counters() -> dict:
    """Host-side counters: workspace allocations, tensor maps encoded, tensor-map cache hits."""
    out = (ctypes.c_ulonglong * 3)()
    rc = library().attn_debug_counters(out, 3)
    if rc != 0:
        raise AttnError(rc, "attn_debug_counters")
    return {"workspace_allocs": out[0], "map_encodes": out[1], "map_hits": out[2]}


def attn_tile_shape(d: int):
    """(rows per query tile, columns per key tile) the kernel uses for head dim d."""
    bm, bn = ctypes.c_int(0), ctypes.c_int(0)
    rc = library().attn_tile_shape(int(d), ctypes.byref(bm), ctypes.byref(bn))
    if rc != 0:
        raise AttnError(rc, "attn_tile_shape")
    return bm.value, bn.value
