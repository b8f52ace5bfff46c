"""The target model's key/value cache around a round (argument marshalling only).

Binding of the ``dt_kv_*``, ``dt_cache_attention`` and ``dt_prompt_attention``
calls of ``include/dtree.h``, which state formulas, layouts and errors.  A round
of a serving loop, per attention layer::

    kv_plan(...)             # pages and slots for a prompt, a token or an accepted path
    prompt_attention(...)    # causal attention of packed prompts
    kv_append(...)           # their keys and values into the 8-bit cache
    cache_attention(...)     # a token, or a drafted tree under its mask, over the cache

``examples/serve_tree.py`` runs them around ``DraftTreeBuilder``.  Nothing here
computes: tensors become pointers, a refused call raises ``DtreeError``.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from ctypes import c_float, c_int, c_int64, c_size_t, c_void_p

from .dtree import DtreeError, load_library

# bits of the status words (DT_KV_*)
KV_SHORT_OF_PAGES = 1
KV_BAD_LENGTH = 2
KV_SHORT_OF_ROWS = 4
KV_BAD_PATH = 8
KV_BAD_INDEX = 16
KV_TIMEOUT = 32


class _Cache(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p),
                ("n_pages", c_int), ("page", c_int), ("n_kv", c_int), ("head_dim", c_int)]


class _Plan(ctypes.Structure):
    _fields_ = [("n_req", c_int), ("max_blocks", c_int), ("page", c_int), ("n_pages", c_int), ("extra", c_int),
                ("path_len", c_int), ("path_rows", c_int), ("max_rows", c_int64)] + \
        [(n, c_void_p) for n in ("len_old", "delta", "path", "ring_in", "block_table", "free_pages", "len_new",
                                 "ring_out", "row_start", "slot_map", "positions", "src_rows", "status")]


class _Append(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("k_row_stride", c_int64), ("k_head_stride", c_int64),
                ("v_row_stride", c_int64), ("v_head_stride", c_int64), ("n_src", c_int64), ("n_rows", c_int64),
                ("slot_map", c_void_p), ("src_rows", c_void_p), ("status", c_void_p)]


class _Attend(ctypes.Structure):
    _fields_ = [("n_req", c_int), ("slots", c_int), ("n_q", c_int), ("max_blocks", c_int), ("scale", c_float),
                ("q", c_void_p), ("q_row_stride", c_int64), ("q_head_stride", c_int64),
                ("k_new", c_void_p), ("v_new", c_void_p), ("k_row_stride", c_int64), ("k_head_stride", c_int64),
                ("v_row_stride", c_int64), ("v_head_stride", c_int64),
                ("block_table", c_void_p), ("length", c_void_p), ("mask", c_void_p),
                ("out", c_void_p), ("out_row_stride", c_int64), ("out_head_stride", c_int64), ("lse", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("status", c_void_p)]


class _Prompt(ctypes.Structure):
    _fields_ = [("n_seq", c_int), ("n_q", c_int), ("n_kv", c_int), ("head_dim", c_int), ("n_rows", c_int64),
                ("scale", c_float), ("q", c_void_p), ("k", c_void_p), ("v", c_void_p), ("out", c_void_p),
                ("q_row_stride", c_int64), ("q_head_stride", c_int64), ("k_row_stride", c_int64),
                ("k_head_stride", c_int64), ("v_row_stride", c_int64), ("v_head_stride", c_int64),
                ("out_row_stride", c_int64), ("out_head_stride", c_int64), ("row_start", c_void_p), ("lse", c_void_p),
                ("status", c_void_p)]


def _packer(cls):
    """Packs a mirror's fields, given in order, to the bytes of the C struct (native alignment): several times
    faster than filling a ctypes.Structure, and a call of a few microseconds notices."""
    codes = {c_int: "i", c_int64: "q", c_float: "f", c_void_p: "P", c_size_t: "N"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in cls._fields_) + "0P")  # (0P: the tail's padding)
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_cache, _pack_plan, _pack_append, _pack_attend, _pack_prompt = map(_packer, (_Cache, _Plan, _Append, _Attend, _Prompt))

_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        for name, res, args in (
                ("dt_kv_plan", c_int, [c_void_p] * 2),
                ("dt_kv_append", c_int, [c_void_p] * 3),
                ("dt_cache_attention", c_int, [c_void_p] * 3),
                ("dt_cache_attention_workspace", c_size_t, [c_int] * 5),
                ("dt_prompt_attention", c_int, [c_void_p] * 2)):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


_cuda = None


def _current_device():
    global _cuda
    if _cuda is None:
        import torch
        _cuda = torch._C
    return _cuda._cuda_getDevice()


def _stream(stream, index):
    """The stream of a call whose tensors are on CUDA device `index`, which must be the current one: the library launches there."""
    import torch
    if _current_device() != index:
        raise ValueError(f"tensors on cuda:{index}, but the current device is cuda:{_current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device_index != index:
        raise ValueError(f"stream: on cuda:{stream.device_index}, the tensors on cuda:{index}")
    return stream.cuda_stream


def _allocating(stream):
    """What a call allocates belongs to the stream that it runs on."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _refused(status, where):
    return DtreeError(status, where + ": " + _lib.dt_last_error().decode(errors="replace"))


def _flat(t, dtype, numel, name, index):
    """Pointer of a contiguous tensor of `numel` elements on CUDA device `index`."""
    if t.dtype is dtype and t.get_device() == index and t.numel() == numel and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the others on cuda:{index}")
    raise ValueError(f"{name}: expected a contiguous tensor of {numel} elements, got {tuple(t.shape)}")


def _heads(t, lead, heads, dim, name, index):
    """Pointer, row stride and head stride of a bf16 tensor [*lead, heads, dim].
    Only rows and heads may be strided: several leading dimensions must fold into
    one row index, and channels must be adjacent.  The stride of a dimension of one
    entry says nothing and is not looked at."""
    import torch
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected torch.bfloat16, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, the others on cuda:{index}")
    if t.shape != (*lead, heads, dim):
        raise ValueError(f"{name}: expected {(*lead, heads, dim)}, got {tuple(t.shape)}")
    st = t.stride()
    if st[-1] != 1 or (len(lead) == 2 and lead[0] > 1 and lead[1] > 1 and st[0] != st[1] * lead[1]):
        raise ValueError(f"{name}: strides {st}: channels must be adjacent and rows evenly spaced")
    return t.data_ptr(), (st[-3] if lead[-1] > 1 else st[0] if lead[0] > 1 else 0), (st[-2] if heads > 1 else 0)


def _on_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    return t.get_device()


class KvCache:
    """One layer's cache: ``k``, ``v`` [n_pages, n_kv, page, head_dim] torch.float8_e4m3fn and
    ``k_scale``, ``v_scale`` [n_pages, n_kv] fp32, caller tensors that are kept alive here."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if k.dim() != 4:
            raise ValueError("k: expected [n_pages, n_kv, page, head_dim]")
        self.index = index = _on_device(k, "k")
        self.n_pages, self.n_kv, self.page, self.head_dim = k.shape
        n, s = k.numel(), self.n_pages * self.n_kv
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.c = _pack_cache(_flat(k, torch.float8_e4m3fn, n, "k", index), _flat(v, torch.float8_e4m3fn, n, "v", index),
                             _flat(k_scale, torch.float32, s, "k_scale", index),
                             _flat(v_scale, torch.float32, s, "v_scale", index),
                             self.n_pages, self.page, self.n_kv, self.head_dim)

    @classmethod
    def empty(cls, n_pages, page, n_kv, head_dim, device="cuda"):
        """A cache of unwritten pages."""
        import torch
        k = torch.empty(n_pages, n_kv, page, head_dim, dtype=torch.float8_e4m3fn, device=device)
        scale = torch.ones(n_pages, n_kv, dtype=torch.float32, device=device)
        return cls(k, torch.empty_like(k), scale, torch.ones_like(scale))


class AttentionWorkspace:
    """Device memory that ``cache_attention`` calls use one after the other (calls that may
    overlap, on several streams, need one each).  It grows with the largest call so far,
    at least to twice its size; what it had before stays with it, since captured graphs may
    work there: keep it as long as the graph.  It does not grow while a stream is being
    captured (its zeros would be the graph's): a call that needs more then has memory of the
    graph's own, zeroed in every replay.  Grow it before, by a call of the captured sizes or by
    ``reserve``, to have neither.  Memory is taken and zeroed in the order of the stream of the call that needs it, and
    goes back only behind the work of every stream that has used it."""

    def __init__(self):
        self.buffer, self.sizes, self.streams, self.outgrown = None, None, set(), []

    def reserve(self, n_req, slots, n_q, n_kv, head_dim, device="cuda", stream=None):
        import torch
        sizes = (n_req, slots, n_q, n_kv, head_dim, device)
        if sizes != self.sizes:
            need = _library().dt_cache_attention_workspace(*sizes[:5])
            if self.buffer is None or self.buffer.numel() < need or self.buffer.device != torch.empty(0, device=device).device:
                with _allocating(stream):
                    if torch.cuda.is_current_stream_capturing():
                        return torch.zeros(max(need, 256), dtype=torch.uint8, device=device)
                    if self.buffer is not None:
                        self.outgrown.append(self.buffer)
                        need = max(need, 2 * self.buffer.numel())
                    self.buffer = torch.zeros(max(need, 256), dtype=torch.uint8, device=device)
                self.streams = {_stream(stream, self.buffer.get_device())}
            self.sizes = sizes
        return self._on(stream, _stream(stream, self.buffer.get_device()))

    def _on(self, stream, raw):
        """The buffer, for work on `stream` (whose handle is `raw`)."""
        if raw not in self.streams:
            import torch
            self.streams.add(raw)
            self.buffer.record_stream(torch.cuda.current_stream(self.buffer.device) if stream is None else stream)
        return self.buffer


def kv_plan(len_old, len_new, block_table, free_pages, ring_in, ring_out, row_start, slot_map, status, *, page,
            delta=None, extra=0, positions=None, path=None, path_rows=0, src_rows=None, stream=None):
    """Block tables and slot maps from request lengths (``dt_kv_plan``).  int32 CUDA tensors but for
    ``slot_map`` (int64): len_old, delta, len_new [n_req], block_table [n_req, max_blocks], free_pages
    [n_pages], ring_in, ring_out [2], row_start [n_req + 1], slot_map, positions, src_rows [max_rows],
    path [n_req, path_len], status [1] (KV_* bits, read it when convenient)."""
    import torch
    lib = _library()
    i32, dev = torch.int32, _on_device(len_old, "len_old")
    n, rows = len_old.numel(), slot_map.numel()
    if block_table.dim() != 2:
        raise ValueError("block_table: expected [n_req, max_blocks]")
    path_len = 0
    if path is not None:
        if path.dim() != 2:
            raise ValueError("path: expected [n_req, path_len]")
        path_len = path.shape[1]
    width = block_table.shape[1]
    a = _pack_plan(n, width, page, free_pages.numel(), extra, path_len, path_rows, rows,
                   _flat(len_old, i32, n, "len_old", dev),
                   0 if delta is None else _flat(delta, i32, n, "delta", dev),
                   # (a path of no width is one all the same: it has no pointer of its own, and nothing is read from it)
                   0 if path is None else _flat(path, i32, n * path_len, "path", dev) or len_old.data_ptr(),
                   _flat(ring_in, i32, 2, "ring_in", dev), _flat(block_table, i32, n * width, "block_table", dev),
                   _flat(free_pages, i32, free_pages.numel(), "free_pages", dev),
                   _flat(len_new, i32, n, "len_new", dev), _flat(ring_out, i32, 2, "ring_out", dev),
                   _flat(row_start, i32, n + 1, "row_start", dev), _flat(slot_map, torch.int64, rows, "slot_map", dev),
                   0 if positions is None else _flat(positions, i32, rows, "positions", dev),
                   0 if src_rows is None else _flat(src_rows, i32, rows, "src_rows", dev),
                   _flat(status, i32, 1, "status", dev))
    err = lib.dt_kv_plan(a, _stream(stream, dev))
    if err:
        raise _refused(err, "dt_kv_plan")


def kv_append(cache, k, v, slot_map, *, src_rows=None, status=None, stream=None):
    """Keys and values of new tokens into the cache (``dt_kv_append``).  k, v: bf16
    [rows, n_kv, head_dim] or [n_req, rows, n_kv, head_dim], rows and heads may be strided."""
    import torch
    lib = _library()
    dev, n = cache.index, slot_map.numel()
    if k.dim() not in (3, 4):
        raise ValueError("k: expected [rows, n_kv, head_dim] or [n_req, rows, n_kv, head_dim]")
    lead = tuple(k.shape[:-2])
    kp, kr, kh = _heads(k, lead, cache.n_kv, cache.head_dim, "k", dev)
    vp, vr, vh = _heads(v, lead, cache.n_kv, cache.head_dim, "v", dev)
    n_src = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    if src_rows is None and n > n_src:
        raise ValueError(f"slot_map: {n} rows, but k has {n_src}")
    a = _pack_append(kp, vp, kr, kh, vr, vh, n_src, n, _flat(slot_map, torch.int64, n, "slot_map", dev),
                     0 if src_rows is None else _flat(src_rows, torch.int32, n, "src_rows", dev),
                     0 if status is None else _flat(status, torch.int32, 1, "status", dev))
    err = lib.dt_kv_append(cache.c, a, _stream(stream, dev))
    if err:
        raise _refused(err, "dt_kv_append")


def cache_attention(cache, q, block_table, length, *, k_new=None, v_new=None, mask=None, scale=None, out=None,
                    lse=None, workspace, status=None, stream=None):
    """Attention of new tokens over the cache (``dt_cache_attention``).  q [n_req, slots, n_q, head_dim] bf16;
    block_table [n_req, max_blocks], length [n_req] int32; k_new, v_new [n_req, slots, n_kv, head_dim] bf16: the
    tokens' own keys and values, seen by mask [n_req, slots, slots] uint8 (``tree_mask``'s) or causally.
    scale: head_dim ** -0.5 unless given.  Returns out [n_req, slots, n_q, head_dim] bf16; lse, if given,
    [n_req, slots, n_q] fp32 is filled."""
    import torch
    lib = _library()
    dev = cache.index
    if q.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q: expected [n_req, slots, n_q, head_dim], block_table: [n_req, max_blocks]")
    n, slots, heads, dim = q.shape
    width = block_table.shape[1]
    if dim != cache.head_dim:
        raise ValueError(f"q: head_dim {dim}, the cache's is {cache.head_dim}")
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new: give both or neither")
    if out is None:
        with _allocating(stream):
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lead = (n, slots)
    kp = kr = kh = vp = vr = vh = 0
    if k_new is not None:
        kp, kr, kh = _heads(k_new, lead, cache.n_kv, dim, "k_new", dev)
        vp, vr, vh = _heads(v_new, lead, cache.n_kv, dim, "v_new", dev)
    qp, qr, qh = _heads(q, lead, heads, dim, "q", dev)
    op, orow, oh = _heads(out, lead, heads, dim, "out", dev)
    raw = _stream(stream, dev)
    sizes = (n, slots, heads, cache.n_kv, dim, dev)
    buf = workspace._on(stream, raw) if workspace.sizes == sizes else workspace.reserve(*sizes, stream)
    a = _pack_attend(n, slots, heads, width, dim ** -0.5 if scale is None else scale, qp, qr, qh, kp, vp, kr, kh, vr, vh,
                     _flat(block_table, torch.int32, n * width, "block_table", dev),
                     _flat(length, torch.int32, n, "length", dev),
                     0 if mask is None else _flat(mask, torch.uint8, n * slots * slots, "mask", dev), op, orow, oh,
                     0 if lse is None else _flat(lse, torch.float32, n * slots * heads, "lse", dev), buf.data_ptr(),
                     buf.numel(), 0 if status is None else _flat(status, torch.int32, 1, "status", dev))
    err = lib.dt_cache_attention(cache.c, a, raw)
    if err:
        raise _refused(err, "dt_cache_attention")
    return out


def prompt_attention(q, k, v, row_start, *, scale=None, out=None, lse=None, status=None, stream=None):
    """Causal attention over packed prompts (``dt_prompt_attention``).  q [rows, n_q, head_dim], k, v
    [rows, n_kv, head_dim] bf16, rows and heads may be strided (slices of one projection's output);
    row_start [n_seq + 1] int32.  Returns out [rows, n_q, head_dim]; lse [rows, n_q] fp32 is filled if given."""
    import torch
    lib = _library()
    dev = _on_device(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k: expected [rows, heads, head_dim]")
    rows, heads, dim = q.shape
    kv = k.shape[1]
    if out is None:
        with _allocating(stream):
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
    lead = (rows,)
    qp, qr, qh = _heads(q, lead, heads, dim, "q", dev)
    kp, kr, kh = _heads(k, lead, kv, dim, "k", dev)
    vp, vr, vh = _heads(v, lead, kv, dim, "v", dev)
    op, orow, oh = _heads(out, lead, heads, dim, "out", dev)
    n = row_start.numel()
    a = _pack_prompt(n - 1, heads, kv, dim, rows, dim ** -0.5 if scale is None else scale, qp, kp, vp, op,
                     qr, qh, kr, kh, vr, vh, orow, oh, _flat(row_start, torch.int32, n, "row_start", dev),
                     0 if lse is None else _flat(lse, torch.float32, rows * heads, "lse", dev),
                     0 if status is None else _flat(status, torch.int32, 1, "status", dev))
    err = lib.dt_prompt_attention(a, _stream(stream, dev))
    if err:
        raise _refused(err, "dt_prompt_attention")
    return out
