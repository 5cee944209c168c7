"""Python binding of the paged cache's calls (include/xq.h): attention of
single tokens and of chunks, rotary positions, pages.

``xq_kv_cache`` and ``xq_rope_plan`` describe tensors that the caller owns and
keep them alive; everything else carries the C names and marshals arguments.
Each call checks on the host that its tensors are device tensors of the types
and shapes it reads and writes. What lies in lengths, tables, positions, slots
and reference counts stays on the device; the kernels check it themselves.
"""

from __future__ import annotations

import ctypes

import torch

from . import _check as _raise
from . import lib as _load

XQ_F32, XQ_BF16, XQ_F16, XQ_E4M3 = range(4)
_L = None


def lib():
    """The loaded library; these calls are a few microseconds, so it is kept at hand."""
    global _L
    if _L is None:
        _L = _load()
    return _L


def _check(status: int, func: str):
    if status:
        _raise(status, func)


def _workspace(ws, index: int):
    """(pointer, bytes) of a workspace tensor; the library holds them against its need."""
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor on device %d" % index)
    return ws.data_ptr(), ws.nbytes


_ROW = {torch.float32: XQ_F32, torch.bfloat16: XQ_BF16, torch.float16: XQ_F16}
_CACHE = {torch.bfloat16: XQ_BF16, torch.float16: XQ_F16, torch.float8_e4m3fn: XQ_E4M3}


class _KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("layers", ctypes.c_int64), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("page", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("k_stride", ctypes.c_int64 * 4), ("v_stride", ctypes.c_int64 * 4),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class _Rope(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("rot", ctypes.c_int64), ("axes", ctypes.c_int64),
                ("adjacent", ctypes.c_int64), ("sections", ctypes.c_int64 * 4)]


def _device(t, what: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s: must be a device tensor" % what)


class xq_kv_cache:
    """A paged cache: ``k`` and ``v`` of shape [pages, kv_heads, page, dim], or
    [layers, pages, kv_heads, page, dim], bfloat16, float16 or float8_e4m3fn,
    any strides with contiguous dims (a pool stored [pages, page, kv_heads,
    dim] is passed transposed). What is stored stands for k * k_scale and
    v * v_scale."""

    def __init__(self, k, v, k_scale: float = 1.0, v_scale: float = 1.0):
        for t, what in ((k, "k"), (v, "v")):
            _device(t, what)
            if t.dim() not in (4, 5):
                raise ValueError("%s: expected [pages, kv_heads, page, dim] or [layers, pages, kv_heads, "
                                 "page, dim], got %d dims" % (what, t.dim()))
            if t.dtype not in _CACHE:
                raise ValueError("%s: a cache of %s is not supported" % (what, t.dtype))
            if t.stride(-1) != 1:
                raise ValueError("%s: the last dim must be contiguous" % what)
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v differ in shape, type or device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, float(k_scale), float(v_scale)
        shape = tuple(k.shape) if k.dim() == 5 else (1, *k.shape)
        self.layers, self.pages, self.kv_heads, self.page, self.dim = shape
        self.index = k.device.index
        # a dim of size 1 has no stride that matters
        def strides(t):
            s = t.stride() if t.dim() == 5 else (0, *t.stride())
            return (ctypes.c_int64 * 4)(*(0 if n == 1 else x for n, x in zip(shape[:4], s)))
        self._c = _KV(k.data_ptr(), v.data_ptr(), *shape, strides(k), strides(v), _CACHE[k.dtype],
                      self.k_scale, self.v_scale)
        self._ref = ctypes.byref(self._c)

    def layer(self, i: int) -> "xq_kv_cache":
        """One layer, for the calls that take one (attention, the append)."""
        if self.k.dim() == 4:
            raise ValueError("this cache has one layer")
        return xq_kv_cache(self.k[i], self.v[i], self.k_scale, self.v_scale)


class xq_rope_plan:
    """Rotary frequencies: ``freq`` device float64[rot/2], one per pair;
    ``sections`` deals the pairs to the axes of the positions in order;
    ``adjacent`` pairs elements 2i, 2i+1 instead of i, i + rot/2."""

    def __init__(self, freq, sections, adjacent: bool = False):
        _device(freq, "freq")
        if freq.dtype != torch.float64 or freq.dim() != 1 or not freq.is_contiguous():
            raise ValueError("freq: expected a contiguous float64 vector")
        sections = [int(n) for n in sections]
        if not 1 <= len(sections) <= 4:
            raise ValueError("sections: expected 1 to 4 axes, got %d" % len(sections))
        self.freq, self.axes, self.rot = freq, len(sections), 2 * freq.numel()
        self._c = _Rope(freq.data_ptr(), self.rot, self.axes, int(bool(adjacent)),
                        (ctypes.c_int64 * 4)(*sections))
        self._ref = ctypes.byref(self._c)


def _raw_stream(stream, index: int):
    """The caller's stream, or the current one of the tensors' device, which
    has to be the current device. (What torch.cuda.current_device and
    current_stream look up, without the objects they make: 0.2 against
    1.4 us a call.)"""
    if torch._C._cuda_getDevice() != index:
        raise ValueError("the tensors are on device %d, the current device is %d"
                         % (index, torch._C._cuda_getDevice()))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rows(t, what: str, index: int):
    """(pointer, type, row stride, head stride) of [rows, heads, dim]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % what)
    if t.get_device() != index:
        raise ValueError("%s: must be on device %d" % (what, index))
    kind = _ROW.get(t.dtype)
    if kind is None:
        raise ValueError("%s: %s is not supported" % (what, t.dtype))
    st = t.stride()
    if len(st) != 3 or st[2] != 1:
        raise ValueError("%s: expected [rows, heads, dim] with contiguous dims" % what)
    shape = t.shape
    return t.data_ptr(), kind, st[0] if shape[0] != 1 else 0, st[1] if shape[1] != 1 else 0


def _ints(t, what: str, index: int, n: int, dtype=torch.int32):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % what)
    if t.get_device() != index or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected %d contiguous %s on device %d" % (what, n, dtype, index))
    return t.data_ptr()


def _table(t, what: str, index: int, rows: int):
    """(pointer, width, stride) of a table of pages."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % what)
    shape, st = t.shape, t.stride()
    if (t.get_device() != index or t.dtype != torch.int32 or len(shape) != 2 or shape[0] != rows
            or (shape[1] > 1 and st[1] != 1)):
        raise ValueError("%s: expected int32 [%d, width] on device %d" % (what, rows, index))
    return t.data_ptr(), shape[1], st[0] if rows != 1 else shape[1]


def xq_attn_decode_workspace_bytes(seqs: int, heads: int, kv: xq_kv_cache, max_len: int,
                                   window: int = 0, sinks: int = 0) -> int:
    return lib().xq_attn_decode_workspace_bytes(seqs, heads, kv._ref, max_len, window, sinks)


def _attention(out, q, kv):
    index = kv.index
    qp, kind, q_row, q_head = _rows(q, "q", index)
    op, out_kind, out_row, out_head = _rows(out, "out", index)
    if out.shape != q.shape or out_kind != kind:
        raise ValueError("out and q differ in shape or type")
    rows, heads, dim = q.shape
    if dim != kv.dim:
        raise ValueError("q has %d dims a head, the cache %d" % (dim, kv.dim))
    return op, qp, kind, rows, heads, out_row, out_head, q_row, q_head


def xq_attn_decode(out, q, kv: xq_kv_cache, tables, lens, scale: float, window: int = 0, sinks: int = 0,
                   max_len: int = None, workspace=None, stream=None) -> None:
    """Attention of one new token per sequence; max_len (the longest length,
    which the host knows) is the tables' room when left out, 2^30 at most."""
    op, qp, kind, seqs, heads, out_row, out_head, q_row, q_head = _attention(out, q, kv)
    index = kv.index
    tp, width, t_stride = _table(tables, "tables", index, seqs)
    if max_len is None:
        max_len = min(width * kv.page, 1 << 30)
    wp, wb = _workspace(workspace, index)
    _check(lib().xq_attn_decode(op, qp, kind, seqs, heads, out_row, out_head, q_row, q_head, kv._ref, tp,
                                width, t_stride, _ints(lens, "lens", index, seqs), scale, window, sinks,
                                max_len, wp, wb, _raw_stream(stream, index)),
           "xq_attn_decode")


def xq_attn_prefill(out, q, kv: xq_kv_cache, tables, lens, starts, max_chunk: int, scale: float,
                    window: int = 0, sinks: int = 0, stream=None) -> None:
    """Attention of a chunk of new tokens per sequence, rows
    starts[b]..starts[b+1]-1 of q the last tokens of sequence b."""
    op, qp, kind, rows, heads, out_row, out_head, q_row, q_head = _attention(out, q, kv)
    index, seqs = kv.index, lens.numel()
    tp, width, t_stride = _table(tables, "tables", index, seqs)
    _check(lib().xq_attn_prefill(op, qp, kind, rows, seqs, heads, out_row, out_head, q_row, q_head, kv._ref,
                                 tp, width, t_stride, _ints(lens, "lens", index, seqs),
                                 _ints(starts, "starts", index, seqs + 1), max_chunk, scale, window, sinks,
                                 _raw_stream(stream, index)),
           "xq_attn_prefill")


def _positions(pos, rope, tokens: int, index: int):
    """(pointer, axis stride): [axes, tokens], or [tokens] for one axis."""
    if not isinstance(pos, torch.Tensor):
        raise TypeError("pos: expected a torch.Tensor")
    shape = tuple(pos.shape)
    if (pos.get_device() != index or pos.dtype != torch.int32 or (tokens > 1 and pos.stride(-1) != 1)
            or shape != (rope.axes, tokens) and (rope.axes != 1 or shape != (tokens,))):
        raise ValueError("pos: expected int32 [%d, %d] on device %d" % (rope.axes, tokens, index))
    if rope.freq.get_device() != index:
        raise ValueError("freq: must be on device %d" % index)
    return pos.data_ptr(), pos.stride(0) if rope.axes > 1 else 0


def xq_rope(out, x, pos, rope: xq_rope_plan, inverse: bool = False, stream=None) -> None:
    """Rotary positions of x [tokens, heads, dim] into out; inverse=True is the
    gradient (out from the gradient of out)."""
    index = x.get_device() if isinstance(x, torch.Tensor) else -1
    if index < 0:
        raise ValueError("x: must be a device tensor")
    xp, x_kind, x_row, x_head = _rows(x, "x", index)
    op, out_kind, out_row, out_head = _rows(out, "out", index)
    if out.shape != x.shape:
        raise ValueError("out and x differ in shape")
    tokens, heads, dim = x.shape
    pp, p_stride = _positions(pos, rope, tokens, index)
    _check(lib().xq_rope(op, out_kind, out_row, out_head, xp, x_kind, x_row, x_head, tokens, heads, dim, pp,
                         p_stride, rope._ref, 1 if inverse else 0, _raw_stream(stream, index)),
           "xq_rope")


def xq_rope_append(q_out, kv: xq_kv_cache, q, k, v, pos, rope: xq_rope_plan, slots, stream=None) -> None:
    """Rotary positions of q into q_out, of k into the cache, and v into the
    cache, at the tokens' slots."""
    index = kv.index
    qp, kind, q_row, q_head = _rows(q, "q", index)
    kp, k_kind, k_row, k_head = _rows(k, "k", index)
    vp, v_kind, v_row, v_head = _rows(v, "v", index)
    op, out_kind, out_row, out_head = _rows(q_out, "q_out", index)
    if not kind == k_kind == v_kind:
        raise ValueError("q, k and v differ in type")
    if q_out.shape != q.shape:
        raise ValueError("q_out and q differ in shape")
    tokens, heads, dim = q.shape
    if dim != kv.dim:
        raise ValueError("q has %d dims a head, the cache %d" % (dim, kv.dim))
    if tuple(k.shape) != (tokens, kv.kv_heads, dim) or tuple(v.shape) != (tokens, kv.kv_heads, dim):
        raise ValueError("k and v: expected [%d, %d, %d]" % (tokens, kv.kv_heads, dim))
    pp, p_stride = _positions(pos, rope, tokens, index)
    _check(lib().xq_rope_append(op, out_kind, out_row, out_head, kv._ref, qp, q_row, q_head, kp, k_row, k_head,
                                vp, v_row, v_head, kind, tokens, heads, pp, p_stride, rope._ref,
                                _ints(slots, "slots", index, tokens, torch.int64),
                                _raw_stream(stream, index)),
           "xq_rope_append")


def xq_cache_workspace_bytes(pages: int, slots: int) -> int:
    return lib().xq_cache_workspace_bytes(pages, slots)


def xq_cache_copy(kv: xq_kv_cache, src, dst, stream=None) -> None:
    """Page src[i] -> page dst[i], in every layer."""
    n = src.numel()
    _check(lib().xq_cache_copy(kv._ref, _ints(src, "src", kv.index, n), _ints(dst, "dst", kv.index, n), n,
                               _raw_stream(stream, kv.index)),
           "xq_cache_copy")


def xq_cache_free(kv: xq_kv_cache, refs, tables, lens, rows, stream=None) -> None:
    """The table rows `rows` give their pages back."""
    index, slots, n = kv.index, lens.numel(), rows.numel()
    tp, width, t_stride = _table(tables, "tables", index, slots)
    _check(lib().xq_cache_free(kv._ref, _ints(refs, "refs", index, kv.pages), tp, slots, width, t_stride,
                               _ints(lens, "lens", index, slots), _ints(rows, "rows", index, n), n,
                               _raw_stream(stream, index)),
           "xq_cache_free")


def xq_cache_fork(kv: xq_kv_cache, refs, tables, lens, parents, children, status, workspace=None,
                  stream=None) -> None:
    """Empty row children[i] becomes a copy of row parents[i]; status is
    [refused forks, free pages lacking]."""
    index, slots, n = kv.index, lens.numel(), children.numel()
    tp, width, t_stride = _table(tables, "tables", index, slots)
    wp, wb = _workspace(workspace, index)
    _check(lib().xq_cache_fork(kv._ref, _ints(refs, "refs", index, kv.pages), tp, slots, width, t_stride,
                               _ints(lens, "lens", index, slots), _ints(parents, "parents", index, n),
                               _ints(children, "children", index, n), n, _ints(status, "status", index, 2),
                               wp, wb, _raw_stream(stream, index)),
           "xq_cache_fork")


def xq_cache_compact(kv: xq_kv_cache, refs, tables, status, workspace=None, stream=None) -> None:
    """The live pages move together at the front; status is [0, live pages]."""
    index, slots = kv.index, tables.shape[0]
    tp, width, t_stride = _table(tables, "tables", index, slots)
    wp, wb = _workspace(workspace, index)
    _check(lib().xq_cache_compact(kv._ref, _ints(refs, "refs", index, kv.pages), tp, slots, width, t_stride,
                                  _ints(status, "status", index, 2), wp, wb, _raw_stream(stream, index)),
           "xq_cache_compact")
