"""A paged KV cache: its pages, the append of new tokens and attention over them (of one new
token per sequence, of chunks of them, differential).

``skv_cache_*`` mirror the C ABI in ``include/skv.h`` one to one; ``PagedCache``
owns the buffers as torch tensors and ``Rope`` the tables of rotary positions.
Nothing here synchronizes but ``PagedCache.status``.
"""
from __future__ import annotations

import ctypes as C
import threading

from . import (SKV_BF16, SKV_E4M3, SKV_ERR_ARG, SkvError, lib)

SKV_NO_PAGE = 0xFFFFFFFF
SKV_ROPE_INTERLEAVED = 1
SKV_CHUNK_FULL = 1


class SkvCache(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("layers", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("page_tokens", C.c_int32), ("max_seqs", C.c_int32),
                ("max_blocks", C.c_int32), ("flags", C.c_int32), ("num_pages", C.c_uint64),
                ("pool", C.c_void_p), ("table", C.c_void_p), ("refs", C.c_void_p),
                ("status", C.c_void_p), ("scale", C.c_void_p)]


class SkvRope(C.Structure):
    _fields_ = [("rotary_dim", C.c_int32), ("axes", C.c_int32), ("flags", C.c_int32),
                ("reserved", C.c_int32), ("freqs", C.c_void_p), ("axis_of_pair", C.c_void_p)]


class SkvTokens(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p),
                ("q_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("k_stride", C.c_int64), ("k_head_stride", C.c_int64),
                ("v_stride", C.c_int64), ("v_head_stride", C.c_int64)]


class SkvChunk(C.Structure):
    _fields_ = [("batch", C.c_int32), ("tokens", C.c_int32), ("max_len", C.c_int32),
                ("window", C.c_int32), ("flags", C.c_int32), ("reserved", C.c_int32),
                ("slots", C.c_void_p), ("lens", C.c_void_p), ("begins", C.c_void_p),
                ("starts", C.c_void_p)]


class SkvDiff(C.Structure):
    _fields_ = [("lambda_", C.c_void_p), ("norm", C.c_void_p), ("eps", C.c_float),
                ("reserved", C.c_int32)]


_vp, _i32, _i64, _u64, _sz = C.c_void_p, C.c_int32, C.c_int64, C.c_uint64, C.c_size_t
_K = C.POINTER(SkvCache)
SIGNATURES = {
    "skv_cache_init": (C.c_int, [_K, _vp]),
    "skv_cache_status": (C.c_int, [_K, _vp]),
    "skv_cache_workspace_bytes": (_sz, [_K, _i32]),
    "skv_cache_reserve": (C.c_int, [_K, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "skv_cache_fork": (C.c_int, [_K, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "skv_cache_free": (C.c_int, [_K, _vp, _i32, _vp]),
    "skv_cache_compact": (C.c_int, [_K, _vp, _vp, _vp, _sz, _vp]),
    "skv_cache_copy_pages": (C.c_int, [_K, _vp, _u64, _vp, _vp, _u64, _vp, _i64, _vp]),
    "skv_cache_append": (C.c_int, [_K, _i32, C.POINTER(SkvRope), C.POINTER(SkvTokens), _vp, _vp,
                                   _vp, _i32, _i32, _vp, _vp]),
    "skv_cache_attend_workspace_bytes": (_sz, [_K, _i32, _i32]),
    "skv_cache_attend": (C.c_int, [_K, _i32, _vp, _vp, _vp, _i32, _vp, _i64, _i64, _i32, C.c_float,
                                   _i32, _vp, _vp, _vp, _sz, _vp]),
    "skv_cache_attend_chunk_workspace_bytes": (_sz, [_K, _i32]),
    "skv_cache_attend_chunk": (C.c_int, [_K, _i32, C.POINTER(SkvChunk), _vp, _i64, _i64, _i32,
                                         C.c_float, _vp, _vp, _vp, _sz, _vp]),
    "skv_cache_attend_diff": (C.c_int, [_K, _i32, C.POINTER(SkvChunk), C.POINTER(SkvDiff), _vp,
                                        _i64, _i64, _i32, C.c_float, _vp, _vp, _vp, _sz, _vp]),
}


# ---- one-to-one wrappers of the C ABI ----

def skv_cache_init(cache, stream):
    return lib().skv_cache_init(C.byref(cache), stream)


def skv_cache_status(cache, stream):
    return lib().skv_cache_status(C.byref(cache), stream)


def skv_cache_workspace_bytes(cache, n):
    return int(lib().skv_cache_workspace_bytes(C.byref(cache), n))


def skv_cache_reserve(cache, slots_ptr, old_ptr, new_ptr, n, ws_ptr, ws_bytes, stream):
    return lib().skv_cache_reserve(C.byref(cache), slots_ptr, old_ptr, new_ptr, n, ws_ptr,
                                   ws_bytes, stream)


def skv_cache_fork(cache, parents_ptr, children_ptr, lens_ptr, n, ws_ptr, ws_bytes, stream):
    return lib().skv_cache_fork(C.byref(cache), parents_ptr, children_ptr, lens_ptr, n, ws_ptr,
                                ws_bytes, stream)


def skv_cache_free(cache, slots_ptr, n, stream):
    return lib().skv_cache_free(C.byref(cache), slots_ptr, n, stream)


def skv_cache_compact(cache, table_out_ptr, refs_out_ptr, ws_ptr, ws_bytes, stream):
    return lib().skv_cache_compact(C.byref(cache), table_out_ptr, refs_out_ptr, ws_ptr, ws_bytes,
                                   stream)


def skv_cache_copy_pages(cache, src_pool_ptr, src_pages, src_ptr, dst_pool_ptr, dst_pages, dst_ptr,
                         n, stream):
    return lib().skv_cache_copy_pages(C.byref(cache), src_pool_ptr, src_pages, src_ptr,
                                      dst_pool_ptr, dst_pages, dst_ptr, n, stream)


def skv_cache_append(cache, layer, rope, tokens, slots_ptr, at_ptr, positions_ptr, n, q_heads,
                     q_out_ptr, stream):
    """rope: an SkvRope or None; tokens: an SkvTokens."""
    return lib().skv_cache_append(C.byref(cache), layer, None if rope is None else C.byref(rope),
                                  C.byref(tokens), slots_ptr, at_ptr, positions_ptr, n, q_heads,
                                  q_out_ptr, stream)


def skv_cache_attend_workspace_bytes(cache, batch, q_heads):
    return int(lib().skv_cache_attend_workspace_bytes(C.byref(cache), batch, q_heads))


def skv_cache_attend(cache, layer, slots_ptr, lens_ptr, begins_ptr, batch, q_ptr, q_stride,
                     q_head_stride, q_heads, softmax_scale, max_len, out_ptr, lse_ptr, ws_ptr,
                     ws_bytes, stream):
    return lib().skv_cache_attend(C.byref(cache), layer, slots_ptr, lens_ptr, begins_ptr, batch,
                                  q_ptr, q_stride, q_head_stride, q_heads, softmax_scale, max_len,
                                  out_ptr, lse_ptr, ws_ptr, ws_bytes, stream)


def skv_cache_attend_chunk_workspace_bytes(cache, q_heads):
    return int(lib().skv_cache_attend_chunk_workspace_bytes(C.byref(cache), q_heads))


def skv_cache_attend_chunk(cache, layer, chunk, q_ptr, q_stride, q_head_stride, q_heads,
                           softmax_scale, out_ptr, lse_ptr, ws_ptr, ws_bytes, stream):
    """chunk: an SkvChunk."""
    return lib().skv_cache_attend_chunk(C.byref(cache), layer, C.byref(chunk), q_ptr, q_stride,
                                        q_head_stride, q_heads, softmax_scale, out_ptr, lse_ptr,
                                        ws_ptr, ws_bytes, stream)


def skv_cache_attend_diff(cache, layer, chunk, diff, q_ptr, q_stride, q_head_stride, q_heads,
                          softmax_scale, out_ptr, lse_ptr, ws_ptr, ws_bytes, stream):
    """chunk: an SkvChunk; diff: an SkvDiff."""
    return lib().skv_cache_attend_diff(C.byref(cache), layer, C.byref(chunk), C.byref(diff), q_ptr,
                                       q_stride, q_head_stride, q_heads, softmax_scale, out_ptr,
                                       lse_ptr, ws_ptr, ws_bytes, stream)


# ---- torch convenience wrappers ----

def _bad(what):
    return SkvError(SKV_ERR_ARG, what)


def _allocator(device):
    """empty(shape, strides, dtype) on the current device, which is `device`: torch's own
    short cut where it has it (1 us a call in place of 3), else torch.empty_strided."""
    import torch
    try:
        from torch._C._dynamo.guards import _empty_strided_cuda
        return _empty_strided_cuda
    except ImportError:
        return lambda shape, strides, dtype: torch.empty_strided(shape, strides, dtype=dtype,
                                                                 device=device)


class Rope:
    """Rotary positions: pair p of a head's first 2 * freqs.numel() channels turns by
    position[axis_of_pair[p]] * freqs[p].

    freqs: float64 [pairs] on the device, for instance base ** (-2 p / rotary_dim);
    axis_of_pair: uint8 [pairs] on the device or None (one axis); interleaved: pairs
    are neighbouring channels instead of the two halves."""

    def __init__(self, freqs, axis_of_pair=None, axes=1, interleaved=False):
        import torch
        if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
            raise _bad("Rope: freqs must be a contiguous float64 vector")
        if axis_of_pair is not None and (axis_of_pair.dtype != torch.uint8 or
                                         axis_of_pair.shape != freqs.shape or
                                         axis_of_pair.device != freqs.device or
                                         not axis_of_pair.is_contiguous()):
            raise _bad("Rope: axis_of_pair must be a contiguous uint8 vector like freqs")
        if not 1 <= axes <= 4 or freqs.numel() % 8:
            raise _bad("Rope: 1 to 4 axes, a multiple of 8 pairs")
        self.freqs, self.axis_of_pair, self.axes = freqs, axis_of_pair, int(axes)
        self.struct = SkvRope(2 * freqs.numel(), self.axes,
                              SKV_ROPE_INTERLEAVED if interleaved else 0, 0, freqs.data_ptr(),
                              None if axis_of_pair is None else axis_of_pair.data_ptr())
        self.ref = C.byref(self.struct)


class PagedCache:
    """The pages, table and counts of a paged KV cache, and the calls on them.

    pool: [num_pages, page_tokens, head_dim] int16 (bf16 patterns) or uint8 (e4m3
    codes); table: int32 [max_seqs, layers, 2, heads, max_blocks] of page numbers
    (-1: none); refs: int32 [num_pages].  Give num_pages, max_seqs and max_blocks
    to have them made (an empty cache), or the tensors themselves.  scale: float32
    [layers, heads], e4m3 only.

    Slots, lengths, places and positions are int32 tensors on the device.  Calls
    run on ``stream`` (a torch stream; default: the current one), outputs are
    allocated there; errors in the data show in ``status()``.  Several threads may
    call at once: each call's kernels are enqueued together (which of two calls comes
    first is theirs to order).  Results carry no gradient, whatever the inputs require."""

    def __init__(self, dtype, layers, heads, head_dim, page_tokens, num_pages=None, max_seqs=None,
                 max_blocks=None, scale=None, device="cuda", pool=None, table=None, refs=None):
        import torch
        self.torch = torch
        if dtype not in (SKV_BF16, SKV_E4M3):
            raise _bad("PagedCache: dtype")
        scalar = torch.int16 if dtype == SKV_BF16 else torch.uint8
        if (table is None) != (refs is None):
            raise _bad("PagedCache: table and refs belong together")
        if pool is None:
            if not num_pages:
                raise _bad("PagedCache: pool or num_pages")
            pool = torch.empty((num_pages, page_tokens, head_dim), dtype=scalar, device=device)
        empty = table is None
        if empty:
            if not max_seqs or not max_blocks:
                raise _bad("PagedCache: table or max_seqs and max_blocks")
            table = torch.empty((max_seqs, layers, 2, heads, max_blocks), dtype=torch.int32,
                                device=pool.device)
            refs = torch.empty(pool.shape[0], dtype=torch.int32, device=pool.device)
        if (pool.dtype != scalar or pool.dim() != 3 or
                tuple(pool.shape[1:]) != (page_tokens, head_dim) or not pool.is_contiguous()):
            raise _bad("PagedCache: pool must be contiguous [pages, page_tokens, head_dim]")
        if (table.dtype != torch.int32 or table.dim() != 5 or
                tuple(table.shape[1:4]) != (layers, 2, heads) or not table.is_contiguous() or
                table.device != pool.device):
            raise _bad("PagedCache: table must be contiguous int32 [seqs, layers, 2, heads, blocks]")
        if (refs.dtype != torch.int32 or tuple(refs.shape) != (pool.shape[0],) or
                not refs.is_contiguous() or refs.device != pool.device):
            raise _bad("PagedCache: refs must be contiguous int32 [pages]")
        if scale is not None and (dtype != SKV_E4M3 or scale.dtype != torch.float32 or
                                  tuple(scale.shape) != (layers, heads) or
                                  not scale.is_contiguous() or scale.device != pool.device):
            raise _bad("PagedCache: scale must be contiguous float32 [layers, heads], e4m3 only")
        if not pool.is_cuda:
            raise _bad("PagedCache: tensors on a CUDA device")
        self.pool, self.table, self.refs, self.scale = pool, table, refs, scale
        self.device = pool.device
        self.layers, self.heads, self.head_dim = layers, heads, head_dim
        self.page_tokens = page_tokens
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.struct = SkvCache(dtype, layers, heads, head_dim, page_tokens, table.shape[0],
                               table.shape[4], 0, pool.shape[0], pool.data_ptr(),
                               table.data_ptr(), refs.data_ptr(), self._status.data_ptr(),
                               None if scale is None else scale.data_ptr())
        self._ref = C.byref(self.struct)
        self._index = self.device.index
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._current_device = torch._C._cuda_getDevice
        self._capturing = torch._C._cuda_isCurrentStreamCapturing
        self._int32, self._bf16, self._f32 = torch.int32, torch.bfloat16, torch.float32
        self._empty = _allocator(self.device)
        self._attend_bytes = {}    # workspace bytes by q_heads
        self._chunk_bytes = {}     # of attend_chunk and attend_diff
        self._pages_bytes = {}     # and of the page operations by n
        self._default_scale = head_dim ** -0.5
        self._lib = lib()
        self._ws = {}
        # held from the look-up of a workspace until its call has enqueued all of its kernels:
        # they hand data on in it, and the library's calls let other threads run
        self._enqueue = threading.Lock()
        if skv_cache_workspace_bytes(self.struct, 0) == 0:
            raise _bad("PagedCache: shape (head_dim a multiple of 8, or 16 for e4m3)")
        if empty:
            self.clear()

    # -- helpers --

    def _stream(self):
        if self._current_device() != self._index:
            raise _bad("PagedCache: its device must be the current one")
        return self._raw_stream(self._index)

    def _on(self, stream, tensors, call):
        """`call` with `stream` current: what it allocates belongs to that stream, and the
        device tensors given stay allocated until the stream is past it."""
        with self.torch.cuda.stream(stream):
            for t in (*tensors, self.pool, self.table, self.refs, self._status, self.scale):
                if t is not None:
                    t.record_stream(stream)
            return call()

    def _workspace(self, kind, stream, nbytes):
        """This stream's workspace of at least nbytes: (address, bytes, tensor)."""
        capturing = self._capturing()
        have = None if capturing else self._ws.get((kind, stream))
        if have is None or have[1] < nbytes:
            ws = self.torch.empty(nbytes, dtype=self.torch.uint8, device=self.device)
            have = ws.data_ptr(), nbytes, ws
            if not capturing:       # a captured one belongs to its graph
                self._ws[kind, stream] = have
        return have

    def _ints(self, what, n, *tensors):
        i32 = self._int32
        for t in tensors:
            if (t.dtype is not i32 or t.dim() != 1 or t.numel() != n or
                    t.get_device() != self._index or not t.is_contiguous()):
                raise _bad("%s: int32 vectors of one length on the cache's device" % what)

    def _heads(self, what, t, n, heads=None):
        """Token and head strides of a [tokens, heads, head_dim] tensor; 0 for a dimension of
        one, where torch keeps any number and the library asks for multiples of 8."""
        shape = t.shape
        st = t.stride()
        if (t.dtype is not self._bf16 or len(shape) != 3 or shape[0] != n or
                shape[2] != self.head_dim or t.get_device() != self._index or
                (heads is not None and shape[1] != heads) or (st[2] != 1 and t.numel())):
            raise _bad("%s: bf16 [tokens, heads, head_dim], channels contiguous" % what)
        return st[0] if n > 1 else 0, st[1] if shape[1] > 1 else 0

    def _numbers(self, what, layer, *counts):
        """ctypes cuts what does not fit its 32 bits without a word."""
        if not 0 <= layer < self.layers or not 0 <= min(counts) <= max(counts) < 1 << 31:
            raise _bad("%s: layer, max_len or window" % what)

    def _check(self, rc, what):
        if rc:
            raise SkvError(rc, what)

    # -- state --

    def clear(self):
        """Empty the cache: no sequence has pages."""
        st = self._stream()
        with self._enqueue:
            rc = self._lib.skv_cache_init(self._ref, st)
        self._check(rc, "skv_cache_init")

    def status(self):
        """Raises the error gathered since the last call, if any.  Synchronizes."""
        self._check(self._lib.skv_cache_status(self._ref, self._stream()), "paged cache")

    def page_of_chunk(self, slot, tokens):
        """The sequence's pages as Codec.decode_range wants them (a container of this
        many tokens): a contiguous int32 vector."""
        blocks = -(-tokens // self.page_tokens)
        return self.table[slot, ..., :blocks].contiguous().view(-1)

    # -- pages --

    def _pages_ws(self, n, stream):
        nb = self._pages_bytes.get(n)
        if nb is None:
            nb = self._pages_bytes[n] = skv_cache_workspace_bytes(self.struct, n)
        return self._workspace("pages", stream, nb)

    def reserve(self, slots, old_len, new_len, stream=None):
        """Pages for the tokens old_len .. new_len - 1 of each sequence."""
        if stream is not None:
            return self._on(stream, (slots, old_len, new_len),
                            lambda: self.reserve(slots, old_len, new_len))
        n = slots.numel()
        self._ints("reserve", n, slots, old_len, new_len)
        st = self._stream()
        with self._enqueue:
            ws = self._pages_ws(n, st)
            rc = self._lib.skv_cache_reserve(self._ref, slots.data_ptr(), old_len.data_ptr(),
                                             new_len.data_ptr(), n, ws[0], ws[1], st)
        self._check(rc, "skv_cache_reserve")

    def fork(self, parents, children, lens, stream=None):
        """Each child becomes a copy of the first tokens of its parent."""
        if stream is not None:
            return self._on(stream, (parents, children, lens),
                            lambda: self.fork(parents, children, lens))
        n = parents.numel()
        self._ints("fork", n, parents, children, lens)
        st = self._stream()
        with self._enqueue:
            ws = self._pages_ws(n, st)
            rc = self._lib.skv_cache_fork(self._ref, parents.data_ptr(), children.data_ptr(),
                                          lens.data_ptr(), n, ws[0], ws[1], st)
        self._check(rc, "skv_cache_fork")

    def free(self, slots, stream=None):
        """Give back the pages of these sequences."""
        if stream is not None:
            return self._on(stream, (slots,), lambda: self.free(slots))
        n = slots.numel()
        self._ints("free", n, slots)
        st = self._stream()
        with self._enqueue:     # not between a fork's check of its parents and their sharing
            rc = self._lib.skv_cache_free(self._ref, slots.data_ptr(), n, st)
        self._check(rc, "skv_cache_free")

    def compact(self, table_out=None, refs_out=None, stream=None):
        """Move the pages in use to the lowest numbers; in place, or with the new table
        and counts in table_out and refs_out."""
        if stream is not None:
            return self._on(stream, (table_out, refs_out),
                            lambda: self.compact(table_out, refs_out))
        if (table_out is None) != (refs_out is None):
            raise _bad("compact: table_out and refs_out belong together")
        for t, own in ((table_out, self.table), (refs_out, self.refs)):
            if t is not None and (t.dtype != own.dtype or t.shape != own.shape or
                                  t.device != own.device or not t.is_contiguous()):
                raise _bad("compact: outputs shaped like the cache's table and refs")
        st = self._stream()
        with self._enqueue:
            ws = self._pages_ws(0, st)
            rc = self._lib.skv_cache_compact(
                self._ref, None if table_out is None else table_out.data_ptr(),
                None if refs_out is None else refs_out.data_ptr(), ws[0], ws[1], st)
        self._check(rc, "skv_cache_compact")

    def copy_pages(self, src, dst, src_pool=None, dst_pool=None, stream=None):
        """Page dst[i] of dst_pool = page src[i] of src_pool (None: the cache's pool; a
        pool may be in pinned host memory, which torch, if it pinned it, keeps until the
        copy is done.  The pools of a copy that is captured into a graph are the caller's to
        keep, like all that a graph uses)."""
        if stream is not None:
            return self._on(stream, [t for t in (src, dst, src_pool, dst_pool)
                                     if t is not None and t.is_cuda],
                            lambda: self.copy_pages(src, dst, src_pool, dst_pool))
        n = src.numel()
        self._ints("copy_pages", n, src, dst)
        for t in (src_pool, dst_pool):
            if t is not None and (t.dtype != self.pool.dtype or t.shape[1:] != self.pool.shape[1:]
                                  or not t.is_contiguous() or not t.numel() or
                                  not (t.device == self.device or t.is_pinned())):
                raise _bad("copy_pages: pools with pages like the cache's, on its device or pinned")
        st = self._stream()
        self._check(self._lib.skv_cache_copy_pages(
            self._ref, None if src_pool is None else src_pool.data_ptr(),
            0 if src_pool is None else src_pool.shape[0], src.data_ptr(),
            None if dst_pool is None else dst_pool.data_ptr(),
            0 if dst_pool is None else dst_pool.shape[0], dst.data_ptr(), n, st),
            "skv_cache_copy_pages")
        if not self._capturing():
            for t in (src_pool, dst_pool):
                if t is not None and not t.is_cuda:
                    self._used(t, st)

    def _used(self, pool, stream):
        """Tell torch's pinned allocator that this stream uses the pool up to here.  Of a
        kernel's accesses it knows nothing, and would give a dropped pool to the next who
        asks; a copy of its own out of it makes it wait.  (An event of our own would have to
        be asked for, which breaks a capture that another thread is at.)"""
        last = self._workspace("last", stream, 16)[2][:pool.element_size()].view(pool.dtype)
        last.copy_(pool.view(-1)[:1], non_blocking=True)

    # -- tokens --

    def append(self, layer, slots, at, q, k, v, rope=None, positions=None, q_out=None,
               stream=None):
        """New tokens of one layer: q [n, q_heads, D], k and v [n, heads, D] bf16 (any
        strides that keep channels contiguous; q may be None) turned by rope at
        positions [axes, n], k and v written to place at[i] of sequence slots[i].
        Returns the turned q."""
        if stream is not None:
            return self._on(stream, (slots, at, q, k, v, positions, q_out,
                                     rope and rope.freqs, rope and rope.axis_of_pair),
                            lambda: self.append(layer, slots, at, q, k, v, rope, positions, q_out))
        n = slots.numel()
        self._numbers("append", layer, n)
        self._ints("append", n, slots, at)
        ks = self._heads("append: k", k, n, self.heads)
        vs = self._heads("append: v", v, n, self.heads)
        qs, q_heads, q_ptr, out_ptr = (0, 0), 0, None, None
        st = self._stream()
        if q is not None:
            qs = self._heads("append: q", q, n)
            q_heads = q.shape[1]
            if q_out is None:
                d = self.head_dim
                q_out = self._empty((n, q_heads, d), (q_heads * d, d, 1), self._bf16)
            else:
                self._heads("append: q_out", q_out, n, q_heads)
                if not q_out.is_contiguous():
                    raise _bad("append: q_out must be contiguous")
            q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
        rope_ref = pos_ptr = None
        if rope is not None:
            if (positions is None or positions.dtype is not self._int32 or
                    tuple(positions.shape) != (rope.axes, n) or
                    positions.get_device() != self._index or
                    rope.freqs.get_device() != self._index or not positions.is_contiguous()):
                raise _bad("append: positions must be contiguous int32 [axes, n]")
            rope_ref, pos_ptr = rope.ref, positions.data_ptr()
        t = SkvTokens(q_ptr, k.data_ptr(), v.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1])
        self._check(self._lib.skv_cache_append(
            self._ref, layer, rope_ref, C.byref(t), slots.data_ptr(), at.data_ptr(), pos_ptr, n,
            q_heads, out_ptr, st), "skv_cache_append")
        return q_out

    def attend(self, layer, slots, lens, q, max_len, begins=None, scale=None, out=None, lse=False,
               stream=None):
        """Attention of one new token per sequence, q [batch, q_heads, D] bf16, over the
        tokens begins[i] .. lens[i] - 1 of sequence slots[i] (max_len: no length is
        larger).  scale: default 1 / sqrt(head_dim).  Returns out [batch, q_heads, D],
        with lse=True also the log of the sum of exponentials [batch, q_heads]."""
        if stream is not None:
            return self._on(stream, (slots, lens, begins, q, out),
                            lambda: self.attend(layer, slots, lens, q, max_len, begins, scale,
                                                out, lse))
        n = slots.numel()
        self._numbers("attend", layer, max_len)
        self._ints("attend", n, slots, lens)
        if begins is not None:
            self._ints("attend", n, begins)
        qs = self._heads("attend: q", q, n)
        q_heads, d = q.shape[1], self.head_dim
        nb = self._attend_bytes.get(q_heads)
        if nb is None:
            nb = skv_cache_attend_workspace_bytes(self.struct, n, q_heads)
            if nb == 0:
                raise _bad("attend: q_heads a multiple of the cache's heads, head_dim up to 256")
            self._attend_bytes[q_heads] = nb
        st = self._stream()
        if out is None:
            out = self._empty((n, q_heads, d), (q_heads * d, d, 1), self._bf16)
        else:
            self._heads("attend: out", out, n, q_heads)
            if not out.is_contiguous():
                raise _bad("attend: out must be contiguous")
        s = self._empty((n, q_heads), (q_heads, 1), self._f32) if lse else None
        with self._enqueue:
            ws = self._workspace("attend", st, nb)
            rc = self._lib.skv_cache_attend(
                self._ref, layer, slots.data_ptr(), lens.data_ptr(),
                None if begins is None else begins.data_ptr(), n, q.data_ptr(), qs[0], qs[1],
                q_heads, self._default_scale if scale is None else scale, max_len, out.data_ptr(),
                None if s is None else s.data_ptr(), ws[0], ws[1], st)
        self._check(rc, "skv_cache_attend")
        return (out, s) if lse else out

    def _floats(self, what, t, n):
        if (t.dtype is not self._f32 or t.dim() != 1 or t.numel() != n or
                t.get_device() != self._index or not t.is_contiguous()):
            raise _bad("%s: a float32 vector of %d on the cache's device" % (what, n))

    def _chunk(self, what, layer, slots, lens, starts, begins, q, max_len, window, causal, scale,
               out, lse, maps, diff):
        """The call that attend_chunk (diff None) and attend_diff share; maps: sums of
        exponentials per row and head."""
        batch, d = slots.numel(), self.head_dim
        self._numbers(what, layer, max_len, window)
        self._ints(what, batch, slots, lens)
        if begins is not None:
            self._ints(what, batch, begins)
        if starts is not None:
            self._ints(what, batch + 1, starts)
        n = q.shape[0] if starts is not None and q.dim() else batch
        qs = self._heads(what + ": q", q, n)
        q_heads = q.shape[1]
        nb = self._chunk_bytes.get(q_heads)
        if nb is None:
            nb = skv_cache_attend_chunk_workspace_bytes(self.struct, q_heads)
            if nb == 0:
                raise _bad("%s: q_heads a multiple of the cache's heads, head_dim up to 256" % what)
            self._chunk_bytes[q_heads] = nb
        st = self._stream()
        if out is None:
            out = self._empty((n, q_heads, d), (q_heads * d, d, 1), self._bf16)
        else:
            self._heads(what + ": out", out, n, q_heads)
            if not out.is_contiguous():
                raise _bad("%s: out must be contiguous" % what)
        s = None
        if lse:
            s = self._empty((n, q_heads), (q_heads, 1), self._f32) if maps == 1 else \
                self._empty((n, q_heads, 2), (2 * q_heads, 2, 1), self._f32)
        k = SkvChunk(batch, n, max_len, window, 0 if causal else SKV_CHUNK_FULL, 0,
                     slots.data_ptr(), lens.data_ptr(),
                     None if begins is None else begins.data_ptr(),
                     None if starts is None else starts.data_ptr())
        if scale is None:
            scale = (d / maps) ** -0.5
        more = () if diff is None else (C.byref(diff),)
        call = self._lib.skv_cache_attend_chunk if diff is None else self._lib.skv_cache_attend_diff
        with self._enqueue:
            ws = self._workspace("chunk", st, nb)
            rc = call(self._ref, layer, C.byref(k), *more, q.data_ptr(), qs[0], qs[1], q_heads,
                      scale, out.data_ptr(), None if s is None else s.data_ptr(), ws[0], ws[1], st)
        self._check(rc, what)
        return (out, s) if lse else out

    def attend_chunk(self, layer, slots, lens, starts, q, max_len, begins=None, window=0,
                     causal=True, scale=None, out=None, lse=False, stream=None):
        """Attention of the new tokens of each sequence, q [tokens, q_heads, D] bf16: rows
        starts[i] .. starts[i + 1] - 1 are the last ones of the lens[i] tokens of sequence
        slots[i] (max_len: no length is larger), whose keys and values are in the pages
        already.  A token at place p sees the tokens begins[i] .. p (causal=False: to the
        sequence's end), with a window those above p - window.  scale: default 1 /
        sqrt(head_dim).  Returns out [tokens, q_heads, D], with lse=True also the log of the
        sum of exponentials [tokens, q_heads]; rows that no sequence names are not
        written."""
        if starts is None:
            raise _bad("attend_chunk: starts")
        if stream is not None:
            return self._on(stream, (slots, lens, starts, begins, q, out),
                            lambda: self.attend_chunk(layer, slots, lens, starts, q, max_len,
                                                      begins, window, causal, scale, out, lse))
        return self._chunk("attend_chunk", layer, slots, lens, starts, begins, q, max_len, window,
                           causal, scale, out, lse, 1, None)

    def attend_diff(self, layer, slots, lens, q, lam, max_len, starts=None, norm=None, eps=1e-5,
                    begins=None, window=0, causal=True, scale=None, out=None, lse=False,
                    stream=None):
        """Differential attention: with q = (q1, q2) and k = (k1, k2) in halves of a head's
        channels, (softmax(q1 k1) - lam[head] softmax(q2 k2)) v of the new tokens of each
        sequence, q [tokens, q_heads, D] bf16.  starts None: one new token per sequence
        (row i); else as in attend_chunk, like the other arguments.  lam: float32
        [q_heads]; norm: float32 [D] or None, with it each head's result is divided by
        the root of its mean square + eps and multiplied by norm.  scale: default 1 /
        sqrt(D / 2).  Returns out [tokens, q_heads, D], with lse=True also the logs of both
        sums of exponentials [tokens, q_heads, 2].  Positions: append with
        Rope(freqs.repeat(2), interleaved=True), freqs those of one half (pairs of channels
        must not lie in both)."""
        if stream is not None:
            return self._on(stream, (slots, lens, q, lam, starts, norm, begins, out),
                            lambda: self.attend_diff(layer, slots, lens, q, lam, max_len, starts,
                                                     norm, eps, begins, window, causal, scale, out,
                                                     lse))
        if q.dim() == 3:
            self._floats("attend_diff: lam", lam, q.shape[1])
        if norm is not None:
            self._floats("attend_diff: norm", norm, self.head_dim)
        diff = SkvDiff(lam.data_ptr(), None if norm is None else norm.data_ptr(), eps, 0)
        return self._chunk("attend_diff", layer, slots, lens, starts, begins, q, max_len, window,
                           causal, scale, out, lse, 2, diff)
