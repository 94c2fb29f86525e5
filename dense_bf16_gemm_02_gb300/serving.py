"""Torch conveniences over the entry points of ``include/hk_gemm.h`` for a batch
that shares its prompts: the pages of the 8-bit cache that its sequences hold
(``Kv8Pool``, ``kv8_arrange``, ``kv8_compact``, ``kv8_copy_pages``), the norm of
each head's query and key with the rotation by its position (``qk_norm_rope``), and
the attention that reads shared pages once (``attention_kv8_shared``).

As in ``low_precision``, this is argument marshalling: every step runs in the CUDA
library, on ``stream`` (default: torch's current stream), nothing is read back, and
the tensors are on torch's current device.

As there, the way through Python is kept short, since a decoding step's calls are a few
microseconds of GPU time each: sizes and strides are taken once, small numbers go to the
library as packed bytes, what a pool's calls need is worked out once per pool.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import hk_gemm as _hk
from .hk_gemm import HK_OK, HKError
from .low_precision import (Kv8Cache, _check_vector, _empty, _f32, _i32, _raw_stream, _read_only, _row_stride, _stream, _strides, _table,
                            _tokens_shape, _type_code, _u8)

_pool_struct = struct.Struct("PPPqq4i").pack       # hk_kv8_pool
_int32s = [struct.Struct(f"{n}i").pack for n in range(5)]
_Tensor = torch.Tensor
_verdicts = {}       # (device, stream) -> what is left of the last 64
_is_capturing = torch._C._cuda_isCurrentStreamCapturing


class Kv8Pool:
    """Which pages of an 8-bit cache (or of several alike: a model's layers) its sequences hold.

    ``refs`` int32 [pages]: table entries that name each page (0: free);
    ``table`` int32 [rows, max_pages]: the block table that kv8_append and
    attention_kv8 take; ``held`` int32 [rows]: tokens whose pages a row has.
    CUDA tensors; ``Kv8Pool.empty`` makes them, with nothing held. None of them can be
    set to another tensor. The object itself may be dropped while work on its tensors is under way or
    captured (the tensors have to live, as any that a kernel works on). ``missing``: what the last
    arrangement lacked that was not captured in a graph."""

    __slots__ = ("_refs", "_table", "_held", "_pages", "_rows", "_max_pages", "_page_size", "_ref", "_missing", "_workspace",
                 "_workspace_stream", "_workspace_size")
    refs, table, held = (_read_only(n) for n in __slots__[:3])
    pages, rows, max_pages, page_size = (_read_only(n) for n in __slots__[3:7])

    def __init__(self, refs, table, held, page_size=64):
        for t, dim in ((refs, 1), (table, 2), (held, 1)):
            if not isinstance(t, torch.Tensor) or t.dtype != _i32 or not t.is_cuda or t.dim() != dim:
                raise TypeError("refs and held must be 1-D, table 2-D int32 CUDA tensors")
        if refs.get_device() != table.get_device() or held.get_device() != table.get_device():
            raise ValueError("a pool's tensors must be on one device")
        rows, max_pages = table.shape
        if held.size(0) != rows:
            raise ValueError(f"table has {rows} rows, held {held.size(0)}")
        if not refs.is_contiguous() or not held.is_contiguous():
            raise ValueError("refs and held must be contiguous")
        self._refs, self._table, self._held = refs, table, held
        self._pages, self._rows, self._max_pages, self._page_size = refs.size(0), rows, max_pages, page_size
        self._ref = _pool_struct(refs.data_ptr(), table.data_ptr(), held.data_ptr(), refs.size(0), _row_stride(table, "table"),
                                 rows, max_pages, page_size, 0)
        self._workspace_size = _hk.load().hk_kv8_arrange_workspace_size(self._ref)
        self._missing = self._workspace = self._workspace_stream = None

    @classmethod
    def empty(cls, pages, rows, max_pages, page_size=64, device="cuda"):
        """A pool of `pages` free pages and `rows` rows that hold nothing."""
        return cls(torch.zeros(pages, dtype=_i32, device=device), torch.zeros(rows, max_pages, dtype=_i32, device=device),
                   torch.zeros(rows, dtype=_i32, device=device), page_size)

    @property
    def missing(self):
        if self._missing is None:            # (no call so far)
            self._missing = torch.zeros((), dtype=_i32, device=self._refs.device)
        return self._missing


def _check_pool(pool):
    if not isinstance(pool, Kv8Pool):
        raise TypeError("pool must be a Kv8Pool")


def _cache_refs(caches, name):
    """The caches' structures side by side, as the entry points take them, and their number."""
    if isinstance(caches, Kv8Cache):
        return caches._ref, 1
    refs = []
    for c in caches:
        if not isinstance(c, Kv8Cache):
            raise TypeError(f"{name} must be Kv8Caches")
        refs.append(c._ref)
    return b"".join(refs), len(refs)


def _verdict(like, raw):
    """A 0-dim int32 tensor that no call has had before, on the device's current stream `raw`. Made 64 at a time: a tensor made
    between launches costs its call 5 us on the GPU's host (as much as the launches), one of 64 less than one."""
    key = like.get_device(), raw
    try:
        return _verdicts[key].pop()
    except (KeyError, IndexError):
        with torch.inference_mode(False):    # (an ordinary tensor wherever the first of them is asked for)
            some = list(torch.empty(64, dtype=_i32, device=like.device).unbind())
        verdict = some.pop()
        _verdicts[key] = some
        return verdict


def kv8_arrange(pool: Kv8Pool, keep, room=None, parents=None, caches=(), copies=None, stream=None):
    """Arrange the pool's rows anew, all at once: row i becomes the first ``keep[i]``
    tokens of what row ``parents[i]`` was (None: of its own), with pages for
    ``room[i]`` tokens (None: keep). int32 CUDA tensors [rows].

    room above what a row holds takes pages, keep below it cuts the row back (0 ends
    it), another parent forks or reorders. Whole pages within keep are shared, the ones
    that will be written are the row's own: copied in each of ``caches`` where they hold
    tokens. Returns a 0-dim int32 tensor of its own: 0; or the pages that lacked, or -1 for
    arguments out of range, and then nothing was changed. What a call frees is free for the next
    one. ``copies``: an int32 tensor [2, rows] that receives the copied pages and their
    copies (-1: none). See hk_kv8_arrange."""
    _check_pool(pool)
    rows = pool._rows
    _check_vector(keep, "keep", rows)
    if room is None:
        room = keep
    else:
        _check_vector(room, "room", rows)
    if parents is not None:
        _check_vector(parents, "parents", rows)
    if copies is not None and (not isinstance(copies, _Tensor) or copies.dtype != _i32 or not copies.is_cuda
                               or tuple(copies.shape) != (2, rows) or not copies.is_contiguous()):
        raise TypeError("copies must be a contiguous int32 CUDA tensor [2, rows]")
    refs, n = _cache_refs(caches, "caches") if caches else (None, 0)
    # The pool keeps a workspace for the stream that it is used on: calls there follow one another, and when the pool is dropped
    # the memory is free for what comes after them on that stream. For a stream that is given, or in a graph, which may
    # run when the pool is gone, it is the call's own.
    if stream is None:
        raw = _raw_stream(keep.get_device())
        captured = raw != 0 and _is_capturing()          # (the default stream cannot be)
    else:
        raw = int(stream.cuda_stream)
        with torch.cuda.stream(stream):
            captured = _is_capturing()
    if stream is None and not captured:
        missing, workspace = _verdict(keep, raw), pool._workspace
        if workspace is None or pool._workspace_stream != raw:
            workspace = _empty(pool._workspace_size, _u8, keep, None)
            if pool._workspace is None:
                pool._workspace, pool._workspace_stream = workspace, raw
    else:
        missing, workspace = _empty((), _i32, keep, stream), _empty(pool._workspace_size, _u8, keep, stream)
    st = _hk.load().hk_kv8_arrange(pool._ref, keep.data_ptr(), room.data_ptr(), None if parents is None else parents.data_ptr(), refs,
                                   n, None if copies is None else copies.data_ptr(), missing.data_ptr(), workspace.data_ptr(),
                                   pool._workspace_size, raw)
    if st != HK_OK:
        raise HKError(st, "hk_kv8_arrange")
    if not captured:
        pool._missing = missing
    return missing


def kv8_compact(pool: Kv8Pool, caches=(), stream=None):
    """Move the pool's pages in use to its first places, in each of ``caches`` and in
    the table. Returns int32 [pages]: where each page is now, -1 where it was free. See
    hk_kv8_compact."""
    _check_pool(pool)
    refs, n = _cache_refs(caches, "caches")
    lib = _hk.load()
    size = lib.hk_kv8_compact_workspace_size(pool._ref)
    workspace = _empty(max(size, 1), _u8, pool._refs, stream)
    moved = _empty(pool._pages, _i32, pool._refs, stream)
    st = lib.hk_kv8_compact(pool._ref, refs, n, moved.data_ptr(), workspace.data_ptr(), size, _stream(stream, moved))
    if st != HK_OK:
        raise HKError(st, "hk_kv8_compact")
    return moved


def kv8_copy_pages(dst, src, dst_pages, src_pages, stream=None) -> None:
    """Copy page ``src_pages[i]`` of each cache of ``src`` to page ``dst_pages[i]`` of
    its counterpart in ``dst`` (one Kv8Cache or several; they may be the same ones): int32
    CUDA tensors; -1 in both leaves the entry out. See hk_kv8_copy_pages."""
    to, n = _cache_refs(dst, "dst")
    of, m = _cache_refs(src, "src")
    if n != m:
        raise ValueError(f"{n} caches to copy to, {m} to copy from")
    if not isinstance(src_pages, torch.Tensor) or src_pages.dim() != 1:
        raise TypeError("src_pages must be a 1-D int32 CUDA tensor")
    _check_vector(src_pages, "src_pages", src_pages.size(0))
    _check_vector(dst_pages, "dst_pages", src_pages.size(0))
    st = _hk.load().hk_kv8_copy_pages(to, of, n, dst_pages.data_ptr(), src_pages.data_ptr(), src_pages.size(0),
                                      _stream(stream, src_pages))
    if st != HK_OK:
        raise HKError(st, "hk_kv8_copy_pages")


def _heads(t, name):
    """Sizes and packed strides of [B, T, heads, head_dim]."""
    if not isinstance(t, _Tensor) or not t.is_cuda or t.dim() != 4:
        raise TypeError(f"{name} must be a CUDA tensor [B, T, heads, head_dim]")
    sb, st, sh, sd = t.stride()
    shape = t.shape
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    return shape, _strides(sb, st, sh)


def _rope_weight(w, name, dtype, D):
    if not isinstance(w, _Tensor) or not w.is_cuda or w.dim() != 1 or w.size(0) != D or not w.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA tensor [{D}]")
    if w.dtype != dtype and w.dtype != _f32:
        raise TypeError(f"{name} must be of q's type or float32")
    return w.data_ptr()


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, sections=None, interleaved=False, out=None,
                 stream=None):
    """Norm of each head's query and key and the rotation by its token's position, in one
    pass: x / sqrt(mean(x²) + eps) · weight, then the pairs (i, i + R/2) of the first R =
    2 · len(inv_freq) elements (``interleaved``: (2i, 2i + 1)) turned by position · inv_freq[i].

    q [B, T, Hq, D], k [B, T, Hk, D] (bf16, fp16 or fp32; any strides with contiguous rows),
    ``positions`` int32 [B, T], or [axes, B, T] with ``sections``: the numbers of successive
    pairs that turn by each axis. ``inv_freq`` float32 [R/2]. Weights [D] of q's type or
    float32, both alike; None: 1. eps None: no norm and no weights. ``out``: (q', k') to write into, q and k
    themselves among others. Returns (q', k'). See hk_qk_norm_rope."""
    (B, T, Hq, D), qs = _heads(q, "q")
    (kB, kT, Hk, kD), ks = _heads(k, "k")
    dtype = q.dtype
    code = _type_code(q, "q")
    if kB != B or kT != T or kD != D or k.dtype != dtype:
        raise ValueError("k must have q's type, batch, tokens and head dimension")
    if not isinstance(inv_freq, _Tensor) or inv_freq.dtype != _f32 or not inv_freq.is_cuda or inv_freq.dim() != 1 \
            or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous 1-D float32 CUDA tensor")
    if not isinstance(positions, _Tensor) or positions.dtype != _i32 or not positions.is_cuda:
        raise TypeError("positions must be an int32 CUDA tensor [B, T] or [axes, B, T]")
    shape, pos = positions.shape, positions.stride()
    if len(shape) == 2:
        axes, pos = 1, (0, *pos)
    elif len(shape) == 3:
        axes = shape[0]
    else:
        raise TypeError("positions must be an int32 CUDA tensor [B, T] or [axes, B, T]")
    if shape[-1] != T or shape[-2] != B:
        raise ValueError(f"positions {tuple(shape)} for {B} sequences of {T} tokens")
    if sections is not None:
        if len(sections) != axes or axes >= len(_int32s):
            raise ValueError(f"{len(sections)} sections for {axes} position axes (at most 4)")
        sections = _int32s[axes](*sections)
    weight_code = code
    qw = kw = None
    if q_weight is not None:
        qw = _rope_weight(q_weight, "q_weight", dtype, D)
        weight_code = _type_code(q_weight, "q_weight")
    if k_weight is not None:
        kw = _rope_weight(k_weight, "k_weight", dtype, D)
        if q_weight is not None and k_weight.dtype != q_weight.dtype:
            raise TypeError("q_weight and k_weight must be of one type")
        weight_code = _type_code(k_weight, "k_weight")
    if eps is None:
        eps = -1.0
    elif eps < 0:
        raise ValueError("eps must not be negative (None: no norm)")
    if out is None:
        qo, ko = _empty((B, T, Hq, D), dtype, q, stream), _empty((B, T, Hk, D), dtype, q, stream)
        row = Hq * D, Hk * D
        qos, kos = _strides(T * row[0], row[0], D), _strides(T * row[1], row[1], D)
    else:
        qo, ko = out
        (qshape, qos), (kshape, kos) = _heads(qo, "out"), _heads(ko, "out")
        if qshape != q.shape or kshape != k.shape or qo.dtype != dtype or ko.dtype != dtype:
            raise ValueError("out must have q's and k's shapes and type")
    st = _hk.load().hk_qk_norm_rope(q.data_ptr(), qs, k.data_ptr(), ks, qo.data_ptr(), qos, ko.data_ptr(), kos, code, B, T, Hq, Hk, D,
                                    qw, kw, weight_code, eps, positions.data_ptr(), _strides(*pos), sections, axes,
                                    inv_freq.data_ptr(), inv_freq.size(0), 1 if interleaved else 0, _stream(stream, q))
    if st != HK_OK:
        raise HKError(st, "hk_qk_norm_rope")
    return qo, ko


def attention_kv8_shared(q, cache: Kv8Cache, block_table, lengths, groups, shared, counts=None, causal=True, scale=None,
                         return_lse=False, out=None, stream=None):
    """attention_kv8 for a batch whose sequences begin with the same tokens in the same
    pages: those are read once per group.

    ``groups`` int32 [G + 1], strictly increasing from 0 to B: group g is the sequences
    groups[g] to groups[g + 1] - 1; ``shared`` int32 [G]: their first so many tokens
    lie in the pages that the table row of the group's first sequence names (as far as they fill
    blocks of 128). CUDA tensors. Everything else as attention_kv8. See
    hk_attention_kv8_shared."""
    B, T, Hq, qs = _tokens_shape(q, "q", cache, False)
    code = _type_code(q, "q")
    if code == _hk.HK_TYPE_FP32:
        raise TypeError("q must be bfloat16 or float16")
    if scale is None:
        scale = 0.0
    elif not ctypes.c_float(scale).value:
        raise ValueError("scale must not be 0, nor round to it in 32 bits")
    ld, pages = _table(block_table, B)
    _check_vector(lengths, "lengths", B)
    if counts is not None:
        _check_vector(counts, "counts", B)
    if not isinstance(shared, torch.Tensor) or shared.dim() != 1:
        raise TypeError("shared must be a 1-D int32 CUDA tensor")
    G = shared.size(0)
    _check_vector(shared, "shared", G)
    _check_vector(groups, "groups", G + 1)
    if out is None:
        out = _empty((B, T, Hq, cache._head_dim), q.dtype, q, stream)
        os = _strides(T * Hq * cache._head_dim, Hq * cache._head_dim, cache._head_dim)
    else:
        if not isinstance(out, torch.Tensor) or out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out must have q's shape and type")
        os = _tokens_shape(out, "out", cache, False)[3]
    lse = _empty((B, T, Hq), _f32, q, stream) if return_lse else None
    lib = _hk.load()
    size = lib.hk_attention_kv8_shared_workspace_size_ex(q.data_ptr(), code, qs, cache._ref, pages, out.data_ptr(), os, B, T, Hq, G, 0)
    workspace = _empty(size, _u8, q, stream) if size else None
    st = lib.hk_attention_kv8_shared(q.data_ptr(), code, qs, cache._ref, block_table.data_ptr(), ld, pages, lengths.data_ptr(),
                                     None if counts is None else counts.data_ptr(), groups.data_ptr(), shared.data_ptr(), G,
                                     out.data_ptr(), os, None if lse is None else lse.data_ptr(), B, T, Hq, 1 if causal else 0,
                                     scale, None if workspace is None else workspace.data_ptr(), size, _stream(stream, q))
    if st != HK_OK:
        raise HKError(st, "hk_attention_kv8_shared")
    return (out, lse) if return_lse else out
