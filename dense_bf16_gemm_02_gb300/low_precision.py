"""Torch conveniences over the low-precision serving entry points of
``include/hk_gemm.h``: matrices in microscaled 4-bit floating point
(``quantize_fp4``, ``dequantize_fp4``, ``gemm_fp4``), and a paged key/value
cache in 8 bits (``Kv8Cache``, ``kv8_append``, ``attention_kv8``).

As in ``hk_gemm``, this is argument marshalling: every step runs in the CUDA
library, on ``stream`` (default: torch's current stream). What a call
allocates comes from torch's allocator, for that stream, and the tensors are on
torch's current device.

A decoding step makes many calls of a few microseconds of GPU time each, so
the way through Python is kept short: one check per condition, no context
managers and no stream object unless a stream is given. Measured in a loop on the
GPU's host: a one-token quantisation 10 us (3 of them its Python, 3 the launch, the
rest what the two and the allocator cost each other in caches), a one-token product
9, an append 7, attention 14; a captured step pays none of it.
"""
from __future__ import annotations

import ctypes
import operator
import struct

import torch

from . import hk_gemm as _hk
from .hk_gemm import HK_OK, HKError

_FORMATS = {"mxfp4": _hk.HK_FP4_MXFP4, "nvfp4": _hk.HK_FP4_NVFP4}
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_TYPES = {torch.bfloat16: _hk.HK_TYPE_BF16, torch.float16: _hk.HK_TYPE_FP16, torch.float32: _hk.HK_TYPE_FP32}
_strides = struct.Struct("3q").pack       # three element strides, as the C entry points take them
_cache_struct = struct.Struct("PPPPq4i").pack      # hk_kv8_cache
_u8, _bf16, _f32, _i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(stream, t):
    return _raw_stream(t.get_device()) if stream is None else int(stream.cuda_stream)


def _empty(shape, dtype, like, stream):
    """Memory that belongs to the call's stream, so that it may be freed as soon as the call is enqueued."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _type_code(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported element type {t.dtype} (bfloat16, float16 or float32)")
    return code


def _row_stride(t, name):
    """Leading dimension of a 2-D tensor whose rows are contiguous and do not overlap."""
    rows, cols = t.shape
    row, col = t.stride()
    if cols > 1 and col != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if rows <= 1:
        return cols
    if row < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return row


def _read_only(slot, doc=None):
    """A property without a setter over a slot: the pointers of an object go to the kernels as it was made with
    them, so that another tensor or size needs another object."""
    return property(operator.attrgetter(slot), doc=doc)


def _checked_global_scale(g, format):
    if format != "nvfp4":
        raise ValueError("only nvfp4 has a global scale")
    if not isinstance(g, torch.Tensor) or g.dtype != _f32 or not g.is_cuda or g.numel() != 1:
        raise TypeError("global_scale must be a float32 CUDA tensor of one element")
    return g


class Fp4Matrix:
    """A rows × cols matrix in ``format`` "mxfp4" or "nvfp4" (see hk_fp4_quantize).

    ``codes``: uint8 [rows, ld], two codes per byte; ``scales``: uint8, the
    block scales in 128×4 tiles; ``global_scale``: a float32 CUDA tensor of one
    element (NVFP4 only) or None. None of them can be set to another tensor or size."""

    __slots__ = ("_codes", "_scales", "_buffer", "_codes_ptr", "_scales_ptr", "_ld", "_rows", "_cols", "_format",
                 "_global_scale")
    rows, cols, format = _read_only("_rows"), _read_only("_cols"), _read_only("_format")
    global_scale = _read_only("_global_scale")

    def __init__(self, codes, scales, rows, cols, format="mxfp4", global_scale=None):
        if format not in _FORMATS:
            raise ValueError(f"unknown 4-bit format {format!r} (mxfp4 or nvfp4)")
        if (not isinstance(codes, torch.Tensor) or not isinstance(scales, torch.Tensor) or codes.dtype != _u8
                or scales.dtype != _u8 or not codes.is_cuda or not scales.is_cuda):
            raise TypeError("codes and scales must be uint8 CUDA tensors")
        if codes.dim() != 2 or codes.size(0) != rows or codes.size(1) < (cols + 31) // 32 * 16:
            raise ValueError("codes must be [rows, at least ceil(cols / 32) * 16]")
        if not scales.is_contiguous() or scales.numel() < self.scales_size(rows, cols, format):
            raise ValueError("scales must be contiguous and hold hk_fp4_scales_size bytes")
        self._ld = _row_stride(codes, "codes")
        self._buffer = None
        self._codes, self._scales, self._rows, self._cols, self._format = codes, scales, rows, cols, format
        self._codes_ptr, self._scales_ptr = codes.data_ptr(), scales.data_ptr()
        self._global_scale = None if global_scale is None else _checked_global_scale(global_scale, format)

    # (quantize_fp4 allocates once for both arrays; what nobody looks at needs no views)
    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._buffer[self._scales_bytes:].view(self.rows, self._ld)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._buffer[: self._scales_bytes]
        return self._scales

    @property
    def _any(self):
        return self._codes if self._buffer is None else self._buffer

    @property
    def _scales_bytes(self):
        return self.scales_size(self.rows, self.cols, self.format)

    @staticmethod
    def scales_size(rows, cols, format):
        """Bytes of the scales (hk_fp4_scales_size)."""
        return (rows + 127) // 128 * 128 * ((cols + 255) // 256 * (256 // _BLOCK[format]))

    @property
    def shape(self):
        return (self._rows, self._cols)

    def scale_matrix(self):
        """The block scales' bytes as [rows, ceil(cols / block)] (UE8M0 or E4M3)."""
        blk = _BLOCK[self.format]
        nb = -(-self.cols // 256) * (256 // blk)
        s = self.scales.view(-1)[: self._scales_bytes]
        s = s.view(-1, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, nb)
        return s[: self.rows, : -(-self.cols // blk)]


def quantize_fp4(x, format="mxfp4", global_scale=None, out=None, stream=None) -> Fp4Matrix:
    """Quantise a 2-D bf16, fp16 or fp32 CUDA tensor; rows contiguous, any row stride.

    ``global_scale`` (NVFP4): the matrix's scale g on the device; its largest
    magnitude / 2688 uses the whole range (None: 1). ``out``: an Fp4Matrix of
    the same shape and format to write into."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise TypeError("x must be a 2-D CUDA tensor")
    code = _type_code(x, "x")
    fmt = _FORMATS.get(format)
    if fmt is None:
        raise ValueError(f"unknown 4-bit format {format!r} (mxfp4 or nvfp4)")
    if global_scale is not None:
        _checked_global_scale(global_scale, format)
    rows, cols = x.shape
    ldx = _row_stride(x, "x")
    if out is None:
        out = Fp4Matrix.__new__(Fp4Matrix)
        out._ld = ld = (cols + 31) // 32 * 16
        size = Fp4Matrix.scales_size(rows, cols, format)      # (a multiple of 1024: the codes behind it are aligned)
        out._buffer = buffer = _empty(size + rows * ld, _u8, x, stream)
        out._codes = out._scales = None
        out._scales_ptr = ptr = buffer.data_ptr()
        out._codes_ptr = ptr + size
        out._rows, out._cols, out._format = rows, cols, format
    elif not isinstance(out, Fp4Matrix):
        raise TypeError("out must be an Fp4Matrix")
    elif out._rows != rows or out._cols != cols or out._format != format:
        raise ValueError("out must have x's shape and the asked format")
    st = _hk.load().hk_fp4_quantize(x.data_ptr(), code, rows, cols, ldx, out._codes_ptr, out._ld, out._scales_ptr, fmt,
                                    None if global_scale is None else global_scale.data_ptr(), _stream(stream, x))
    if st != HK_OK:
        raise HKError(st, "hk_fp4_quantize")
    out._global_scale = global_scale
    return out


def dequantize_fp4(q: Fp4Matrix, dtype=None, out=None, stream=None):
    """The values of a quantised matrix (default bf16)."""
    if not isinstance(q, Fp4Matrix):
        raise TypeError("q must be an Fp4Matrix (see quantize_fp4)")
    if out is None:
        out = _empty((q._rows, q._cols), dtype or _bf16, q._any, stream)
    elif tuple(out.shape) != q.shape or (dtype is not None and out.dtype != dtype) or not out.is_cuda:
        raise ValueError("out must be a CUDA tensor of the matrix's shape and the asked type")
    g = q._global_scale
    st = _hk.load().hk_fp4_dequantize(q._codes_ptr, q._ld, q._scales_ptr, _FORMATS[q._format],
                                      None if g is None else g.data_ptr(), q._rows, q._cols, out.data_ptr(),
                                      _type_code(out, "out"), _row_stride(out, "out"), _stream(stream, out))
    if st != HK_OK:
        raise HKError(st, "hk_fp4_dequantize")
    return out


def gemm_fp4(a: Fp4Matrix, b: Fp4Matrix, out=None, stream=None):
    """C = A·Bᵀ in bf16 for quantised A (M×K) and B (N×K) of one format."""
    if not isinstance(a, Fp4Matrix) or not isinstance(b, Fp4Matrix):
        raise TypeError("a and b must be Fp4Matrix (see quantize_fp4)")
    if a._cols != b._cols or a._format != b._format:
        raise ValueError(f"a [{a._rows}, {a._cols}] {a._format} and b [{b._rows}, {b._cols}] {b._format} do not match")
    M, N = a._rows, b._rows
    if out is None:
        out = _empty((M, N), _bf16, a._any, stream)
        ldc = N
    else:
        if tuple(out.shape) != (M, N) or out.dtype != _bf16 or not out.is_cuda:
            raise ValueError("out must be a bfloat16 CUDA tensor [a.rows, b.rows]")
        ldc = _row_stride(out, "out")
    ga, gb = a._global_scale, b._global_scale
    st = _hk.load().hk_gemm_fp4(a._codes_ptr, a._scales_ptr, b._codes_ptr, b._scales_ptr, out.data_ptr(), M, N, a._cols, a._ld, b._ld, ldc, _FORMATS[a._format],
                                None if ga is None else ga.data_ptr(), None if gb is None else gb.data_ptr(),
                                _stream(stream, out))
    if st != HK_OK:
        raise HKError(st, "hk_gemm_fp4")
    return out


class Kv8Cache:
    """A paged key/value cache in E4M3 with a power-of-two scale per page and head.

    ``k``, ``v``: uint8 [pages, heads, page_size, head_dim]; ``k_scale``,
    ``v_scale``: float32 [pages, heads]; all contiguous CUDA tensors.
    ``Kv8Cache.empty`` makes them. None of them can be set to another tensor: a
    larger pool is a new Kv8Cache over tensors that the old ones were copied to."""

    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_pages", "_heads", "_page_size", "_head_dim", "_ref")
    k, v, k_scale, v_scale = (_read_only(n) for n in __slots__[:4])
    pages, heads, page_size, head_dim = (_read_only(n) for n in __slots__[4:8])

    def __init__(self, k, v, k_scale, v_scale):
        for t, dtype in ((k, _u8), (v, _u8), (k_scale, _f32), (v_scale, _f32)):
            if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
                raise TypeError("k and v must be uint8, k_scale and v_scale float32 CUDA tensors")
            if not t.is_contiguous():
                raise ValueError("a cache's tensors must be contiguous")
        shape = tuple(k.shape)
        if len(shape) != 4 or tuple(v.shape) != shape or tuple(k_scale.shape) != shape[:2] or tuple(v_scale.shape) != shape[:2]:
            raise ValueError("k and v must be [pages, heads, page_size, head_dim], the scales [pages, heads]")
        self._k, self._v, self._k_scale, self._v_scale = k, v, k_scale, v_scale
        self._pages, self._heads, self._page_size, self._head_dim = shape
        self._ref = _cache_struct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *shape, 0)

    @classmethod
    def empty(cls, pages, heads, head_dim, page_size=64, device="cuda"):
        """A cache of `pages` pages; nothing needs to be initialised."""
        shape = (pages, heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=_u8, device=device), torch.empty(shape, dtype=_u8, device=device),
                   torch.empty(shape[:2], dtype=_f32, device=device), torch.empty(shape[:2], dtype=_f32, device=device))


def _tokens_shape(t, name, cache, all_heads):
    """(B, T, heads) and packed strides of [B, T, heads, head_dim]."""
    if not isinstance(cache, Kv8Cache):
        raise TypeError("cache must be a Kv8Cache")
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4:
        raise TypeError(f"{name} must be a CUDA tensor [B, T, heads, head_dim]")
    B, T, H, D = t.shape
    sb, st, sh, sd = t.stride()
    if D != cache._head_dim or (all_heads and H != cache._heads):
        raise ValueError(f"{name} {tuple(t.shape)} does not fit the cache ({cache._heads} heads of {cache._head_dim})")
    if sd != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    return B, T, H, _strides(sb, st, sh)


def _check_vector(t, name, B):
    if not isinstance(t, torch.Tensor) or t.dtype != _i32 or not t.is_cuda or t.dim() != 1:
        raise TypeError(f"{name} must be a 1-D int32 CUDA tensor")
    if t.size(0) != B or (B > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be {B} contiguous entries")


def _table(t, B):
    """(row stride, pages per sequence) of a block table."""
    if not isinstance(t, torch.Tensor) or t.dtype != _i32 or not t.is_cuda or t.dim() != 2:
        raise TypeError("block_table must be a 2-D int32 CUDA tensor")
    if t.size(0) != B:
        raise ValueError(f"block_table has {t.size(0)} rows for {B} sequences")
    return _row_stride(t, "block_table"), t.size(1)


def kv8_append(cache: Kv8Cache, k, v, block_table, starts, counts=None, stream=None) -> None:
    """Append k, v [B, T, heads, head_dim] (bf16, fp16 or fp32) to B sequences
    that hold ``starts`` tokens; ``counts``: of each sequence's T tokens the first
    so many (None: all). ``block_table`` [B, max_pages], ``starts``, ``counts``
    [B]: int32. See hk_kv8_append for the scales."""
    B, T, _, ks = _tokens_shape(k, "k", cache, True)
    vb, vt, _, vs = _tokens_shape(v, "v", cache, True)
    if vb != B or vt != T or v.dtype != k.dtype:
        raise ValueError("v must have k's shape and type")
    ld, pages = _table(block_table, B)
    _check_vector(starts, "starts", B)
    if counts is not None:
        _check_vector(counts, "counts", B)
    st = _hk.load().hk_kv8_append(cache._ref, k.data_ptr(), v.data_ptr(), _type_code(k, "k"), B, T, ks, vs,
                                  block_table.data_ptr(), ld, pages, starts.data_ptr(),
                                  None if counts is None else counts.data_ptr(), _stream(stream, k))
    if st != HK_OK:
        raise HKError(st, "hk_kv8_append")


def attention_kv8(q, cache: Kv8Cache, block_table, lengths, counts=None, causal=True, scale=None, return_lse=False,
                  out=None, stream=None):
    """softmax(scale · q·Kᵀ)·V over the cached tokens of each sequence.

    q [B, T, Hq, head_dim] (bf16 or fp16, any strides with contiguous rows),
    ``lengths`` [B] int32: cached tokens, the queries' own among them; with
    ``causal`` query t stands at position lengths - counts + t (``counts`` [B]
    int32: valid queries of each sequence, None: T). Queries that see no token,
    or lie past ``counts``, give zeros. Returns o [B, T, Hq, head_dim] (and the
    fp32 log-sum-exp [B, T, Hq] with ``return_lse``). ``scale``: 1/sqrt(head_dim)."""
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
    if out is None:
        out = _empty((B, T, Hq, cache._head_dim), q.dtype, q, stream)
        os = _strides(T * Hq * cache._head_dim, Hq * cache._head_dim, cache._head_dim)
    else:
        if not isinstance(out, torch.Tensor) or out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out must have q's shape and type")
        os = _tokens_shape(out, "out", cache, False)[3]
    lse = _empty((B, T, Hq), _f32, q, stream) if return_lse else None
    lib = _hk.load()
    size = lib.hk_attention_kv8_workspace_size(cache._ref, B, T, Hq, pages)
    if size:               # (enough for any type and strides; this call may need less)
        size = lib.hk_attention_kv8_workspace_size_ex(q.data_ptr(), code, qs, cache._ref, pages, out.data_ptr(), os, B, T, Hq, 0)
    workspace = _empty(size, _u8, q, stream) if size else None
    st = lib.hk_attention_kv8(q.data_ptr(), code, qs, cache._ref, block_table.data_ptr(), ld, pages, lengths.data_ptr(),
                              None if counts is None else counts.data_ptr(), out.data_ptr(), os,
                              None if lse is None else lse.data_ptr(), B, T, Hq, 1 if causal else 0, scale,
                              None if workspace is None else workspace.data_ptr(), size, _stream(stream, q))
    if st != HK_OK:
        raise HKError(st, "hk_attention_kv8")
    return (out, lse) if return_lse else out
