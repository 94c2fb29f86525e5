"""Torch conveniences over the low-precision serving entry points of
``include/hk_gemm.h``: matrices in microscaled 4-bit floating point
(``quantize_fp4``, ``dequantize_fp4``, ``gemm_fp4``), and a paged key/value
cache in 8 bits (``Kv8Cache``, ``kv8_append``, ``attention_kv8``).

As in ``hk_gemm``, this is argument marshalling: every step runs in the CUDA
library, on ``stream`` (default: torch's current stream). What a call
allocates comes from torch's allocator, for that stream.
"""
from __future__ import annotations

import contextlib

from . import hk_gemm as _hk
from .hk_gemm import HK_OK, HKError, _stream_handle

_FORMATS = {"mxfp4": _hk.HK_FP4_MXFP4, "nvfp4": _hk.HK_FP4_NVFP4}
_FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}


def _on(stream):
    """Allocations inside belong to `stream`, so that they may be freed as soon as the call is enqueued."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _type_code(dtype):
    import torch
    code = {torch.bfloat16: _hk.HK_TYPE_BF16, torch.float16: _hk.HK_TYPE_FP16, torch.float32: _hk.HK_TYPE_FP32}.get(dtype)
    if code is None:
        raise TypeError(f"unsupported element type {dtype} (bfloat16, float16 or float32)")
    return code


def _row_stride(t, name):
    """Leading dimension of a 2-D tensor whose rows are contiguous."""
    if t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if t.size(0) <= 1:
        return t.size(1)
    if t.stride(0) < t.size(1):
        raise ValueError(f"{name}'s rows must not overlap")
    return t.stride(0)


def _check(status, where):
    if status != HK_OK:
        raise HKError(status, where)


class Fp4Matrix:
    """A rows × cols matrix in ``format`` "mxfp4" or "nvfp4" (see hk_fp4_quantize).

    ``codes``: uint8 [rows, ld], two codes per byte; ``scales``: uint8, the
    block scales in 128×4 tiles; ``global_scale``: a float32 CUDA tensor of one
    element (NVFP4 only) or None."""

    __slots__ = ("codes", "scales", "rows", "cols", "format", "global_scale")

    def __init__(self, codes, scales, rows, cols, format="mxfp4", global_scale=None):
        import torch
        if format not in _FORMATS:
            raise ValueError(f"unknown 4-bit format {format!r} (mxfp4 or nvfp4)")
        for t, name in ((codes, "codes"), (scales, "scales")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or not t.is_cuda:
                raise TypeError(f"{name} must be a uint8 CUDA tensor")
        if codes.dim() != 2 or codes.size(0) != rows or codes.size(1) < -(-cols // 32) * 16:
            raise ValueError("codes must be [rows, at least ceil(cols / 32) * 16]")
        _row_stride(codes, "codes")
        if not scales.is_contiguous() or scales.numel() < self.scales_size(rows, cols, format):
            raise ValueError("scales must be contiguous and hold hk_fp4_scales_size bytes")
        self.codes, self.scales, self.rows, self.cols, self.format = codes, scales, rows, cols, format
        self.global_scale = _checked_global_scale(global_scale, format)

    @staticmethod
    def scales_size(rows, cols, format):
        """Bytes of the scales (hk_fp4_scales_size)."""
        return -(-rows // 128) * 128 * (-(-cols // 256) * (256 // _FP4_BLOCK[format]))

    @property
    def shape(self):
        return (self.rows, self.cols)

    def scale_matrix(self):
        """The block scales' bytes as [rows, ceil(cols / block)] (UE8M0 or E4M3)."""
        nb = -(-self.cols // 256) * (256 // _FP4_BLOCK[self.format])
        s = self.scales[: self.scales_size(self.rows, self.cols, self.format)]
        s = s.view(-1, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, nb)
        return s[: self.rows, : -(-self.cols // _FP4_BLOCK[self.format])]


def _checked_global_scale(g, format):
    import torch
    if g is None:
        return None
    if format != "nvfp4":
        raise ValueError("only nvfp4 has a global scale")
    if not isinstance(g, torch.Tensor) or g.dtype != torch.float32 or not g.is_cuda or g.numel() != 1:
        raise TypeError("global_scale must be a float32 CUDA tensor of one element")
    return g


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def quantize_fp4(x, format="mxfp4", global_scale=None, out=None, stream=None) -> Fp4Matrix:
    """Quantise a 2-D bf16, fp16 or fp32 CUDA tensor; rows contiguous, any row stride.

    ``global_scale`` (NVFP4): the matrix's scale g on the device; its largest
    magnitude / 2688 uses the whole range (None: 1). ``out``: an Fp4Matrix of
    the same shape and format to write into."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise TypeError("x must be a 2-D CUDA tensor")
    code = _type_code(x.dtype)
    if format not in _FORMATS:
        raise ValueError(f"unknown 4-bit format {format!r} (mxfp4 or nvfp4)")
    rows, cols = x.shape
    ldx = _row_stride(x, "x")
    if out is None:
        with _on(stream):
            out = Fp4Matrix(torch.empty((rows, -(-cols // 32) * 16), dtype=torch.uint8, device=x.device),
                            torch.empty(Fp4Matrix.scales_size(rows, cols, format), dtype=torch.uint8, device=x.device),
                            rows, cols, format, global_scale)
    else:
        if out.shape != (rows, cols) or out.format != format:
            raise ValueError("out must have x's shape and the asked format")
        out.global_scale = _checked_global_scale(global_scale, format)
    _check(_hk.hk_fp4_quantize(x.data_ptr(), code, rows, cols, ldx, out.codes.data_ptr(), _row_stride(out.codes, "codes"),
                               out.scales.data_ptr(), _FORMATS[format], _ptr(global_scale), _stream_handle(stream)),
           "hk_fp4_quantize")
    return out


def dequantize_fp4(q: Fp4Matrix, dtype=None, out=None, stream=None):
    """The values of a quantised matrix (default bf16)."""
    import torch
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=dtype or torch.bfloat16, device=q.codes.device)
    elif tuple(out.shape) != q.shape or (dtype is not None and out.dtype != dtype) or not out.is_cuda:
        raise ValueError("out must be a CUDA tensor of the matrix's shape and the asked type")
    _check(_hk.hk_fp4_dequantize(q.codes.data_ptr(), _row_stride(q.codes, "codes"), q.scales.data_ptr(), _FORMATS[q.format],
                                 _ptr(q.global_scale), q.rows, q.cols, out.data_ptr(), _type_code(out.dtype),
                                 _row_stride(out, "out"), _stream_handle(stream)),
           "hk_fp4_dequantize")
    return out


def gemm_fp4(a: Fp4Matrix, b: Fp4Matrix, out=None, stream=None):
    """C = A·Bᵀ in bf16 for quantised A (M×K) and B (N×K) of one format."""
    import torch
    if not isinstance(a, Fp4Matrix) or not isinstance(b, Fp4Matrix):
        raise TypeError("a and b must be Fp4Matrix (see quantize_fp4)")
    if a.cols != b.cols or a.format != b.format:
        raise ValueError(f"a [{a.rows}, {a.cols}] {a.format} and b [{b.rows}, {b.cols}] {b.format} do not match")
    if out is None:
        with _on(stream):
            out = torch.empty((a.rows, b.rows), dtype=torch.bfloat16, device=a.codes.device)
    elif tuple(out.shape) != (a.rows, b.rows) or out.dtype != torch.bfloat16 or not out.is_cuda:
        raise ValueError("out must be a bfloat16 CUDA tensor [a.rows, b.rows]")
    _check(_hk.hk_gemm_fp4(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                           out.data_ptr(), a.rows, b.rows, a.cols, _row_stride(a.codes, "codes"), _row_stride(b.codes, "codes"),
                           _row_stride(out, "out"), _FORMATS[a.format], _ptr(a.global_scale), _ptr(b.global_scale),
                           _stream_handle(stream)),
           "hk_gemm_fp4")
    return out


class Kv8Cache:
    """A paged key/value cache in E4M3 with a power-of-two scale per page and head.

    ``k``, ``v``: uint8 [pages, heads, page_size, head_dim]; ``k_scale``,
    ``v_scale``: float32 [pages, heads]; all contiguous CUDA tensors.
    ``Kv8Cache.empty`` makes them."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "_c")

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        for t, name, dtype, dims in ((k, "k", torch.uint8, 4), (v, "v", torch.uint8, 4),
                                     (k_scale, "k_scale", torch.float32, 2), (v_scale, "v_scale", torch.float32, 2)):
            if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or t.dim() != dims:
                raise TypeError(f"{name} must be a {dims}-D {dtype} CUDA tensor")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if v.shape != k.shape or k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2]:
            raise ValueError("v must have k's shape, the scales [pages, heads]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        pages, heads, page_size, head_dim = k.shape
        self._c = _hk.hk_kv8_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads,
                                   page_size, head_dim, 0)

    @classmethod
    def empty(cls, pages, heads, head_dim, page_size=64, device="cuda"):
        """A cache of `pages` pages; nothing needs to be initialised."""
        import torch
        shape = (pages, heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=torch.uint8, device=device), torch.empty(shape, dtype=torch.uint8, device=device),
                   torch.empty(shape[:2], dtype=torch.float32, device=device),
                   torch.empty(shape[:2], dtype=torch.float32, device=device))

    pages = property(lambda self: self.k.size(0))
    heads = property(lambda self: self.k.size(1))
    page_size = property(lambda self: self.k.size(2))
    head_dim = property(lambda self: self.k.size(3))


def _check_tokens(t, name, cache, heads):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4:
        raise TypeError(f"{name} must be a CUDA tensor [B, T, heads, head_dim]")
    if t.size(3) != cache.head_dim or (heads and t.size(2) != heads):
        raise ValueError(f"{name} {tuple(t.shape)} does not fit the cache ({cache.heads} heads of {cache.head_dim})")
    if t.stride(3) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def _check_index(t, name, shape_dims, B):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or t.dim() != shape_dims:
        raise TypeError(f"{name} must be a {shape_dims}-D int32 CUDA tensor")
    if t.size(0) != B:
        raise ValueError(f"{name} has {t.size(0)} entries for {B} sequences")
    if t.size(-1) > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")


def kv8_append(cache: Kv8Cache, k, v, block_table, starts, counts=None, stream=None) -> None:
    """Append k, v [B, T, heads, head_dim] (bf16, fp16 or fp32) to B sequences
    that hold ``starts`` tokens; ``counts``: of each sequence's T tokens the first
    so many (None: all). ``block_table`` [B, max_pages], ``starts``, ``counts``
    [B]: int32. See hk_kv8_append for the scales."""
    _check_tokens(k, "k", cache, cache.heads)
    _check_tokens(v, "v", cache, cache.heads)
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("v must have k's shape and type")
    B, T = k.shape[:2]
    _check_index(block_table, "block_table", 2, B)
    _check_index(starts, "starts", 1, B)
    if counts is not None:
        _check_index(counts, "counts", 1, B)
    _check(_hk.hk_kv8_append(cache._c, k.data_ptr(), v.data_ptr(), _type_code(k.dtype), B, T, k.stride()[:3],
                             v.stride()[:3], block_table.data_ptr(), block_table.stride(0), block_table.size(1),
                             starts.data_ptr(), _ptr(counts), _stream_handle(stream)),
           "hk_kv8_append")


def attention_kv8(q, cache: Kv8Cache, block_table, lengths, counts=None, causal=True, scale=None, return_lse=False,
                  out=None, stream=None):
    """softmax(scale · q·Kᵀ)·V over the cached tokens of each sequence.

    q [B, T, Hq, head_dim] (bf16 or fp16, any strides with contiguous rows),
    ``lengths`` [B] int32: cached tokens, the queries' own among them; with
    ``causal`` query t stands at position lengths - counts + t (``counts`` [B]
    int32: valid queries of each sequence, None: T). Queries that see no token,
    or lie past ``counts``, give zeros. Returns o [B, T, Hq, head_dim] (and the
    fp32 log-sum-exp [B, T, Hq] with ``return_lse``). ``scale``: 1/sqrt(head_dim)."""
    import torch
    _check_tokens(q, "q", cache, 0)
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q must be bfloat16 or float16")
    if scale is not None and not scale:
        raise ValueError("scale must not be 0")
    B, T, Hq = q.shape[:3]
    _check_index(block_table, "block_table", 2, B)
    _check_index(lengths, "lengths", 1, B)
    if counts is not None:
        _check_index(counts, "counts", 1, B)
    size = _hk.hk_attention_kv8_workspace_size(cache._c, B, T, Hq, block_table.size(1))
    with _on(stream):
        if out is None:
            out = torch.empty((B, T, Hq, cache.head_dim), dtype=q.dtype, device=q.device)
        elif out.shape != q.shape or out.dtype != q.dtype or not out.is_cuda or out.stride(3) != 1:
            raise ValueError("out must have q's shape and type, rows contiguous")
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    _check(_hk.hk_attention_kv8(q.data_ptr(), _type_code(q.dtype), q.stride()[:3], cache._c, block_table.data_ptr(),
                                block_table.stride(0), block_table.size(1), lengths.data_ptr(), _ptr(counts),
                                out.data_ptr(), out.stride()[:3], _ptr(lse), B, T, Hq, int(causal),
                                0.0 if scale is None else scale, workspace.data_ptr(), size, _stream_handle(stream)),
           "hk_attention_kv8")
    return (out, lse) if return_lse else out
