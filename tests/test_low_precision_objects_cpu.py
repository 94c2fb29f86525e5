"""Quantised matrices and caches keep the pointers that the kernels get: what
they were made with cannot be exchanged behind those."""
import pytest


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "pages", "heads", "page_size", "head_dim"])
def test_a_cache_keeps_its_tensors_and_sizes(name):
    from dense_bf16_gemm_02_gb300 import Kv8Cache
    cache = Kv8Cache.__new__(Kv8Cache)
    with pytest.raises(AttributeError):
        setattr(cache, name, 1)
    setattr(cache, "_" + name, 7)
    assert getattr(cache, name) == 7


@pytest.mark.parametrize("name", ["rows", "cols", "format", "global_scale", "codes", "scales"])
def test_a_quantised_matrix_keeps_its_tensors_and_sizes(name):
    from dense_bf16_gemm_02_gb300 import Fp4Matrix
    q = Fp4Matrix.__new__(Fp4Matrix)
    with pytest.raises(AttributeError):
        setattr(q, name, 1)
    setattr(q, "_" + name, 7)
    assert getattr(q, name) == 7


@pytest.mark.parametrize("scale", [0, 0.0, -0.0, 1e-50, -1e-60])
def test_a_scale_that_is_0_in_32_bits_is_refused(scale, monkeypatch):
    """(0 asks the entry point for its default, so it must not be what a small scale rounds to)"""
    import torch

    from dense_bf16_gemm_02_gb300 import Kv8Cache, low_precision
    monkeypatch.setattr(low_precision, "_tokens_shape", lambda *a: (1, 1, 1, b""))
    with pytest.raises(ValueError, match="scale"):
        low_precision.attention_kv8(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), Kv8Cache.__new__(Kv8Cache), None, None,
                                    scale=scale)


def test_an_output_whose_rows_overlap_is_refused():
    import ctypes

    from dense_bf16_gemm_02_gb300 import build, hk_gemm as h
    build.build()
    lib, P, I3 = h.load(), 1 << 20, ctypes.c_int64 * 3
    cache = h.hk_kv8_cache(k_codes=P, v_codes=P, k_scale=P, v_scale=P, num_pages=4, heads=2, page_size=64, head_dim=64)

    def call(strides, B=2, T=3, Hq=4):
        return lib.hk_attention_kv8(P, 0, I3(768, 256, 64), ctypes.byref(cache), P, 4, 4, P, None, P, I3(*strides), None, B, T, Hq,
                                    1, 0.0, P, 1 << 40, None)
    for bad in ((0, 256, 64), (768, 0, 64), (768, 256, 0), (768, 256, 63), (768, -32, 64), (1, 256, 64)):
        assert call(bad) == h.HK_ERR_INVALID_ARG, bad
    for good in ((768, 256, 64), (64, 128, 384), (-768, 256, 64)):
        assert call(good) != h.HK_ERR_INVALID_ARG, good
    assert call((0, 256, 64), B=1) != h.HK_ERR_INVALID_ARG and call((64, 1, 128), B=2, T=1) != h.HK_ERR_INVALID_ARG
