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
