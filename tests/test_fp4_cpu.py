"""The 4-bit entry points without a GPU: refusals, sizes, and the plain
reference that the GPU tests compare with, pinned by the formats' own tables."""
import numpy as np
import pytest

import fp4_ref as ref


@pytest.fixture(scope="module")
def lib():
    from dense_bf16_gemm_02_gb300 import build
    build.build()
    from dense_bf16_gemm_02_gb300 import hk_gemm
    return hk_gemm.load()


P = 1 << 20      # a 16-byte aligned address that is never read on these paths


def test_quantize_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED

    def q(X=P, t=0, rows=4, cols=64, ldx=64, codes=P, ld=32, scales=P, fmt=0, g=None):
        return lib.hk_fp4_quantize(X, t, rows, cols, ldx, codes, ld, scales, fmt, g, None)
    assert q(rows=0, X=None, codes=None, scales=None) == h.HK_OK and q(cols=0, ldx=0, ld=0) == h.HK_OK
    assert q(rows=-1) == INV and q(cols=-1) == INV and q(rows=1 << 31) == INV
    assert q(fmt=2) == INV and q(t=3) == INV and q(t=-1) == INV
    assert q(ldx=63) == INV and q(ld=16) == INV and q(cols=65, ldx=65, ld=32) == INV
    assert q(X=None) == INV and q(codes=None) == INV and q(scales=None) == INV
    assert q(ld=40) == MIS and q(codes=P + 8) == MIS and q(scales=P + 4) == MIS and q(X=P + 1) == MIS
    assert q(fmt=0, g=P) == INV and q(fmt=1, g=P + 2) == MIS

    def d(codes=P, ld=32, scales=P, fmt=0, g=None, rows=4, cols=64, Y=P, t=0, ldy=64):
        return lib.hk_fp4_dequantize(codes, ld, scales, fmt, g, rows, cols, Y, t, ldy, None)
    assert d(rows=0) == h.HK_OK and d(ldy=60) == INV and d(Y=None) == INV and d(t=7) == INV and d(Y=P + 1) == MIS
    assert d(fmt=-1) == INV and d(ld=24) == INV and d(codes=P + 4) == MIS


def test_product_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED

    def g(A=P, SA=P, B=P, SB=P, C=P, M=8, N=8, K=64, lda=32, ldb=32, ldc=8, fmt=1, ga=None, gb=None, flags=0,
          kernel=0, split=0):
        return lib.hk_gemm_fp4_ex(A, SA, B, SB, C, M, N, K, lda, ldb, ldc, fmt, ga, gb, kernel, split, flags, 0, None)
    assert g(M=0, A=None) == h.HK_OK and g(N=0, ldc=0, B=None) == h.HK_OK
    assert g(M=-1) == INV and g(K=-1) == INV and g(K=1 << 31) == INV and g(ldc=7) == INV
    assert g(lda=16) == INV and g(ldb=16) == INV and g(lda=40) == MIS and g(ldb=40) == MIS
    assert g(A=None) == INV and g(SA=None) == INV and g(B=None) == INV and g(SB=None) == INV and g(C=None) == INV
    assert g(A=P + 8) == MIS and g(SA=P + 8) == MIS and g(B=P + 8) == MIS and g(SB=P + 8) == MIS and g(C=P + 1) == MIS
    assert g(fmt=0, ga=P) == INV and g(fmt=0, gb=P) == INV and g(ga=P + 1) == MIS and g(fmt=5) == INV
    assert g(flags=2) == INV and g(kernel=2) == INV and g(kernel=9) == INV and g(split=3) == INV and g(split=16) == INV
    assert lib.hk_gemm_fp4(P, P, P, P, P, 8, 8, 64, 32, 32, 7, 0, None, None, None) == INV


def test_scales_size(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    assert h.hk_fp4_scales_size(1, 1, 0) == 128 * 8 and h.hk_fp4_scales_size(1, 1, 1) == 128 * 16
    assert h.hk_fp4_scales_size(129, 257, 0) == 256 * 16 and h.hk_fp4_scales_size(129, 257, 1) == 256 * 32
    assert h.hk_fp4_scales_size(0, 5, 0) == 0 and h.hk_fp4_scales_size(5, 5, 9) == 0
    assert h.hk_fp4_scales_size(1 << 30, 1 << 20, 1) == (1 << 30) * ((1 << 20) // 16)     # passes 32 bits
    for rows, cols in ((1, 1), (300, 1000), (128, 256)):
        for fmt, code in (("mxfp4", 0), ("nvfp4", 1)):
            byte = np.ones((rows, -(-cols // ref.BLOCK[fmt])), dtype=np.uint8)
            t = ref.tile_scales(byte, cols, fmt)
            assert t.size == h.hk_fp4_scales_size(rows, cols, code) and int(t.sum()) == byte.size


def test_reference_rounds_to_the_formats_tables():
    # every E4M3 number is its own rounding, and halves go to the even one
    all_e4m3 = ref.e4m3_value(np.arange(0x7F))
    assert np.array_equal(ref.half_even(all_e4m3, 3, -6, 448.0), all_e4m3)
    assert np.array_equal(ref.e4m3_byte(all_e4m3), np.arange(0x7F, dtype=np.uint8))
    mid = (all_e4m3[:-1] + all_e4m3[1:]) / 2
    assert np.array_equal(ref.e4m3_byte(ref.half_even(mid, 3, -6, 448.0)) % 2, np.zeros(len(mid)))
    mid = (ref.GRID[:-1] + ref.GRID[1:]) / 2
    assert np.array_equal(ref.half_even(mid, 1, 0, 6.0), [0, 1, 1, 2, 2, 4, 4])
    assert np.array_equal(ref.half_even([7, 100, -9], 1, 0, 6.0), [6, 6, -6])
    code, byte = ref.quantize(np.array([[8.0] + [1.0] * 31], dtype=np.float32), "mxfp4")
    assert byte[0, 0] == 128 and code[0, 0] == 6 and code[0, 1] == 1       # 2^1: 8 -> 4, 1 -> 0.5
    v = ref.values(code, byte, "mxfp4")
    assert v[0, 0] == 8.0 and v[0, 1] == 1.0
    code, byte = ref.quantize(np.array([[12.0] + [1.0] * 15], dtype=np.float32), "nvfp4", 1.0)
    assert byte[0, 0] == 0x40 and code[0, 0] == 7 and code[0, 1] == 1


def test_python_refusals():
    import torch

    import dense_bf16_gemm_02_gb300 as hk
    with pytest.raises(TypeError):
        hk.quantize_fp4(torch.zeros(4, 64))                    # not on the GPU
    with pytest.raises(ValueError):
        hk.Fp4Matrix(None, None, 1, 1, "fp4")
    with pytest.raises(TypeError):
        hk.Fp4Matrix(torch.zeros(1, 16, dtype=torch.uint8), torch.zeros(2048, dtype=torch.uint8), 1, 1)
    with pytest.raises(TypeError):
        hk.gemm_fp4(None, None)


def test_what_is_no_quantised_matrix_is_refused():
    import torch

    from dense_bf16_gemm_02_gb300 import dequantize_fp4, gemm_fp4
    x = torch.zeros(4, 32)
    for f in (lambda: dequantize_fp4(x), lambda: dequantize_fp4(None), lambda: gemm_fp4(x, x)):
        with pytest.raises(TypeError):
            f()
