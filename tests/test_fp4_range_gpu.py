"""NVFP4 with global scales down to fp32's smallest numbers.

A power of two times the matrix and its global scale changes no code and no block
scale, so the codes are those of the same matrix 2^64 times as large, whose fp32
steps leave nothing to the subnormal numbers. The values on the way back are
code · s · g in 64 bits; they are off by the rounding of s·g (2^-24), the product's
(2^-24), where they are fp32's subnormals by half of 2^-149 for each of two
roundings, and by half a step of the output's type, which below its normal numbers
is 2^-150 (fp32), 2^-134 (bf16) or 2^-25 (fp16)."""
from __future__ import annotations

import numpy as np
import pytest

import fp4_ref as ref
from test_fp4_gpu import hk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

SCALES = [2.0 ** -58, 2.0 ** -60, 2.0 ** -61, 1.7e-30, 1.1e-38, 4e-39, 1e-41, 7e-45, 1.4e-45]


def _matrix(g, dtype, seed):
    """Zeros, values that use the whole range of g and values far below it, in fp32 (rounded to dtype)."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((9, 100)) * np.exp2(rng.integers(-14, 10, (9, 1))) * g
    x[rng.random(x.shape) < 0.1] = 0
    x[3, :32] = 0
    x[4, 7] = np.nan
    x[5, 40] = 3e38                    # saturates: 448 and 6
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("g", SCALES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_with_a_small_global_scale(hk, g, dtype):  # noqa: F811
    import torch
    x = _matrix(g, getattr(torch, dtype), 3)
    gt = torch.tensor([g], dtype=torch.float32, device="cuda")
    g = float(gt.double().item())
    q = hk.quantize_fp4(x.cuda(), format="nvfp4", global_scale=gt)
    with np.errstate(over="ignore", invalid="ignore"):
        lifted = np.clip(x.double().numpy() * 2.0 ** 64, -3e38, 3e38).astype(np.float32)    # (the clipped saturate too)
    code, byte = ref.quantize(lifted, "nvfp4", np.float32(g * 2.0 ** 64))
    want = ref.pack(code)
    got = q.codes.cpu().numpy()
    assert np.array_equal(q.scale_matrix().cpu().numpy(), byte)
    assert np.array_equal(got, want), f"{(got != want).sum()} of {want.size} bytes differ"
    for out, half, least in ((torch.float32, 2.0 ** -24, 2.0 ** -150), (torch.bfloat16, 2.0 ** -8, 2.0 ** -134),
                             (torch.float16, 2.0 ** -11, 2.0 ** -25)):
        y = hk.dequantize_fp4(q, dtype=out).double().cpu().numpy()
        v = ref.values(code, byte, "nvfp4", g)
        assert np.array_equal(np.isnan(y), np.isnan(v))
        ok = np.abs(y - v) <= (half + 2.0 ** -23) * np.abs(v) + least + 2.0 ** -149
        assert (ok | np.isnan(v)).all()
    torch.cuda.synchronize()
    assert hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK


# products of global scales that fp32 does not hold, or barely, and sums that bring them back or do not
PRODUCTS = [(1e-23, 1e-22, 0), (3e-39, 2e30, 0), (1.4e-45, 1e38, 0), (1e-20, 1e-19, 0), (2e-25, 2e-25, 0), (1e25, 1e9, 0),
            (1e22, 3e17, 0), (1e22, 1e22, -8), (2e38, 1e-38, 0), (1e-30, 1e-30, 0), (1e30, 1e30, 0), (0.37, 1.9, 0), (1e-23, 1e-22, 8),
            (1e-24, 1e-22, 8), (3e-30, 2e-18, 8), (1.4e-45, 1e0, 8)]


@pytest.mark.parametrize("ga,gb,span", PRODUCTS)
@pytest.mark.parametrize("M,split", [(3, 1), (3, 4), (100, 2), (300, 0)])
def test_product_with_small_and_large_global_scales(hk, ga, gb, span, M, split):  # noqa: F811
    """Tolerance: test_fp4_gpu.py's, and half a step of bf16's and fp32's smallest numbers (2^-134, 2^-149)."""
    import torch
    from test_fp4_gpu import _forced
    N, K = 130, 2048
    rng = np.random.default_rng(M)

    def matrix(rows, g):
        code = rng.integers(0, 16, (rows, K)).astype(np.uint8)
        byte = rng.integers(0x28, 0x50, (rows, K // 16)).astype(np.uint8)
        if span:
            byte[:] = 1 if span < 0 else 0x7E                 # every block's scale E4M3's smallest, or its largest number
        gt = torch.tensor([g], dtype=torch.float32, device="cuda")
        m = hk.Fp4Matrix(torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(ref.tile_scales(byte, K, "nvfp4")).cuda(),
                         rows, K, "nvfp4", gt)
        return m, ref.values(code, byte, "nvfp4", float(gt.double().item()))
    (a, av), (b, bv) = matrix(M, ga), matrix(N, gb)
    got = _forced(hk, a, b, 4 if split else 1, split).double().cpu().numpy()
    want = av @ bv.T
    tol = 2.0 ** -8 * np.abs(want) + (K * 2.0 ** -27 + 2.0 ** -22) * (np.abs(av) @ np.abs(bv).T) + 2.0 ** -134 + 2.0 ** -149
    top = 2.0 ** 127 * (2 - 2.0 ** -8)                        # half a step above bf16's largest
    huge = np.abs(want) > top * (1 + 2.0 ** -7)
    near = ~huge & (np.abs(want) > top * (1 - 2.0 ** -7))      # may round to either
    assert np.array_equal(got[huge], np.sign(want[huge]) * np.inf)
    ok = np.abs(got - want) <= tol
    assert (ok | huge | near).all(), (got[~(ok | huge | near)][:4], want[~(ok | huge | near)][:4])
