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
