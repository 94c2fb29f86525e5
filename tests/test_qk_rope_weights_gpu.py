"""Weights belong to the norm: without it (eps None, below 0 in C) they are not looked at."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,pairs", [(64, 32), (128, 24), (16, 0)])
def test_no_norm_takes_no_weights(dtype, interleaved, D, pairs):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    g = torch.Generator(device="cuda").manual_seed(D + pairs)
    q, k = (torch.randn(2, 5, h, D, generator=g, device="cuda").to(getattr(torch, dtype)) for h in (6, 2))
    pos = torch.randint(0, 4000, (2, 5), generator=g, device="cuda", dtype=torch.int32)
    freq = torch.rand(pairs, generator=g, device="cuda")
    plain = hk.qk_norm_rope(q, k, pos, freq, eps=None, interleaved=interleaved)
    for weights in ((torch.full((D,), 3.0, device="cuda"), torch.full((D,), float("nan"), device="cuda")),
                    (torch.full((D,), 0.5, device="cuda", dtype=q.dtype), None)):
        got = hk.qk_norm_rope(q, k, pos, freq, *weights, eps=None, interleaved=interleaved)
        assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    assert torch.equal(plain[0][..., 2 * pairs:], q[..., 2 * pairs:])         # (what is not turned is as it was)
