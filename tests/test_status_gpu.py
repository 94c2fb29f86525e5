"""A captured launch whose wait ran out, and what later replays say."""
from __future__ import annotations

import pytest

from test_fp4_gpu import _random_matrix, hk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 300])
def test_every_replay_that_fails_is_reported(hk, M):  # noqa: F811
    """The launch drops a stage's arrival each time; the status is read, and so reset, between the replays."""
    import torch
    a, _ = _random_matrix(hk, M, 4096, "mxfp4", 1)
    b, _ = _random_matrix(hk, 256, 4096, "mxfp4", 2)
    out = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")
    hk.gemm_fp4(a, b, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert hk.hk_gemm_fp4_ex(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                                 out.data_ptr(), M, 256, 4096, 2048, 2048, 256, hk.HK_FP4_MXFP4,
                                 flags=hk.HK_FLAG_FAULT_DROP_ARRIVE, timeout_ns=5_000_000,
                                 stream=torch.cuda.current_stream().cuda_stream) == hk.HK_OK
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert hk.hk_gemm_last_device_status(0) == hk.HK_ERR_TIMEOUT
    hk.gemm_fp4(a, b, out=out)
    torch.cuda.synchronize()
    assert hk.hk_gemm_last_device_status(0) == hk.HK_OK


def _slow(hk):  # noqa: F811
    """What launches a product that takes 3 ms on one SM."""
    import torch
    K = 1 << 22
    codes = torch.zeros(128, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(hk.Fp4Matrix.scales_size(128, K, "mxfp4"), dtype=torch.uint8, device="cuda")
    out = torch.empty(1, 128, dtype=torch.bfloat16, device="cuda")

    def launch():
        assert hk.hk_gemm_fp4_ex(codes.data_ptr(), scales.data_ptr(), codes.data_ptr(), scales.data_ptr(), out.data_ptr(), 1, 128,
                                 K, K // 2, K // 2, 128, hk.HK_FP4_MXFP4, kernel=4, split_k=1,
                                 stream=torch.cuda.current_stream().cuda_stream) == hk.HK_OK
    return launch


@pytest.mark.parametrize("M,kernel", [(1, 4), (300, 1)])
def test_the_time_limit_does_not_count_the_kernel_before(hk, M, kernel):  # noqa: F811
    """A product launched early behind one of 3 ms on one SM, with waits of at most 0.5 ms."""
    import torch
    slow = _slow(hk)
    a, _ = _random_matrix(hk, M, 4096, "mxfp4", 1)
    b, _ = _random_matrix(hk, 256, 4096, "mxfp4", 2)
    want, out = hk.gemm_fp4(a, b), torch.zeros(M, 256, dtype=torch.bfloat16, device="cuda")
    ptr, stream = lambda *t: [x.data_ptr() for x in t], torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        slow()
        assert hk.hk_gemm_fp4_ex(*ptr(a.codes, a.scales, b.codes, b.scales, out), M, 256, 4096, 2048, 2048, 256,
                                 hk.HK_FP4_MXFP4, kernel=kernel, timeout_ns=500_000, stream=stream) == hk.HK_OK
        torch.cuda.synchronize()
        assert hk.hk_gemm_last_device_status(0) == hk.HK_OK
        assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()


@pytest.mark.parametrize("kernel", [1, 2, 3, 4, 5, 6, 7])
def test_the_time_limit_of_a_bf16_product_does_not_count_the_kernel_before(hk, kernel):  # noqa: F811
    import torch
    slow = _slow(hk)
    A, B = (torch.randn(n, 256, device="cuda").to(torch.bfloat16) for n in (300, 520))
    out = torch.empty(300, 520, dtype=torch.bfloat16, device="cuda")
    want = hk.Plan(300, 520, 256, kernel=kernel).run(A, B, out).clone()
    plan = hk.Plan(300, 520, 256, kernel=kernel, timeout_ns=500_000)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        slow()
        plan.run(A, B, out)
        torch.cuda.synchronize()
        assert plan.device_status() == hk.HK_OK and torch.equal(out, want)
    assert hk.hk_gemm_last_device_status(0) == hk.HK_OK
