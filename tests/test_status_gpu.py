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
