"""hk_kv8_copy_pages: -1 in both lists leaves an entry out; any other index out of range is said, and not followed."""
import pytest

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 - 1


@pytest.mark.parametrize("src,dst,ok", [(-1, -1, True), (-2, -2, False), (-1, -3, False), (-3, -1, False), (-FAR - 1, -FAR - 1, False),
                                        (-1, 0, False), (0, -1, False), (5, 0, False), (0, 5, False), (FAR, FAR, False)])
def test_indexes_out_of_range(src, dst, ok):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    cache = hk.Kv8Cache.empty(5, 2, 64, 16)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(0, 256, t.shape, device="cuda", dtype=torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.rand(t.shape, device="cuda"))
    tensors = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    want = [t.clone() for t in tensors]
    lists = [torch.tensor([a, b, -1], dtype=torch.int32, device="cuda") for a, b in ((src, 3), (dst, 1))]
    hk.kv8_copy_pages(cache, cache, lists[1], lists[0])
    for t, w in zip(tensors, want):
        w[1] = w[3]                          # (the entry beside it is copied)
        assert torch.equal(t, w)
    assert (hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK) == ok
