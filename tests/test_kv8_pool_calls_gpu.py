"""Calls on one pool: what each of them found stays what it was, and no call works in memory that another may get."""
import pytest

pytestmark = pytest.mark.gpu


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_what_a_call_lacked_outlives_the_next_call():
    import dense_bf16_gemm_02_gb300 as hk
    pool = hk.Kv8Pool.empty(4, 3, 4, 16)
    first = hk.kv8_arrange(pool, _i32([0, 0, 0]), _i32([64, 33, 0]))          # 7 pages of 4
    second = hk.kv8_arrange(pool, _i32([0, 0, 0]), _i32([17, 1, 0]))
    bad = hk.kv8_arrange(pool, _i32([18, 1, 0]))                              # more than the row holds
    last = hk.kv8_arrange(pool, _i32([17, 1, 0]))
    assert [t.item() for t in (first, second, bad, last)] == [3, 0, -1, 0]
    assert last is pool.missing and pool.held.tolist() == [17, 1, 0]
    assert hk.hk_gemm_last_device_status(0) == hk.HK_ERR_INVALID_ARG


def test_what_captured_calls_lacked():
    """Two calls of one graph, and a call between replays."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    pool = hk.Kv8Pool.empty(4, 2, 8, 16)
    none, rooms = _i32([0, 0]), [_i32([0, 0]) for _ in range(2)]
    assert pool.missing.item() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = hk.kv8_arrange(pool, none, rooms[0])
        b = hk.kv8_arrange(pool, none, rooms[1])
    assert pool.missing.item() == 0                     # (of calls outside a graph)
    for want, (x, y) in (((6, 0), ([100, 40], [16, 16])), ((0, 2), ([0, 0], [96, 0])), ((0, 0), ([0, 16], [16, 0]))):
        rooms[0].copy_(_i32(x))
        rooms[1].copy_(_i32(y))
        graph.replay()
        assert hk.kv8_arrange(pool, none).item() == 0
        assert (a.item(), b.item()) == want
    assert hk.hk_gemm_last_device_status(0) == hk.HK_OK


def test_a_pool_says_what_its_last_call_lacked():
    import dense_bf16_gemm_02_gb300 as hk
    pool, other = hk.Kv8Pool.empty(4, 1, 8, 16), hk.Kv8Pool.empty(4, 1, 8, 16)
    assert pool.missing.item() == 0 and pool.missing.dim() == 0
    for room, lack in ((80, 1), (64, 0), (128, 4)):
        got = hk.kv8_arrange(pool, _i32([0]), _i32([room]))
        assert hk.kv8_arrange(other, _i32([0]), _i32([16])).item() == 0
        hk.kv8_arrange(other, _i32([0]))
        assert pool.missing is got and got.item() == lack
        hk.kv8_arrange(pool, _i32([0]))


@pytest.mark.parametrize("inference", [False, True])
def test_verdicts_are_each_calls_own(inference):
    """More calls than verdicts are made at a time, on two streams, all of them kept."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    side, got = torch.cuda.Stream(), []
    for i in range(200):
        with torch.inference_mode(inference), torch.cuda.stream(side if i % 3 == 0 else torch.cuda.current_stream()):
            pool = hk.Kv8Pool.empty(4, 1, 300, 16)
            got.append(hk.kv8_arrange(pool, _i32([0]), _i32([16 * (4 + i)])))
    torch.cuda.synchronize()
    assert len({t.data_ptr() for t in got}) == 200
    assert [t.item() for t in got] == list(range(200))
    got[0].add_(5)                                       # (ordinary tensors, wherever they come from)
    got[1].add_(got[0])
    assert got[1].item() == 6 and [t.item() for t in got[2:]] == list(range(2, 200))
