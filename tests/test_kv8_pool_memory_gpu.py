"""A pool dropped while work on its tensors is under way or captured: the call's scratch memory is nobody else's until it has
run. A pool object may be made for one call around tensors that live longer."""
import random

import pytest

import pages_ref as ref

pytestmark = pytest.mark.gpu

PAGES, ROWS, WIDTH, PAGE = 300, 20, 12, 16


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Recorder:
    """The library, but for one entry point, which only writes down its workspace and where it says what lacked."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def hk_kv8_arrange(self, pool, keep, room, parents, caches, n, copies, missing, workspace, size, stream):
        self.calls.append((workspace, size))
        return 0


def _tensors():
    import torch
    return (torch.zeros(PAGES, dtype=torch.int32, device="cuda"), torch.zeros(ROWS, WIDTH, dtype=torch.int32, device="cuda"),
            torch.zeros(ROWS, dtype=torch.int32, device="cuda"))


def _others(size, n=40):
    """Memory that the current stream gets now."""
    import torch
    return [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(n)]


def _overlap(others, start, size):
    return any(t.data_ptr() < start + size and start < t.data_ptr() + t.numel() for t in others)


@pytest.mark.parametrize("how", ["argument", "current"])
def test_scratch_of_another_stream(how, monkeypatch):
    """Nothing is launched here: the addresses tell."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    from dense_bf16_gemm_02_gb300 import serving
    lib = Recorder(hk.load())
    monkeypatch.setattr(serving._hk, "load", lambda: lib)
    keep, side = _i32([0] * ROWS), torch.cuda.Stream()
    pool = hk.Kv8Pool(*_tensors(), PAGE)
    if how == "argument":
        hk.kv8_arrange(pool, keep, stream=side)
    else:
        with torch.cuda.stream(side):
            hk.kv8_arrange(pool, keep)
    del pool
    assert len(lib.calls) == 1 and lib.calls[0][1] > 0
    assert not _overlap(_others(lib.calls[0][1]), *lib.calls[0])


def test_scratch_of_a_captured_call(monkeypatch):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    from dense_bf16_gemm_02_gb300 import serving
    lib = Recorder(hk.load())
    monkeypatch.setattr(serving._hk, "load", lambda: lib)
    keep, count = _i32([0] * ROWS), _i32([0])
    pool = hk.Kv8Pool(*_tensors(), PAGE)
    hk.kv8_arrange(pool, keep)               # (one outside before, which may leave the pool scratch memory of its own)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        count.add_(1)
        hk.kv8_arrange(pool, keep)
    del pool
    assert not _overlap(_others(lib.calls[1][1]), *lib.calls[1])
    graph.replay()


def test_calls_of_one_stream_share_scratch(monkeypatch):
    """(They follow one another: nothing is allocated for the second.)"""
    import dense_bf16_gemm_02_gb300 as hk
    from dense_bf16_gemm_02_gb300 import serving
    lib = Recorder(hk.load())
    monkeypatch.setattr(serving._hk, "load", lambda: lib)
    pool, keep = hk.Kv8Pool(*_tensors(), PAGE), _i32([0] * ROWS)
    hk.kv8_arrange(pool, keep)
    hk.kv8_arrange(pool, keep)
    assert lib.calls[0] == lib.calls[1]


def _expect(tensors, state):
    refs, table, held = state
    assert tensors[0].tolist() == refs and tensors[2].tolist() == held
    got = tensors[1].tolist()
    for i, h in enumerate(held):
        n = ref.slots(h, PAGE)
        assert got[i][:n] == table[i][:n], i


@pytest.mark.parametrize("captured", [False, True])
def test_a_pool_dropped_right_after_its_call(captured):
    """Whatever memory of the pool's is free again is written by the first stream before the call runs."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    rng = random.Random(3)
    tensors = _tensors()
    state = [0] * PAGES, [[0] * WIDTH for _ in range(ROWS)], [0] * ROWS
    cache = hk.Kv8Cache.empty(PAGES, 1, 64, PAGE)
    for t in (cache.k, cache.v):
        t.copy_(torch.randint(0, 256, t.shape, device="cuda", dtype=torch.uint8))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    want = cache.k.clone()
    size = hk.hk_kv8_arrange_workspace_size(hk.hk_kv8_pool(num_pages=PAGES, table_stride=WIDTH, rows=ROWS, max_pages=WIDTH, page_size=PAGE))
    side = torch.cuda.Stream()
    keep, room, parents = _i32([0] * ROWS), _i32([0] * ROWS), _i32(list(range(ROWS)))
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        pool = hk.Kv8Pool(*tensors, PAGE)
        with torch.cuda.graph(graph):
            missing = hk.kv8_arrange(pool, keep, room, parents, cache)
        del pool
    for _ in range(8):
        k, r, p = ref.random_call(rng, state[2], PAGE, WIDTH)
        p = list(range(ROWS)) if p is None else p
        for t, v in ((keep, k), (room, r), (parents, p)):
            t.copy_(_i32(v))
        torch.cuda.synchronize()
        if captured:
            others = [t.fill_(1) for t in _others(size)]
            graph.replay()
        else:
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)
            missing = hk.kv8_arrange(hk.Kv8Pool(*tensors, PAGE), keep, room, parents, cache, stream=side)
            others = [t.fill_(1) for t in _others(size)]
        torch.cuda.synchronize()
        refs, table, held, copied, lack = ref.arrange(*state, k, r, p, PAGE)
        state = refs, table, held
        for a, b in copied.values():
            want[b] = want[a]
        assert missing.item() == lack and torch.equal(cache.k, want)
        _expect(tensors, state)
        assert all((t == 1).all() for t in others)
    assert hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK
