"""Pools of more than 256 x 4096 pages, whose counts are added up in more than one step. Most pages are somebody else's
(references that no row's entries account for)."""
import random

import pytest

import pages_ref as ref

pytestmark = pytest.mark.gpu

PAGES = 2 * 256 * 4096 + 70000


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("free", [[(0, 5), (1048000, 1050000), (PAGES - 300, PAGES)], [(2097100, 2097300), (PAGES - 3000, PAGES - 10)],
                                  [(4095, 4097), (1048575, 1048577), (2097151, 2097153), (PAGES - 1, PAGES)], [(0, PAGES)]])
def test_free_pages_far_apart(free):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    rng = random.Random(len(free))
    rows, width, page = 5, 300, 16
    refs = [2] * PAGES
    for a, b in free:
        refs[a:b] = [0] * (b - a)
    pool = hk.Kv8Pool(_i32(refs), torch.zeros(rows, width, dtype=torch.int32, device="cuda"), _i32([0] * rows), page)
    table, held = [[0] * width for _ in range(rows)], [0] * rows
    lacked = 0
    for step in range(6):
        keep, room, parents = ref.random_call(rng, held, page, width)
        if step == 0:
            keep, room, parents = [0] * rows, [width * page // (1 if len(free) != 3 else 3)] * rows, None
        missing = hk.kv8_arrange(pool, _i32(keep), _i32(room), None if parents is None else _i32(parents))
        refs, table, held, _, lack = ref.arrange(refs, table, held, keep, room, parents, page)
        assert missing.item() == lack and pool.held.tolist() == held
        assert torch.equal(pool.refs.cpu(), torch.tensor(refs, dtype=torch.int32))
        lacked += lack > 0
        for i, h in enumerate(held):
            n = ref.slots(h, page)
            assert pool.table[i, :n].tolist() == table[i][:n]
        if step % 3 == 1:
            moved = hk.kv8_compact(pool)
            refs, table, to = ref.compact(refs, table, held, page)
            assert torch.equal(moved.cpu(), torch.tensor(to, dtype=torch.int32))
            assert torch.equal(pool.refs.cpu(), torch.tensor(refs, dtype=torch.int32))
            for i, h in enumerate(held):
                n = ref.slots(h, page)
                assert pool.table[i, :n].tolist() == table[i][:n]
    assert lacked == 0 or len(free) == 4
    assert hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK
