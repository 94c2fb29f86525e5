"""Arranging, compacting and copying pages on the GPU against the plain reference
(tests/pages_ref.py): whole numbers and codes, equal in every place."""
import random

import numpy as np
import pytest

import pages_ref as ref

pytestmark = pytest.mark.gpu


def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _caches(n, pages, page, seed=0, H=2, D=64):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(n):
        c = hk.Kv8Cache.empty(pages, H, D, page)
        for t in (c.k, c.v):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        for t in (c.k_scale, c.v_scale):
            t.copy_(torch.rand(t.shape, generator=g, device="cuda"))
        out.append(c)
    return out


def _tensors(caches):
    return [t for c in caches for t in (c.k, c.v, c.k_scale, c.v_scale)]


def _status_ok():
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    return hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK


def _same_rows(got, want, held, page):
    for i, h in enumerate(held):
        n = ref.slots(h, page)
        assert got[i][:n] == want[i][:n], i


@pytest.mark.parametrize("page,rows,width,pages,layers,H,D", [
    (16, 6, 8, 60, 1, 2, 64), (32, 1, 5, 7, 2, 1, 128), (64, 40, 5, 150, 1, 1, 64), (128, 9, 30, 9000, 0, 1, 64),
    (16, 300, 20, 4096, 1, 1, 64), (16, 3, 700, 1500, 17, 1, 64),
])
def test_arrange_and_compact_follow_the_reference(page, rows, width, pages, layers, H, D):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    rng = random.Random(page * rows + width)
    caches = _caches(layers, pages, page, rows, H, D)
    store = torch.zeros(rows, width + 3, dtype=torch.int32, device="cuda")       # (rows with a stride)
    pool = hk.Kv8Pool(torch.zeros(pages, dtype=torch.int32, device="cuda"), store[:, :width],
                      torch.zeros(rows, dtype=torch.int32, device="cuda"), page)
    refs, table, held = [0] * pages, [[0] * width for _ in range(rows)], [0] * rows
    for step in range(25):
        keep, room, parents = ref.random_call(rng, held, page, width)
        want = [t.clone() for t in _tensors(caches)]
        copies = torch.full((2, rows), 7, dtype=torch.int32, device="cuda")
        missing = hk.kv8_arrange(pool, _i32(keep), _i32(room), None if parents is None else _i32(parents), caches, copies=copies)
        refs, table, held, copied, lack = ref.arrange(refs, table, held, keep, room, parents, page)
        assert missing.item() == lack
        assert pool.refs.tolist() == refs and pool.held.tolist() == held
        _same_rows(pool.table.tolist(), table, held, page)
        assert copies.tolist() == [[copied[i][k] if i in copied else -1 for i in range(rows)] for k in (0, 1)]
        if copied:
            a, b = (torch.tensor([c[k] for c in copied.values()], device="cuda") for k in (0, 1))
            for t in want:
                t[b] = t[a]
        for t, w in zip(_tensors(caches), want):
            assert torch.equal(t, w)
        if step % 4 == 3:
            moved = hk.kv8_compact(pool, caches)
            before = refs
            refs, table, to = ref.compact(refs, table, held, page)
            assert moved.tolist() == to and pool.refs.tolist() == refs
            _same_rows(pool.table.tolist(), table, held, page)
            pairs = [(p, q) for p, q in enumerate(to) if q >= 0 and q != p]
            if pairs:
                a, b = (torch.tensor([c[k] for c in pairs], device="cuda") for k in (0, 1))
                for t in want:
                    t[b] = t[a]
            for t, w in zip(_tensors(caches), want):
                assert torch.equal(t, w)
            assert sorted(before) == sorted(refs)
    assert (store[:, width:] == 0).all()
    assert _status_ok()


def test_a_call_that_lacks_pages_changes_nothing():
    import dense_bf16_gemm_02_gb300 as hk
    pool, caches = hk.Kv8Pool.empty(4, 3, 4, 16), _caches(1, 4, 16)
    assert hk.kv8_arrange(pool, _i32([0, 0, 0]), _i32([17, 1, 0]), caches=caches).item() == 0
    state = [t.clone() for t in (pool.refs, pool.table, pool.held, *_tensors(caches))]
    lack = hk.kv8_arrange(pool, _i32([17, 1, 1]), _i32([33, 1, 17]), _i32([0, 1, 1]), caches)
    assert lack.item() == 2 and lack is pool.missing
    other = hk.Kv8Pool.empty(4, 3, 4, 16)
    assert hk.kv8_arrange(other, _i32([0, 0, 0])).item() == 0 and lack.item() == 2
    assert all((a == b).all() for a, b in zip(state, (pool.refs, pool.table, pool.held, *_tensors(caches))))
    assert hk.kv8_arrange(pool, _i32([17, 0, 0])).item() == 0          # (room: keep)
    assert pool.refs.sum().item() == 2 and pool.held.tolist() == [17, 0, 0]
    assert _status_ok()


@pytest.mark.parametrize("what", ["parent", "parent-", "keep", "keep-", "room", "room+", "held", "held-", "entry", "entry-"])
def test_arguments_out_of_range_change_nothing(what):
    """One bad row: the call says so, and follows nothing."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    pool, caches = hk.Kv8Pool.empty(20, 3, 4, 16), _caches(1, 20, 16)
    assert hk.kv8_arrange(pool, _i32([0, 0, 0]), _i32([20, 33, 1]), caches=caches).item() == 0
    keep, room, parents = [20, 33, 20], [21, 34, 21], [0, 1, 0]
    if what.startswith("parent"):
        parents[2] = 3 if what == "parent" else -1
    elif what.startswith("keep"):
        keep[2] = 21 if what == "keep" else -1
    elif what == "room":
        room[1] = 32
    elif what == "room+":
        room[1] = 65
    elif what.startswith("held"):
        pool.held[0] = 65 if what == "held" else -5
    else:
        pool.table[0, 1] = 20 if what == "entry" else -1
    state = [t.clone() for t in (pool.refs, pool.table, pool.held, *_tensors(caches))]
    assert hk.kv8_arrange(pool, _i32(keep), _i32(room), _i32(parents), caches).item() == -1
    assert all(torch.equal(a, b) for a, b in zip(state, (pool.refs, pool.table, pool.held, *_tensors(caches))))
    assert not _status_ok() and _status_ok()


def test_compacting_leaves_entries_out_of_range():
    import dense_bf16_gemm_02_gb300 as hk
    pool = hk.Kv8Pool.empty(10, 3, 4, 16)
    pool.refs[3] = pool.refs[7] = pool.refs[9] = 1
    pool.table[0, :2] = _i32([7, 10])
    pool.table[1, :2] = _i32([-1, 9])
    pool.held.copy_(_i32([32, 32, 999]))
    moved = hk.kv8_compact(pool)
    assert moved.tolist() == [-1, -1, -1, 0, -1, -1, -1, 1, -1, 2]
    assert pool.table[:2, :2].tolist() == [[1, 10], [-1, 2]] and pool.refs.tolist() == [1, 1, 1] + [0] * 7
    assert not _status_ok()


@pytest.mark.parametrize("pages", [1, 31, 4096, 4097, 20000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 1.0])
def test_compacting_pools_of_every_size(pages, share):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    rng = np.random.default_rng(pages)
    refs = np.where(rng.random(pages) < share, rng.integers(1, 4, pages), 0).astype(np.int32)
    used = np.flatnonzero(refs)
    pool = hk.Kv8Pool(_i32(refs.tolist()), _i32(rng.permutation(used).tolist() or [0]).view(1, -1), _i32([64 * len(used)]), 64)
    caches = _caches(1, pages, 64, H=1)
    want = [t.clone() for t in _tensors(caches)]
    new, table, moved = ref.compact(refs.tolist(), pool.table.tolist(), pool.held.tolist(), 64)
    assert hk.kv8_compact(pool, caches[0]).tolist() == moved
    assert pool.refs.tolist() == new and pool.table.tolist() == table
    m = torch.tensor(moved, device="cuda")
    a = ((m >= 0) & (m != torch.arange(pages, device="cuda"))).nonzero().flatten()
    for t, w in zip(_tensors(caches), want):
        w[m[a]] = w[a]
        assert torch.equal(t, w)
    assert _status_ok()


@pytest.mark.parametrize("H,D,page", [(1, 64, 16), (3, 128, 64), (8, 128, 128)])
def test_copying_to_a_larger_pool(H, D, page):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    src, dst = _caches(2, 11, page, 1, H, D), _caches(2, 30, page, 2, H, D)
    want = [t.clone() for t in _tensors(dst)]
    a, b = [3, -1, 10, 0, 3], [29, -1, 0, 7, 8]
    hk.kv8_copy_pages(dst, src, _i32(b), _i32(a))
    for t, w, s in zip(_tensors(dst), want, _tensors(src)):
        for x, y in zip(a, b):
            if x >= 0:
                w[y] = s[x]
        assert torch.equal(t, w)
    assert _status_ok()
    for x, y in ((11, 1), (1, 30), (-1, 2), (2, -1), (-2, 3)):          # not followed, said
        hk.kv8_copy_pages(dst, src, _i32([y]), _i32([x]))
        assert not _status_ok()
    hk.kv8_copy_pages(dst, src, _i32([]), _i32([]))
    assert all(torch.equal(t, w) for t, w in zip(_tensors(dst), want))


def test_a_captured_step_and_another_stream():
    """Fork and growth captured once and replayed: each replay goes on where the last one ended."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    page, R, M, P = 16, 5, 12, 80
    caches = _caches(3, P, page)
    pool = hk.Kv8Pool.empty(P, R, M, page)
    refs, table, held = [0] * P, [[0] * M for _ in range(R)], [0] * R
    keep, room, parents = _i32([0] * R), _i32([0] * R), _i32(list(range(R)))
    stream = torch.cuda.Stream()
    hk.kv8_arrange(pool, keep, room, parents, caches, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        missing = hk.kv8_arrange(pool, keep, room, parents, caches)
        moved = hk.kv8_compact(pool, caches)
    rng = random.Random(1)
    want = [t.clone() for t in _tensors(caches)]
    for _ in range(12):
        k, r, p = ref.random_call(rng, held, page, M)
        p = list(range(R)) if p is None else p
        for t, v in ((keep, k), (room, r), (parents, p)):
            t.copy_(_i32(v))
        graph.replay()
        refs, table, held, copied, lack = ref.arrange(refs, table, held, k, r, p, page)
        for a, b in copied.values():
            for t in want:
                t[b] = t[a]
        refs, table, to = ref.compact(refs, table, held, page)
        assert missing.item() == lack and moved.tolist() == to
        for a, b in sorted((x, y) for x, y in enumerate(to) if y >= 0 and x != y):
            for t in want:
                t[b] = t[a]
        assert pool.refs.tolist() == refs and pool.held.tolist() == held
        _same_rows(pool.table.tolist(), table, held, page)
        assert all(torch.equal(t, w) for t, w in zip(_tensors(caches), want))
    assert _status_ok()


def test_wrong_shapes_are_refused():
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    pool, (cache,) = hk.Kv8Pool.empty(20, 3, 4, 16), _caches(1, 20, 16)
    three = _i32([0, 0, 0])
    for bad in (_i32([0, 0]), three.view(3, 1), three.float(), three.cpu(), None):
        with pytest.raises((TypeError, ValueError)):
            hk.kv8_arrange(pool, bad)
        with pytest.raises((TypeError, ValueError)):
            hk.kv8_arrange(pool, three, three, parents=bad if bad is not None else 3)
    with pytest.raises(TypeError):
        hk.kv8_arrange(pool, three, copies=three)
    with pytest.raises(TypeError):
        hk.kv8_arrange(pool, three, caches=[pool])
    for other in (hk.Kv8Cache.empty(21, 2, 64, 16), hk.Kv8Cache.empty(20, 2, 64, 32)):
        with pytest.raises(hk.HKError):
            hk.kv8_arrange(pool, three, caches=[cache, other])
        with pytest.raises(hk.HKError):
            hk.kv8_compact(pool, other)
    with pytest.raises(ValueError):
        hk.kv8_copy_pages([cache, cache], cache, three, three)
    with pytest.raises(ValueError):
        hk.kv8_copy_pages(cache, cache, three, _i32([1]))
    with pytest.raises(hk.HKError):
        hk.kv8_copy_pages(cache, hk.Kv8Cache.empty(20, 1, 64, 16), three, three)
    with pytest.raises(ValueError):
        hk.Kv8Pool(pool.refs, pool.table, _i32([0, 0]), 16)
    with pytest.raises(hk.HKError):
        hk.kv8_arrange(hk.Kv8Pool(pool.refs, pool.table, pool.held, 24), three)
    assert pool.refs.sum().item() == 0 and torch.cuda.is_available()


@pytest.mark.parametrize("rows,width,page", [(5, 700, 16), (40, 6, 64), (1, 3, 128)])
def test_what_the_rows_hold_as_an_argument(rows, width, page):
    """keep or room may be the pool's own tensor, which the call writes."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    rng = random.Random(rows * width)
    pages = rows * width + 3
    pool = hk.Kv8Pool.empty(pages, rows, width, page_size=page)
    refs, table, held = [0] * pages, [[0] * width for _ in range(rows)], [0] * rows
    caches = _caches(1, pages, page)
    even = [rng.randrange(1, width * page // 2)] * rows
    calls = [("keep", even, None)]
    for _ in range(6):
        calls += [("keep", [rng.randrange(0, 3 * page) for _ in range(rows)], None), ("room", None, None)]
    for how, more, _ in calls:
        if how == "keep":                    # all that is held, and room for more
            keep, room = list(held), [min(width * page, h + m) for h, m in zip(held, more)]
            missing = hk.kv8_arrange(pool, pool.held, _i32(room), caches=caches)
        else:                                # part of it, with as much room as before
            keep, room = [rng.randrange(0, h + 1) for h in held], list(held)
            missing = hk.kv8_arrange(pool, _i32(keep), pool.held, caches=caches)
        refs, table, held, _, lack = ref.arrange(refs, table, held, keep, room, None, page)
        assert missing.item() == lack == 0
        assert pool.refs.tolist() == refs and pool.held.tolist() == held
        _same_rows(pool.table.tolist(), table, held, page)
    parents = list(range(rows))[::-1]
    room = [max(held)] * rows
    assert hk.kv8_arrange(pool, _i32([0] * rows), _i32(room)).item() == 0
    refs, table, held, _, _ = ref.arrange(refs, table, held, [0] * rows, room, None, page)
    missing = hk.kv8_arrange(pool, pool.held, pool.held, parents=_i32(parents), caches=caches)
    refs, table, held, _, lack = ref.arrange(refs, table, held, list(held), list(held), parents, page)
    assert missing.item() == lack and pool.refs.tolist() == refs
    _same_rows(pool.table.tolist(), table, held, page)
    assert _status_ok()


def test_two_captured_calls_of_one_pool():
    """Graphs that were captured before either ran, replayed in turn: they share the pool's workspace."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    pages, rows, width, page = 400, 20, 12, 16
    pool = hk.Kv8Pool.empty(pages, rows, width, page_size=page)
    caches = _caches(2, pages, page)
    keep, room = _i32([0] * rows), _i32([0] * rows)
    back, parents = _i32([0] * rows), _i32(list(range(rows)))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        hk.kv8_arrange(pool, keep, room, caches=caches)
    with torch.cuda.graph(graphs[1]):
        hk.kv8_arrange(pool, back, back, parents=parents, caches=caches)
    refs, table, held = [0] * pages, [[0] * width for _ in range(rows)], [0] * rows
    rng = random.Random(7)
    for _ in range(12):
        k = [rng.randrange(0, h + 1) for h in held]
        r = [min(width * page, x + rng.randrange(0, 40)) for x in k]
        keep.copy_(_i32(k))
        room.copy_(_i32(r))
        graphs[0].replay()
        refs, table, held, _, lack = ref.arrange(refs, table, held, k, r, None, page)
        assert lack == 0 and pool.missing.item() == 0
        p = [rng.randrange(rows) for _ in range(rows)]
        b = [rng.randrange(0, held[x] + 1) for x in p]
        back.copy_(_i32(b))
        parents.copy_(_i32(p))
        graphs[1].replay()
        refs, table, held, _, lack = ref.arrange(refs, table, held, b, b, p, page)
        assert pool.missing.item() == lack == 0
        assert pool.refs.tolist() == refs and pool.held.tolist() == held
        _same_rows(pool.table.tolist(), table, held, page)
    assert _status_ok()
