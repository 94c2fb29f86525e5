"""The pool's entry points without a GPU: refusals and sizes, and pins of the plain
reference that the GPU tests compare with."""
import ctypes
import random

import pytest

import pages_ref as ref


@pytest.fixture(scope="module")
def lib():
    from dense_bf16_gemm_02_gb300 import build
    build.build()
    from dense_bf16_gemm_02_gb300 import hk_gemm
    return hk_gemm.load()


A = 1 << 20      # a 256-byte aligned address that is never read on these paths


def _pool(**kw):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    f = dict(refs=A, table=A, held=A, num_pages=40, table_stride=8, rows=4, max_pages=8, page_size=64)
    f.update(kw)
    return h.hk_kv8_pool(**f)


def _cache(**kw):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    f = dict(k_codes=A, v_codes=A, k_scale=A, v_scale=A, num_pages=40, heads=2, page_size=64, head_dim=64)
    f.update(kw)
    return h.hk_kv8_cache(**f)


def _array(*caches):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    return (h.hk_kv8_cache * max(1, len(caches)))(*caches)


BAD_POOLS = [dict(refs=None), dict(table=None), dict(held=None), dict(num_pages=0), dict(num_pages=(1 << 30) + 1), dict(rows=0),
             dict(rows=-1), dict(max_pages=0), dict(page_size=48), dict(page_size=0), dict(table_stride=7),
             dict(max_pages=1 << 26, table_stride=1 << 26), dict(rows=1 << 20, max_pages=1 << 12, table_stride=1 << 12)]
BAD_CACHES = [dict(head_dim=96), dict(page_size=32), dict(heads=0), dict(num_pages=39), dict(k_codes=None), dict(v_codes=None),
              dict(k_scale=None), dict(v_scale=None)]


def test_arrange_and_compact_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS, WS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED, h.HK_ERR_WORKSPACE

    def arr(pool=None, keep=A, room=A, parents=None, caches=(), copies=None, missing=A, ws=A, wsb=1 << 40):
        return lib.hk_kv8_arrange(ctypes.byref(pool or _pool()), keep, room, parents, _array(*caches), len(caches), copies, missing,
                                  ws, wsb, None)

    def com(pool=None, caches=(), moved=A, ws=A, wsb=1 << 40):
        return lib.hk_kv8_compact(ctypes.byref(pool or _pool()), _array(*caches), len(caches), moved, ws, wsb, None)
    assert lib.hk_kv8_arrange(None, A, A, None, None, 0, None, A, A, 1 << 40, None) == INV
    assert lib.hk_kv8_compact(None, None, 0, A, A, 1 << 40, None) == INV
    for bad in BAD_POOLS:
        assert arr(_pool(**bad)) == INV and com(_pool(**bad)) == INV, bad
    for bad in BAD_CACHES:
        assert arr(caches=(_cache(), _cache(**bad))) == INV and com(caches=(_cache(**bad),)) == INV, bad
    for name in ("refs", "table", "held"):
        assert arr(_pool(**{name: A + 2})) == MIS and com(_pool(**{name: A + 2})) == MIS
    assert arr(caches=(_cache(k_codes=A + 8),)) == MIS and com(caches=(_cache(v_scale=A + 1),)) == MIS
    assert arr(keep=None) == INV and arr(room=None) == INV and arr(missing=None) == INV and com(moved=None) == INV
    assert arr(keep=A + 1) == MIS and arr(parents=A + 2) == MIS and arr(copies=A + 2) == MIS and com(moved=A + 2) == MIS
    assert lib.hk_kv8_arrange(ctypes.byref(_pool()), A, A, None, None, 2, None, A, A, 1 << 40, None) == INV
    assert lib.hk_kv8_arrange(ctypes.byref(_pool()), A, A, None, None, -1, None, A, A, 1 << 40, None) == INV
    need = lib.hk_kv8_arrange_workspace_size(ctypes.byref(_pool()))
    assert arr(wsb=need - 1) == WS and arr(ws=None) == WS and arr(ws=A + 128) == WS
    need = lib.hk_kv8_compact_workspace_size(ctypes.byref(_pool()))
    assert com(wsb=need - 1) == WS and com(ws=None) == WS and com(ws=A + 128) == WS
    assert lib.hk_kv8_arrange_workspace_size(None) == 0 and lib.hk_kv8_compact_workspace_size(ctypes.byref(_pool(rows=0))) == 0


def test_workspaces_hold_what_the_kernels_use(lib):
    for pages, rows, width in ((1, 1, 1), (4096, 3, 7), (4097, 1000, 33), (1 << 20, 64, 4096)):
        pool = ctypes.byref(_pool(num_pages=pages, rows=rows, max_pages=width, table_stride=width))
        words = -(-pages // 4096) * 128
        assert lib.hk_kv8_arrange_workspace_size(pool) >= 4 * (2 * words + pages + 5 * rows + rows * width + -(-pages // 4096))
        assert lib.hk_kv8_compact_workspace_size(pool) >= 4 * (words + 3 * pages + -(-pages // 4096) + 2)


def test_copy_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED

    def cp(dst=(None,), src=(None,), d=A, s=A, n=3):
        dst, src = ([x or _cache() for x in y] for y in (dst, src))
        return lib.hk_kv8_copy_pages(_array(*dst), _array(*src), len(dst), d, s, n, None)
    assert cp(n=0) == h.HK_OK and cp((), ()) == h.HK_OK
    assert cp(n=-1) == INV and cp(n=1 << 31) == INV and cp(d=None) == INV and cp(s=None) == INV
    assert cp(d=A + 2) == MIS and cp(s=A + 1) == MIS
    for bad in (dict(heads=3), dict(page_size=32), dict(head_dim=128)):
        assert cp((_cache(**bad),)) == INV, bad
    assert cp((None, _cache(num_pages=41)), (None, None)) == INV and cp((None, None), (None, _cache(num_pages=41))) == INV
    assert lib.hk_kv8_copy_pages(None, None, 1, A, A, 1, None) == INV


def test_python_refusals(lib):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        hk.Kv8Pool(z, z.view(2, 2), z)                      # not on the GPU
    with pytest.raises(TypeError):
        hk.kv8_arrange(None, z)
    with pytest.raises(TypeError):
        hk.kv8_compact("pool")
    with pytest.raises(TypeError):
        hk.kv8_copy_pages([z], [z], z, z)
    pool = hk.Kv8Pool.__new__(hk.Kv8Pool)
    for name in ("refs", "table", "held", "pages", "rows", "max_pages", "page_size", "missing"):
        with pytest.raises(AttributeError):
            setattr(pool, name, 1)


@pytest.mark.parametrize("seed", range(6))
def test_the_reference_keeps_its_promises(seed):
    """References are what the tables name, no page that will be written is named twice, and what a row kept is
    what its parent had."""
    rng = random.Random(seed)
    page, R, M, P = 16, 6, 8, 60
    refs, table, held = [0] * P, [[0] * M for _ in range(R)], [0] * R
    contents = {}                            # page -> tokens (who wrote them)
    texts = [[] for _ in range(R)]
    for step in range(60):
        keep, room, parents = ref.random_call(rng, held, page, M)
        # (what is kept was appended: rows fill the room that they take)
        before = [list(r) for r in table], list(held)
        refs, table, held, copies, missing = ref.arrange(refs, table, held, keep, room, parents, page)
        if missing:
            assert (table, held) == before
            continue
        par = list(range(R)) if parents is None else parents
        texts = [texts[par[i]][: keep[i]] for i in range(R)]
        assert refs == ref.counted(table, held, P, page)
        old = {p: list(t) for p, t in contents.items()}
        for i, (a, b) in copies.items():
            contents[b] = list(old[a])
        for i in range(R):
            for s in range(ref.slots(held[i], page)):
                if (s + 1) * page > keep[i]:
                    assert refs[table[i][s]] == 1
                have = contents.get(table[i][s], [])
                want = texts[i][s * page:(s + 1) * page]
                assert have[: len(want)] == want
        for i in range(R):                   # append up to the room
            for at in range(keep[i], room[i]):
                texts[i].append((step, i, at))
                p = contents.setdefault(table[i][at // page], [None] * page)
                p[at % page] = texts[i][-1]
        if rng.random() < 0.3:
            a = [[contents.get(table[i][s]) for s in range(ref.slots(held[i], page))] for i in range(R)]
            was = refs
            refs, table, moved = ref.compact(refs, table, held, page)
            contents = {q: contents[p] for p, q in enumerate(moved) if q >= 0 and p in contents}
            assert refs == ref.counted(table, held, P, page) and sorted(was, reverse=True) == sorted(refs, reverse=True)
            assert all(n > 0 for n in refs[: sum(n > 0 for n in refs)])
            assert a == [[contents.get(table[i][s]) for s in range(ref.slots(held[i], page))] for i in range(R)]
