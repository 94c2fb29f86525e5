"""Attention over the 8-bit cache on either of its forms, whatever the call's shape
would choose: the few-row kernels (a block or cluster for each unit, or all tiles over the
GPU) and the many-row form (a pass to bf16, then the attention-forward kernel).

Tolerances as in test_kv8_gpu.py, the weights' rounding taken from the form that runs:
2^-11 where they are f16 (few rows), 2^-8 where they are bf16 (many)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import kv8_ref as ref
from test_kv8_gpu import _filled, _garbage_cache, _host, _i32, _status, _table, _tokens, hk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

FEW, MANY = 0x10, 0x20
FORMS = pytest.mark.parametrize("form", [FEW, MANY], ids=["few", "many"])


def _strides(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def _attend(hk, form, q, cache, table, lengths, counts=None, causal=True, scale=0.0, out=None, fill=0xFF, timeout_ns=0,  # noqa: F811
            flags=0):
    """(o, lse) through the entry point that takes a form; the workspace is full of `fill` before."""
    import torch
    B, T, Hq, D = q.shape
    out = torch.full_like(q, 3.0) if out is None else out
    lse = torch.full((B, T, Hq), 3.0, dtype=torch.float32, device="cuda")
    kind = hk.HK_TYPE_BF16 if q.dtype == torch.bfloat16 else hk.HK_TYPE_FP16
    lib = hk.load()
    size = lib.hk_attention_kv8_workspace_size_ex(q.data_ptr(), kind, _strides(q), cache._ref, table.size(1), out.data_ptr(),
                                                  _strides(out), B, T, Hq, form)
    workspace = torch.full((max(size, 1),), fill, dtype=torch.uint8, device="cuda")
    n, c = _i32(lengths), None if counts is None else _i32(counts)
    st = lib.hk_attention_kv8_ex(q.data_ptr(), kind, _strides(q), cache._ref, table.data_ptr(), table.stride(0), table.size(1),
                                 n.data_ptr(), None if c is None else c.data_ptr(), out.data_ptr(), _strides(out), lse.data_ptr(),
                                 B, T, Hq, 1 if causal else 0, scale, workspace.data_ptr(), size, form | flags, timeout_ns,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == hk.HK_OK, hk.hk_gemm_last_error_string()
    torch.cuda.synchronize()
    _attend.workspace = workspace
    return out, lse


def _assert(hk, form, q, cache, table, lengths, counts=None, causal=True, scale=0.0, **kw):  # noqa: F811
    import torch
    o, lse = _attend(hk, form, q, cache, table[1], lengths, counts, causal, scale, **kw)
    assert _status(hk) == hk.HK_OK
    n = [q.size(1)] * q.size(0) if counts is None else counts
    want, wlse, mag = ref.attention(q.double().cpu().numpy(), *_host(cache), table[0], lengths, n, causal,
                                    scale or q.size(3) ** -0.5)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    tol = half * np.abs(want) + ((2.0 ** -11 if form == FEW else 2.0 ** -8) + 2.0 ** -12) * mag + 2.0 ** -25
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, first {np.argwhere(bad)[:4].tolist()}: {got[bad][:4]} for "
                           f"{want[bad][:4]}")
    none = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(gl), none) and (got[none] == 0).all()
    assert (np.abs(gl[~none] - wlse[~none]) <= 2.0 ** -16 * np.maximum(1, np.abs(wlse[~none]))).all()
    return o


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 7, 8])
def test_single_queries(hk, form, D, page, group):  # noqa: F811
    import torch
    rng = np.random.default_rng(D + page + group)
    lengths = [1, 0, 31, 32, 33, 127, 128, 129, 700]
    cache, table = _filled(hk, rng, lengths, 2, D, page)
    _assert(hk, form, _tokens(rng, len(lengths), 1, 2 * group, D, torch.bfloat16, 1), cache, table, lengths)


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("T,group", [(2, 8), (5, 1), (33, 3), (40, 7), (70, 8), (130, 1), (257, 2), (600, 1)])
def test_several_queries(hk, form, T, group, causal, D):  # noqa: F811
    """Queries at the end of each sequence; more queries than tokens, counts below T, nothing at all."""
    import torch
    rng = np.random.default_rng(T * group + D)
    lengths = [T, T + 1, 200 + T, 1, max(T - 3, 0), 0]
    cache, table = _filled(hk, rng, lengths, 2, D, 64)
    q = _tokens(rng, len(lengths), T, 2 * group, D, torch.bfloat16, 1)
    _assert(hk, form, q, cache, table, lengths, None, causal)
    _assert(hk, form, q, cache, table, lengths, [T, 1, T // 2, 0, min(T, 2), T], causal)


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,T,length", [(1, 256, 30), (1, 256, 128), (4, 64, 5), (8, 40, 3), (1, 700, 129)])
def test_first_rows_that_see_nothing(hk, form, D, group, T, length):  # noqa: F811
    """The first query tile of a pair without a key, the second with some: fewer tokens than queries."""
    import torch
    rng = np.random.default_rng(T + length)
    lengths = [length, T + 50, length, 0]
    cache, table = _filled(hk, rng, lengths, 2, D, 32)
    _assert(hk, form, _tokens(rng, 4, T, 2 * group, D, torch.bfloat16, 1), cache, table, lengths)


@FORMS
@pytest.mark.parametrize("T", [1, 10, 150])
def test_strided_queries_and_output(hk, form, T):  # noqa: F811
    import torch
    rng = np.random.default_rng(T)
    H, group, D, lengths = 2, 4, 128, [77, 300]
    cache, table = _filled(hk, rng, lengths, H, D, 32)
    heads = _tokens(rng, 2, H * group, T, D, torch.bfloat16, 1)
    q = heads.transpose(1, 2)
    out = torch.full((2, H * group, T, D), 5.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    _assert(hk, form, q, cache, table, lengths, out=out)
    fused = torch.zeros(2, T, H * group + 5, D, dtype=torch.bfloat16, device="cuda")     # rows among others
    fused[:, :, 3:3 + H * group] = q
    store = torch.full((2, T, H * group + 2, D), 5.0, dtype=torch.bfloat16, device="cuda")
    _assert(hk, form, fused[:, :, 3:3 + H * group], cache, table, lengths, out=store[:, :, 1:-1])
    assert bool((store[:, :, 0] == 5.0).all()) and bool((store[:, :, -1] == 5.0).all())


@FORMS
@pytest.mark.parametrize("D", [64, 128])
def test_pages_of_very_different_scale(hk, form, D):  # noqa: F811
    import torch
    rng = np.random.default_rng(11)
    n, page = 330, 16
    k = torch.from_numpy(rng.standard_normal((1, n, 1, D)) * 0.3).to(torch.bfloat16).cuda()
    e = np.repeat(rng.integers(-30, 31, -(-n // page)), page)[:n]
    e[160:176] = -1000
    v = torch.from_numpy(rng.standard_normal((1, n, 1, D)) * np.exp2(e)[None, :, None, None]).to(torch.bfloat16).cuda()
    cache = _garbage_cache(hk, 24, 1, D, page, 1)
    table = _table(rng, 1, 21, 24)
    hk.kv8_append(cache, k, v, table[1], _i32([0]))
    for T in (1, 64, 200):
        _assert(hk, form, _tokens(rng, 1, T, 4, D, torch.bfloat16, 1), cache, table, [n])


@FORMS
@pytest.mark.parametrize("T", [1, 140])
def test_queries_and_scales_of_very_different_size(hk, form, T):  # noqa: F811
    import torch
    rng = np.random.default_rng(12)
    cache, table = _filled(hk, rng, [200], 1, 64, 16)
    q = _tokens(rng, 1, T, 8, 64, torch.bfloat16, 0)
    q = q * torch.tensor([2.0 ** -120, 2.0 ** -60, 1e-30, 1e-3, 1.0, 3.0, 0.0, 2.0 ** -133], device="cuda").view(1, 1, 8, 1)
    _assert(hk, form, q.to(torch.bfloat16), cache, table, [200])
    q = _tokens(rng, 1, T, 8, 64, torch.bfloat16, 0)
    for scale in (2.0 ** -30, 0.7, 5.0):
        _assert(hk, form, q, cache, table, [200], scale=scale)


@FORMS
@pytest.mark.parametrize("T", [1, 150])
def test_nan_keys_and_queries_stay_with_their_head_and_rows(hk, form, T):  # noqa: F811
    import torch
    rng = np.random.default_rng(13)
    H, group, D, n = 2, 2, 64, 400
    cache, table = _filled(hk, rng, [n, n], H, D, 32)
    p = int(table[0][0][12])
    cache.k[p, 1, 5, 7] = 0x7F              # token 389 of sequence 0, KV head 1
    q = _tokens(rng, 2, T, H * group, D, torch.bfloat16, 1)
    o = _attend(hk, form, q, cache, table[1], [n, n])[0].isnan()
    first = max(0, 389 - (n - T))           # queries before it do not see it
    assert bool(o[0, first:, 2:].all()) and int(o.sum()) == (T - first) * 2 * D
    q[1, 0, 1, 3] = float("nan")
    cache.k[p, 1, 5, 7] = 0
    o = _attend(hk, form, q, cache, table[1], [n, n])[0].isnan()
    assert bool(o[1, 0, 1].all()) and int(o.sum()) == D


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 48, 150])
def test_pages_and_lengths_out_of_range_are_reported(hk, form, D, T):  # noqa: F811
    import torch
    rng = np.random.default_rng(14)
    H, page = 2, 64
    lengths = [300, 200, 160]
    cache, table = _filled(hk, rng, lengths, H, D, page)
    q = _tokens(rng, 3, T, H, D, torch.bfloat16, 1)
    want = _assert(hk, form, q, cache, table, lengths)
    for bad in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):
        t = table[1].clone()
        t[0, 1] = bad
        o = _attend(hk, form, q, cache, t, lengths)[0]
        assert _status(hk) == hk.HK_ERR_INVALID_ARG and torch.equal(o[1:], want[1:])
    for bad, counts in (([-5, 200, 160], None), ([10 ** 9, 200, 160], None), (lengths, [-1, T, T]), (lengths, [T + 1, T, T])):
        o = _attend(hk, form, q, cache, table[1], bad, counts)[0]
        assert _status(hk) == hk.HK_ERR_INVALID_ARG and torch.equal(o[1:], want[1:])
    assert torch.equal(_attend(hk, form, q, cache, table[1], lengths)[0], want) and _status(hk) == hk.HK_OK


@FORMS
@pytest.mark.parametrize("D", [64, 128])
def test_long_and_wide_tables(hk, form, D):  # noqa: F811
    """Tables with room for far more tokens than there are; units that several warps share."""
    import torch
    rng = np.random.default_rng(15)
    B, H, page = 3, 2, 64
    lengths = [9000, 0, 41]
    cache, table = _filled(hk, rng, lengths, H, D, page)
    wide = np.full((B, 6000), -7, dtype=np.int32)
    wide[:, : table[0].shape[1]] = table[0]
    table = (wide, torch.from_numpy(wide).cuda())
    for T, counts in ((1, None), (9, [9, 2, 7]), (70, [70, 0, 70])):
        q = _tokens(rng, B, T, H * 3, D, torch.bfloat16, 1)
        want = _assert(hk, form, q, cache, table, lengths, counts, fill=0)
        for fill in (0x7F, 0xFF):
            assert torch.equal(_attend(hk, form, q, cache, table[1], lengths, counts, fill=fill)[0], want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("B,H,group", [(3, 2, 4), (20, 8, 1), (50, 8, 4), (100, 8, 8), (200, 8, 2)])
def test_blocks_of_every_size(hk, D, dtype, B, H, group):  # noqa: F811
    """6 to 1600 units over a short table: blocks of 8, 4, 2 and 1 warps."""
    import torch
    rng = np.random.default_rng(B)
    lengths = [int(x) for x in rng.integers(0, 190, B)]
    cache, table = _filled(hk, rng, lengths, H, D, 64)
    _assert(hk, FEW, _tokens(rng, B, 1, H * group, D, getattr(torch, dtype), 1), cache, table, lengths)
    assert _attend.workspace.numel() == 1


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_tiles_spread_over_the_gpu(hk, D, dtype):  # noqa: F811
    import torch
    rng = np.random.default_rng(23)
    lengths = [30000, 40, 0, 3000]
    cache, table = _filled(hk, rng, lengths, 2, D, 64)
    wide = np.full((4, 2100), -1, dtype=np.int32)            # (more tiles than a cluster of 16 blocks takes)
    wide[:, : table[0].shape[1]] = table[0]
    table = (wide, torch.from_numpy(wide).cuda())
    for T, counts in ((1, None), (9, [9, 1, 9, 6]), (40, [40, 1, 40, 37])):
        _assert(hk, FEW, _tokens(rng, 4, T, 6, D, getattr(torch, dtype), 1), cache, table, lengths, counts, fill=0xFF)
        assert not bool((_attend.workspace == 0xFF).all())   # sums went through memory


@pytest.mark.parametrize("D", [64, 128])
def test_more_sequences_than_are_widened_at_a_time(hk, D):  # noqa: F811
    """A table so wide that the workspace holds one or two sequences: one round of launches after another."""
    import torch
    rng = np.random.default_rng(27)
    B, H, T = 3, 8, 30
    lengths, counts = [500, 20, 290], [30, 30, 7]
    cache, table = _filled(hk, rng, lengths, H, D, 128)
    wide = np.full((B, 1024), -1, dtype=np.int32)
    wide[:, : table[0].shape[1]] = table[0]
    table = (wide, torch.from_numpy(wide).cuda())
    q = _tokens(rng, B, T, H * 4, D, torch.bfloat16, 1)
    _assert(hk, MANY, q, cache, table, lengths, counts)
    t = table[1].clone()
    t[1, 0] = cache.pages
    want = _attend(hk, MANY, q, cache, table[1], lengths, counts)[0]
    o = _attend(hk, MANY, q, cache, t, lengths, counts)[0]
    assert _status(hk) == hk.HK_ERR_INVALID_ARG and torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


@FORMS
@pytest.mark.parametrize("T", [1, 40])
def test_cache_beyond_32_bit_offsets(hk, form, T):  # noqa: F811
    import torch
    rng = np.random.default_rng(16)
    pages, H, page, D, n = 34000, 8, 64, 128, 150            # 2.2e9 codes of keys, as many of values
    cache = hk.Kv8Cache.empty(pages, H, D, page)
    t = np.array([[pages - 1, 0, pages - 2]], dtype=np.int32)
    k = _tokens(rng, 1, n, H, D, torch.bfloat16, 0)
    hk.kv8_append(cache, k * 0.2, k, torch.from_numpy(t).cuda(), _i32([0]))
    q = _tokens(rng, 1, T, H, D, torch.bfloat16, 0)
    o = _attend(hk, form, q, cache, torch.from_numpy(t).cuda(), [n])[0]
    small = hk.Kv8Cache(*(x[t[0].tolist()].contiguous() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    again = (np.array([[0, 1, 2]], dtype=np.int32), _i32([[0, 1, 2]]))
    assert torch.equal(_assert(hk, form, q, small, again, [n]), o)


@FORMS
@pytest.mark.parametrize("T", [1, 5, 150])
def test_repeats_exactly_and_in_graphs(hk, form, T):  # noqa: F811
    import torch
    rng = np.random.default_rng(17)
    lengths = [3000, 180, 800]
    H, D = 2, 128
    cache, table = _filled(hk, rng, [3000, 3000, 3000], H, D, 64)
    q = _tokens(rng, 3, T, H * 8, D, torch.bfloat16, 1)
    want, wlse = _attend(hk, form, q, cache, table[1], lengths)
    for _ in range(3):
        o, lse = _attend(hk, form, q, cache, table[1], lengths)
        assert torch.equal(o, want) and torch.equal(lse, wlse)
    lib, n = hk.load(), _i32(lengths)
    out = torch.empty_like(q)
    size = lib.hk_attention_kv8_workspace_size_ex(q.data_ptr(), 0, _strides(q), cache._ref, table[1].size(1), out.data_ptr(),
                                                  _strides(out), 3, T, H * 8, form)
    workspace = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert lib.hk_attention_kv8_ex(q.data_ptr(), 0, _strides(q), cache._ref, table[1].data_ptr(), table[1].stride(0),
                                       table[1].size(1), n.data_ptr(), None, out.data_ptr(), _strides(out), None, 3, T, H * 8, 1,
                                       0.0, workspace.data_ptr(), size, form, 0,
                                       torch.cuda.current_stream().cuda_stream) == hk.HK_OK
    for other in (lengths, [200, 2900, 151], lengths):
        n.copy_(_i32(other))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _attend(hk, form, q, cache, table[1], other)[0])
    assert _status(hk) == hk.HK_OK
