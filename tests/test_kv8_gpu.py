"""The paged 8-bit cache: appends bit for bit against their definition, and
attention over it against 64-bit sums.

Tolerances of attention. The cached values are taken as they are in the cache
(their rounding is the append's). The weights P are rounded before P·V by at
most half a step of each, finfo.eps / 2: 2^-11 where they are f16 (few query
rows), 2^-8 where they are bf16 (many bf16 rows), so the output moves by at most
that times Σ P|V| / Σ P; scores, exponentials and sums in fp32 add less than
2^-12 of that (scores here are below 2^6 and err by at most 2^-18); the
output's own rounding is half a step, 2^-8 (bf16) or 2^-11 (fp16) of it. The
log-sum-exp is fp32: 2^-16 of max(1, |lse|)."""
from __future__ import annotations

import numpy as np
import pytest

import kv8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import dense_bf16_gemm_02_gb300 as pkg
    pkg.load()
    return pkg


def _status(hk):
    import torch
    torch.cuda.synchronize()
    return hk.hk_gemm_last_device_status(torch.cuda.current_device())


def _garbage_cache(hk, pages, H, D, page, seed):
    """Pages full of NaN codes and NaN scales: nothing that no append wrote may be used."""
    c = hk.Kv8Cache.empty(pages, H, D, page)
    c.k.fill_(0x7F)
    c.v.fill_(0xFF)
    c.k_scale.fill_(float("nan"))
    c.v_scale.fill_(float("nan"))
    return c


def _table(rng, B, width, pages):
    import torch
    t = rng.permutation(pages)[: B * width].reshape(B, width).astype(np.int32)
    return t, torch.from_numpy(t).cuda()


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _host(c):
    return [x.cpu().numpy().copy() for x in (c.k, c.k_scale, c.v, c.v_scale)]


def _appended(hk, cache, k, v, table, starts, counts, host):
    """Append on the GPU and by definition on `host` (k codes, k scale, v codes, v scale), and compare."""
    import torch
    t_np, t = table
    hk.kv8_append(cache, k, v, t, _i32(starts), None if counts is None else _i32(counts))
    n = [k.size(1)] * k.size(0) if counts is None else counts
    ref.append(host[0], host[1], k.double().cpu().numpy(), t_np, starts, n)
    ref.append(host[2], host[3], v.double().cpu().numpy(), t_np, starts, n)
    assert _status(hk) == hk.HK_OK
    for got, want, name in zip(_host(cache), host, ("k codes", "k scale", "v codes", "v scale")):
        same = (got == want) | ((got != got) & (want != want))
        if name.endswith("codes"):     # NaN is one value of either sign
            same |= ((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)
        assert same.all(), f"{name} differ at {np.argwhere(~same)[:4].tolist()}"


def _tokens(rng, B, T, H, D, dtype, spread=4):
    import torch
    x = rng.standard_normal((B, T, H, D)) * np.exp2(rng.integers(-spread, spread + 1, (B, T, H, 1)))
    return torch.from_numpy(x).to(dtype).cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_append_in_steps(hk, D, page, dtype):
    """Prompts of several lengths, then single tokens, then a chunk: pages that
    end inside a call, keep their scale, or must round their codes again."""
    import torch
    rng = np.random.default_rng(page + D)
    B, H = 3, 2
    width = -(-300 // page) + 1
    cache = _garbage_cache(hk, B * width + 2, H, D, page, 1)
    table = _table(rng, B, width, B * width + 2)
    host = _host(cache)
    at = np.zeros(B, dtype=int)
    for T, counts in ((7, None), (90, [90, 1, 33]), (1, None), (1, None), (2, [0, 2, 1]), (130, [130, 17, 128]), (1, None)):
        k, v = (_tokens(rng, B, T, H, D, getattr(torch, dtype)) for _ in range(2))
        _appended(hk, cache, k, v, table, at.copy(), counts, host)
        at += np.asarray([T] * B if counts is None else counts)


def test_append_special_values_and_repetition(hk):
    import torch
    rng = np.random.default_rng(5)
    B, T, H, D, page = 1, 12, 1, 64, 16
    cache = _garbage_cache(hk, 4, H, D, page, 1)
    table = _table(rng, B, 2, 4)
    host = _host(cache)
    k, v = (_tokens(rng, B, T, H, D, torch.float32) for _ in range(2))
    k[0, 3, 0, 5] = float("inf")
    k[0, 4, 0, 6] = float("-inf")
    k[0, 5, 0, 7] = float("nan")
    v.zero_()
    _appended(hk, cache, k, v, table, [0], None, host)
    before = _host(cache)
    _appended(hk, cache, k, v, table, [0], None, host)
    assert all(np.array_equal(a, b, equal_nan=a.dtype.kind == "f") for a, b in zip(before, _host(cache)))
    k = torch.full((B, 1, H, D), 448.0, device="cuda")      # the largest that the smallest scale above holds
    v = torch.full((B, 1, H, D), 1e-44, device="cuda")
    _appended(hk, cache, k, v, table, [12], None, host)
    k.fill_(3e38)
    v.fill_(-448.1)
    _appended(hk, cache, k, v, table, [13], None, host)


def test_append_from_strided_views(hk):
    import torch
    rng = np.random.default_rng(6)
    B, T, H, D, page = 2, 40, 3, 64, 32
    cache = _garbage_cache(hk, 8, H, D, page, 1)
    table = _table(rng, B, 3, 8)
    host = _host(cache)
    base = _tokens(rng, B, H, T, 2 * D + 1, torch.bfloat16)
    k = base[..., :D].transpose(1, 2)                       # [B, H, T, ·] storage, rows of odd length
    v = base[..., D + 1:].transpose(1, 2)
    assert k.shape == (B, T, H, D)
    _appended(hk, cache, k, v, table, [9, 0], None, host)


def _filled(hk, rng, lengths, H, D, page, spread=2, extra=3, width=None, scale=1.0):
    import torch
    B = len(lengths)
    width = width or max(1, max(-(-n // page) for n in lengths))
    cache = _garbage_cache(hk, B * width + extra, H, D, page, 1)
    table = _table(rng, B, width, B * width + extra)
    T = max(max(lengths), 1)
    k, v = (_tokens(rng, B, T, H, D, torch.bfloat16, spread) * scale for _ in range(2))
    k = k / k.float().abs().amax((2, 3), keepdim=True).to(k.dtype)       # scores of moderate size
    hk.kv8_append(cache, k.to(torch.bfloat16), v, table[1], _i32([0] * B), _i32(lengths))
    return cache, table


def _assert_attention(hk, q, cache, table, lengths, counts, causal, scale=None, **kw):
    import torch
    o, lse = hk.attention_kv8(q, cache, table[1], _i32(lengths), counts=None if counts is None else _i32(counts),
                              causal=causal, scale=scale, return_lse=True, **kw)
    assert _status(hk) == hk.HK_OK
    n = [q.size(1)] * q.size(0) if counts is None else counts
    host = _host(cache)
    want, wlse, mag = ref.attention(q.double().cpu().numpy(), host[0], host[1], host[2], host[3], table[0], lengths, n,
                                    causal, scale if scale is not None else q.size(3) ** -0.5)
    got = o.double().cpu().numpy()
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    rows = q.size(1) * q.size(2) // cache.heads
    weight = 2.0 ** -11 if q.dtype == torch.float16 or rows <= 64 else 2.0 ** -8
    tol = half * np.abs(want) + (weight + 2.0 ** -12) * mag + 2.0 ** -25
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} off, first {np.argwhere(bad)[:4].tolist()}: {got[bad][:4]} for "
                           f"{want[bad][:4]}")
    gl = lse.double().cpu().numpy()
    empty = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    assert (np.abs(gl[~empty] - wlse[~empty]) <= 2.0 ** -16 * np.maximum(1, np.abs(wlse[~empty]))).all()
    return o


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_decode(hk, D, page, group):
    import torch
    rng = np.random.default_rng(D + page + group)
    H = 2
    lengths = [1, 0, 31, 32, 33, 64, 129, 700]
    cache, table = _filled(hk, rng, lengths, H, D, page)
    for dtype in (torch.bfloat16, torch.float16):
        q = _tokens(rng, len(lengths), 1, H * group, D, dtype, 1)
        _assert_attention(hk, q, cache, table, lengths, None, True)


@pytest.mark.parametrize("T,group", [(2, 8), (3, 5), (5, 1), (5, 8), (17, 1), (33, 2), (70, 4), (130, 1), (40, 7)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_several_queries(hk, T, group, causal, D):
    """Queries at the end of each sequence; sequences shorter than the queries leave rows empty."""
    import torch
    rng = np.random.default_rng(T * group + D)
    H, page = 2, 64
    lengths = [T, T + 1, 200 + T, 1, max(T - 3, 0), 0]
    cache, table = _filled(hk, rng, lengths, H, D, page)
    q = _tokens(rng, len(lengths), T, H * group, D, torch.bfloat16, 1)
    _assert_attention(hk, q, cache, table, lengths, None, causal)
    counts = [T, 1, T // 2, 0, min(T, 2), T]
    _assert_attention(hk, q, cache, table, lengths, counts, causal)


@pytest.mark.parametrize("T", [1, 10, 40])
def test_strided_queries_and_output(hk, T):
    import torch
    rng = np.random.default_rng(T)
    H, group, D, lengths = 2, 4, 128, [77, 300]
    cache, table = _filled(hk, rng, lengths, H, D, 32)
    heads = _tokens(rng, 2, H * group, T, D, torch.bfloat16, 1)          # [B, H, T, D] storage
    q = heads.transpose(1, 2)
    out = torch.full((2, H * group, T, D), 5.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    a = _assert_attention(hk, q, cache, table, lengths, None, True, out=out)
    assert a is out
    odd = torch.empty(2, T, H * group, D + 1, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:] = q
    _assert_attention(hk, odd[..., 1:], cache, table, lengths, None, True)
    out = torch.full((2, T, H * group, D + 1), 5.0, dtype=torch.bfloat16, device="cuda")
    _assert_attention(hk, q, cache, table, lengths, None, True, out=out[..., :D])
    assert bool((out[..., D] == 5.0).all())
    one = q[:, :, :1].expand(-1, -1, H * group, -1)                      # one row for every head
    _assert_attention(hk, one, cache, table, lengths, None, True)


@pytest.mark.parametrize("T", [1, 64])
def test_pages_of_very_different_scale(hk, T):
    """Values from 2^-30 to 2^30 from page to page, and pages of zeros: the
    page's scale meets the sums in fp32, never a 16-bit weight."""
    import torch
    rng = np.random.default_rng(11)
    H, group, D, page = 1, 4, 128, 16
    n = 330
    k = torch.from_numpy(rng.standard_normal((1, n, H, D)) * 0.3).to(torch.bfloat16).cuda()
    e = np.repeat(rng.integers(-30, 31, -(-n // page)), page)[:n]
    e[160:176] = -1000
    v = torch.from_numpy(rng.standard_normal((1, n, H, D)) * np.exp2(e)[None, :, None, None]).to(torch.bfloat16).cuda()
    cache = _garbage_cache(hk, 24, H, D, page, 1)
    table = _table(rng, 1, 21, 24)
    hk.kv8_append(cache, k, v, table[1], _i32([0]))
    q = _tokens(rng, 1, T, H * group, D, torch.bfloat16, 1)
    _assert_attention(hk, q, cache, table, [n], None, True)


@pytest.mark.parametrize("T", [1, 64])
def test_queries_of_very_different_size(hk, T):
    import torch
    rng = np.random.default_rng(12)
    lengths = [100]
    cache, table = _filled(hk, rng, lengths, 1, 64, 16)
    q = _tokens(rng, 1, T, 8, 64, torch.bfloat16, 0)
    q = q * torch.tensor([2.0 ** -120, 2.0 ** -60, 1e-30, 1e-3, 1.0, 3.0, 0.0, 2.0 ** -133], device="cuda").view(1, 1, 8, 1)
    _assert_attention(hk, q.to(torch.bfloat16), cache, table, lengths, None, True)
    big = (q[:, :, 4:5].expand(-1, -1, 8, -1) * 2.0 ** 100).to(torch.bfloat16)      # a scale brings them back
    _assert_attention(hk, big.contiguous(), cache, table, lengths, None, True, scale=2.0 ** -103)


@pytest.mark.parametrize("T", [1, 64])
def test_nan_stays_with_its_head_and_rows(hk, T):
    import torch
    rng = np.random.default_rng(13)
    H, group, D, n = 2, 2, 64, 200
    cache, table = _filled(hk, rng, [n, n], H, D, 32)
    p = int(table[0][0][2])
    cache.k[p, 1, 5, 7] = 0x7F              # token 69 of sequence 0, KV head 1
    q = _tokens(rng, 2, T, H * group, D, torch.bfloat16, 1)
    o = hk.attention_kv8(q, cache, table[1], _i32([n, n])).isnan()
    assert bool(o[0, :, 2:].all()) and not bool(o[0, :, :2].any()) and not bool(o[1].any())
    q[1, 0, 1, 3] = float("nan")
    cache.k[p, 1, 5, 7] = 0
    o = hk.attention_kv8(q, cache, table[1], _i32([n, n])).isnan()
    assert bool(o[1, 0, 1].all()) and int(o.sum()) == D


@pytest.mark.parametrize("T", [1, 48, 100])
def test_pages_and_lengths_out_of_range_are_reported(hk, T):
    """They are never followed: the other sequences are right and the status says so."""
    import torch
    rng = np.random.default_rng(14)
    H, D, page = 2, 128, 64
    lengths = [300, 200, 100]
    cache, table = _filled(hk, rng, lengths, H, D, page)
    q = _tokens(rng, 3, T, H, D, torch.bfloat16, 1)
    want = hk.attention_kv8(q, cache, table[1], _i32(lengths))
    assert _status(hk) == hk.HK_OK
    for bad in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):
        t = table[1].clone()
        t[0, 1] = bad
        o = hk.attention_kv8(q, cache, t, _i32(lengths))
        assert _status(hk) == hk.HK_ERR_INVALID_ARG
        assert torch.equal(o[1:], want[1:])
        k = _tokens(rng, 3, 1, H, D, torch.bfloat16)
        before = _host(cache)
        hk.kv8_append(cache, k, k, t, _i32([64, 0, 0]), _i32([1, 0, 0]))
        assert _status(hk) == hk.HK_ERR_INVALID_ARG
        assert all(np.array_equal(a, b, equal_nan=a.dtype.kind == "f") for a, b in zip(before, _host(cache)))
    for bad in ([-5, 200, 100], [10 ** 9, 200, 100]):
        o = hk.attention_kv8(q, cache, table[1], _i32(bad))
        assert _status(hk) == hk.HK_ERR_INVALID_ARG
        assert torch.equal(o[1:], want[1:])
    for starts, counts in (([-1, 0, 0], [1, 0, 0]), ([10 ** 6, 0, 0], [1, 0, 0]), ([0, 0, 0], [2, 0, 0]), ([0, 0, 0], [-1, 0, 0])):
        hk.kv8_append(cache, q[:, :1], q[:, :1], table[1], _i32(starts), _i32(counts))
        assert _status(hk) == hk.HK_ERR_INVALID_ARG
    assert torch.equal(hk.attention_kv8(q, cache, table[1], _i32(lengths)), want)
    assert _status(hk) == hk.HK_OK


def test_table_wider_than_needed_and_many_sequences(hk):
    """A table with room for far more tokens than there are; more sequences than one launch takes."""
    import torch
    rng = np.random.default_rng(15)
    H, D, page, B = 1, 64, 16, 1100
    lengths = [int(x) for x in rng.integers(0, 40, B)]
    cache, table = _filled(hk, rng, lengths, H, D, page, width=3)
    wide = np.full((B, 500), -7, dtype=np.int32)             # entries past the tokens are not read
    for b, n in enumerate(lengths):
        wide[b, : -(-n // page)] = table[0][b, : -(-n // page)]
    q = _tokens(rng, B, 1, 2, D, torch.bfloat16, 1)
    _assert_attention(hk, q, cache, (wide, torch.from_numpy(wide).cuda()), lengths, None, True)


@pytest.mark.parametrize("T", [1, 40, 100])
def test_cache_beyond_32_bit_offsets(hk, T):
    import torch
    rng = np.random.default_rng(16)
    pages, H, page, D = 34000, 8, 64, 128                    # 2.2e9 codes of keys, as many of values
    cache = hk.Kv8Cache.empty(pages, H, D, page)
    n = 150
    t = np.array([[pages - 1, 0, pages - 2]], dtype=np.int32)
    table = (t, torch.from_numpy(t).cuda())
    k = _tokens(rng, 1, n, H, D, torch.bfloat16, 0)
    hk.kv8_append(cache, k * 0.2, k, table[1], _i32([0]))
    q = _tokens(rng, 1, T, H, D, torch.bfloat16, 0)
    o = hk.attention_kv8(q, cache, table[1], _i32([n]))
    assert _status(hk) == hk.HK_OK
    small = hk.Kv8Cache(*(x[t[0].tolist()].contiguous() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    again = (np.array([[0, 1, 2]], dtype=np.int32), _i32([[0, 1, 2]]))
    assert torch.equal(_assert_attention(hk, q, small, again, [n], None, True), o)


@pytest.mark.parametrize("T", [1, 5, 100])
def test_repeats_exactly_on_streams_and_in_graphs(hk, T):
    import torch
    rng = np.random.default_rng(17)
    lengths = [3000, 5, 800]
    H, D = 2, 128
    cache, table = _filled(hk, rng, lengths, H, D, 64)
    q = _tokens(rng, 3, T, H * 8, D, torch.bfloat16, 1)
    n = _i32(lengths)
    want = hk.attention_kv8(q, cache, table[1], n)
    for _ in range(3):
        assert torch.equal(hk.attention_kv8(q, cache, table[1], n), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hk.attention_kv8(q, cache, table[1], n, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = hk.attention_kv8(q, cache, table[1], n)
    n.copy_(_i32([100, 700, 20]))
    graph.replay()
    torch.cuda.synchronize()
    # (sequence 1 now reads what no append wrote, NaN among it: compared as bits)
    again = hk.attention_kv8(q, cache, table[1], _i32([100, 700, 20]))
    assert torch.equal(captured.view(torch.int16), again.view(torch.int16))
    assert _status(hk) == hk.HK_OK


@pytest.mark.parametrize("T,dtype", [(1, "bfloat16"), (9, "float16"), (70, "float16")])
def test_workspace_contents_do_not_matter(hk, T, dtype):
    """Long tables, whose units several warps share: every record and sum that is read was written by the call."""
    import ctypes

    import torch
    rng = np.random.default_rng(23)
    lengths, counts = [66000, 40, 0, 3000], [T, 1, T, max(T - 3, 0)]
    H, D, group = 2, 64, 3
    cache, table = _filled(hk, rng, lengths, H, D, 64)
    q = _tokens(rng, 4, T, H * group, D, getattr(torch, dtype), 1)
    want = _assert_attention(hk, q, cache, table, lengths, counts, True)
    lib = hk.load()
    size = lib.hk_attention_kv8_workspace_size(cache._ref, 4, T, H * group, table[1].size(1))
    assert size > 0
    n, c = _i32(lengths), _i32(counts)
    strides = (ctypes.c_int64 * 3)(*q.stride()[:3])
    for fill in (0, 0x7F, 0xFF):
        workspace = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        assert lib.hk_attention_kv8(q.data_ptr(), hk.HK_TYPE_BF16 if dtype == "bfloat16" else hk.HK_TYPE_FP16, strides,
                                    cache._ref, table[1].data_ptr(), table[1].stride(0), table[1].size(1), n.data_ptr(),
                                    c.data_ptr(), out.data_ptr(), strides, None, 4, T, H * group, 1, 0.0,
                                    workspace.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == hk.HK_OK
        assert _status(hk) == hk.HK_OK
        assert torch.equal(out, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,group,lengths", [(1, 1, 8, [9000]), (1, 8, 4, [4100]), (2, 4, 16, [2500, 33]), (1, 4, 1, [2100]),
                                               (5, 3, 2, [3000, 0, 1, 2000, 64])])
def test_few_units_over_many_blocks(hk, D, B, H, group, lengths):
    """Units that clusters of 2 to 16 blocks share, parts without tokens among them."""
    import torch
    rng = np.random.default_rng(31)
    cache, table = _filled(hk, rng, lengths, H, D, 64)
    q = _tokens(rng, B, 1, H * group, D, torch.bfloat16, 1)
    _assert_attention(hk, q, cache, table, lengths, None, True)
