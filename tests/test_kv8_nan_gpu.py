"""NaN among the cached values: a query that does not see a token is not touched by
it, one that does gets NaN in the dimensions that hold it. Finite values are held to
the tolerances of test_kv8_gpu.py."""
from __future__ import annotations

import numpy as np
import pytest

import kv8_ref as ref
from test_kv8_gpu import _filled, _host, _i32, _status, _tokens, hk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def _check(hk, B, H, group, T, D, page, lengths, counts, causal, spots, wide=0, weight=2.0 ** -11, seed=1):  # noqa: F811
    """spots: (sequence, token, head, dimension) of the values that are NaN."""
    import torch
    rng = np.random.default_rng(seed)
    cache, (t_np, t) = _filled(hk, rng, lengths, H, D, page)
    for b, j, h, d in spots:
        cache.v[int(t_np[b][j // page]), h, j % page, d] = 0x7F if d & 1 else 0xFF
    if wide:
        w = np.full((B, wide), -1, dtype=np.int32)
        w[:, : t_np.shape[1]] = t_np
        t_np, t = w, torch.from_numpy(w).cuda()
    q = _tokens(rng, B, T, H * group, D, torch.bfloat16, 1)
    o, lse = hk.attention_kv8(q, cache, t, _i32(lengths), counts=None if counts is None else _i32(counts), causal=causal,
                              return_lse=True)
    assert _status(hk) == hk.HK_OK
    host = _host(cache)
    with np.errstate(invalid="ignore"):
        want, wlse, mag = ref.attention(q.double().cpu().numpy(), *host, t_np, lengths, counts or [T] * B, causal, D ** -0.5)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    wrong = np.isnan(got) != np.isnan(want)
    assert not wrong.any(), (f"{wrong.sum()} values are NaN and should not be, or the other way round: "
                             f"{np.argwhere(wrong)[:4].tolist()}")
    assert np.isnan(want).any() == bool(spots)
    ok = np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (weight + 2.0 ** -12) * mag + 2.0 ** -25
    assert (ok | np.isnan(want)).all()
    none = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(gl), none) and (got[none] == 0).all()
    assert (np.abs(gl[~none] - wlse[~none]) <= 2.0 ** -16 * np.maximum(1, np.abs(wlse[~none]))).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("page,group,T,n", [(16, 8, 2, 300), (64, 4, 4, 301), (32, 1, 16, 97), (128, 3, 5, 64), (64, 8, 9, 32)])
def test_few_queries_that_do_not_see_a_token_are_not_touched_by_it(hk, D, wide, page, group, T, n):  # noqa: F811
    """The last tokens, one at a time to each sequence; a block for each unit, and tiles over the whole GPU."""
    B, H = 3, 2
    spots = [(0, n - 1, 0, 3), (0, n - 1, 0, D - 2), (1, n - 2, 1, 0), (2, n - T // 2 - 1, 0, 17), (2, 0, 1, 40)]
    _check(hk, B, H, group, T, D, page, [n] * B, None, True, spots, wide)


@pytest.mark.parametrize("D", [64, 128])
def test_one_warp_that_has_tiles_before_the_one_with_nan(hk, D):  # noqa: F811
    """720 units, a warp each: rows that see the first three tiles and nothing, or not all, of the last."""
    n = 97
    _check(hk, 90, 8, 1, 16, D, 32, [n] * 90, None, True, [(0, n - 1, 0, 3), (1, n - 2, 1, 5), (2, n - 9, 2, 7), (3, 40, 3, 0)])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("wide", [0, 3000])
@pytest.mark.parametrize("causal", [True, False])
def test_few_queries_past_the_count_and_before_the_first_token_stay_zero(hk, D, wide, causal):  # noqa: F811
    lengths, counts = [200, 3, 100], [2, 6, 1]
    _check(hk, 3, 2, 4, 6, D, 32, lengths, counts, causal, [(0, 198, 0, 5), (1, 1, 1, 9), (2, 50, 0, 63)], wide)


# (sizes at which a call runs on the attention-forward kernel: many rows of many heads)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,T,n", [(8, 100, 300), (3, 300, 400), (1, 700, 700)])
def test_many_queries_that_do_not_see_a_token_are_not_touched_by_it(hk, D, group, T, n):  # noqa: F811
    spots = [(0, n - 1, 0, 3), (0, n - 40, 1, D - 2), (0, n - 40, 1, D - 1), (1, n - T // 2, 7, 0), (1, 5, 2, 17)]
    _check(hk, 2, 8, group, T, D, 64, [n, n], None, True, spots, weight=2.0 ** -8)


@pytest.mark.parametrize("causal", [True, False])
def test_many_queries_past_the_count_and_before_the_first_token_stay_zero(hk, causal):  # noqa: F811
    _check(hk, 3, 8, 4, 150, 128, 32, [200, 60, 3], [70, 150, 1], causal, [(0, 198, 0, 5), (1, 1, 1, 9), (1, 59, 3, 8), (2, 2, 7, 63)],
           weight=2.0 ** -8)


def test_many_queries_without_nan_after_a_call_with_it(hk):  # noqa: F811
    _check(hk, 2, 8, 8, 100, 64, 16, [300, 90], None, True, [], weight=2.0 ** -8)


def test_calls_after_one_with_nan_are_as_fast_as_before(hk):  # noqa: F811
    """16384 tokens of 8 heads: looking through them for NaN, once one was seen, took some 390 us of a call of 420."""
    import torch
    rng = np.random.default_rng(5)
    n, H, D = 16384, 8, 128
    cache = hk.Kv8Cache.empty(n // 64, H, D, 64)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").view(1, -1)
    x = torch.randn(1, n, H, D, device="cuda").to(torch.bfloat16)
    hk.kv8_append(cache, x, x, table, _i32([0]))
    q = _tokens(rng, 1, 512, 32, D, torch.bfloat16, 0)
    length = _i32([n])

    def least():
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            hk.attention_kv8(q, cache, table, length)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    least()
    before = least()
    kept = cache.v[3].clone()
    cache.v[3, :, 7] = 0x7F
    assert bool(hk.attention_kv8(q, cache, table, length).isnan().all())
    cache.v[3] = kept
    assert not bool(hk.attention_kv8(q, cache, table, length).isnan().any())
    after = least()
    assert after <= 1.3 * before + 0.02, (before, after)
