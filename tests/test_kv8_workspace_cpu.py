"""The workspace of the cache attention is what the kernels that run the call need."""
import ctypes

import pytest

from test_kv8_cpu import P, S3, _cache, lib  # noqa: F401  (a fixture)


def _call(lib, c, size, flags=0, type=0, Q=P, qs=S3, O=P, os=S3, B=2, T=4000, Hq=8, pages=4000):  # noqa: F811
    return lib.hk_attention_kv8_ex(Q, type, qs, ctypes.byref(c), P, pages, pages, P, None, O, os, None, B, T, Hq, 1, 0.0, P,
                                   size, flags, 0, None)


def _size(lib, c, flags=0, type=0, Q=P, qs=S3, O=P, os=S3, B=2, T=4000, Hq=8, pages=4000):  # noqa: F811
    return lib.hk_attention_kv8_workspace_size_ex(Q, type, qs, ctypes.byref(c), pages, O, os, B, T, Hq, flags)


def test_calls_on_the_few_row_kernels_ask_for_no_widened_keys(lib):  # noqa: F811
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    c = _cache()
    most = h.hk_attention_kv8_workspace_size(c, 2, 4000, 8, 4000)
    assert most > 100 << 20
    odd, one = (ctypes.c_int64 * 3)(257, 129, 65), (ctypes.c_int64 * 3)(256, 128, 0)
    few = 1 << 25
    for kw in (dict(type=1), dict(qs=odd), dict(os=odd), dict(qs=one), dict(Q=P + 2), dict(O=P + 8)):
        assert 0 < _size(lib, c, **kw) <= few, kw
        assert _call(lib, c, few, **kw) != h.HK_ERR_WORKSPACE, kw
        assert _call(lib, c, _size(lib, c, **kw) - 1, **kw) == h.HK_ERR_WORKSPACE, kw
    assert _size(lib, c) == most and _call(lib, c, most - 1) == h.HK_ERR_WORKSPACE
    assert _size(lib, c, type=1, pages=4, T=1) == 0 and _size(lib, c, type=1, T=0) == 0 and _size(lib, c, qs=None) == 0


@pytest.mark.parametrize("B,T,Hq,pages", [(1, 1, 2, 4), (2, 4000, 8, 1000), (64, 1, 64, 512), (3, 100, 14, 10000), (1100, 9, 6, 30)])
def test_the_size_without_a_type_is_enough_for_every_one(lib, B, T, Hq, pages):  # noqa: F811
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    c = _cache(num_pages=1 << 20)
    most = h.hk_attention_kv8_workspace_size(c, B, T, Hq, pages)
    assert all(_size(lib, c, type=t, B=B, T=T, Hq=Hq, pages=pages) <= most for t in (0, 1))


def test_either_form_can_be_asked_for(lib):  # noqa: F811
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    c = _cache()
    few, many = h.HK_KV8_FEW_ROWS, h.HK_KV8_MANY_ROWS
    wide = 2 * 2 * 4000 * 64 * 2 * 64 * 2
    for T in (1, 4000):
        assert _size(lib, c, many, T=T) == wide and 0 < _size(lib, c, few, T=T) <= 1 << 25
        assert _call(lib, c, wide - 1, many, T=T) == h.HK_ERR_WORKSPACE
        assert _call(lib, c, 1 << 25, few, T=T) != h.HK_ERR_WORKSPACE
    assert _call(lib, c, wide, many, type=1) == h.HK_ERR_INVALID_ARG
    assert _call(lib, c, wide, many, O=P + 2) == h.HK_ERR_INVALID_ARG
    assert _call(lib, c, wide, few | many) == h.HK_ERR_INVALID_ARG
    for other in (0x1, 0x2, 0x8, 0x80, 0x100, 0x80000000):
        assert _call(lib, c, wide, other) == h.HK_ERR_INVALID_ARG


def test_a_wide_table_does_not_cost_a_round_for_each_sequence(lib):  # noqa: F811
    """64 sequences, 32 queries of 32 heads each: together they fill the GPU with 256-row items; where the table's
    width lets only a few be widened at a time, items of one sequence alone would leave most SMs idle."""
    c = _cache(num_pages=1 << 20, heads=8, head_dim=128)
    kw = dict(B=64, T=32, Hq=32)
    one = 2 * 8 * 128 * 2                                      # bytes of a widened token
    assert _size(lib, c, pages=32, **kw) == 64 * 2048 * one    # 2048 tokens: all at once, on the many-row form
    assert _size(lib, c, pages=512, **kw) < 64 << 20           # 32768: the few-row form
    assert _size(lib, c, pages=2048, **kw) < 64 << 20          # 131072
    assert _size(lib, c, pages=2048, B=64, T=2048, Hq=32) == 131072 * one      # whole prompts: still many rows
