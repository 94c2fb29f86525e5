"""The paged 8-bit cache's entry points without a GPU: refusals and sizes, and
pins of the plain reference that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import kv8_ref as ref


@pytest.fixture(scope="module")
def lib():
    from dense_bf16_gemm_02_gb300 import build
    build.build()
    from dense_bf16_gemm_02_gb300 import hk_gemm
    return hk_gemm.load()


P = 1 << 20      # a 256-byte aligned address that is never read on these paths
S3 = (ctypes.c_int64 * 3)(256, 128, 64)


def _cache(**kw):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    f = dict(k_codes=P, v_codes=P, k_scale=P, v_scale=P, num_pages=4, heads=2, page_size=64, head_dim=64)
    f.update(kw)
    return h.hk_kv8_cache(**f)


BAD_CACHES = [dict(head_dim=96), dict(head_dim=0), dict(page_size=48), dict(page_size=256), dict(page_size=0),
              dict(heads=0), dict(heads=-1), dict(num_pages=0), dict(num_pages=1 << 31), dict(k_codes=None),
              dict(v_codes=None), dict(k_scale=None), dict(v_scale=None)]


def test_append_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED

    def ap(cache=None, K=P, V=P, type=0, B=2, T=3, ks=S3, vs=S3, table=P, stride=4, pages=4, starts=P, counts=None):
        return lib.hk_kv8_append(ctypes.byref(cache or _cache()), K, V, type, B, T, ks, vs, table, stride, pages, starts,
                                 counts, None)
    assert ap(B=0, K=None) == h.HK_OK and ap(T=0, table=None) == h.HK_OK
    assert lib.hk_kv8_append(None, P, P, 0, 1, 1, S3, S3, P, 4, 4, P, None, None) == INV
    for bad in BAD_CACHES:
        assert ap(_cache(**bad)) == INV, bad
    assert ap(_cache(k_codes=P + 8)) == MIS and ap(_cache(v_scale=P + 2)) == MIS
    assert ap(type=3) == INV and ap(B=-1) == INV and ap(T=-1) == INV and ap(B=1 << 31) == INV
    assert ap(K=None) == INV and ap(V=None) == INV and ap(ks=None) == INV and ap(table=None) == INV and ap(starts=None) == INV
    assert ap(pages=0) == INV and ap(stride=3) == INV and ap(pages=1 << 26) == INV
    assert ap(K=P + 1) == MIS and ap(type=2, V=P + 2) == MIS and ap(starts=P + 2) == MIS and ap(table=P + 1) == MIS


def test_attention_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS, WS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED, h.HK_ERR_WORKSPACE

    def at(cache=None, Q=P, type=0, qs=S3, table=P, stride=4, pages=4, lengths=P, counts=None, O=P, os=S3, lse=None, B=2,
           T=1, Hq=8, causal=1, scale=0.0, ws=P, wsb=1 << 40, flags=0):
        return lib.hk_attention_kv8_ex(Q, type, qs, ctypes.byref(cache or _cache()), table, stride, pages, lengths, counts, O,
                                       os, lse, B, T, Hq, causal, scale, ws, wsb, flags, 0, None)
    assert at(B=0, Q=None) == h.HK_OK and at(T=0) == h.HK_OK and at(Hq=0) == h.HK_OK
    for bad in BAD_CACHES:
        assert at(_cache(**bad)) == INV, bad
    assert at(type=2) == INV and at(Hq=7) == INV and at(B=-1) == INV and at(T=-1) == INV and at(Hq=-2) == INV
    assert at(scale=float("nan")) == INV and at(scale=float("inf")) == INV and at(scale=-1.0) == INV and at(flags=1) == INV
    assert at(Q=None) == INV and at(O=None) == INV and at(qs=None) == INV and at(os=None) == INV
    assert at(table=None) == INV and at(lengths=None) == INV and at(pages=0) == INV and at(stride=2) == INV
    assert at(T=1 << 30) == INV
    assert at(Q=P + 1) == MIS and at(O=P + 1) == MIS and at(lse=P + 2) == MIS and at(counts=P + 1) == MIS
    c = _cache()
    long = dict(pages=4000, stride=4000)
    need = h.hk_attention_kv8_workspace_size(c, 2, 1, 8, 4000)
    assert need > 0 and at(wsb=need - 1, **long) == WS and at(ws=None, **long) == WS and at(ws=P + 128, **long) == WS
    assert h.hk_attention_kv8_workspace_size(c, 2, 1, 8, 4) == 0         # short: nothing is left in memory
    wide = h.hk_attention_kv8_workspace_size(c, 2, 4000, 8, 1000)        # bf16 keys and values of two sequences
    assert wide == 2 * 2 * 1000 * 64 * 2 * 64 * 2
    assert h.hk_attention_kv8_workspace_size(c, 64, 4000, 8, 4000) <= 512 << 20
    assert h.hk_attention_kv8_workspace_size(c, 64, 4000, 8, 100000) == 2 * 100000 * 64 * 2 * 64 * 2
    assert h.hk_attention_kv8_workspace_size(c, 0, 1, 8, 4) == 0
    assert lib.hk_attention_kv8(P, 0, S3, ctypes.byref(c), P, 4, 4, P, None, P, S3, None, 2, 1, 7, 1, 0.0, P, need, None) == INV


def test_python_refusals():
    import torch

    import dense_bf16_gemm_02_gb300 as hk
    z = torch.zeros(2, 1, 64, 64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        hk.Kv8Cache(z, z, torch.zeros(2, 1), torch.zeros(2, 1))


def test_reference_append_by_hand():
    codes = np.full((2, 1, 16, 64), 0x7F, dtype=np.uint8)
    scale = np.full((2, 1), np.nan, dtype=np.float32)
    x = np.zeros((1, 2, 1, 64))
    x[0, 0, 0, 0], x[0, 1, 0, 1] = 448.0, 1.0
    ref.append(codes, scale, x, [[1]], [0], [2])
    assert scale[1, 0] == 1.0 and codes[1, 0, 0, 0] == 0x7E and codes[1, 0, 1, 1] == 0x38 and codes[1, 0, 2, 0] == 0x7F
    ref.append(codes, scale, np.full((1, 1, 1, 64), -449.0), [[1]], [2], [1])
    assert scale[1, 0] == 2.0 and codes[1, 0, 0, 0] == 0x76 and codes[1, 0, 1, 1] == 0x30
    assert np.all(ref.values(codes, scale, [1], 3)[0, 2] == -448.0)      # 224.5 is nearest 224
    ref.append(codes, scale, np.full((1, 1, 1, 64), 1.0), [[1]], [3], [1])
    assert scale[1, 0] == 2.0 and np.all(ref.values(codes, scale, [1], 4)[0, 3] == 1.0)


def test_reference_attention_by_hand():
    codes = np.full((1, 1, 16, 64), 0x38, dtype=np.uint8)               # 1.0 everywhere
    scale = np.ones((1, 1), dtype=np.float32)
    v = codes.copy()
    v[0, 0, 1] = 0x40                                                    # token 1 holds 2.0
    q = np.zeros((1, 3, 1, 64))
    o, lse, _ = ref.attention(q, codes, scale, v, scale, [[0]], [2], [3], True, 1.0)
    assert np.all(o[0, 0] == 0) and np.isneginf(lse[0, 0, 0])            # stands before the first token
    assert np.all(o[0, 1] == 1.0) and np.allclose(o[0, 2], 1.5) and np.isclose(lse[0, 2, 0], np.log(2))


def test_sizes_that_pass_64_bits_are_refused(lib):
    """Shapes whose products (rows x heads x head_dim) pass what 64 bits hold: refused, and no bytes asked for."""
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV = h.HK_ERR_INVALID_ARG

    def at(cache, T, Hq, pages):
        return lib.hk_attention_kv8(P, 0, S3, ctypes.byref(cache), P, pages, pages, P, None, P, S3, None, 1, T, Hq, 1, 0.0,
                                    P, 1 << 40, None)
    many_heads = _cache(num_pages=1, heads=1 << 27, page_size=16, head_dim=128)
    assert h.hk_attention_kv8_workspace_size(many_heads, 1, 128, 1 << 27, 1 << 26) == 0
    assert at(many_heads, 128, 1 << 27, 1 << 26) == INV
    one_page = _cache(num_pages=1, heads=65535, page_size=128, head_dim=128)
    assert h.hk_attention_kv8_workspace_size(one_page, 1, 4096, 65535, (1 << 24) - 1) > 1 << 40    # (huge, but a size)
    assert h.hk_attention_kv8_workspace_size(one_page, 1, 4096, 65535, 1 << 24) == 0               # 2^31 tokens
    assert at(one_page, 4096, 65535, 1 << 24) == INV
    for bad in BAD_CACHES:
        if all(v is not None for v in bad.values()):
            assert h.hk_attention_kv8_workspace_size(_cache(**bad), 2, 4000, 8, 4000) == 0, bad
    assert h.hk_attention_kv8_workspace_size(_cache(), 2, 1 << 40, 8, 4000) == 0
    assert h.hk_attention_kv8_workspace_size(_cache(), 1 << 40, 1, 8, 4000) == 0


def test_what_is_no_cache_is_refused():
    import torch

    from dense_bf16_gemm_02_gb300 import attention_kv8, kv8_append
    t, table, n = torch.zeros(1, 1, 1, 64), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for cache in (None, (t, t, t, t)):
        with pytest.raises(TypeError):
            kv8_append(cache, t, t, table, n)
        with pytest.raises(TypeError):
            attention_kv8(t, cache, table, n)
