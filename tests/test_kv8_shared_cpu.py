"""hk_attention_kv8_shared without a GPU: refusals and sizes."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from dense_bf16_gemm_02_gb300 import build
    build.build()
    from dense_bf16_gemm_02_gb300 import hk_gemm
    return hk_gemm.load()


A = 1 << 20      # a 256-byte aligned address that is never read on these paths
S3 = (ctypes.c_int64 * 3)(4096, 512, 64)


def _cache(**kw):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    f = dict(k_codes=A, v_codes=A, k_scale=A, v_scale=A, num_pages=4, heads=2, page_size=64, head_dim=64)
    f.update(kw)
    return h.hk_kv8_cache(**f)


def test_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS, WS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED, h.HK_ERR_WORKSPACE

    def at(cache=None, Q=A, type=0, qs=S3, table=A, stride=4, pages=4, lengths=A, counts=None, groups=A, shared=A, G=2, O=A, os=S3,
           lse=None, B=4, T=1, Hq=8, causal=1, scale=0.0, ws=A, wsb=1 << 40, flags=0):
        return lib.hk_attention_kv8_shared_ex(Q, type, qs, ctypes.byref(cache or _cache()), table, stride, pages, lengths, counts,
                                              groups, shared, G, O, os, lse, B, T, Hq, causal, scale, ws, wsb, flags, 0, None)
    assert at(B=0, Q=None) == h.HK_OK and at(T=0) == h.HK_OK and at(Hq=0) == h.HK_OK
    for bad in (dict(head_dim=96), dict(page_size=48), dict(heads=0), dict(num_pages=0), dict(k_codes=None), dict(v_scale=None)):
        assert at(_cache(**bad)) == INV, bad
    assert at(_cache(v_codes=A + 8)) == MIS
    assert at(type=2) == INV and at(Hq=7) == INV and at(B=-1) == INV and at(T=1 << 31) == INV
    assert at(G=0) == INV and at(G=5) == INV and at(groups=None) == INV and at(shared=None) == INV
    assert at(groups=A + 2) == MIS and at(shared=A + 1) == MIS
    assert at(scale=float("nan")) == INV and at(scale=-1.0) == INV and at(flags=1) == INV
    assert at(flags=0x30) == INV and at(flags=0x20, Q=A + 2) == INV
    assert at(flags=0x20, B=130, G=65) == INV                    # more groups than the tensor-core kernel plans for
    assert at(Q=None) == INV and at(O=None) == INV and at(qs=None) == INV and at(os=None) == INV
    assert at(table=None) == INV and at(lengths=None) == INV and at(pages=0) == INV and at(stride=2) == INV
    assert at(os=(ctypes.c_int64 * 3)(4096, 512, 32)) == INV and at(T=1 << 28) == INV
    assert at(pages=1 << 24, stride=1 << 24, B=512, Hq=2) == INV                 # more tiles than are counted
    assert at(Q=A + 1) == MIS and at(O=A + 1) == MIS and at(lse=A + 2) == MIS and at(counts=A + 1) == MIS
    c = _cache()
    for T in (1, 100, 300):                  # (1024 rows of a sequence and more: what attention_kv8 needs)
        need = lib.hk_attention_kv8_shared_workspace_size_ex(A, 0, S3, ctypes.byref(c), 4000, A, S3, 4, T, 8, 2, 0)
        assert 0 < need <= h.hk_attention_kv8_shared_workspace_size(c, 4, T, 8, 4000, 2)
        assert at(T=T, pages=4000, stride=4000, wsb=need - 1) == WS and at(T=T, pages=4000, stride=4000, ws=None) == WS
        assert at(T=T, pages=4000, stride=4000, ws=A + 128) == WS
    assert h.hk_attention_kv8_shared_workspace_size(c, 4, 300, 8, 4000, 2) == h.hk_attention_kv8_workspace_size(c, 4, 300, 8, 4000)
    assert at(T=300, pages=4000, stride=4000, flags=0x10) == INV and at(T=300, pages=4000, stride=4000, flags=0x20) == INV
    # (what attention_kv8 needs fits wherever it is chosen)
    for T in (1, 3, 20, 64, 200, 255):
        for pages in (1, 5, 40, 400, 4000):
            for B, G in ((1, 1), (4, 1), (64, 1), (64, 64), (700, 3)):
                need = h.hk_attention_kv8_shared_workspace_size(c, B, T, 8, pages, G)
                for type, at_q in ((0, A), (0, A + 2), (1, A), (1, A + 2)):
                    for flags in (0, 0x10, 0x20)[: 3 if at_q == A else 2]:
                        assert lib.hk_attention_kv8_shared_workspace_size_ex(at_q, type, S3, ctypes.byref(c), pages, A, S3, B, T, 8, G,
                                                                             flags) <= need
    assert lib.hk_attention_kv8_shared_workspace_size_ex(A, 0, S3, ctypes.byref(c), 4, A, S3, 2, 1, 8, 1, 0) == 0      # a small call
    for args in ((0, 1, 8, 4, 1), (4, 1, 7, 4, 1), (4, 1, 8, 4, 5), (4, 1, 8, 4, 0), (4, 1, 8, 0, 1)):
        assert h.hk_attention_kv8_shared_workspace_size(c, *args) == 0
    # (bounded by the rows of a launch, whatever the batch is)
    assert h.hk_attention_kv8_shared_workspace_size(c, 1 << 20, 1, 128, 4, 1) < 256 << 20


def test_python_refusals(lib):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        hk.attention_kv8_shared(torch.zeros(1, 1, 2, 64), None, z, z, z, z)
