"""hk_qk_norm_rope without a GPU: what it refuses, and what it does with nothing to do."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from dense_bf16_gemm_02_gb300 import build
    build.build()
    from dense_bf16_gemm_02_gb300 import hk_gemm
    return hk_gemm.load()


A = 1 << 20      # an aligned address that is never read on these paths
I3 = ctypes.c_int64 * 3
S = I3(4096, 1024, 128)


def test_refusals(lib):
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    INV, MIS = h.HK_ERR_INVALID_ARG, h.HK_ERR_MISALIGNED

    def rope(Q=A, qs=S, K=A + (1 << 16), ks=S, QO=A + (1 << 17), qos=S, KO=A + (1 << 18), kos=S, type=0, B=2, T=3, Hq=4, Hk=2, D=128,
             qw=None, kw=None, wt=0, eps=1e-6, pos=A, ps=I3(0, 3, 1), sections=None, axes=1, freq=A, pairs=64, il=0):
        sec = (ctypes.c_int32 * len(sections))(*sections) if sections is not None else None
        return lib.hk_qk_norm_rope(Q, qs, K, ks, QO, qos, KO, kos, type, B, T, Hq, Hk, D, qw, kw, wt, eps, pos, ps, sec, axes, freq,
                                   pairs, il, None)
    assert rope(B=0, Q=None) == h.HK_OK and rope(T=0, pos=None) == h.HK_OK and rope(Hq=0, Hk=0) == h.HK_OK
    assert rope(type=3) == INV and rope(type=-1) == INV and rope(wt=1) == INV and rope(wt=3) == INV
    assert rope(B=-1) == INV and rope(T=1 << 31) == INV and rope(Hq=-1) == INV and rope(Hk=65536) == INV
    assert rope(B=1 << 30, T=1 << 30) == INV
    for D in (0, 4, 100, 264, -8):
        assert rope(D=D, pairs=0) == INV, D
    for pairs in (-8, 4, 63, 72):
        assert rope(pairs=pairs) == INV, pairs
    assert rope(eps=float("nan")) == INV and rope(eps=float("inf")) == INV
    assert rope(axes=0) == INV and rope(axes=5, sections=[16, 16, 16, 8, 8]) == INV
    assert rope(axes=3) == INV and rope(axes=3, sections=[16, 24, 23]) == INV and rope(axes=3, sections=[16, 24, 25]) == INV
    assert rope(axes=2, sections=[-8, 72]) == INV and rope(sections=[63]) == INV
    assert rope(axes=2, sections=[2147483647, 2147483647]) == INV
    assert rope(Q=None) == INV and rope(K=None) == INV and rope(QO=None) == INV and rope(KO=None) == INV
    assert rope(qs=None) == INV and rope(kos=None) == INV and rope(pos=None) == INV and rope(ps=None) == INV and rope(freq=None) == INV
    assert rope(Q=A + 1) == MIS and rope(type=2, wt=2, KO=A + 2) == MIS and rope(pos=A + 2) == MIS and rope(freq=A + 1) == MIS
    assert rope(qw=A + 1) == MIS and rope(wt=2, kw=A + 2) == MIS
    assert rope(qos=I3(4096, 1024, 64)) == INV and rope(kos=I3(4096, 64, 128)) == INV and rope(qos=I3(0, 1024, 128)) == INV
    assert rope(QO=A, qos=I3(8192, 1024, 128)) == INV            # over its input, with other strides


def test_python_refusals(lib):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q = torch.zeros(1, 2, 3, 64)
    with pytest.raises(TypeError):
        hk.qk_norm_rope(q, q, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(32))
