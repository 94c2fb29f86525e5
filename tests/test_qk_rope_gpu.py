"""hk_qk_norm_rope against the formula in 64 bits.

Tolerance, with u = 2^-24: the sum of D <= 256 squares is a chain of 8 and a tree of 5, and with
the products, the mean, eps, the root, the quotient and the two factors an element of
the normalised row is off by at most 24 u of itself. A turn is off by 2^-31 of a turn and by
the rounding of its top 32 bits to 24 (together below 2^-22.6 radians), sincospi by another
2^-23. So before the last rounding an output a cos t - b sin t is off by less than
(|a| + |b|) (24 u + 2^-22 + 4 u) < (|a| + |b|) 2^-19; the last rounding adds half a
step: eps / 2 of the value, in fp16 at least 2^-25."""
import math

import pytest

pytestmark = pytest.mark.gpu

DT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _reference(x, weight, eps, positions, freq, sections, interleaved):
    """(value, |a| + |b|) in 64 bits; positions [axes, B, T]."""
    import torch
    x = x.double()
    if eps is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            x = x * weight.double()
    n = len(freq)
    axis = [a for a, m in enumerate(sections) for _ in range(m)]
    pos = positions.long()
    out, mag = x.clone(), x.abs()
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # whole turns in exact arithmetic: a float64 holds position times a 24-bit frequency exactly
        t = (pos[axis[i]].double() * float(freq[i])).unsqueeze(-1)
        c, s = torch.cos(t), torch.sin(t)
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return out, mag


def _check(got, x, weight, eps, positions, freq, sections, interleaved):
    import torch
    want, mag = _reference(x, weight, eps, positions, freq, sections, interleaved)
    half = torch.finfo(got.dtype).eps / 2
    tol = half * want.abs() + mag * 2.0 ** -19 + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (off - tol).max().item()


def _inputs(dtype, B, T, Hq, Hk, D, seed=0, views=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, T, Hq + 2 * Hk + 1, D, generator=g, device="cuda") * 3
    x = x.to(getattr(torch, DT[dtype]))
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    if not views:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(x.dtype) for _ in range(2)]
    return q, k, w


def _freq(pairs, base=10000.0):
    import torch
    return (base ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / max(pairs, 1))).float()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,pairs,sections,interleaved", [
    (1, 1, 1, 1, 64, 32, None, False), (64, 1, 64, 8, 128, 64, None, False), (2, 37, 7, 1, 128, 48, [16, 16, 16], False),
    (1, 5003, 3, 3, 128, 64, [10, 31, 23], True), (3, 11, 28, 4, 80, 40, None, False), (3, 11, 6, 2, 80, 16, [9, 7], True),
    (2, 9, 4, 4, 256, 128, None, False), (2, 9, 5, 3, 256, 64, [1, 2, 60, 1], False), (5, 3, 3, 2, 96, 24, None, True),
    (1, 2, 300, 0, 8, 0, None, False), (1, 7, 0, 5, 16, 8, None, False), (2, 3, 4, 4, 24, 8, None, False),
    (4, 1000, 64, 8, 128, 64, None, False),
])
def test_values(dtype, B, T, Hq, Hk, D, pairs, sections, interleaved):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q, k, (wq, wk) = _inputs(dtype, B, T, Hq, Hk, D)
    axes = len(sections) if sections else 1
    pos = torch.randint(0, 100000, (axes, B, T), device="cuda", dtype=torch.int32)
    freq = _freq(pairs)
    qo, ko = hk.qk_norm_rope(q, k, pos if sections else pos[0], freq, wq, wk, sections=sections, interleaved=interleaved)
    assert qo.shape == q.shape and ko.shape == k.shape and qo.dtype == q.dtype
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        if x.numel():
            _check(got, x, w, 1e-6, pos, freq.tolist(), sections or [pairs], interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_far_positions_and_odd_frequencies(dtype):
    """The whole range of int32, frequencies from 0 to 1000, negative ones among them. (A float64 product of a
    position and a 24-bit frequency is exact; its reduction in cos() too.)"""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q, k, _ = _inputs(dtype, 2, 6, 3, 1, 64)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1000003], [5, 131072, -77, 2 ** 30 + 1, 99999999, -2 ** 30]],
                       dtype=torch.int32, device="cuda")
    freq = _freq(32)
    freq[3], freq[5], freq[7], freq[8], freq[9], freq[10] = 0.0, -0.37, 1e-30, 1e-45, -1e-8, 1.0
    qo, ko = hk.qk_norm_rope(q, k, pos, freq, eps=1e-5)
    for got, x in ((qo, q), (ko, k)):
        _check(got, x, None, 1e-5, pos[None], freq.tolist(), [32], False)
    # frequencies above 1: near positions, as 2^e costs e bits of 64 (1000 x 2^20: 2^-34 of a turn)
    freq[0], freq[1] = 1000.0, -123.456
    near = pos % (1 << 20)
    qo, ko = hk.qk_norm_rope(q, k, near, freq, eps=1e-5)
    for got, x in ((qo, q), (ko, k)):
        _check(got, x, None, 1e-5, near[None], freq.tolist(), [32], False)
    freq[4] = float("inf")
    freq[6] = float("nan")
    qo, _ = hk.qk_norm_rope(q, k, near, freq, eps=1e-5)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[4, 6, 36, 38]] = True
    assert torch.equal(qo.isnan(), bad.expand_as(qo))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_without_norm_without_weights_with_fp32_weights(dtype):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q, k, (wq, wk) = _inputs(dtype, 2, 5, 4, 2, 128, 3)
    pos = torch.arange(10, device="cuda", dtype=torch.int32).view(2, 5)
    freq = _freq(64)
    for eps, a, b in ((None, None, None), (0.0, None, None), (1e-6, wq.float(), wk.float()), (1e-6, None, wk), (0.5, wq, None)):
        qo, ko = hk.qk_norm_rope(q, k, pos, freq, a, b, eps=eps)
        _check(qo, q, a, eps, pos[None], freq.tolist(), [64], False)
        _check(ko, k, b, eps, pos[None], freq.tolist(), [64], False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_alignment_and_in_place(dtype):
    """Rows at odd addresses, permuted dimensions, broadcast inputs, outputs inside other tensors, over the inputs."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    dt = getattr(torch, DT[dtype])
    B, T, Hq, Hk, D = 3, 5, 6, 2, 64
    pos = torch.randint(0, 5000, (B, T), device="cuda", dtype=torch.int32)
    freq = _freq(32)
    flat = torch.randn(B * T * (Hq + Hk) * (D + 1) + 9, device="cuda").to(dt)
    q = flat[1:].as_strided((B, T, Hq, D), (T * Hq * (D + 1), D + 1, T * (D + 1), 1))           # odd, heads outside tokens
    k = flat[3:].as_strided((B, T, Hk, D), (0, D + 1, T * (D + 1), 1))                          # one batch for all
    store = torch.full((B, Hq + Hk, T, D + 5), 9.0, device="cuda").to(dt)
    out = (store[:, :Hq, :, 3:3 + D].transpose(1, 2), store[:, Hq:, :, 3:3 + D].transpose(1, 2))
    got = hk.qk_norm_rope(q, k, pos, freq, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for y, x in zip(out, (q, k)):
        _check(y, x, None, 1e-6, pos[None], freq.tolist(), [32], False)
    assert (store[..., :3] == 9).all() and (store[..., 3 + D:] == 9).all()
    x = torch.randn(B, T, Hq + 2 * Hk, D, device="cuda").to(dt)
    kept = x.clone()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    hk.qk_norm_rope(q, k, pos, freq, out=(q, k))
    _check(q, kept[:, :, :Hq], None, 1e-6, pos[None], freq.tolist(), [32], False)
    _check(k, kept[:, :, Hq:Hq + Hk], None, 1e-6, pos[None], freq.tolist(), [32], False)
    assert torch.equal(x[:, :, Hq + Hk:], kept[:, :, Hq + Hk:])
    with pytest.raises(hk.HKError):
        hk.qk_norm_rope(q, k, pos, freq, out=(q.transpose(0, 1).contiguous().transpose(0, 1)[:, :, :1].expand(B, T, Hq, D), k))


def test_rows_of_nothing_infinities_and_nan():
    """A row of zeros stays zeros, a NaN takes its own row, an infinity makes its row 0 or NaN as the formula does."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q, k, _ = _inputs("bf16", 1, 4, 2, 1, 128, views=False)
    q[0, 0, 0] = 0
    q[0, 1, 1, 77] = float("nan")
    q[0, 2, 0, 5] = float("inf")
    pos = torch.arange(4, device="cuda", dtype=torch.int32).view(1, 4)
    freq = _freq(32)                     # half of each row is not turned
    y, _ = hk.qk_norm_rope(q, k, pos, freq)
    assert (y[0, 0, 0] == 0).all() and y[0, 1, 1].isnan().all()
    assert y[0, 2, 0, 5].isnan() and (y[0, 2, 0, 64:] == 0).all()
    rest = torch.ones(4, 2, dtype=torch.bool)
    rest[1, 1] = rest[2, 0] = False
    assert y[0][rest].isfinite().all()
    y, _ = hk.qk_norm_rope(q, k, pos, freq, eps=None)        # no norm: what is not turned is as it was, and the others' pairs
    assert y[0, 1, 1, 77].isnan() and y[0, 1, 1].isnan().sum() == 1
    assert not y[0, 2, 0, :5].isnan().any() and torch.equal(y[0, :, :, 64:].nan_to_num(), q[0, :, :, 64:].nan_to_num())


def test_a_captured_call_and_another_stream():
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q, k, (wq, wk) = _inputs("bf16", 4, 1, 8, 2, 128, views=False)
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    freq = _freq(64)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    a = hk.qk_norm_rope(q, k, pos, freq, wq, wk, stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = hk.qk_norm_rope(q, k, pos, freq, wq, wk)
    graph.replay()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    pos.add_(70001)
    graph.replay()
    _check(b[0], q, wq, 1e-6, pos[None], freq.tolist(), [64], False)
    assert math.isfinite(b[1].float().sum().item())


def test_refusals():
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    q, k, (wq, wk) = _inputs("bf16", 2, 3, 4, 2, 64)
    pos, freq = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), _freq(32)
    bad = [dict(k=k.float()), dict(k=k[:1]), dict(k=k[..., :32]), dict(positions=pos.long()), dict(positions=pos[:, :2]),
           dict(positions=pos.cpu()), dict(inv_freq=freq.double()), dict(inv_freq=freq[::2]), dict(q_weight=wq[:32]),
           dict(q_weight=wq.half()), dict(q_weight=wq.float()), dict(eps=-1.0), dict(sections=[16, 16]),
           dict(positions=pos.expand(2, 2, 3)), dict(positions=pos.expand(2, 2, 3), sections=[16, 15]), dict(inv_freq=_freq(40)),
           dict(inv_freq=_freq(12)), dict(out=(q, q)), dict(q=q.transpose(2, 3)), dict(q=q.double()), dict(q=q[0])]
    for change in bad:
        args = {**dict(q=q, k=k, positions=pos, inv_freq=freq, q_weight=wq, k_weight=wk), **change}
        with pytest.raises((TypeError, ValueError, hk.HKError)):
            hk.qk_norm_rope(**args)
    assert hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK
