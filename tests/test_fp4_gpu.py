"""Microscaled 4-bit quantisation and product against plain 64-bit forms.

Tolerances. Quantisation is compared bit for bit: MXFP4 scales are powers of
two, so every step before the rounding is exact, and NVFP4's fp32 steps are
repeated in the same order. A product's entry is off by its rounding to bf16
(half a step: 2^-8 of the value) plus the fp32 sums: each of the at most K / 16
additions of the tensor core may lose 2^-23 of the largest partial sum, at most
K · 2^-27 · Σ|a·b|, and the global scale's product and its application 2^-23."""
from __future__ import annotations

import numpy as np
import pytest

import fp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hk():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("no CUDA device")
    import dense_bf16_gemm_02_gb300 as pkg
    pkg.load()
    return pkg


def _status_ok(hk):
    import torch
    torch.cuda.synchronize()
    assert hk.hk_gemm_last_device_status(torch.cuda.current_device()) == hk.HK_OK


def _input(rows, cols, dtype, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
    x[rng.random((rows, cols)) < 0.02] *= 50
    x[rng.random((rows, cols)) < 0.05] = 0
    # values on the borders between codes, in blocks whose scale is 1
    t = torch.from_numpy(x).to(dtype)
    if cols >= 64:
        t[0, :32] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5,
                                  -5.0, 7.0] * 2).to(dtype)
    return t


def _assert_quantised(hk, q, x, fmt, g):
    code, byte = ref.quantize(x.float().numpy(), fmt, g)
    want = ref.pack(code)
    got = q.codes.cpu().numpy()
    assert np.array_equal(got[:, : want.shape[1]], want), f"codes differ at {np.argwhere(got[:, :want.shape[1]] != want)[:5]}"
    tiles = ref.tile_scales(byte, x.shape[1], fmt)
    assert np.array_equal(q.scales.cpu().numpy()[: tiles.size], tiles)
    assert np.array_equal(q.scale_matrix().cpu().numpy(), byte)


SHAPES = [(1, 1), (1, 8192), (3, 15), (2, 16), (5, 17), (7, 31), (4, 32), (4, 33), (127, 255), (128, 256), (129, 257),
          (300, 1000), (2, 1025), (40, 5003), (1000, 64)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_matches_definition(hk, fmt, dtype, rows, cols):
    import torch
    x = _input(rows, cols, getattr(torch, dtype), rows * 1000 + cols)
    g = float(x.float().abs().max()) / 2688 if fmt == "nvfp4" else None
    gt = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    g = None if gt is None else float(gt.item())
    q = hk.quantize_fp4(x.cuda(), format=fmt, global_scale=gt)
    _assert_quantised(hk, q, x, fmt, g)
    for out_dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = hk.dequantize_fp4(q, dtype=out_dtype).cpu()
        code, byte = ref.quantize(x.float().numpy(), fmt, g)
        s = ref.scale_value(byte, fmt)
        if g is not None:
            s = (s.astype(np.float32) * np.float32(g)).astype(np.float64)     # scale · g rounds once
        v = ref.GRID[code & 7] * np.where(code & 8, -1.0, 1.0) * np.repeat(s, ref.BLOCK[fmt], axis=1)[:, :cols]
        want = torch.from_numpy(v.astype(np.float32)).to(out_dtype)
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
    _status_ok(hk)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_strided_and_unaligned_rows(hk, fmt):
    import torch
    store = _input(70, 1100, torch.bfloat16, 5).cuda()
    for off, cols in ((0, 1024), (1, 1000), (3, 33), (8, 512)):
        x = store[:, off:off + cols]
        for rows in (slice(None), slice(1, None, 2)):
            q = hk.quantize_fp4(x[rows], format=fmt)
            _assert_quantised(hk, q, x[rows].cpu(), fmt, None)
    # codes written into a wider buffer leave the rest of its rows alone
    codes = torch.full((70, 600), 0xAB, dtype=torch.uint8, device="cuda")
    x = store[:, :1000]
    scales = torch.empty(hk.Fp4Matrix.scales_size(70, 1000, fmt), dtype=torch.uint8, device="cuda")
    q = hk.Fp4Matrix(codes[:, :576], scales, 70, 1000, fmt)
    if codes.stride(0) % 16 == 8:
        with pytest.raises(hk.HKError):
            hk.quantize_fp4(x, format=fmt, out=q)
    codes = torch.full((70, 608), 0xAB, dtype=torch.uint8, device="cuda")
    q = hk.Fp4Matrix(codes[:, :576], scales, 70, 1000, fmt)
    hk.quantize_fp4(x, format=fmt, out=q)
    _assert_quantised(hk, q, x.cpu(), fmt, None)
    assert bool((codes[:, 512:] == 0xAB).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_special_values(hk, fmt):
    import torch
    x = torch.zeros(6, 96, dtype=torch.float32)
    x[0] = torch.linspace(-3, 3, 96)
    x[0, 5] = float("nan")
    x[1] = torch.linspace(-3, 3, 96)
    x[1, 40] = float("inf")
    x[1, 95] = float("-inf")
    x[2] = 1e-44                       # subnormals
    x[3] = 3.3e38
    x[3, ::2] = -3.3e38
    x[4, ::7] = 2.0 ** -126
    x[5] = -0.0
    q = hk.quantize_fp4(x.cuda(), format=fmt)
    _assert_quantised(hk, q, x, fmt, None)
    y = hk.dequantize_fp4(q, dtype=torch.float32).cpu()
    blk = ref.BLOCK[fmt]
    assert bool(y[0, 5 // blk * blk:(5 // blk + 1) * blk].isnan().all()) and not bool(y[0, blk:].isnan().any())
    assert bool(y[1, 40 // blk * blk:(40 // blk + 1) * blk].isnan().all())


def _random_matrix(hk, rows, K, fmt, seed, g=None, spread=3):
    """A quantised matrix of random codes and scales: the library's object, codes and scale bytes."""
    import torch
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    nblk = -(-K // ref.BLOCK[fmt])
    if fmt == "mxfp4":
        byte = rng.integers(127 - spread, 128 + spread, (rows, nblk)).astype(np.uint8)
    else:
        byte = rng.integers(0x28, 0x50, (rows, nblk)).astype(np.uint8)
    gt = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    m = hk.Fp4Matrix(torch.from_numpy(ref.pack(code)).cuda(),
                     torch.from_numpy(ref.tile_scales(byte, K, fmt)).cuda(), rows, K, fmt, gt)
    return m, ref.values(code, byte, fmt, g)


def _assert_product(C, a, b, K):
    got = C.float().cpu().numpy().astype(np.float64)
    want = a @ b.T
    tol = 2.0 ** -8 * np.abs(want) + (K * 2.0 ** -27 + 2.0 ** -22) * (np.abs(a) @ np.abs(b).T) + 1e-300
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} entries off, first {np.argwhere(bad)[:4].tolist()}: "
                           f"{got[bad][:4]} for {want[bad][:4]}")


PRODUCTS = [(1, 1, 1), (1, 8, 31), (1, 130, 256), (3, 128, 257), (16, 300, 512), (17, 129, 1000), (33, 256, 2080),
            (64, 640, 768), (65, 257, 320), (128, 384, 1024), (129, 128, 512), (200, 1001, 1025), (256, 256, 4096),
            (300, 515, 255), (513, 770, 640), (1, 1024, 8192), (5, 200, 16384)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(hk, fmt, M, N, K):
    g = (0.37, 1.9) if fmt == "nvfp4" else (None, None)
    a, av = _random_matrix(hk, M, K, fmt, M + N + K, g[0])
    b, bv = _random_matrix(hk, N, K, fmt, M + N + K + 1, g[1])
    C = hk.gemm_fp4(a, b)
    _status_ok(hk)
    _assert_product(C, av, bv, K)


def _forced(hk, a, b, kernel, split):
    import torch
    M, N, K = a.rows, b.rows, a.cols
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ptr = lambda t: 0 if t is None else t.data_ptr()
    st = hk.hk_gemm_fp4_ex(a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                           out.data_ptr(), M, N, K, a.codes.stride(0), b.codes.stride(0), N,
                           hk.HK_FP4_MXFP4 if a.format == "mxfp4" else hk.HK_FP4_NVFP4, ptr(a.global_scale),
                           ptr(b.global_scale), kernel=kernel, split_k=split,
                           stream=torch.cuda.current_stream().cuda_stream)
    assert st == hk.HK_OK, hk.hk_gemm_last_error_string()
    return out


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 2304), (17, 130, 2048), (50, 129, 3000), (100, 640, 2100), (260, 513, 4096),
                                   (777, 1000, 1536)])
def test_every_kernel_and_split(hk, fmt, M, N, K):
    """4 = HK_KERNEL_SINGLE_128x128 with each K split, 1 = HK_KERNEL_PAIR_256x256."""
    a, av = _random_matrix(hk, M, K, fmt, M + N)
    b, bv = _random_matrix(hk, N, K, fmt, M + K)
    for kernel, split in ((4, 1), (4, 2), (4, 4), (4, 8), (1, 0)):
        _assert_product(_forced(hk, a, b, kernel, split), av, bv, K)
    _status_ok(hk)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(2560, 2100, 256), (5000, 2900, 320), (2304, 4352, 512)])
def test_product_of_several_rounds(hk, fmt, M, N, K):
    """More tiles than CTA pairs: accumulators take turns, the last round runs in halves."""
    a, av = _random_matrix(hk, M, K, fmt, 5)
    b, bv = _random_matrix(hk, N, K, fmt, 6)
    for _ in range(2):
        _assert_product(hk.gemm_fp4(a, b), av, bv, K)
    _status_ok(hk)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_scales_reach_their_rows_and_blocks(hk, fmt, M):
    """One code and one scale in each row of A, everything else 0 and scale 1:
    any scale read for another row or block shows."""
    import torch
    N, K = 260, 768
    blk = ref.BLOCK[fmt]
    one = 127 if fmt == "mxfp4" else 0x38
    for side in ("a", "b"):
        rows = M if side == "a" else N
        other = N if side == "a" else M
        code = np.zeros((rows, K), dtype=np.uint8)
        byte = np.full((rows, K // blk), one, dtype=np.uint8)
        r = np.arange(rows)
        at = (r * 37) % K
        code[r, at] = 2                                     # 1.0
        if fmt == "mxfp4":
            byte[r, at // blk] = 120 + r % 15
        else:
            byte[r, at // blk] = 0x20 + r % 60
        ones = np.full((other, K), 2, dtype=np.uint8)
        oneb = np.full((other, K // blk), one, dtype=np.uint8)

        def make(c, s, n):
            return hk.Fp4Matrix(torch.from_numpy(ref.pack(c)).cuda(),
                                torch.from_numpy(ref.tile_scales(s, K, fmt)).cuda(), n, K, fmt)
        x, y = make(code, byte, rows), make(ones, oneb, other)
        C = hk.gemm_fp4(x, y) if side == "a" else hk.gemm_fp4(y, x)
        want = ref.values(code, byte, fmt).sum(1)
        got = C.float().cpu().numpy()
        assert np.array_equal(got if side == "a" else got.T, np.repeat(want[:, None], other, 1).astype(np.float32))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_integer_sums_are_exact(hk, fmt):
    import torch
    M, N, K = 70, 200, 1000
    rng = np.random.default_rng(3)
    code = [rng.choice([0, 2, 4, 5, 10, 12, 13], (n, K)).astype(np.uint8) for n in (M, N)]
    byte = [np.full((n, -(-K // ref.BLOCK[fmt])), 127 if fmt == "mxfp4" else 0x38, dtype=np.uint8) for n in (M, N)]
    a, b = (hk.Fp4Matrix(torch.from_numpy(ref.pack(c)).cuda(), torch.from_numpy(ref.tile_scales(s, K, fmt)).cuda(),
                         c.shape[0], K, fmt) for c, s in zip(code, byte))
    want = torch.from_numpy(ref.values(code[0], byte[0], fmt) @ ref.values(code[1], byte[1], fmt).T).to(torch.bfloat16)
    assert torch.equal(hk.gemm_fp4(a, b).cpu(), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M", [2, 300])
def test_product_nan_scale_stays_in_its_row(hk, fmt, M):
    import torch
    N, K = 140, 700
    a, av = _random_matrix(hk, M, K, fmt, 1)
    b, bv = _random_matrix(hk, N, K, fmt, 2)
    nb = -(-K // 256) * (256 // ref.BLOCK[fmt])
    r, blkno = 1, 3
    at = (blkno // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + blkno % 4
    assert at < 128 * nb
    a.scales[at] = 255 if fmt == "mxfp4" else 0x7F
    C = hk.gemm_fp4(a, b).float().cpu().numpy()
    assert np.isnan(C[1]).all() and np.isfinite(np.delete(C, 1, 0)).all()


@pytest.mark.parametrize("M", [1, 100, 400])
def test_product_into_strided_output(hk, M):
    import torch
    N, K = 203, 512
    a, av = _random_matrix(hk, M, K, "nvfp4", 7, 0.5)
    b, bv = _random_matrix(hk, N, K, "nvfp4", 8)
    for off, width in ((0, 203), (8, 216), (1, 209)):
        store = torch.full((M + 2, width + off), 7.0, dtype=torch.bfloat16, device="cuda")
        out = store[1:M + 1, off:off + N]
        hk.gemm_fp4(a, b, out=out)
        _assert_product(out, av, bv, K)
        keep = store.clone()
        keep[1:M + 1, off:off + N] = 7.0
        assert bool((keep == 7.0).all()), "wrote outside the output"


def test_product_empty(hk):
    import torch
    a, _ = _random_matrix(hk, 5, 64, "mxfp4", 1)
    b = hk.quantize_fp4(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert hk.gemm_fp4(a, b).shape == (5, 0) and hk.gemm_fp4(b, a).shape == (0, 5)
    z = hk.quantize_fp4(torch.zeros(5, 0, dtype=torch.bfloat16, device="cuda"))
    w = hk.quantize_fp4(torch.zeros(9, 0, dtype=torch.bfloat16, device="cuda"))
    assert bool((hk.gemm_fp4(z, w, out=torch.ones(5, 9, dtype=torch.bfloat16, device="cuda")) == 0).all())


def test_quantize_then_product_on_a_stream_and_in_a_graph(hk):
    import torch
    M, N, K = 20, 384, 1024
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    w = hk.quantize_fp4(torch.randn(N, K, device="cuda", dtype=torch.bfloat16))
    want = hk.gemm_fp4(hk.quantize_fp4(x), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = hk.gemm_fp4(hk.quantize_fp4(x, stream=side), w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = hk.gemm_fp4(hk.quantize_fp4(x), w)
    x.copy_(torch.randn_like(x))
    graph.replay()
    assert torch.equal(captured, hk.gemm_fp4(hk.quantize_fp4(x), w))
    _status_ok(hk)


@pytest.mark.parametrize("M", [1, 300])
def test_product_wait_that_runs_out_is_reported(hk, M):
    import torch
    a, av = _random_matrix(hk, M, 4096, "mxfp4", 1)
    b, bv = _random_matrix(hk, 256, 4096, "mxfp4", 2)
    out = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")
    args = (a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(), out.data_ptr(), M, 256,
            4096, 2048, 2048, 256, hk.HK_FP4_MXFP4)
    assert hk.hk_gemm_fp4_ex(*args, flags=hk.HK_FLAG_FAULT_DROP_ARRIVE, timeout_ns=5_000_000,
                             stream=torch.cuda.current_stream().cuda_stream) == hk.HK_OK
    torch.cuda.synchronize()
    assert hk.hk_gemm_last_device_status(0) == hk.HK_ERR_TIMEOUT
    _assert_product(hk.gemm_fp4(a, b), av, bv, 4096)     # the context is usable, the next call right
    _status_ok(hk)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,split", [(100, 8200, 1500, 1), (128, 1030, 2048, 4), (90, 2000, 4096, 2), (128, 300, 4096, 8),
                                         (200, 130, 600, 1), (333, 520, 1024, 2), (1000, 257, 300, 1)])
def test_product_tiles_of_fewer_tokens_than_there_are(hk, fmt, M, N, K, split):
    """Several tiles along M whose scales lie in one tile of 128 rows."""
    from dense_bf16_gemm_02_gb300 import hk_gemm as h
    a, av = _random_matrix(hk, M, K, fmt, 11)
    b, bv = _random_matrix(hk, N, K, fmt, 12)
    _assert_product(_forced(hk, a, b, h.HK_KERNEL_SINGLE_128x128, split), av, bv, K)
    _assert_product(_forced(hk, a, b, h.HK_KERNEL_SINGLE_128x128, 0), av, bv, K)
    _status_ok(hk)


def test_out_that_is_no_quantised_matrix_is_refused(hk):
    import torch
    x = torch.zeros(4, 32, device="cuda")
    for out in (x, (4, 32)):
        with pytest.raises(TypeError):
            hk.quantize_fp4(x, out=out)
