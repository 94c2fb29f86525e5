"""Attention over the 8-bit cache with pages that sequences share, against 64-bit sums
over what each sequence sees.

Tolerances as in test_kv8_gpu.py: the weights are rounded by at most half a step before they
meet V (2^-11 of them where they are f16, 2^-8 where they are bf16: blocks of shared units on the
tensor-core kernel where values' scales are more than 2^7 above the first ones or 2^14 below the largest), fp32 scores, exponentials and sums add less
than 2^-12 of the weighted |V|, the output is rounded by half a step, and the log-sum-exp
is fp32: 2^-16 of max(1, |lse|)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

FEW, MANY = 0x10, 0x20         # units of 16 rows, shared units of 128 rows
FORMS = pytest.mark.parametrize("form", [FEW, MANY], ids=["few", "many"])


def _i32(x):
    import torch
    return x if isinstance(x, torch.Tensor) else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Batch:
    """Groups of sequences [(shared tokens, [own tokens, ...]), ...] over a cache whose other places hold NaN."""

    def __init__(self, groups, H=2, D=64, page=16, seed=0, spare=3, scales=(0.0625, 0.03125)):
        import torch
        import dense_bf16_gemm_02_gb300 as hk
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.shared = [s for s, _ in groups]
        self.lengths = [s + n for s, own in groups for n in own]
        self.offsets = np.cumsum([0] + [len(own) for _, own in groups]).tolist()
        B, width = len(self.lengths), max(1, max(-(-n // page) for n in self.lengths))
        table = np.full((B, width), -1, dtype=np.int64)
        at = 0
        for (s, own), b0 in zip(groups, self.offsets):
            for i, n in enumerate(own):
                whole, slots = (s // page if i else 0), -(-(s + n) // page)
                table[b0 + i, :whole] = table[b0, :whole]
                table[b0 + i, whole:slots] = np.arange(at, at + slots - whole)
                at += slots - whole
        perm = rng.permutation(at + spare)
        table = np.where(table >= 0, perm[table], -1)
        pages = at + spare
        self.cache = c = hk.Kv8Cache.empty(pages, H, D, page)
        self.page, self.H, self.D, self.B = page, H, D, B
        for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
            codes.fill_(0x7F)
            scale.fill_(float("nan"))
            x = (torch.randn(pages, H, page, D, generator=g, device="cuda") * 16).to(torch.float8_e4m3fn).view(torch.uint8)
            pick = torch.tensor(scales, device="cuda")[torch.randint(0, len(scales), (pages, H), generator=g, device="cuda")]
            filled = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
            for b, n in enumerate(self.lengths):
                ids = torch.tensor(table[b, : -(-n // page)], device="cuda")
                place = torch.arange(len(ids) * page, device="cuda").view(-1, page) < n
                filled[ids] |= place
            codes.copy_(torch.where(filled[:, None, :, None], x, codes))
            scale.copy_(torch.where(filled.any(1)[:, None], pick, scale))
            for (s, own), b0 in zip(groups, self.offsets):        # the shared tokens of a page that is not all shared
                if s % page:
                    for b in range(b0 + 1, b0 + len(own)):
                        a, z = table[b0, s // page], table[b, s // page]
                        codes[z, :, : s % page] = codes[a, :, : s % page]
                        scale[z] = scale[a]
        self.np_table = table
        self.table = _i32(table)

    def values(self, b):
        """k, v float64 [H, n, D]."""
        import torch
        n = self.lengths[b]
        ids = torch.tensor(self.np_table[b, : -(-n // self.page)], device="cuda")
        return [(codes[ids].view(torch.float8_e4m3fn).double() * scale[ids].double()[:, :, None, None]).transpose(0, 1)
                .reshape(self.H, -1, self.D)[:, :n] for codes, scale in ((self.cache.k, self.cache.k_scale),
                                                                        (self.cache.v, self.cache.v_scale))]

    def reference(self, q, counts, causal, scale):
        """(o, lse, sum of p |v|), float64."""
        import torch
        B, T, Hq, D = q.shape
        o = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
        mag, lse = o.clone(), torch.full((B, T, Hq), -np.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(self.lengths):
            if n == 0:
                continue
            k, v = self.values(b)
            for t in range(counts[b]):
                seen = max(0, n - counts[b] + t + 1) if causal else n
                if seen == 0:
                    continue
                x = q[b, t].double().view(self.H, -1, D)
                s = torch.einsum("hgd,hld->hgl", x, k[:, :seen]) * scale
                p = torch.softmax(s, -1)
                o[b, t] = torch.einsum("hgl,hld->hgd", p, v[:, :seen]).reshape(Hq, D)
                mag[b, t] = torch.einsum("hgl,hld->hgd", p, v[:, :seen].abs()).reshape(Hq, D)
                lse[b, t] = torch.logsumexp(s, -1).view(Hq)
        return o, lse, mag


def _strides(t):
    return (ctypes.c_int64 * 3)(*t.stride()[:3])


def _attend(batch, q, counts=None, causal=True, scale=0.0, form=0, out=None, fill=0xFF, flags=0, timeout_ns=0, shared=None,
            offsets=None, lengths=None, wait=True):
    """(o, lse) through the entry point with controls; the workspace is full of `fill` before."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    B, T, Hq, D = q.shape
    lib = hk.load()
    out = torch.full_like(q, 3.0) if out is None else out
    lse = torch.full((B, T, Hq), 3.0, dtype=torch.float32, device="cuda")
    offsets, shared = _i32(batch.offsets if offsets is None else offsets), _i32(batch.shared if shared is None else shared)
    size = lib.hk_attention_kv8_shared_workspace_size(batch.cache._ref, B, T, Hq, batch.table.size(1), len(shared))
    workspace = torch.full((max(size, 1),), fill, dtype=torch.uint8, device="cuda")
    n, c = _i32(batch.lengths if lengths is None else lengths), None if counts is None else _i32(counts)
    st = lib.hk_attention_kv8_shared_ex(
        q.data_ptr(), hk.HK_TYPE_BF16 if q.dtype == torch.bfloat16 else hk.HK_TYPE_FP16, _strides(q), batch.cache._ref,
        batch.table.data_ptr(), batch.table.stride(0), batch.table.size(1), n.data_ptr(), None if c is None else c.data_ptr(),
        offsets.data_ptr(), shared.data_ptr(), len(shared), out.data_ptr(), _strides(out), lse.data_ptr(), B, T, Hq,
        1 if causal else 0, scale, workspace.data_ptr(), size, form | flags, timeout_ns, torch.cuda.current_stream().cuda_stream)
    assert st == hk.HK_OK, hk.hk_gemm_last_error_string()
    if wait:
        torch.cuda.synchronize()
    return out, lse


def _status():
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    torch.cuda.synchronize()
    return hk.hk_gemm_last_device_status(torch.cuda.current_device())


def _check(batch, q, got, counts=None, causal=True, scale=0.0, form=0, rows=None, weight=2.0 ** -11):
    import torch
    o, lse = got
    counts = [q.size(1)] * q.size(0) if counts is None else counts
    want, wlse, mag = batch.reference(q, counts, causal, scale or q.size(3) ** -0.5)
    half = torch.finfo(q.dtype).eps / 2
    tol = half * want.abs() + (weight + 2.0 ** -12) * mag + 2.0 ** -25
    off = (o.double() - want).abs()
    rows = slice(None) if rows is None else rows
    bad = ~(off <= tol)[rows]
    assert not bad.any(), (int(bad.sum()), (off - tol)[rows].max().item(), bad.nonzero()[:4].tolist())
    assert torch.equal(lse[rows] == -np.inf, wlse[rows] == -np.inf)
    near = (lse.double() - wlse).abs() <= 2.0 ** -16 * wlse.abs().clamp(min=1)
    assert (near | (wlse == -np.inf))[rows].all()


def _q(B, T, Hq, D, dtype="bf16", seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    return torch.randn(B, T, Hq, D, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float16)


@FORMS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,page,H,group,T,groups", [
    (64, 16, 1, 1, 1, [(128, [1, 5])]),
    (128, 64, 8, 8, 1, [(1000, [60, 1, 24, 33])]),
    (64, 32, 2, 7, 1, [(300, [20] * 9), (127, [1, 200]), (0, [5]), (700, [1]), (128, [128, 1, 63])]),
    (128, 128, 1, 4, 3, [(513, [3, 9, 70]), (256, [3])]),
    (64, 128, 4, 2, 5, [(2000, list(range(5, 45)))]),
    (128, 16, 2, 1, 1, [(3000, [7] * 130)]),
    (128, 32, 1, 16, 2, [(5003, [2 + i % 50 for i in range(33)])]),
    (64, 64, 1, 1, 1, [(2 + 40 * i, [1 + i, 3]) for i in range(40)]),
])
def test_values(form, dtype, D, page, H, group, T, groups):
    batch = Batch(groups, H, D, page)
    q = _q(batch.B, T, H * group, D, dtype)
    _check(batch, q, _attend(batch, q, form=form), form=form)
    _check(batch, q, _attend(batch, q, causal=False, scale=0.05, form=form), causal=False, scale=0.05, form=form)
    assert _status() == 0


@FORMS
@pytest.mark.parametrize("D,page,B,H,group", [(64, 32, 3, 1, 2), (128, 64, 20, 8, 4), (64, 16, 40, 8, 1), (128, 128, 90, 8, 2),
                                              (64, 64, 200, 8, 1)])
def test_own_parts_short_and_long(form, D, page, B, H, group):
    """Own parts of one token to thousands, in blocks of eight to one warps and, where they are long, spread over the GPU."""
    own = [(37 * i * i + 1) % 90 + 1 for i in range(B)]
    own[1], own[B // 2] = 9000, 2500
    cut = B // 3
    batch = Batch([(700, own[:cut]), (130, own[cut:])], H, D, page)
    q = _q(batch.B, 1, H * group, D)
    _check(batch, q, _attend(batch, q, form=form), form=form)
    assert _status() == 0


@FORMS
def test_counts_empty_sequences_and_queries_inside_what_is_shared(form):
    """Sequences that hold nothing or ask nothing, first sequences shorter than the shared part, queries that do not see
    all of it: those read their own tables."""
    import torch
    batch = Batch([(400, [0, 0, 4, 9]), (256, [0, 3, 3])], 2, 64, 32)
    q = _q(batch.B, 4, 8, 64)
    for lengths, counts in (([400, 400, 404, 409, 256, 259, 259], [1, 4, 4, 0, 4, 2, 3]),
                            ([0, 0, 404, 409, 256, 0, 259], [1, 0, 2, 4, 1, 1, 4]),
                            ([150, 400, 404, 17, 256, 2, 259], [4, 4, 1, 4, 0, 3, 4]),
                            ([400, 130, 3, 409, 200, 100, 50], [4, 4, 4, 4, 4, 4, 4])):
        batch.lengths = lengths
        for causal in (True, False):
            got = _attend(batch, q, counts, causal, form=form)
            _check(batch, q, got, counts, causal, form=form)
            for b, n in enumerate(counts):
                assert (got[0][b, n:] == 0).all() and (got[1][b, n:] == -np.inf).all()
    assert _status() == 0 and torch.isfinite(got[0]).all()


@FORMS
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_strided_queries_and_output(form, dtype):
    import torch
    batch = Batch([(300, [9, 40, 2]), (140, [3, 3])], 2, 64, 16)
    wide = _q(batch.B, 2, 11, 64, dtype)
    q = wide[:, :, 1:7]                                           # 6 heads of a fused row
    store = torch.full((batch.B, 6, 2, 70), 5.0, dtype=q.dtype, device="cuda")
    out = store[..., 3:67].transpose(1, 2)                        # odd rows, heads outside tokens
    _check(batch, q, _attend(batch, q, form=form, out=out), form=form)
    assert (store[..., :3] == 5).all() and (store[..., 67:] == 5).all()
    flat = torch.randn(batch.B * 2 * 6 * 65 + 1, device="cuda").to(q.dtype)
    q = flat[1:].view(batch.B, 2, 6, 65)[..., :64]                # rows at odd addresses
    if form == MANY:                                              # (refused there, chosen otherwise without a form)
        with pytest.raises(AssertionError, match="16-byte"):
            _attend(batch, q, form=form)
    _check(batch, q, _attend(batch, q, form=form & FEW), form=FEW)
    q = _q(1, 1, 6, 64, dtype).expand(batch.B, 2, 6, 64)          # one row for all
    _check(batch, q, _attend(batch, q, form=form), form=form)


@FORMS
def test_many_sequences_and_groups(form):
    """More sequences and groups than one launch plans for, groups that the launches cut."""
    groups = [(130 + (i % 3) * 128, [1 + (i * 7 + j) % 5 for j in range(1 + i % 4)]) for i in range(520)]
    batch = Batch(groups, 1, 64, 128)
    q = _q(batch.B, 1, 2, 64)
    assert batch.B > 1024 and len(groups) > 512
    _check(batch, q, _attend(batch, q, form=form & FEW), form=FEW)
    assert _status() == 0
    for groups in ([(640, [3] * 700)], [(640, [3] * 300), (0, [9]), (300, [7] * 280), (400, [5, 2500] * 60)]):
        batch = Batch(groups, 1, 64, 64)
        q = _q(batch.B, 1, 2, 64)
        _check(batch, q, _attend(batch, q, form=form), form=form)
    assert _status() == 0


@FORMS
def test_pages_and_queries_of_very_different_size(form):
    batch = Batch([(1024, [40, 9, 100])], 2, 128, 16, scales=(2.0 ** -4, 2.0 ** -40, 2.0 ** -9))
    q = _q(batch.B, 1, 8, 128)
    weight = 2.0 ** -11 if form == FEW else 2.0 ** -8
    _check(batch, q, _attend(batch, q, form=form), form=form, weight=weight)
    q = q.clone()
    q[0] *= 2.0 ** -90
    q[1, 0, 3] *= 2.0 ** 20
    q[2, 0, 1] = 0
    _check(batch, q, _attend(batch, q, scale=2.0 ** -24, form=form), scale=2.0 ** -24, form=form, weight=weight)
    batch = Batch([(1500, [40, 9, 100])], 2, 64, 32, scales=(2.0 ** 9, 2.0 ** 6, 2.0 ** 20, 2.0 ** -126))      # (bf16 ends at 2^127)
    q = _q(batch.B, 1, 8, 64)
    _check(batch, q, _attend(batch, q, scale=2.0 ** -26, form=form), scale=2.0 ** -26, form=form, weight=weight)
    # scales that all lie within what f16 values take, and pages that grow from block to block
    for D, scales in ((64, (2.0 ** -8, 2.0 ** -11, 2.0 ** -15)), (128, (2.0 ** 7, 2.0 ** 0, 2.0 ** 4))):
        batch = Batch([(1500, [40, 9, 100])], 2, D, 32, scales=scales)
        q = _q(batch.B, 1, 8, D)
        _check(batch, q, _attend(batch, q, scale=2.0 ** -12, form=form), scale=2.0 ** -12, form=form)
    batch = Batch([(2560, [40, 9, 100])], 2, 64, 128)
    q = _q(batch.B, 1, 8, 64)
    for step in (1, 6, -1, -6):
        for slot in range(20):
            page = batch.np_table[0, slot]
            batch.cache.v_scale[page] = 2.0 ** (step * slot)
        _check(batch, q, _attend(batch, q, form=form), form=form, weight=weight)


@FORMS
def test_nan_stays_with_the_queries_that_see_it(form):
    """A NaN among a shared token's values reaches its dimension in every query of the group that sees it, one of a
    sequence's own tokens that sequence alone; one among a query only its head."""
    import torch
    batch = Batch([(384, [5, 9, 30]), (256, [4, 4])], 2, 64, 64)
    c = batch.cache
    q = _q(batch.B, 1, 4, 64)
    clean, _ = _attend(batch, q, form=form)
    c.v[batch.np_table[0, 2], 1, 7, 33] = 0x7F           # a shared token of group 0, KV head 1
    c.v[batch.np_table[2, 6], 0, 3, 5] = 0xFF            # sequence 2's own
    got, lse = _attend(batch, q, form=form)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[:3, 0, 2:, 33] = True
    nan[2, 0, :2, 5] = True
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], clean[~nan]) and not lse.isnan().any()
    # a sequence whose queries do not see the token (it is past them) reads its own table
    lengths = list(batch.lengths)
    batch.lengths[1] = 100
    got, lse = _attend(batch, q, form=form)
    assert torch.equal(got.isnan()[[0, 2, 3, 4]], nan[[0, 2, 3, 4]]) and not got[1].isnan().any()
    batch.lengths = lengths
    q[4, 0, 3, 11] = float("nan")
    got, lse = _attend(batch, q, form=form)
    assert got[4, 0, 3].isnan().all() and lse[4, 0, 3].isnan() and not got[4, 0, :3].isnan().any() and not got[3].isnan().any()
    c.k[batch.np_table[3, 1], 0, 5, 1] = 0x7F            # a shared key of group 1: its scores are NaN for every query
    got, lse = _attend(batch, q, form=form)
    assert got[3:, 0, :2].isnan().all() and not got[3, 0, 2:].isnan().any()
    assert _status() == 0


@FORMS
def test_arguments_out_of_range_are_reported(form):
    """Groups out of order: every sequence reads its own table and is right; a page out of range spoils its sequences alone."""
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(384, [5, 9, 30]), (256, [4, 4])], 2, 64, 64)
    q = _q(batch.B, 1, 4, 64)
    for offsets, shared in (([0, 3, 4], [384, 256]), ([1, 3, 5], [384, 256]), ([0, 0, 5], [384, 256]), ([0, 6, 5], [384, 256]),
                            ([0, -1, 5], [384, 256]), ([0, 3, 5], [-1, 256]), ([0, 5, 3], [384, 256]),
                            ([0, 5, 3, 5], [384, 384, 256]), ([0, 2 ** 31 - 1, 5], [384, 256])):
        got = _attend(batch, q, form=form, offsets=offsets, shared=shared)
        assert _status() == hk.HK_ERR_INVALID_ARG
        _check(batch, q, got, form=form)
    got = _attend(batch, q, form=form, shared=[1 << 30, 2 ** 31 - 1])       # more than there is: what there is
    assert _status() == hk.HK_OK
    good = batch.table.clone()
    for bad in (-1, batch.cache.pages, 2 ** 31 - 1):
        batch.table.copy_(good)
        batch.table[0, 1] = bad
        got = _attend(batch, q, form=form)
        assert _status() == hk.HK_ERR_INVALID_ARG
        _check(batch, q, got, form=form, rows=[3, 4])
    batch.table.copy_(good)
    lengths = list(batch.lengths)
    for bad in (-1, 100000):
        got = _attend(batch, q, form=form, lengths=lengths[:4] + [bad])
        assert _status() == hk.HK_ERR_INVALID_ARG
        _check(batch, q, got, form=form, rows=[0, 1, 2, 3])


@FORMS
def test_repeats_exactly_on_streams_and_in_graphs(form):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(2000, [5, 9, 30, 80]), (256, [4, 4]), (0, [900])], 2, 128, 64)
    q = _q(batch.B, 1, 8, 128)
    a, la = _attend(batch, q, form=form)
    for fill in (0, 0x7F, 0xFF):
        b, lb = _attend(batch, q, form=form, fill=fill)
        assert torch.equal(a, b) and torch.equal(la, lb)
    n, offsets, shared = _i32(batch.lengths), _i32(batch.offsets), _i32(batch.shared)
    same = dict(form=form, lengths=n, offsets=offsets, shared=shared, wait=False)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c, _ = _attend(batch, q, **same)
    stream.synchronize()
    assert torch.equal(a, c)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = _attend(batch, q, **same)
        graphs.append((graph, *got))
    for graph, _, _ in graphs:
        graph.replay()
    for _, d, ld in graphs:
        assert torch.equal(a, d) and torch.equal(la, ld)
    # other lengths and another sharing in the captured call: all of it is read on the device
    n[0] = 1800
    shared[0] = 1000
    graphs[0][0].replay()
    batch.lengths[0] = 1800
    _check(batch, q, graphs[0][1:], form=form)
    assert _status() == hk.HK_OK


@FORMS
def test_two_calls_at_once(form):
    """Calls on two streams, and a GEMM on a third, beside one another."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    jobs = []
    for seed, (groups, H, group, D) in enumerate((([(3000, [50] * 20)], 4, 8, 128), ([(900, [7, 2000, 60]), (1300, [5] * 30)], 2, 4, 64))):
        batch = Batch(groups, H, D, 64, seed=seed)
        q = _q(batch.B, 1, H * group, D)
        same = dict(form=form, lengths=_i32(batch.lengths), offsets=_i32(batch.offsets), shared=_i32(batch.shared), wait=False)
        jobs.append((batch, q, same, _attend(batch, q, form=form)))
    a = torch.randn(2048, 2048, device="cuda").to(torch.bfloat16)
    product = hk.gemm(a, a)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for (batch, q, same, _), stream in zip(jobs, streams):
            with torch.cuda.stream(stream):
                got.append(_attend(batch, q, **same))
        with torch.cuda.stream(streams[2]):
            got.append(hk.gemm(a, a))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        if i % 3 == 2:
            assert torch.equal(x, product)
        else:
            assert torch.equal(x[0], jobs[i % 3][3][0]) and torch.equal(x[1], jobs[i % 3][3][1])
    assert _status() == hk.HK_OK


def test_python_on_streams_and_in_graphs():
    """A size that each form takes by itself."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    for groups, H, group, D in (([(200, [5, 9])], 2, 4, 64), ([(2000, [3] * 64)], 4, 1, 64), ([(6000, [40] * 48)], 8, 8, 128)):
        batch = Batch(groups, H, D, 64)
        q = _q(batch.B, 1, H * group, D)
        args = (q, batch.cache, batch.table, _i32(batch.lengths), _i32(batch.offsets), _i32(batch.shared))
        a, la = hk.attention_kv8_shared(*args, return_lse=True)
        _check(batch, q, (a, la))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        out = torch.empty_like(q)
        c = hk.attention_kv8_shared(*args, stream=stream, out=out)
        stream.synchronize()
        assert c is out and torch.equal(a, c)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d, ld = hk.attention_kv8_shared(*args, return_lse=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, d) and torch.equal(la, ld)
    assert _status() == hk.HK_OK


@FORMS
@pytest.mark.parametrize("D", [64, 128])
def test_an_arrival_that_never_comes_is_reported(form, D):
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(2000, [5, 9, 30, 80]), (256, [4, 4])], 2, D, 64)
    q = _q(batch.B, 1, 8, D)
    for fill in (0, 0x7F, 0xFF):
        _attend(batch, q, form=form, fill=fill, timeout_ns=3_000_000, flags=hk.HK_KV8_FAULT_DROP_ARRIVE)
        assert _status() == hk.HK_ERR_TIMEOUT
        assert _status() == hk.HK_OK
    _check(batch, q, _attend(batch, q, form=form), form=form)


@FORMS
@pytest.mark.parametrize("T,group,dtype", [(40, 8, "bf16"), (63, 16, "bf16"), (40, 8, "fp16"), (341, 3, "bf16")])
def test_many_queries_of_each_sequence(form, T, group, dtype):
    batch = Batch([(1300, [T, T + 9, T + 100]), (500, [T, T + 1])], 2, 64, 32)
    q = _q(batch.B, T, 2 * group, 64, dtype)
    _check(batch, q, _attend(batch, q, form=form), form=form)
    counts = [T, 1, T // 2, 0, T - 1]
    _check(batch, q, _attend(batch, q, counts, form=form), counts, form=form)
    assert _status() == 0


@pytest.mark.parametrize("T,dtype,tokens", [(1, "bf16", 300), (1, "fp16", 300), (128, "bf16", 300), (128, "fp16", 300)])
def test_small_calls_and_many_queries_are_attention_kv8s(T, dtype, tokens):
    """Where reading everything again costs less than joining, and from 1024 rows of a sequence and KV head on."""
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(tokens, [T, T + 9])], 1, 64, 32)
    q = _q(batch.B, T, 8, 64, dtype)
    got = _attend(batch, q)
    _check(batch, q, got)
    o, lse = hk.attention_kv8(q, batch.cache, batch.table, _i32(batch.lengths), return_lse=True)
    assert torch.equal(o, got[0]) and torch.equal(lse, got[1])


@FORMS
def test_cache_beyond_32_bit_offsets(form):
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    small = Batch([(1024, [40, 9, 100])], 8, 128, 128, scales=(0.0625,))
    pages = (1 << 32) // (8 * 128 * 128) + small.cache.pages + 5
    big = hk.Kv8Cache.empty(pages, 8, 128, 128)
    move = pages - small.cache.pages
    for a, b in zip((small.cache.k, small.cache.v, small.cache.k_scale, small.cache.v_scale), (big.k, big.v, big.k_scale, big.v_scale)):
        b[move:] = a
    q = _q(small.B, 1, 64, 128)
    want = _attend(small, q, form=form)
    small.cache, small.table = big, torch.where(small.table >= 0, small.table + move, small.table)
    small.np_table = np.where(small.np_table >= 0, small.np_table + move, small.np_table)
    got = _attend(small, q, form=form)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_refusals():
    import torch
    import dense_bf16_gemm_02_gb300 as hk
    batch = Batch([(384, [5, 9, 30]), (256, [4, 4])], 2, 64, 64)
    q = _q(batch.B, 1, 4, 64)
    n, o, s = _i32(batch.lengths), _i32(batch.offsets), _i32(batch.shared)
    good = dict(q=q, cache=batch.cache, block_table=batch.table, lengths=n, groups=o, shared=s)
    for change in (dict(q=q.float()), dict(q=q[..., :32]), dict(cache=None), dict(block_table=batch.table.long()), dict(lengths=n[:3]),
                   dict(groups=o[:2]), dict(groups=s), dict(shared=s.float()), dict(shared=s[:1]), dict(shared=None), dict(groups=o.cpu()),
                   dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0), dict(out=q.half()), dict(counts=n[:2]),
                   dict(groups=_i32([0]), shared=_i32([])), dict(groups=_i32(list(range(7))), shared=_i32([0] * 6))):
        with pytest.raises((TypeError, ValueError, hk.HKError)):
            hk.attention_kv8_shared(**{**good, **change})
    assert torch.isfinite(hk.attention_kv8_shared(**good)).all()
