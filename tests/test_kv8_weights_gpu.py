"""Small softmax weights of the cache attention's few-row kernels.

One token takes most of the weight and tens of thousands share the rest, each with a
weight far below f16's normal numbers (2^-14) when the largest is 1. The first
token's value is 0, so the output is the tail's share alone. Tolerance, relative: each
weight is held to 11 bits (2^-11 of it); scores and exponentials in fp32 add 2^-16 (scores up to
2^5 in units of log2, 2^-19 absolute each); the sums of up to n tokens, split over
many warps, at most 2^-12; the output's own rounding is half a step."""
from __future__ import annotations

import math

import numpy as np
import pytest

from test_kv8_gpu import _i32, _status, hk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,width", [(3000, 3000), (40000, 40000), (40000, 400000)])
@pytest.mark.parametrize("low", [13.3, 15.6, 17.7, 20.4, 24.9, 26.3, 28.2])
def test_a_tail_of_small_weights_keeps_its_mass(hk, D, n, width, low):  # noqa: F811
    """The tail's weights are 2^-low of the first token's; a short table, a long one, a wide one."""
    import torch
    page, group = 64, 4
    pages = -(-n // page)
    cache = hk.Kv8Cache.empty(pages, 1, D, page)
    k = torch.zeros(1, n, 1, D, device="cuda")
    k[0, 0, 0, 0] = 1.0
    v = torch.ones(1, n, 1, D, device="cuda")
    v[0, 0] = 0
    table = torch.full((1, -(-width // page)), -1, dtype=torch.int32, device="cuda")
    table[0, :pages] = torch.arange(pages, device="cuda")
    hk.kv8_append(cache, k, v, table, _i32([0]))
    for dtype, half in ((torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -8)):
        q = torch.zeros(1, 1, group, D, dtype=dtype, device="cuda")
        q[..., 0] = 1
        scale = float(np.float32(low * math.log(2)))
        o, lse = hk.attention_kv8(q, cache, table, _i32([n]), scale=scale, return_lse=True)
        assert _status(hk) == hk.HK_OK
        tail = (n - 1) * math.exp(-scale)
        want = tail / (1 + tail)
        off = (o.double() / want - 1).abs().max().item()
        assert off <= half + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -16, (off, want)
        assert (lse.double() - (scale + math.log1p(tail))).abs().max().item() <= 2.0 ** -16 * max(1, scale)
