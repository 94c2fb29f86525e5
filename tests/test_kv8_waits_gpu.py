"""Bounded waits of the cache attention that run out: every form gives up, reports it
and leaves the context usable, whatever the workspace held before."""
from __future__ import annotations

import numpy as np
import pytest

from test_kv8_forms_gpu import FEW, MANY, _assert, _attend
from test_kv8_gpu import _filled, _status, _tokens, hk  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

# form, sequences, heads, queries, tokens, table's pages: many rows; blocks of 8, 4, 2 and 1 warps, a cluster, tiles spread
# over the GPU
CASES = [(MANY, 2, 2, 40, 300, 0), (FEW, 19, 8, 1, 150, 0), (FEW, 38, 8, 1, 150, 0), (FEW, 50, 8, 2, 150, 0),
         (FEW, 100, 8, 1, 150, 0), (FEW, 1, 1, 1, 9000, 0), (FEW, 3, 2, 9, 5000, 2100)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", CASES, ids=["many", "block8", "block4", "block2", "block1", "cluster", "spread"])
def test_an_arrival_that_never_comes_is_reported(hk, D, case):  # noqa: F811
    import torch
    form, B, H, T, n, wide = case
    rng = np.random.default_rng(B)
    lengths = [n] * B
    cache, table = _filled(hk, rng, lengths, H, D, 64)
    if wide:
        w = np.full((B, wide), -1, dtype=np.int32)
        w[:, : table[0].shape[1]] = table[0]
        table = (w, torch.from_numpy(w).cuda())
    q = _tokens(rng, B, T, H * 4, D, torch.bfloat16, 1)
    for fill in (0, 0x7F, 0xFF):
        _attend(hk, form, q, cache, table[1], lengths, fill=fill, timeout_ns=3_000_000, flags=hk.HK_KV8_FAULT_DROP_ARRIVE)
        assert _status(hk) == hk.HK_ERR_TIMEOUT
        assert _status(hk) == hk.HK_OK
    _assert(hk, form, q, cache, table, lengths)
