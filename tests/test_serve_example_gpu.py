"""The serving example runs its four operators together: a ragged prefill and
captured decoding steps, against the same block in fp32.

What this test is for is how the operators are put together (the split views of
the fused projection, positions, counts, the captured step); how exact each of
them is, the tests of each say. The bound: a rounding to the format leaves a
relative error e in Gaussian data (0.095 NVFP4, 0.115 MXFP4). A product of two
rounded operands is off by sqrt(2) e, so q, k and v are. Scores of unit variance
carry the errors of q and k (4 e^2) into the softmax weights, v adds 2 e^2, the
output product 2 e^2, and the 8-bit cache its keys' and values' 2 * 2^-8. A tenth is
left for the roundings to bf16 and for terms of higher order. A mask that is off by
one token leaves the block without any rounding 0.39 (one too many) or 0.51 (one too
few) away, heads, positions or k and v mixed up 0.9 and more."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("format,e", [("nvfp4", 0.0952), ("mxfp4", 0.1150)])
@pytest.mark.parametrize("batch,prompt,heads,kv_heads", [(3, 70, 8, 2), (1, 300, 4, 4)])
def test_serve_example(format, e, batch, prompt, heads, kv_heads):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_low_precision.py")
    spec = importlib.util.spec_from_file_location("serve_low_precision", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    error = example.run(hidden=512, heads=heads, kv_heads=kv_heads, head_dim=64, batch=batch, prompt=prompt, steps=20,
                        format=format, verbose=False)
    assert 0 < error < 1.1 * math.sqrt(8 * e * e + 2 * 2.0 ** -8)
