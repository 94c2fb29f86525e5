"""The shared-prompt example runs the operators of a forked batch together: fork, growth (and beams' reordering) in a
captured step, head norm and rotation, append, attention over the shared prompt, ending rows and compaction,
against the same block in fp32.

The bound. E4M3 rounds a key's or a value's elements by at most 2^-4 of each, 2^-4 / sqrt(3) in the root mean square
over a uniform mantissa's steps at most; keys' errors reach the scores (of unit variance: two normed rows) and so the
weights by as much again, values' the output. So the update is off by less than 2^-4 sqrt(2 / 3) = 0.051 of itself, and
the roundings to bf16 (activations, projections, queries, weights, output: ten of them, 2^-8 at most each) add less than
sqrt(10) 2^-8 = 0.013. A row that reads another row's tokens, a page copied late or a position off by one leaves the
block without any rounding more than 0.3 away."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beams", [False, True])
@pytest.mark.parametrize("answers,prompt,heads,kv_heads,head_dim,page_size", [(4, 150, 8, 2, 64, 16), (10, 700, 8, 2, 128, 64),
                                                                            (3, 37, 4, 4, 64, 32)])
def test_shared_prompt_example(answers, prompt, heads, kv_heads, head_dim, page_size, beams):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_shared_prompt.py")
    spec = importlib.util.spec_from_file_location("serve_shared_prompt", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    error = example.run(hidden=512, heads=heads, kv_heads=kv_heads, head_dim=head_dim, answers=answers, prompt=prompt, steps=20,
                        beams=beams, page_size=page_size, verbose=False)
    assert 0 < error < 0.064
