"""tcgen05.commit tracks what the executing thread issued, and which lane elect.sync
picks is not specified: in the 4-bit products all of a warp's MMAs, scale copies and commits
stand under elect_one()."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_bf16_gemm_02_gb300", "csrc",
                      "fp4_gemm.cuh")


def _guards(text, at):
    """The statement that holds position `at`, and the headers of the blocks around it."""
    heads = [text[max(text.rfind(c, 0, at) for c in ";{}") + 1:at]]
    depth = 0
    for i in range(at - 1, -1, -1):
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth:
                depth -= 1
            else:
                heads.append(text[max(text.rfind(c, 0, i) for c in ";{}") + 1:i])
    return heads


@pytest.mark.parametrize("call", ["mma_commit_one(", "mma_commit_pair_mask(", "mma_fp4<", "tmem_cp_128x16b(", "tmem_cp_128x16b_pair("])
def test_every_tensor_core_operation_is_issued_by_the_elected_lane(call):
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    text = text[text.index("gemm_fp4_single_kernel("):]
    places = [m.start() for m in re.finditer(re.escape(call), text)]
    assert places
    for at in places:
        assert any("elect_one()" in g for g in _guards(text, at)), text[at - 80:at + 40]
