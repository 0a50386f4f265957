"""The MXFP4 block example at a small size: every new entry point together, eager and from a graph."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt", [5, 70])
def test_block_agrees_with_its_plain_form(prompt):
    print(f"example block, prompt of {prompt}", flush=True)
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import mxfp4_moe_block as ex
    pre, dec, _ = ex.run(hidden=512, inner=256, experts=4, topk=2, prompt=prompt, tokens=4)
    # BF16 roundings of relative size 2^-9 rms at most: of h (shared), of the logits (2^-9 of up to 8 moves a
    # softmax weight by 2 %, and the experts are about a tenth of y), of the inner product and of y
    assert pre < 0.01 and dec < 0.01
