"""The feed-forward example runs the operators together as a block would."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_ffn_block_example():
    """Decode, prompt and gradient of a small block against 64 bits.  Each bf16
    rounding on the way (a, y; da, dh, W twice, dx) has a relative 2-norm error of
    at most 2^-8 / sqrt 3 = 0.0023; two in the forward pass, six in the backward
    pass, as independent errors, and a factor 1.5 for the activation's slope."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import ffn_block
        out = ffn_block.main(hidden=512, width=1408, tokens=256)
    finally:
        sys.path.pop(0)
    assert out["decode"] <= 1.5 * 2 ** 0.5 * 0.0023
    assert out["prompt"] <= 1.5 * 2 ** 0.5 * 0.0023
    assert out["gradient"] <= 1.5 * 6 ** 0.5 * 0.0023
