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


def test_ffn_block_takes_any_row_count():
    """Ragged row counts share the block's workspace, forward and backward; the bounds
    of the test above."""
    import torch
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import ffn_block
    finally:
        sys.path.pop(0)
    block = ffn_block.FeedForward(512, 1408, 256)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for rows in (3, 77, 129, 255):
        x, dy = (torch.randn((rows, 512), device="cuda", generator=gen).bfloat16() for _ in range(2))
        y, h = block.forward(x, save=True)
        dx = block.backward(dy, h)
        xr = x.double().requires_grad_()
        want = block.reference(xr)
        want.backward(dy.double())
        assert ffn_block.relative(y, want.detach()) <= 1.5 * 2 ** 0.5 * 0.0023
        assert ffn_block.relative(dx, xr.grad) <= 1.5 * 6 ** 0.5 * 0.0023
