"""A W4A16 feed-forward block with the fused linear operators: decoding, a prompt
and a training step through frozen int4 weights.

    y = x + (silu(x . Wg) * (x . Wu)) . Wd

    python examples/ffn_block.py [--hidden 4096 --width 14336 --tokens 2048]

The weights are random int4 codes with bf16 scales (group 128) and zero points,
prepacked once; every step below is one call of the library.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import weight_only_quantized_amd as w4  # noqa: E402


def quantized(K, N, gen):
    """Random weights W [K][N] in the library's plain form and prepacked; the
    plain tensors are kept for checking only."""
    dev = gen.device
    w = torch.randint(0, 256, (K, N // 2), device=dev, dtype=torch.uint8, generator=gen)
    zero = torch.randint(6, 10, (K // 128, N), device=dev, dtype=torch.uint8, generator=gen)
    zero = zero[:, 0::2] | (zero[:, 1::2] << 4)
    scale = ((torch.rand((K // 128, N), device=dev, generator=gen) + 0.5) / (4.6 * K ** 0.5)).bfloat16()
    packed = torch.empty(w4.w4a16_prepacked_bytes(1, K, N), device=dev, dtype=torch.uint8)
    w4.w4a16_prepack(w, packed, 1, K, N, 0)
    return w4.linear(K, N, packed, scale, zero), (w, scale, zero)


def dequantized(plain):
    """W in 64 bits (for checking)."""
    w, scale, zero = plain
    q = torch.stack((w & 15, w >> 4), -1).flatten(1).double()
    z = torch.stack((zero & 15, zero >> 4), -1).flatten(1).double()
    return (q - z.repeat_interleave(128, 0)) * scale.double().repeat_interleave(128, 0)


class FeedForward:
    """The block's weights and one workspace for all of its calls of up to max_tokens rows."""

    def __init__(self, hidden, width, max_tokens, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.width, self.device = hidden, width, device
        self.w13, self.plain13 = quantized(hidden, 2 * width, gen)
        self.w2, self.plain2 = quantized(width, hidden, gen)
        # (a size is not monotonic in the row count, since fewer rows may be cut into more
        # slices: the largest of all counts up to max_tokens)
        self.ws_bytes = max(q(lin, m) for m in range(1, max_tokens + 1) for lin, qs in (
            (self.w13, (w4.w4a16_glu_gemm_workspace_bytes, w4.w4a16_glu_gemm_backward_workspace_bytes)),
            (self.w2, (w4.w4a16_gemm_ep_workspace_bytes, w4.w4a16_gemm_ep_backward_workspace_bytes))) for q in qs)
        self.ws = torch.empty(max(self.ws_bytes, 16), device=device, dtype=torch.uint8)

    def new(self, rows, cols):
        return torch.empty((rows, cols), device=self.device, dtype=torch.bfloat16)

    def forward(self, x, save=False):
        """y, and what backward needs when `save` is set."""
        M = x.shape[0]
        h = self.new(M, 2 * self.width) if save else None
        a, y = self.new(M, self.width), self.new(M, self.hidden)
        ws = dict(workspace=self.ws, workspace_bytes=self.ws_bytes)
        w4.w4a16_glu_gemm(x, self.w13, a, M, w4.W4A16_ACT_SILU, h, **ws)
        w4.w4a16_gemm_ep(a, self.w2, y, M, w4.W4A16_ACT_NONE, residual=x, **ws)
        return y, h

    def backward(self, dy, h):
        """dx of the whole block; h is overwritten with its gradient."""
        M = dy.shape[0]
        da, dx = self.new(M, self.width), self.new(M, self.hidden)
        ws = dict(workspace=self.ws, workspace_bytes=self.ws_bytes)
        w4.w4a16_gemm_ep_backward(dy, None, self.w2, da, M, w4.W4A16_ACT_NONE, **ws)
        w4.w4a16_glu_gemm_backward(da, h, self.w13, dx, M, w4.W4A16_ACT_SILU, dh=h, addend=dy, **ws)
        return dx

    def reference(self, x):
        """The block in 64 bits, differentiable."""
        g, u = (x @ dequantized(self.plain13)).chunk(2, 1)
        return x + (g * torch.sigmoid(g) * u) @ dequantized(self.plain2)


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def main(hidden=4096, width=14336, tokens=2048, check_tokens=64):
    block = FeedForward(hidden, width, tokens)
    gen = torch.Generator(device="cuda").manual_seed(1)
    out = {}
    # decode: a few tokens, one at a time, against the 64-bit block
    x = torch.randn((check_tokens, hidden), device="cuda", generator=gen).bfloat16()
    want = block.reference(x.double())
    step = torch.cat([block.forward(x[i:i + 1])[0] for i in range(4)])
    out["decode"] = relative(step, want[:4])
    # prompt and training step: the same rows at once, then the gradient
    y, h = block.forward(x, save=True)
    out["prompt"] = relative(y, want)
    dy = torch.randn((check_tokens, hidden), device="cuda", generator=gen).bfloat16()
    dx = block.backward(dy, h)
    xr = x.double().requires_grad_()
    block.reference(xr).backward(dy.double())
    out["gradient"] = relative(dx, xr.grad)
    # time of a decode step and of a training step
    for name, rows, train in (("decode_us", 1, False), ("train_us", tokens, True)):
        xs = torch.randn((rows, hidden), device="cuda", generator=gen).bfloat16()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for i in range(13):
            if i == 3:
                begin.record()
            ys, hs = block.forward(xs, save=train)
            if train:
                block.backward(xs, hs)
        end.record()
        torch.cuda.synchronize()
        out[name] = begin.elapsed_time(end) * 100.0
    for k, v in out.items():
        print(f"{k:10s} {v:.4g}")
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for flag, default in (("hidden", 4096), ("width", 14336), ("tokens", 2048)):
        ap.add_argument("--" + flag, type=int, default=default)
    main(**vars(ap.parse_args()))
