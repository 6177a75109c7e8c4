"""A mixture-of-experts layer with int8 experts: routing with its balance loss, the
experts' products on the tokens' 8-bit codes, a shared expert beside them, and the
router's training step.

    y = sum_k w_k expert_k(x) + shared(x),   expert(x) = (silu(x . Wg) * (x . Wu)) . Wd

    python examples/moe_layer.py [--hidden 2048 --width 1408 --experts 64 --topk 8 --tokens 512]

The weights are random int8 codes with one fp32 scale per column, prepacked once; the
router's weights are fp32 and its logits one torch product.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import weight_only_quantized_amd as w4  # noqa: E402


class Int8:
    """E matrices [K][N] of int8 codes with fp32 column scales, prepacked (the plain codes are
    kept for checking only)."""

    def __init__(self, E, K, N, gen):
        self.codes = (torch.randn((E, K, N), device=gen.device, generator=gen) * 36).round().clamp(-127, 127).to(torch.int8)
        self.scale = (torch.rand((E, N), device=gen.device, generator=gen) + 0.5) / (36 * K ** 0.5)
        self.packed = torch.empty(w4.w8a16_prepacked_bytes(E, K, N), device=gen.device, dtype=torch.uint8)
        w4.w8a16_prepack(self.codes, self.packed, E, K, N, 1)
        self.E, self.K, self.N = E, K, N

    def dense(self, e):
        return self.codes[e].double() * self.scale[e].double()


class MoeLayer:
    def __init__(self, hidden, width, experts, topk, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.width, self.experts, self.topk, self.device = hidden, width, experts, topk, device
        self.gate = torch.randn((hidden, experts), device=device, generator=gen) / hidden ** 0.5
        self.w13, self.w2 = Int8(experts, hidden, 2 * width, gen), Int8(experts, width, hidden, gen)
        self.shared13, self.shared2 = Int8(1, hidden, 2 * width, gen), Int8(1, width, hidden, gen)

    def new(self, *shape, dtype=torch.bfloat16):
        return torch.empty(shape, device=self.device, dtype=dtype)

    def workspace(self, nbytes):
        return dict(workspace=self.new(nbytes, dtype=torch.uint8), workspace_bytes=nbytes)

    def route(self, x):
        """Experts and weights of the tokens, per-expert counts and the balance loss."""
        T, E = x.shape[0], self.experts
        r = {"logits": x.float() @ self.gate, "ids": self.new(T, self.topk, dtype=torch.int32),
             "w": self.new(T, self.topk, dtype=torch.float32), "counts": self.new(E + 1, dtype=torch.int32),
             "loss": self.new(1, dtype=torch.float32)}
        w4.w4a16_moe_route(r["logits"], T, E, self.topk, r["ids"], r["w"], counts=r["counts"], loss=r["loss"],
                           **self.workspace(w4.w4a16_moe_route_workspace_bytes(T, E)))
        return r

    def forward(self, x):
        """y, and the intermediates for the router's backward pass."""
        T, E, H, I = x.shape[0], self.experts, self.hidden, self.width
        R = T * self.topk
        r = self.route(x)
        off, srt, row_of = (self.new(n, dtype=torch.int32) for n in (E + 1, R, R))
        w4.w4a16_moe_align(r["ids"], T, self.topk, E, off, srt, row_of)
        ws = self.workspace(w4.w8a8_grouped_workspace_bytes(R, max(H, I)))
        h, a, o, y = self.new(R, 2 * I), self.new(R, I), self.new(R, H), self.new(T, H)
        w4.w8a8_grouped_gemm(x, off, self.w13.packed, self.w13.scale, h, E, R, H, 2 * I, sorted_ids=srt, topk=self.topk, **ws)
        w4.w4a16_silu_and_mul(h, off[E:], R, I, a)
        w4.w8a8_grouped_gemm(a, off, self.w2.packed, self.w2.scale, o, E, R, I, H, **ws)
        w4.w4a16_moe_sum(o, row_of, r["w"], T, self.topk, H, y)
        # the shared expert
        ws = self.workspace(w4.w8a8_workspace_bytes(T, max(H, I)))
        hs, as_, ys = self.new(T, 2 * I), self.new(T, I), self.new(T, H)
        w4.w8a8_gemm(x, self.shared13.packed, self.shared13.scale, hs, T, H, 2 * I, **ws)
        w4.w4a16_silu_and_mul(hs, None, T, I, as_)
        w4.w8a8_gemm(as_, self.shared2.packed, self.shared2.scale, ys, T, I, H, **ws)
        r.update(x=x, o=o, row_of=row_of, a=a, routed=off[E:])
        return y + ys, r

    def router_gradient(self, dy, r, balance=0.01):
        """Gradient of the router's weights for the output gradient dy plus the balance loss."""
        T = dy.shape[0]
        picked = r["o"][r["row_of"].long().clamp(min=0)].view(T, self.topk, self.hidden)
        dw = torch.bmm(picked.float(), dy.float()[..., None])[..., 0].contiguous()
        dlogits = torch.empty_like(r["logits"])
        w4.w4a16_moe_route_backward(r["logits"], r["ids"], r["w"], dlogits, T, self.experts, self.topk,
                                    counts=r["counts"], dtopk_w=dw, dloss=torch.full((1,), balance, device=self.device))
        return r["x"].float().t() @ dlogits

    # ---- checks in 64 bits -------------------------------------------------------

    def reference(self, x, r):
        """The layer without activation quantization, for the experts that the router chose."""
        x = x.double()

        def expert(w13, w2, e, rows):
            g, u = (rows @ w13.dense(e)).chunk(2, 1)
            return (g * torch.sigmoid(g) * u) @ w2.dense(e)
        y = expert(self.shared13, self.shared2, 0, x)
        for e in range(self.experts):
            t, k = torch.where(r["ids"] == e)
            if len(t):
                y.index_add_(0, t, expert(self.w13, self.w2, e, x[t]) * r["w"][t, k].double()[:, None])
        return y

    def reference_gradient(self, dy, r, balance=0.01):
        gate = self.gate.double().requires_grad_()
        T, E = dy.shape[0], self.experts
        p = torch.softmax(r["x"].double() @ gate, 1)
        w = p.gather(1, r["ids"].long())
        w = w / w.sum(1, keepdim=True)
        picked = r["o"][r["row_of"].long()].view(T, self.topk, self.hidden).double()
        c = r["counts"][:E].double()
        loss = E * (c / c.sum() * p.mean(0)).sum()
        total = (w[..., None] * picked * dy.double()[:, None]).sum() + balance * loss
        return torch.autograd.grad(total, gate)[0]


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def main(hidden=2048, width=1408, experts=64, topk=8, tokens=512, check_tokens=64):
    layer = MoeLayer(hidden, width, experts, topk)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((check_tokens, hidden), device="cuda", generator=gen).bfloat16()
    y, r = layer.forward(x)
    out = {"balance_loss": float(r["loss"]), "layer": relative(y, layer.reference(x, r))}
    dy = torch.randn((check_tokens, hidden), device="cuda", generator=gen).bfloat16()
    out["gradient"] = relative(layer.router_gradient(dy, r), layer.reference_gradient(dy, r))
    for name, rows in (("decode_us", 4), ("prompt_us", tokens)):
        xs = torch.randn((rows, hidden), device="cuda", generator=gen).bfloat16()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for i in range(13):
            if i == 3:
                begin.record()
            layer.forward(xs)
        end.record()
        torch.cuda.synchronize()
        out[name] = begin.elapsed_time(end) * 100.0
    for k, v in out.items():
        print(f"{k:12s} {v:.4g}")
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for flag, default in (("hidden", 2048), ("width", 1408), ("experts", 64), ("topk", 8), ("tokens", 512)):
        ap.add_argument("--" + flag, type=int, default=default)
    main(**vars(ap.parse_args()))
