"""Router, routed int8 products and the MoE chain's operators run together."""
import os
import sys

import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import moe_layer
    finally:
        sys.path.pop(0)
    return moe_layer


@pytest.mark.parametrize("T,E,topk", [(1, 8, 2), (5, 16, 4), (70, 8, 2), (333, 24, 6)])
def test_chain_stage_by_stage(T, E, topk):
    """Every stage against the 64-bit formula on what the stage before it wrote."""
    H, I, R = 256, 384, T * topk
    g = torch.Generator().manual_seed(T)
    z = torch.randn((T, E), generator=g) * 1.5
    mask = (torch.rand(T, generator=g) > 0.1).to(torch.uint8)
    mask[0] = 1
    x = torch.randn((T, H), generator=g).bfloat16()
    w13, w2 = (torch.randint(-127, 128, s, generator=g).to(torch.int8) for s in ((E, H, 2 * I), (E, I, H)))
    s13, s2 = torch.rand((E, 2 * I), generator=g) * 1e-3, torch.rand((E, H), generator=g) * 1e-3

    def new(*shape, dtype=torch.bfloat16):
        return torch.full(shape, 3, dtype=dtype, device=DEV)

    def ws(n):
        return dict(workspace=new(max(n, 16), dtype=torch.uint8), workspace_bytes=n)
    ids, wt = new(T, topk, dtype=torch.int32), new(T, topk, dtype=torch.float32)
    cnt, loss = new(E + 1, dtype=torch.int32), new(1, dtype=torch.float32)
    w4.w4a16_moe_route(z.to(DEV), T, E, topk, ids, wt, counts=cnt, loss=loss, token_mask=mask.to(DEV),
                       **ws(w4.w4a16_moe_route_workspace_bytes(T, E)))
    off, srt, row_of = (new(n, dtype=torch.int32) for n in (E + 1, R, R))
    w4.w4a16_moe_align(ids, T, topk, E, off, srt, row_of)
    h, a, o, y = new(R, 2 * I), new(R, I), new(R, H), new(T, H)
    xd, k13, k2 = x.to(DEV), ref.pack8(w13).to(DEV), ref.pack8(w2).to(DEV)
    w4.w8a8_grouped_gemm(xd, off, k13, s13.to(DEV), h, E, R, H, 2 * I, sorted_ids=srt, topk=topk,
                         **ws(w4.w8a8_grouped_workspace_bytes(R, H)))
    w4.w4a16_silu_and_mul(h, off[E:], R, I, a)
    w4.w8a8_grouped_gemm(a, off, k2, s2.to(DEV), o, E, R, I, H, **ws(w4.w8a8_grouped_workspace_bytes(R, I)))
    w4.w4a16_moe_sum(o, row_of, wt, T, topk, H, y)

    ri, _, rc, _ = ref.route(z, topk, True, mask)
    assert torch.equal(ids.cpu(), ri) and torch.equal(cnt.cpu(), rc)
    o0 = off.cpu().tolist()
    assert [o0[e + 1] - o0[e] for e in range(E)] == rc[:E].tolist()
    tok = (srt.cpu().long() // topk)
    for e in range(E):
        rows = slice(o0[e], o0[e + 1])
        if o0[e + 1] > o0[e]:
            for got, src, w, s in ((h[rows], x[tok[rows]], w13[e], s13[e]), (o[rows], a[rows].cpu(), w2[e], s2[e])):
                q, sx = ref.quantize(src)
                want, part = ref.gemm(q, sx, w, s)
                assert bool(((got.cpu().double() - want).abs() <= ref.gemm_bound(want, part, torch.bfloat16)).all())
    assert bool((h[o0[E]:] == 3).all()) and bool((o[o0[E]:] == 3).all())
    rr = row_of.cpu().view(T, topk)
    want = (torch.where((rr >= 0)[..., None], o.cpu()[rr.long().clamp(min=0)].double(), torch.zeros(())) *
            wt.cpu().double()[..., None])
    # topk fused multiply-adds in fp32, then one rounding
    bound = want.abs().sum(1) * (topk + 1) * ref.U32 + want.sum(1).abs() * ref.half_step(torch.bfloat16) + 2.0 ** -133
    assert bool(((y.cpu().double() - want.sum(1)).abs() <= bound * (1 + 2.0 ** -8)).all())
    assert bool((y[mask.to(DEV) == 0] == 0).all())


def test_example():
    """The layer against 64 bits without activation quantization, and the router's gradient.

    A code is off by s / sqrt 12 in the mean square (uniform within a step), so quantizing rows costs
    sqrt(mean s^2 / 12) / rms in relative 2-norm, here taken from the data: of x for the first
    products, of a for the second ones.  bf16 rounds h, a, o and y by 2^-8 / sqrt 3 each at most.  As
    independent errors, with a factor 2 for the activation's slope and the gated product's two
    factors.  The gradient sees fp32 products of `hidden` and `tokens` terms and the bf16 outputs
    as they are: (2 sqrt(terms) + 16) half steps of fp32, against cancellation by a factor of 32."""
    moe_layer = example()
    out = moe_layer.main(hidden=256, width=384, experts=16, topk=4, tokens=64, check_tokens=48)
    layer = moe_layer.MoeLayer(256, 384, 16, 4)
    x = torch.randn((48, 256), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).bfloat16()
    _, r = layer.forward(x)

    def cost(v):
        v = v.double()
        return float(((v.abs().amax(1) / 127) ** 2 / 12).mean().sqrt() / v.pow(2).mean().sqrt())
    n = int(r["routed"][0])
    assert out["layer"] <= 2 * (cost(x) ** 2 + cost(r["a"][:n]) ** 2 + 4 * (2.0 ** -8) ** 2 / 3) ** 0.5
    assert out["gradient"] <= 32 * (2 * 256 ** 0.5 + 16) * ref.U32
    assert 0.9 < out["balance_loss"] < 16


@pytest.mark.parametrize("T", [1, 3, 130])
def test_example_layer_takes_any_token_count(T):
    moe_layer = example()
    layer = moe_layer.MoeLayer(256, 128, 8, 2)
    x = torch.randn((T, 256), device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).bfloat16()
    y, r = layer.forward(x)
    # Row by row, so that no row is lost or misplaced: a row's largest value is at most sqrt(K) times its
    # rms, so quantizing costs sqrt(K) / (127 sqrt 12) at most: 0.036 (x), 0.026 (a); with bf16's four
    # roundings and the factor 2 of the test above 0.09 in the mean square, 0.15 for any row
    want = layer.reference(x, r)
    assert float(((y.double() - want).norm(dim=1) / want.norm(dim=1)).max()) < 0.15
    grad = layer.router_gradient(x, r)
    assert moe_layer.relative(grad, layer.reference_gradient(x, r)) <= 32 * (2 * 256 ** 0.5 + 16) * ref.U32


def test_two_graphs_and_two_streams():
    """Two captured calls with workspaces of their own replayed at once on two streams; each gives what
    it gives alone."""
    K, N = 1024, 2048
    g = torch.Generator().manual_seed(9)
    w = torch.randint(-127, 128, (1, K, N), generator=g).to(torch.int8)
    packed, sw = ref.pack8(w).to(DEV), (torch.rand(N, generator=g) * 1e-3).to(DEV)
    calls = []
    for M in (3, 60, 200):
        x = torch.randn((M, K), generator=g).bfloat16().to(DEV)
        nb = w4.w8a8_workspace_bytes(M, K)
        ws, y = torch.empty(nb, dtype=torch.uint8, device=DEV), torch.empty((M, N), dtype=torch.bfloat16, device=DEV)

        def run(M=M, x=x, nb=nb, ws=ws, y=y):
            w4.w8a8_gemm(x, packed, sw, y, M, K, N, workspace=ws, workspace_bytes=nb)
        run()
        torch.cuda.synchronize()
        want, graph, side = y.clone(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            run()
        calls.append((graph, side, y, want, run))      # (run keeps x and the workspace alive)
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, side, y, _, _ in calls:
            with torch.cuda.stream(side):
                y.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for _, _, y, want, _ in calls:
            assert torch.equal(y, want)
