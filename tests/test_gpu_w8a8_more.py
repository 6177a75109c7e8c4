"""8-bit products on the GPU: calls that the sizes and strides of the other files leave out."""
import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4
from test_gpu_w8a8 import check_gemm, dev, packed, problem, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = ref.F16, ref.BF16


def test_two_entries_per_token_past_32_bits():
    """Codes of the tokens pass 2^32 bytes, every token goes to two experts or one: the rows that the
    experts hold, and the last rows of y, which no expert holds, as they were."""
    K, N, E, X, topk, dt = 130944, 64, 3, 32850, 2, BF16
    assert X * K > 1 << 32
    _, w, sw, _ = problem(1, K, N, dt, E=E)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((X, K), dtype=torch.bfloat16, device=DEV, generator=g)
    ids = torch.stack((torch.randint(0, 2, (X,), device=DEV, generator=g), torch.full((X,), 2, device=DEV)), 1)
    ids[torch.rand((X, topk), device=DEV, generator=g) < 0.1] = -1
    R = X * topk
    off, srt, row_of = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E + 1, R, R))
    w4.w4a16_moe_align(ids.to(torch.int32), X, topk, E, off, srt, row_of)
    nb = w4.w8a8_grouped_workspace_bytes(R, K)
    y = torch.full((R, N), 9.0, dtype=torch.bfloat16, device=DEV)
    w4.w8a8_grouped_gemm(x, off, packed(w), dev(sw), y, E, R, K, N, sorted_ids=srt, topk=topk, dt=dt,
                         workspace=torch.empty(nb, dtype=torch.uint8, device=DEV), workspace_bytes=nb)
    o = off.cpu().tolist()
    assert 0 < o[E] < R and bool((y[o[E]:] == 9.0).all())
    for e in range(E):
        for a, b in ((o[e], o[e] + 3), (o[e + 1] - 20, o[e + 1])):
            check_gemm(y[a:b], x[srt[a:b].long() // topk].cpu(), w[e], sw[e], None)


def test_one_workspace_for_all_row_counts():
    """A workspace for up to 1100 rows serves every call, whose results are those of a workspace of its own."""
    K, N, dt = 2048, 192, BF16
    x, w, sw, b = problem(1100, K, N, dt, bias=True)
    xd, wp, swd, bd = dev(x), packed(w), dev(sw), dev(b)
    nb = w4.w8a8_max_workspace_bytes(1100, K)
    ws = workspace(nb)
    for M in (1100, 1, 16, 70, 300, 1024, 1025):
        y = torch.full((M, N), 9.0, dtype=x.dtype, device=DEV)
        w4.w8a8_gemm(xd, wp, swd, y, M, K, N, bias=bd, dt=dt, workspace=ws, workspace_bytes=nb)
        check_gemm(y, x[:M], w[0], sw[0], b)


@pytest.fixture
def config():
    yield w4.w4a16_test_w8a8_config
    w4.w4a16_test_w8a8_config(-1)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("kernel", [3, 4, 5, 6, 7])
@pytest.mark.parametrize("M,slices", [(33, 4), (300, 2), (700, 8)])
def test_slices_between_gaps(config, M, slices, kernel, dt):
    """Products cut into slices of K whose rows of x and y lie in wider buffers: what lies between stays."""
    K, N = 2048, 192
    x, w, sw, b = problem(M, K, N, dt, seed=7, bias=True)
    wide = torch.full((M, K + 24), float("nan"), dtype=x.dtype)
    wide[:, :K] = x
    config(kernel + 100 * slices)
    assert w4.w4a16_test_w8a8_plan(M, K, N, 0) == kernel + 100 * slices
    y = torch.full((M, N + 40), 9.0, dtype=x.dtype, device=DEV)
    nb = w4.w8a8_workspace_bytes(M, K)
    w4.w8a8_gemm(dev(wide), packed(w), dev(sw), y, M, K, N, bias=dev(b), dt=dt, ldx=K + 24, ldy=N + 40,
                 workspace=workspace(nb), workspace_bytes=nb)
    check_gemm(y[:, :N], x, w[0], sw[0], b)
    assert bool((y[:, N:] == 9.0).all())


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,topk,E", [(6, 4, 16), (150, 2, 6)])
def test_grouped_call_in_a_graph(T, topk, E, gather):
    """Captured, then replayed on other tokens and another routing, with eager work between the replays."""
    K, N, R, dt = 256, 192, T * topk, BF16
    _, w, sw, _ = problem(1, K, N, dt, E=E)
    wp, swd, nb = packed(w), dev(sw), w4.w8a8_grouped_workspace_bytes(R, K)
    g = torch.Generator().manual_seed(T)

    def routing():
        ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(T)])
        ids[torch.rand((T, topk), generator=g) < 0.1] = -1
        off, srt, row_of = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E + 1, R, R))
        w4.w4a16_moe_align(ids.to(torch.int32).to(DEV), T, topk, E, off, srt, row_of)
        return torch.randn((T if gather else R, K), generator=g).to(torch.bfloat16).to(DEV), off, srt

    def call(x, off, srt, y, ws):
        w4.w8a8_grouped_gemm(x, off, wp, swd, y, E, R, K, N, sorted_ids=srt if gather else None, topk=topk, dt=dt,
                             workspace=ws, workspace_bytes=nb)
    inputs = [routing() for _ in range(3)]
    want = []
    for v in inputs:
        want.append(torch.full((R, N), 9.0, dtype=torch.bfloat16, device=DEV))
        call(*v, want[-1], workspace(nb))
        for e in range(E):
            a, b = int(v[1][e]), int(v[1][e + 1])
            rows = v[0][v[2][a:b].long() // topk] if gather else v[0][a:b]
            if b > a:
                check_gemm(want[-1][a:b], rows.cpu(), w[e], sw[e], None)
    static, y, ws = [t.clone() for t in inputs[0]], torch.zeros_like(want[0]), workspace(nb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*static, y, ws)
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1, 0):
        for s, t in zip(static, inputs[i]):
            s.copy_(t)
        y.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        other = torch.full_like(y, 9.0)
        call(*inputs[2 - i], other, workspace(nb))
        assert torch.equal(other, want[2 - i])
