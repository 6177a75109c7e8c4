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
