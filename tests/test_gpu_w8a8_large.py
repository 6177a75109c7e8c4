"""8-bit products and the router where offsets pass 32 bits."""
import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4
from test_gpu_route import run, run_bwd
from test_gpu_w8a8 import check_gemm, dev, packed, problem, run_gemm, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = ref.BF16


@pytest.mark.parametrize("X", [32799, 32850])
def test_gathered_rows_on_either_side_of_32_bits(X):
    """Codes of X tokens take just under and just over 2^32 bytes."""
    K, N, E = 130944, 64, 2
    assert (X * K < 2 ** 32) == (X == 32799)
    _, w, sw, _ = problem(1, K, N, BF16, E=E)
    g = torch.Generator(device=DEV).manual_seed(X)
    x = torch.randn((X, K), dtype=torch.bfloat16, device=DEV, generator=g)
    srt = torch.randperm(X, device=DEV, generator=g).to(torch.int32)
    half = X // 2 + 5
    off = torch.tensor([0, half, X], dtype=torch.int32, device=DEV)
    nb = w4.w8a8_grouped_workspace_bytes(X, K)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    y = torch.full((X, N), 9.0, dtype=torch.bfloat16, device=DEV)
    w4.w8a8_grouped_gemm(x, off, packed(w), dev(sw), y, E, X, K, N, sorted_ids=srt, topk=1, dt=BF16, workspace=ws,
                         workspace_bytes=nb)
    # the rows of the last tokens, the first, and some in between
    at = torch.empty(X, dtype=torch.int64, device=DEV)
    at[srt.long()] = torch.arange(X, device=DEV)
    rows = at[torch.cat((torch.arange(X - 20, X), torch.arange(4), torch.arange(16380, 16410))).to(DEV)]
    for e in range(E):
        r = rows[(rows < half) if e == 0 else (rows >= half)]
        check_gemm(y[r], x[srt[r].long()].cpu(), w[e], sw[e], None)


def test_rows_of_y_behind_two_to_the_31():
    M, K, N = 40000, 128, 57344
    x, w, sw, _ = problem(M, K, N, BF16)
    assert M * N > 2 ** 31
    wp, swd = packed(w), dev(sw[0])
    y = run_gemm(dev(x), wp, swd, None, N, BF16)
    for a in (0, 37440, M - 70):
        assert torch.equal(y[a:a + 70], run_gemm(dev(x[a:a + 70]), wp, swd, None, N, BF16))
    check_gemm(y[-8:], x[-8:], w[0], sw[0], None)


def test_logits_behind_two_to_the_31():
    T, E, topk = 2_100_000, 1024, 2
    assert T * E > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.randn((T, E), dtype=torch.bfloat16, device=DEV, generator=g)
    ids, w, cnt, _ = run(z, topk, True, BF16)
    assert int(cnt[E]) == T and int(cnt[:E].sum()) == T * topk
    dw = torch.randn((T, topk), device=DEV, generator=g)
    dz = run_bwd(z, ids, w, cnt, dw, None, topk, True, BF16)
    for a in (0, 2 ** 21 - 100, T - 200):
        s = slice(a, a + 200)
        i, v, c, _ = run(z[s].clone(), topk, True, BF16)
        assert torch.equal(ids[s], i) and torch.equal(w[s], v)
        assert torch.equal(dz[s], run_bwd(z[s].clone(), i, v, c, dw[s].clone(), None, topk, True, BF16))
