"""W8A8 products on the GPU against 64-bit references: codes bit for bit,
results within the rounding of the formula's fp32 steps."""
import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = ref.F16, ref.BF16


def quantize(x, dt, row_count=None, ldx=0, M=None, K=None):
    M, K = M if M is not None else x.shape[0], K or x.shape[1]
    qx = torch.full((M, K), 55, dtype=torch.int8, device=DEV)
    sx = torch.full((M,), -7.0, device=DEV)
    w4.w8a8_quantize(x, qx, sx, M, K, dt, row_count=row_count, ldx=ldx)
    return qx, sx


def check_codes(x, qx, sx):
    q, s = ref.quantize(x.cpu())
    assert torch.equal(sx.cpu().view(torch.int32)[~torch.isnan(s)], s.view(torch.int32)[~torch.isnan(s)])
    assert torch.equal(torch.isnan(sx.cpu()), torch.isnan(s))
    assert torch.equal(qx.cpu().double(), q)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (5, 1408), (2, 8192), (33, 2048), (2, 14336), (1, 130944)])
def test_codes(dt, M, K):
    g = torch.Generator().manual_seed(M * 7 + K)
    x = (torch.randn((M, K), generator=g) * torch.logspace(-3, 2, M)[:, None]).to(ref.TORCH[dt]).to(DEV)
    check_codes(x, *quantize(x, dt))


@pytest.mark.parametrize("dt", [F16, BF16])
def test_codes_at_borders(dt):
    """Rows whose scale is a power of two, with quotients of exactly k + 1/2 (ties to the
    even code), and rows of the same values scaled to either end of the type's range."""
    td = ref.TORCH[dt]
    k = torch.arange(-127, 127, dtype=torch.float32)
    base = torch.cat((torch.tensor([127.0]), (k + 0.5), torch.zeros(1)))          # 256 values, largest 127
    exps = [-14, -5, 0, 3, 8] if dt == F16 else [-133, -126, -120, -60, 0, 60, 120]
    rows = torch.stack([(base.double() * 2.0 ** e).to(td) for e in exps])
    rows = torch.cat((rows, (rows.double() * 0.7).to(td)))
    check_codes(rows, *quantize(rows.to(DEV), dt))


@pytest.mark.parametrize("dt", [F16, BF16])
def test_codes_of_unusual_rows(dt):
    td = ref.TORCH[dt]
    x = torch.randn((9, 384), generator=torch.Generator().manual_seed(5)).to(td)
    x[0] = 0
    x[1, 200] = float("inf")
    x[2, 0] = float("-inf")
    x[3, 383] = float("nan")
    x[4] = 0
    x[4, 17] = torch.finfo(td).smallest_normal * torch.finfo(td).eps              # the smallest subnormal alone
    x[5] = torch.finfo(td).max
    x[6] = -torch.finfo(td).max
    x[7] = x[7] * torch.finfo(td).smallest_normal                                  # subnormals
    x[8] = -0.0
    qx, sx = quantize(x.to(DEV), dt)
    check_codes(x, qx, sx)


def test_quantize_strided_rows_and_row_count():
    x = torch.randn((7, 512 + 24), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    qx, sx = quantize(x, BF16, ldx=536, K=512)
    check_codes(x[:, :512], qx, sx)
    for n in (0, 1, 4, 7, 9):
        cnt = torch.tensor([n], dtype=torch.int32, device=DEV)
        qx, sx = quantize(x, BF16, row_count=cnt, ldx=536, K=512)
        m = min(n, 7)
        check_codes(x[:m, :512], qx[:m], sx[:m]) if m else None
        assert bool((qx[m:] == 55).all()) and bool((sx[m:] == -7).all())


# ---- dense -------------------------------------------------------------------------

def problem(M, K, N, dt, seed=0, E=1, bias=False):
    g = torch.Generator().manual_seed(seed * 1000 + M * 3 + K + N)
    td = ref.TORCH[dt]
    x = (torch.randn((M, K), generator=g) * (1 + 19 * (torch.rand(K, generator=g) < 0.01))).to(td)
    w = torch.randint(-128, 128, (E, K, N), generator=g).to(torch.int8)
    sw = (torch.rand((E, N), generator=g) + 0.5) * 1e-3
    b = torch.randn(N, generator=g).to(td) if bias else None
    return x, w, sw, b


def dev(t):
    return None if t is None else t.to(DEV)


def packed(w):
    E, K, N = w.shape
    wd = w.to(DEV)
    out = torch.empty(w4.w8a16_prepacked_bytes(E, K, N), dtype=torch.uint8, device=DEV)
    w4.w8a16_prepack(wd, out, E, K, N, 1)
    return out


def workspace(nbytes):
    return torch.full((nbytes,), 0xA5, dtype=torch.uint8, device=DEV)


def run_gemm(x, wp, sw, b, N, dt, ldx=0, ldy=0, M=None, K=None, y=None):
    M, K = M or x.shape[0], K or x.shape[1]
    nb = w4.w8a8_workspace_bytes(M, K)
    y = torch.full((M, ldy or N), 9.0, dtype=ref.TORCH[dt], device=DEV) if y is None else y
    w4.w8a8_gemm(x, wp, sw, y, M, K, N, bias=b, dt=dt, ldx=ldx, ldy=ldy, workspace=workspace(nb), workspace_bytes=nb)
    return y


def check_gemm(y, x, w, sw, b):
    q, s = ref.quantize(x)
    want, part = ref.gemm(q, s, w, sw, b)
    bound = ref.gemm_bound(want, part, x.dtype)
    err = (y.cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


SIZES = [(1, 128, 64), (1, 4096, 320), (2, 256, 256), (3, 14336, 64), (7, 640, 192), (16, 2048, 512), (17, 128, 1088),
         (31, 1408, 256), (33, 384, 64), (48, 512, 128), (64, 2048, 192), (65, 256, 320), (100, 1152, 448),
         (128, 1024, 256), (129, 128, 576), (200, 640, 1024), (255, 2048, 256), (257, 384, 192), (300, 256, 2048),
         (513, 512, 320), (1025, 128, 64), (777, 896, 1216)]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_gemm(M, K, N, dt):
    x, w, sw, b = problem(M, K, N, dt, bias=(M + N // 64) % 2 == 0)
    y = run_gemm(dev(x), packed(w), dev(sw), dev(b), N, dt)
    check_gemm(y, x, w[0], sw[0], b)


@pytest.mark.parametrize("M", [1, 20, 70, 300])
def test_gemm_strides(M):
    """Rows of x and y inside wider buffers; what lies between stays."""
    K, N, dt = 384, 192, BF16
    x, w, sw, b = problem(M, K, N, dt, seed=3, bias=True)
    wide = torch.full((M, K + 40), float("nan"), dtype=x.dtype)
    wide[:, :K] = x
    y = run_gemm(dev(wide), packed(w), dev(sw), dev(b), N, dt, ldx=K + 40, ldy=N + 24, M=M, K=K)
    check_gemm(y[:, :N], x, w[0], sw[0], b)
    assert bool((y[:, N:] == 9.0).all())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_largest_sums(M):
    """Codes of -128 and 127 over the longest K: the sums come within 2^21 of 2^31."""
    K, N = 130944, 64
    qx = torch.full((M, K), -128, dtype=torch.int8)
    qx[-1] = 127
    w = torch.full((1, K, N), -128, dtype=torch.int8)
    w[0, :, 1] = 127
    y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    sx, sw = torch.full((M,), 2.0 ** -20), torch.full((1, N), 0.5)
    w4.w8a8_gemm_prequant(dev(qx), dev(sx), packed(w), dev(sw), y, M, K, N)
    want = torch.empty((M, N), dtype=torch.float64)
    for r, c in ((0, -128), (M - 1, 127)):
        want[r] = c * -128 * K
        want[r, 1] = c * 127 * K
    want *= 2.0 ** -21
    for r in (0, M - 1):
        assert bool(((y[r].cpu().double() - want[r]).abs() <= want[r].abs() * (2.0 ** -8 + 2.0 ** -20)).all())


def test_scales_outside_fp32():
    """s_m sw_n leaves fp32's range while y stays inside bf16's: too small for fp32 where the
    sum brings it back, and too large where the sum is 0."""
    M, K, N = 4, 1024, 64
    x, w, _, _ = problem(M, K, N, BF16)
    q = ref.quantize(x)[0].to(torch.int8)
    q[1] = 0
    for sx, f in ((1e-42, 1e-4), (1e-38, 1e-5), (3e38, 1e-40), (1e30, 1e-30)):
        sx, f = torch.full((M,), sx), torch.full((N,), f)
        y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
        w4.w8a8_gemm_prequant(dev(q), dev(sx), packed(w), dev(f), y, M, K, N)
        want, part = ref.gemm(q, sx, w[0], f)
        assert float(want[0].abs().max()) > 0
        assert bool(((y.cpu().double() - want).abs() <= ref.gemm_bound(want, part, torch.bfloat16)).all())
    y = torch.ones((M, N), dtype=torch.bfloat16, device=DEV)
    w4.w8a8_gemm_prequant(dev(q), dev(torch.full((M,), 3e38)), packed(w), dev(torch.full((N,), 2e3)), y, M, K, N)
    assert bool((y[1] == 0).all()) and bool(torch.isinf(y[[0, 2, 3]]).any(1).all()) and not bool(torch.isnan(y).any())


@pytest.mark.parametrize("M", [5, 70, 300])
def test_rows_without_a_scale(M):
    K, N = 512, 128
    x, w, sw, b = problem(M, K, N, F16, bias=True)
    x[1, 3] = float("inf")
    x[3, 511] = float("nan")
    x[4] = 0
    y = run_gemm(dev(x), packed(w), dev(sw), dev(b), N, F16)
    assert bool(torch.isnan(y[[1, 3]]).all())
    keep = [r for r in range(M) if r not in (1, 3)]
    check_gemm(y[keep], x[keep], w[0], sw[0], b)
    assert torch.equal(y[4].cpu(), b)


@pytest.mark.parametrize("dt", [F16, BF16])
def test_a_row_does_not_depend_on_its_batch(dt):
    K, N = 1152, 320
    x, w, sw, b = problem(600, K, N, dt, bias=True)
    wp, xd, swd, bd = packed(w), dev(x), dev(sw), dev(b)
    full = run_gemm(xd, wp, swd, bd, N, dt)
    for M in (1, 2, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512):
        assert torch.equal(run_gemm(xd[:M], wp, swd, bd, N, dt), full[:M]), M


# ---- grouped -----------------------------------------------------------------------

def offsets_of(rows):
    return torch.cat((torch.zeros(1, dtype=torch.int64), torch.tensor(rows).cumsum(0))).to(torch.int32)


ROWS = [[1], [3, 0, 5], [0, 0, 17, 0], [16, 1, 33, 64, 2], [130, 0, 1, 65, 300, 7], [1] * 70, [0] * 64 + [9, 0, 40]]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("K,N", [(128, 64), (640, 320)])
def test_grouped(rows, K, N, dt):
    """Rows in the experts' order, three more rows in x and y than the experts hold."""
    E, R = len(rows), sum(rows) + 3
    x, w, sw, _ = problem(R, K, N, dt, E=E)
    off = offsets_of(rows)
    nb = w4.w8a8_grouped_workspace_bytes(R, K)
    y = torch.full((R, N), 9.0, dtype=x.dtype, device=DEV)
    w4.w8a8_grouped_gemm(dev(x), dev(off), packed(w), dev(sw), y, E, R, K, N, dt=dt, workspace=workspace(nb),
                         workspace_bytes=nb)
    assert bool((y[sum(rows):] == 9.0).all())
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if b > a:
            check_gemm(y[a:b], x[a:b], w[e], sw[e], None)


@pytest.mark.parametrize("T,topk,E", [(1, 1, 4), (4, 8, 64), (37, 3, 70), (200, 2, 5), (150, 8, 16)])
def test_grouped_reads_tokens(T, topk, E):
    """Routed as w4a16_moe_align orders it, some entries without an expert; bit for bit
    what the gathered rows give."""
    K, N, dt, R = 256, 192, BF16, T * topk
    x, w, sw, _ = problem(T, K, N, dt, E=E)
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(T)])
    ids[torch.rand((T, topk), generator=g) < 0.1] = -1
    off, srt, row_of = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (E + 1, R, R))
    w4.w4a16_moe_align(ids.to(torch.int32).to(DEV), T, topk, E, off, srt, row_of)
    nb = w4.w8a8_grouped_workspace_bytes(R, K)
    wp, xd, swd = packed(w), dev(x), dev(sw)
    y, z = (torch.full((R, N), 9.0, dtype=x.dtype, device=DEV) for _ in range(2))
    w4.w8a8_grouped_gemm(xd, off, wp, swd, y, E, R, K, N, sorted_ids=srt, topk=topk, dt=dt, workspace=workspace(nb),
                         workspace_bytes=nb)
    gathered = xd[srt.long() // topk].contiguous()
    w4.w8a8_grouped_gemm(gathered, off, wp, swd, z, E, R, K, N, dt=dt, workspace=workspace(nb), workspace_bytes=nb)
    assert torch.equal(y, z)
    o, rows = off.cpu(), gathered.cpu()
    for e in range(E):
        a, b = int(o[e]), int(o[e + 1])
        if b > a:
            check_gemm(y[a:b], rows[a:b], w[e], sw[e], None)
    assert bool((y[int(o[E]):] == 9.0).all())


def test_stream_and_graph():
    """On a side stream, then captured and replayed with eager work between the replays."""
    M, K, N = 40, 1024, 512
    x, w, sw, b = problem(M, K, N, BF16, bias=True)
    wp, swd, bd = packed(w), dev(sw), dev(b)
    xs = [dev(x * f) for f in (1, -2, 0.5)]
    want = [run_gemm(v, wp, swd, bd, N, BF16) for v in xs]
    static, y, nb = xs[0].clone(), torch.zeros_like(want[0]), w4.w8a8_workspace_bytes(M, K)
    ws = workspace(nb)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(run_gemm(xs[1], wp, swd, bd, N, BF16), want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            w4.w8a8_gemm(static, wp, swd, y, M, K, N, bias=bd, workspace=ws, workspace_bytes=nb)
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1, 0):
        static.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        y.zero_()
        assert torch.equal(run_gemm(xs[2 - i], wp, swd, bd, N, BF16), want[2 - i])


@pytest.fixture
def config():
    yield w4.w4a16_test_w8a8_config
    w4.w4a16_test_w8a8_config(-1)


@pytest.mark.parametrize("idx", [n * 100 + i for i in range(w4.w4a16_test_w8a8_config(-1)) for n in (0, 2, 3, 8)])
@pytest.mark.parametrize("M,K,N", [(1, 128, 64), (37, 256, 320), (150, 384, 192), (300, 1024, 576), (520, 2688, 64)])
def test_every_kernel(config, M, K, N, idx):
    """Each kernel that a size may pick, whole and in slices, on sizes that end inside its tiles
    and on short K."""
    x, w, sw, b = problem(M, K, N, BF16, bias=True)
    config(idx)
    check_gemm(run_gemm(dev(x), packed(w), dev(sw), dev(b), N, BF16), x, w[0], sw[0], b)


@pytest.mark.parametrize("idx", range(w4.w4a16_test_w8a8_config(-1)))
@pytest.mark.parametrize("rows", [[1], [16, 1, 0, 33, 300], [1] * 70])
def test_every_grouped_kernel(config, rows, idx):
    config(idx)
    test_grouped(rows, 640, 320, F16)
    test_grouped_reads_tokens(37, 3, 70)
