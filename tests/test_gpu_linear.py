"""Fused linear operators on the GPU against the 64-bit reference."""
import math

import pytest
import torch

import linear_ref as ref
import weight_only_quantized_amd as w4
from linear_ref import BF16, F16, GELU, GELU_TANH, NONE, RELU, SILU

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GAP = 24          # unused elements per row of a strided tensor


class Dev:
    """A layer on the GPU, prepacked."""

    def __init__(self, L):
        self.L = L
        raw = L.packed_plain().to(DEV)
        self.packed = torch.empty(w4.w4a16_prepacked_bytes(1, L.K, L.N), dtype=torch.uint8, device=DEV)
        w4.w4a16_prepack(raw, self.packed, 1, L.K, L.N, int(L.zero is None))
        z = L.zero_packed()
        self.lin = w4.linear(L.K, L.N, self.packed, L.scale.to(DEV), None if z is None else z.to(DEV),
                             None if L.bias is None else L.bias.to(DEV), L.group)


def put(t, strided):
    """t on the GPU, as a slice of a wider buffer whose gaps hold NaN."""
    if t is None:
        return None, 0
    if not strided:
        return t.to(DEV), 0
    b = torch.full((t.shape[0], t.shape[1] + GAP), math.nan, dtype=t.dtype, device=DEV)
    b[:, :t.shape[1]] = t.to(DEV)
    return b, b.shape[1]


def out(M, width, dt, strided):
    b = torch.full((M, width + (GAP if strided else 0)), 777.0, dtype=ref.TD[dt], device=DEV)
    return b, b.shape[1] if strided else 0


def untouched(b, width):
    assert (b[:, width:] == 777.0).all()


def workspace(n):
    return (torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) if n else None), n     # NaN bytes


def run_ep(D, x, a, residual=None, save=False, strided=False):
    L, M = D.L, x.shape[0]
    xd, ldx = put(x, strided)
    rd, ldr = put(residual, strided)
    y, ldy = out(M, L.N, L.dt, strided)
    p = torch.empty((M, L.N), dtype=ref.TD[L.dt], device=DEV) if save else None
    ws, nb = workspace(w4.w4a16_gemm_ep_workspace_bytes(D.lin, M))
    w4.w4a16_gemm_ep(xd, D.lin, y, M, a, rd, p, L.dt, ldx=ldx, ldr=ldr, ldy=ldy, workspace=ws, workspace_bytes=nb)
    untouched(y, L.N)
    return y[:, :L.N], p


def run_glu(D, x, a, save=False, strided=False):
    L, M = D.L, x.shape[0]
    xd, ldx = put(x, strided)
    y, lda = out(M, L.N // 2, L.dt, strided)
    h = torch.empty((M, L.N), dtype=ref.TD[L.dt], device=DEV) if save else None
    ws, nb = workspace(w4.w4a16_glu_gemm_workspace_bytes(D.lin, M))
    w4.w4a16_glu_gemm(xd, D.lin, y, M, a, h, L.dt, ldx=ldx, lda=lda, workspace=ws, workspace_bytes=nb)
    untouched(y, L.N // 2)
    return y[:, :L.N // 2], h


def run_bwd(D, glu, dy, h, a, addend=None, dbias=True, strided=False):
    """dx, d (None for the plain product without an activation), dbias."""
    L, M = D.L, dy.shape[0]
    dyd, lddy = put(dy, strided)
    ad, ldadd = put(addend, strided)
    dx, lddx = out(M, L.K, L.dt, strided)
    through = glu or a != NONE
    d = torch.empty((M, L.N), dtype=ref.TD[L.dt], device=DEV) if through else None
    db = torch.full((L.N,), 777.0, device=DEV) if dbias else None
    q = w4.w4a16_glu_gemm_backward_workspace_bytes if glu else w4.w4a16_gemm_ep_backward_workspace_bytes
    ws, nb = workspace(q(D.lin, M))
    if glu:
        w4.w4a16_glu_gemm_backward(dyd, h.to(DEV), D.lin, dx, M, a, d, db, ad, L.dt, ldda=lddy, ldadd=ldadd,
                                   lddx=lddx, workspace=ws, workspace_bytes=nb)
    else:
        w4.w4a16_gemm_ep_backward(dyd, h.to(DEV) if through else None, D.lin, dx, M, a, d, db, ad, L.dt, lddy=lddy,
                                  ldadd=ldadd, lddx=lddx, workspace=ws, workspace_bytes=nb)
    untouched(dx, L.K)
    return dx[:, :L.K], d, db


# rows around every tile and wave boundary; widths that end inside a 256-column
# tile and inside its waves; one and many groups; K cut into slices
FORWARD = [
    # M, K, N, group, dt, zero, act, residual, strided
    (1, 128, 64, 128, BF16, False, NONE, False, False),
    (1, 4096, 192, 128, BF16, True, SILU, True, False),
    (3, 2176, 320, 128, F16, False, GELU, False, True),
    (16, 1024, 704, 256, F16, True, RELU, True, True),
    (17, 640, 256, 128, BF16, False, GELU_TANH, True, False),
    (33, 384, 128, 384, BF16, True, SILU, False, True),
    (64, 256, 448, 128, F16, True, NONE, True, False),
    (65, 256, 64, 128, BF16, False, GELU, True, True),
    (65, 4096, 320, 128, F16, True, RELU, True, False),
    (128, 2048, 192, 512, BF16, True, NONE, True, True),
    (129, 128, 576, 128, BF16, False, SILU, False, False),
    (257, 768, 832, 256, F16, False, GELU_TANH, True, True),
    (511, 1152, 256, 1152, BF16, True, GELU, True, False),
    (1030, 256, 1088, 128, F16, True, SILU, False, False),
]


@pytest.mark.parametrize("M,K,N,group,dt,zero,a,residual,strided", FORWARD)
def test_ep_matches_reference(M, K, N, group, dt, zero, a, residual, strided):
    L = ref.layer(K, N, group, dt, zero, bias=M % 2 == 1, seed=M + K)
    x = ref.normal(M, K, 1.0, dt, 1)
    r = ref.normal(M, N, 1.0, dt, 2) if residual else None
    y, p = run_ep(Dev(L), x, a, r, save=True, strided=strided)
    yr, pr = ref.ep(x, L, a, r)
    ref.close(p, pr, ref.tol_ep(pr, pr, dt), f"pre {M} {K} {N}")
    ref.close(y, yr, ref.tol_ep(yr, pr, dt), f"ep {M} {K} {N}")


@pytest.mark.parametrize("M,K,N,group,dt,zero,a,residual,strided", [c for c in FORWARD if c[2] % 128 == 0])
def test_glu_matches_reference(M, K, N, group, dt, zero, a, residual, strided):
    L = ref.layer(K, N, group, dt, zero, bias=M % 2 == 1, seed=M + K)
    x = ref.normal(M, K, 1.0, dt, 1)
    y, h = run_glu(Dev(L), x, a, save=True, strided=strided)
    yr, hr = ref.glu(x, L, a)
    ref.close(h, hr, ref.tol_ep(hr, hr, dt), f"h {M} {K} {N}")
    ref.close(y, yr, ref.tol_glu(yr, hr, dt), f"glu {M} {K} {N}")


@pytest.mark.parametrize("M,K,N,dt", [(1, 256, 128, BF16), (40, 512, 384, F16), (100, 2048, 640, BF16), (300, 384, 1152, F16)])
def test_every_activation(M, K, N, dt):
    L = ref.layer(K, N, 128, dt, True, True, seed=9)
    x = ref.normal(M, K, 1.0, dt, 1)
    D = Dev(L)
    for a in ref.ACTS:
        y, _ = run_ep(D, x, a)
        yr, pr = ref.ep(x, L, a)
        ref.close(y, yr, ref.tol_ep(yr, pr, dt), f"ep act {a}")
        y, _ = run_glu(D, x, a)
        yr, hr = ref.glu(x, L, a)
        ref.close(y, yr, ref.tol_glu(yr, hr, dt), f"glu act {a}")


BACKWARD = [
    # M, K, N, group, dt, zero, act, addend, strided
    (1, 128, 64, 128, BF16, False, NONE, False, False),
    (1, 4096, 128, 128, F16, True, SILU, True, True),
    (5, 256, 1024, 256, BF16, True, GELU, True, False),
    (63, 384, 192, 128, BF16, False, RELU, False, True),
    (64, 128, 2048, 128, F16, False, GELU_TANH, True, False),
    (66, 640, 448, 128, BF16, True, NONE, True, True),
    (129, 256, 1152, 128, F16, True, SILU, False, False),
    (258, 1152, 256, 384, BF16, False, GELU, True, True),
    (515, 512, 1088, 512, F16, False, NONE, True, False),
    # few rows: one block of columns, odd blocks, N cut into slices
    (2, 128, 64, 128, F16, True, GELU, False, True),
    (17, 384, 320, 384, BF16, False, NONE, True, True),
    (32, 128, 4224, 128, BF16, True, SILU, True, False),
    (31, 256, 6528, 256, F16, False, RELU, False, True),
]


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("M,K,N,group,dt,zero,a,addend,strided", BACKWARD)
def test_backward_matches_reference(glu, M, K, N, group, dt, zero, a, addend, strided):
    N = N + 64 if glu and N % 128 else N
    L = ref.layer(K, N, group, dt, zero, seed=M + K)
    dy = ref.normal(M, N // 2 if glu else N, 0.5, dt, 1)
    h = ref.normal(M, N, 1.5, dt, 2)
    r = ref.normal(M, K, 0.5, dt, 3) if addend else None
    dx, d, db = run_bwd(Dev(L), glu, dy, h, a, r, strided=strided)
    rx, rd, rb = (ref.glu_backward if glu else ref.ep_backward)(dy, h, L, a, r)
    if d is not None:
        ref.close(d, rd, ref.tol_d(rd, dt), f"d {M} {K} {N}")
    ref.close(dx, rx, ref.tol_dx(rx, rd, L, dt), f"dx {M} {K} {N}")
    # fp32 sums of M values, each within a few 2^-23 of its factors' size
    ref.close(db, rb, 2.0 ** -20 * (rd.abs().sum(0) + rd.abs().amax()), f"dbias {M} {K} {N}")


@pytest.mark.parametrize("a", ref.ACTS)
@pytest.mark.parametrize("glu", [False, True])
def test_gradients_match_differences(glu, a):
    """The kernels' gradients along random directions against central
    differences of the 64-bit forward function.  The direction's error is that
    of dx: independent errors of tol_dx / 6 standard deviations."""
    M, K, N, e = 70, 256, 256, 2.0 ** -14
    L = ref.layer(K, N, 128, F16, True, seed=21)
    x = ref.normal(M, K, 1.0, F16, 1)
    f = ref.glu if glu else ref.ep
    h = f(x, L, a)[1].to(torch.float16)             # the kernels read it rounded: so does the reference below
    dy = ref.normal(M, N // 2 if glu else N, 1.0, F16, 2)
    dx, d, _ = run_bwd(Dev(L), glu, dy, h, a)
    W = L.weights()
    for seed in range(4):
        v = torch.randn((M, K), dtype=torch.float64, generator=torch.Generator().manual_seed(seed))

        def loss(t):
            p = h.double() + t * (v @ W)
            if glu:
                g, u = p.chunk(2, 1)
                return (ref.act(g, a)[0] * u * dy.double()).sum()
            return (ref.act(p, a)[0] * dy.double()).sum()

        num = (loss(e) - loss(-e)) / (2 * e)
        rx, rd, _ = (ref.glu_backward if glu else ref.ep_backward)(dy, h, L, a)
        sd = (ref.tol_dx(rx, rd, L, F16) * v).square().sum().sqrt()
        got = (dx.double().cpu() * v).sum()
        # RELU: steps of 2^-14 cross a few kinks, each by at most e |vW| |dy|
        kink = 0.0
        if a == RELU:
            g = (h.double().chunk(2, 1)[0] if glu else h.double())
            vw = (v @ W)[:, :g.shape[1]]
            w = dy.double().abs() * (h.double().chunk(2, 1)[1].abs() if glu else 1.0)
            kink = ((g.abs() <= e * vw.abs()) * vw.abs() * w).sum()
        assert abs(num - got) <= sd + kink, (seed, num, got, sd)


@pytest.fixture
def plan():
    """Forces a tile shape and slice count; back to the choice by size after the test."""
    yield w4.w4a16_test_linear_plan
    w4.w4a16_test_linear_plan(-1, 0)


SHAPES = 4


@pytest.mark.parametrize("slices", [1, 3])
@pytest.mark.parametrize("shape", range(SHAPES))
@pytest.mark.parametrize("dt", [F16, BF16])
def test_every_tile_shape(plan, shape, slices, dt):
    """Each tile shape, whole and in slices, on rows and columns that end inside
    it: one row, a few, more than one tile; an odd number of 64-column stages in
    the transposed product; scale groups of one and several 128-row groups."""
    assert plan(-1, 0) == SHAPES
    for M, K, N, group, zero in ((1, 768, 128, 128, True), (70, 768, 448, 384, False), (300, 1152, 640, 128, True)):
        L = ref.layer(K, N, group, dt, zero, seed=M)
        D = Dev(L)
        plan(shape, slices)
        x, r = ref.normal(M, K, 1.0, dt, 1), ref.normal(M, N, 1.0, dt, 2)
        y, p = run_ep(D, x, GELU, r, save=True)
        yr, pr = ref.ep(x, L, GELU, r)
        ref.close(p, pr, ref.tol_ep(pr, pr, dt), "pre")
        ref.close(y, yr, ref.tol_ep(yr, pr, dt), "ep")
        h = ref.normal(M, N, 1.5, dt, 3)
        dx, d, db = run_bwd(D, False, r, h, SILU)
        rx, rd, rb = ref.ep_backward(r, h, L, SILU)
        ref.close(dx, rx, ref.tol_dx(rx, rd, L, dt), "dx")
        ref.close(db, rb, 2.0 ** -20 * (rd.abs().sum(0) + rd.abs().amax()), "dbias")
        if N % 128 == 0:
            y, h = run_glu(D, x, SILU, save=True)
            yr, hr = ref.glu(x, L, SILU)
            ref.close(y, yr, ref.tol_glu(yr, hr, dt), "glu")
            ref.close(h, hr, ref.tol_ep(hr, hr, dt), "h")


@pytest.mark.parametrize("shape", range(SHAPES))
@pytest.mark.parametrize("M,n", [(3, 1), (65, 2), (33, 3), (130, 5), (40, 7)])
def test_short_and_uneven_contractions(plan, shape, M, n):
    """Contractions of one to seven 128-row groups forward and of one to seven
    64-column stages transposed: the second wave group of a 128-column tile gets
    a smaller share or none."""
    K, N = 128 * n, 64 * n
    L = ref.layer(K, N, 128, BF16, True, seed=n)
    D = Dev(L)
    plan(shape, 1)
    x, r = ref.normal(M, K, 1.0, BF16, 1), ref.normal(M, N, 1.0, BF16, 2)
    y, _ = run_ep(D, x, SILU, r, save=True)
    yr, pr = ref.ep(x, L, SILU, r)
    ref.close(y, yr, ref.tol_ep(yr, pr, BF16), "ep")
    h = ref.normal(M, N, 1.5, BF16, 3)
    dx, _, _ = run_bwd(D, False, r, h, SILU)
    rx, rd, _ = ref.ep_backward(r, h, L, SILU)
    ref.close(dx, rx, ref.tol_dx(rx, rd, L, BF16), "dx")


@pytest.mark.parametrize("shape", range(SHAPES))
def test_every_tile_shape_holds_its_scales(plan, shape):
    """The unit change of the tile kernel's sums (zero, tiny and huge scales) in
    every shape, in whole calls and slices that start inside a scale group."""
    K, N, M = 1024, 256, 150
    for group, slices in ((128, 1), (512, 4)):
        L = ref.layer(K, N, group, BF16, True, bias=False, seed=8)
        s = L.scale.clone()
        s[0, :16], s[-1, 8:32] = 0, 0
        s[0, 32:48], s[-1, 40:56] = 2.0 ** 20, 2.0 ** -100
        s[:, 64:96] *= torch.tensor([-1.0, 1.0]).repeat(16).to(s.dtype)
        L.scale = s
        plan(shape, slices)
        x = ref.normal(M, K, 1.0, BF16, 1)
        y, _ = run_ep(Dev(L), x, NONE)
        yr, _ = ref.ep(x, L, NONE)
        size = (x.double().square() @ L.weights().square()).sqrt()
        ref.close(y, yr, ref.ULP[BF16] * 1.01 * yr.abs() + 8 * ref.SUM * size + 2.0 ** -134, "scales")


def test_in_place_residual_and_gradients():
    """y may be the residual, dpre the saved pre, dx the addend."""
    for M in (9, 200):
        L = ref.layer(256, 256, 128, BF16, True, seed=4)
        D = Dev(L)
        x, r = ref.normal(M, 256, 1.0, BF16, 1), ref.normal(M, 256, 1.0, BF16, 2)
        y = r.to(DEV)
        ws, nb = workspace(w4.w4a16_gemm_ep_workspace_bytes(D.lin, M))
        w4.w4a16_gemm_ep(x.to(DEV), D.lin, y, M, SILU, y, None, BF16, workspace=ws, workspace_bytes=nb)
        yr, pr = ref.ep(x, L, SILU, r)
        ref.close(y, yr, ref.tol_ep(yr, pr, BF16), "in place y")
        for glu in (False, True):
            dy = ref.normal(M, 128 if glu else 256, 1.0, BF16, 3)
            h, g = ref.normal(M, 256, 1.0, BF16, 5).to(DEV), r.to(DEV)
            rx, rd, _ = (ref.glu_backward if glu else ref.ep_backward)(dy, h.cpu(), L, GELU, r)
            q = w4.w4a16_glu_gemm_backward_workspace_bytes if glu else w4.w4a16_gemm_ep_backward_workspace_bytes
            ws, nb = workspace(q(D.lin, M))
            f = w4.w4a16_glu_gemm_backward if glu else w4.w4a16_gemm_ep_backward
            f(dy.to(DEV), h, D.lin, g, M, GELU, h, None, g, BF16, workspace=ws, workspace_bytes=nb)
            ref.close(h, rd, ref.tol_d(rd, BF16), "in place d")
            ref.close(g, rx, ref.tol_dx(rx, rd, L, BF16), "in place dx")


@pytest.mark.parametrize("glu", [False, True])
def test_no_rows_gives_zero_bias_gradient(glu):
    L = ref.layer(128, 128)
    db = torch.full((128,), 5.0, device=DEV)
    f = w4.w4a16_glu_gemm_backward if glu else w4.w4a16_gemm_ep_backward
    f(None, None, Dev(L).lin, None, 0, SILU, None, db)
    assert (db == 0).all()


@pytest.mark.parametrize("M", [2, 20, 90, 300])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_scales_of_any_size_and_sign(M, dt):
    """Zero, negative, tiny and huge scales next to ordinary ones, group by
    group: the tile kernel holds its sums in units of the running scale."""
    K, N = 1024, 128
    L = ref.layer(K, N, 128, dt, True, bias=False, seed=8)
    s = L.scale.clone()
    s[0, 0:16] = 0
    s[3, 8:24] = 0
    s[7, 0:32] = 0
    s[:, 32:40] = 0                                  # a column without any weight
    s[2, 40:64] *= -1
    lo, hi = (2.0 ** -24, 16.0) if dt == F16 else (2.0 ** -120, 2.0 ** 20)
    s[0, 64:72], s[4, 64:72] = lo, lo
    s[1, 72:80], s[5, 72:80] = hi, lo
    s[:, 80:84] = lo                                 # nothing but tiny scales
    L.scale = s
    x = ref.normal(M, K, 1.0, dt, 1)
    y, _ = run_ep(Dev(L), x, NONE)
    yr, _ = ref.ep(x, L, NONE)
    w2 = L.weights().square()
    # per element: fp32 sums relative to the terms' own sizes, one rounding, fp16 subnormals
    size = (x.double().square() @ w2).sqrt()
    tiny = 2.0 ** -25 if dt == F16 else 2.0 ** -134
    ref.close(y, yr, ref.ULP[dt] * 1.01 * yr.abs() + 8 * ref.SUM * size + tiny, "scales")
    assert (y[:, 32:40] == 0).all()


@pytest.mark.parametrize("M", [12, 40, 100, 300])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_rows_do_not_mix(M, dt):
    """A NaN or an infinity in one row of x (or dy) reaches no other row; the
    last row repeats past M inside the kernels."""
    L = ref.layer(256, 192, 128, dt, True, seed=8)
    D = Dev(L)
    x = ref.normal(M, 256, 1.0, dt, 1)
    clean, _ = run_ep(D, x, SILU)
    x[M - 1, 7], x[2, 200] = math.nan, math.inf
    y, _ = run_ep(D, x, SILU)
    keep = [m for m in range(M) if m not in (2, M - 1)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[M - 1]).all() and not torch.isfinite(y[2]).all()
    dy = ref.normal(M, 192, 1.0, dt, 3)
    h = ref.normal(M, 192, 1.0, dt, 4)
    cx, _, _ = run_bwd(D, False, dy, h, GELU_TANH)
    dy[M - 1, 5] = math.nan
    gx, _, db = run_bwd(D, False, dy, h, GELU_TANH)
    assert torch.equal(gx[:M - 1], cx[:M - 1]) and torch.isnan(gx[M - 1]).all()
    assert torch.isnan(db[5]) and torch.isfinite(db[:5]).all() and torch.isfinite(db[6:]).all()


@pytest.mark.parametrize("a", ref.ACTS)
def test_saturated_pre_activations(a):
    """Large, zero and NaN pre-activations: finite gradients where the true
    ones are, NaN where they are NaN."""
    M, N = 6, 128
    L = ref.layer(128, N, 128, BF16, bias=False, seed=2)
    h = ref.normal(M, N, 1.0, BF16, 2)
    h[0] = 0.0
    h[1], h[2] = 300.0, -300.0
    h[3], h[4] = 3e37, -3e37
    h[5, 0] = math.nan
    dy = ref.normal(M, N, 0.5, BF16, 1)
    _, d, _ = run_bwd(Dev(L), False, dy, h, a) if a != NONE else (None, dy.to(DEV), None)
    rd = dy.double() if a == NONE else dy.double() * ref.act(h.double().clamp(-300, 300), a)[1]
    assert a == NONE or torch.isnan(d[5, 0])
    ok = torch.isfinite(rd)
    ref.close(d[ok.to(DEV)], rd[ok], ref.tol_d(rd[ok], BF16), f"saturated act {a}")


def test_equal_calls_give_equal_bits():
    L = ref.layer(2048, 640, 128, BF16, True, seed=6)
    D = Dev(L)
    for M in (7, 50, 130, 520):
        x, dy = ref.normal(M, 2048, 1.0, BF16, 1), ref.normal(M, 320, 1.0, BF16, 2)
        h = ref.normal(M, 640, 1.0, BF16, 3)
        first = run_glu(D, x, SILU)[0].clone(), *run_bwd(D, True, dy, h, SILU)
        again = run_glu(D, x, SILU)[0], *run_bwd(D, True, dy, h, SILU)
        for p, q in zip(first, again):
            assert torch.equal(p, q)


def test_on_another_stream_and_in_a_graph():
    """The calls enqueue on the stream they are given, and a captured block
    gives the eager result on every replay, with eager work in between."""
    L1, L2 = ref.layer(512, 1024, 128, BF16, True, seed=1), ref.layer(512, 512, 128, BF16, True, seed=2)
    D1, D2 = Dev(L1), Dev(L2)
    M = 100
    x = ref.normal(M, 512, 1.0, BF16, 1).to(DEV)
    a = torch.empty((M, 512), dtype=torch.bfloat16, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    da = torch.empty_like(a)
    h = torch.empty((M, 1024), dtype=torch.bfloat16, device=DEV)
    dh, db = torch.empty_like(h), torch.empty(1024, device=DEV)
    sizes = [w4.w4a16_glu_gemm_workspace_bytes(D1.lin, M), w4.w4a16_gemm_ep_workspace_bytes(D2.lin, M),
             w4.w4a16_glu_gemm_backward_workspace_bytes(D1.lin, M), w4.w4a16_gemm_ep_backward_workspace_bytes(D2.lin, M)]
    ws, nb = workspace(max(sizes))

    def block():
        w4.w4a16_glu_gemm(x, D1.lin, a, M, SILU, h, workspace=ws, workspace_bytes=nb)
        w4.w4a16_gemm_ep(a, D2.lin, y, M, NONE, x, workspace=ws, workspace_bytes=nb)
        w4.w4a16_gemm_ep_backward(y, None, D2.lin, da, M, NONE, workspace=ws, workspace_bytes=nb)
        w4.w4a16_glu_gemm_backward(da, h, D1.lin, dx, M, SILU, dh, db, y, workspace=ws, workspace_bytes=nb)

    block()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dh, db)]
    s = torch.cuda.Stream()
    for t in (y, dx, dh, db):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (y, dx, dh, db)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block()
    for _ in range(4):
        for t in (y, dx, dh, db):
            t.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, (y, dx, dh, db)))
        block()
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31 and byte offsets 2^32: a wide
    stride, few rows."""
    M, K, N, ld = 1040, 128, 64, 1 << 22
    L = ref.layer(K, N, 128, F16, False, seed=3)
    D = Dev(L)
    big = torch.empty(M * ld, dtype=torch.float16, device=DEV)           # 8.7 GB
    rows = big.view(M, ld)
    x = ref.normal(M, K, 1.0, F16, 1)
    rows[:, :K] = x.to(DEV)
    y = rows[:, 4096:4096 + N]
    ws, nb = workspace(w4.w4a16_gemm_ep_workspace_bytes(D.lin, M))
    w4.w4a16_gemm_ep(big, D.lin, y, M, NONE, None, None, F16, ldx=ld, ldy=ld, workspace=ws, workspace_bytes=nb)
    yr, pr = ref.ep(x, L, NONE)
    ref.close(y, yr, ref.tol_ep(yr, pr, F16), "wide stride ep")
    dx = rows[:, 8192:8192 + K]
    ws, nb = workspace(w4.w4a16_gemm_ep_backward_workspace_bytes(D.lin, M))
    w4.w4a16_gemm_ep_backward(y, None, D.lin, dx, M, NONE, dt=F16, lddy=ld, lddx=ld, workspace=ws, workspace_bytes=nb)
    rx, rd, _ = ref.ep_backward(y.cpu(), None, L, NONE)
    ref.close(dx, rx, ref.tol_dx(rx, rd, L, F16), "wide stride dx")


def on_device(L):
    """The layer with its tensors on the GPU: the 64-bit reference of a large one."""
    return ref.Layer(L.K, L.N, L.group, L.dt, *(t if t is None else t.to(DEV) for t in (L.q, L.scale, L.zero, L.bias)))


# decode kernel: column blocks per workgroup (1 by default, 2 and 4 for wide
# matrices), and K in slices (few rows of 13 to 80 million weights and more)
@pytest.mark.parametrize("glu,M,K,N,group,dt,slices", [
    (False, 3, 256, 7168, 128, BF16, 1), (False, 20, 384, 7168, 384, F16, 1),
    (False, 1, 256, 14336, 128, F16, 1), (False, 16, 384, 14336, 128, BF16, 1), (False, 32, 128, 14336, 128, BF16, 1),
    (True, 1, 256, 14336, 128, BF16, 1), (True, 16, 384, 14336, 384, F16, 1), (True, 32, 256, 14336, 128, BF16, 1),
    (False, 5, 14336, 4096, 128, BF16, 4), (False, 17, 14336, 4096, 512, F16, 4), (False, 32, 14336, 4096, 256, BF16, 4),
    (False, 16, 53376, 512, 128, F16, 8), (False, 19, 26752, 512, 128, BF16, 8),
    (True, 5, 40960, 2048, 128, F16, 8), (True, 16, 40960, 2048, 256, BF16, 8), (True, 17, 20608, 2048, 128, BF16, 8),
])
def test_decode_blocks_and_slices(glu, M, K, N, group, dt, slices):
    L = ref.layer(K, N, group, dt, True, seed=M)
    D, dev = Dev(L), on_device(L)
    query = w4.w4a16_glu_gemm_workspace_bytes if glu else w4.w4a16_gemm_ep_workspace_bytes
    assert query(D.lin, M) == (slices * M * N * 4 if slices > 1 else 0)
    # sums of about the size that K = 256 gives: the activation is then not saturated
    x, r = ref.normal(M, K, 16.0 / K ** 0.5, dt, 1), ref.normal(M, N, 1.0, dt, 2)
    if glu:
        y, h = run_glu(D, x, SILU, save=True)
        yr, hr = (t.cpu() for t in ref.glu(x.to(DEV), dev, SILU))
        ref.close(y, yr, ref.tol_glu(yr, hr, dt), "glu")
    else:
        y, h = run_ep(D, x, GELU, r, save=True)
        yr, hr = (t.cpu() for t in ref.ep(x.to(DEV), dev, GELU, r.to(DEV)))
        ref.close(y, yr, ref.tol_ep(yr, hr, dt), "ep")
    ref.close(h, hr, ref.tol_ep(hr, hr, dt), "pre")


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("M,dt", [(64, BF16), (75, F16)])
def test_transposed_decode_slices_of_several_row_groups(glu, M, dt):
    """Rows past 32 with N in slices: seven of them, which no tile plan has; the
    bias gradient is formed once."""
    K, N = 128, 14336
    L = ref.layer(K, N, 128, dt, True, seed=5)
    D = Dev(L)
    query = w4.w4a16_glu_gemm_backward_workspace_bytes if glu else w4.w4a16_gemm_ep_backward_workspace_bytes
    rows = 4 * N * ((M + 3) // 4)                    # partial column sums, one row per block of four
    assert query(D.lin, M) == rows + 7 * M * K * 4
    dy = ref.normal(M, N // 2 if glu else N, 0.5, dt, 1)
    h, r = ref.normal(M, N, 1.5, dt, 2), ref.normal(M, K, 0.5, dt, 3)
    dx, d, db = run_bwd(D, glu, dy, h, SILU, r)
    rx, rd, rb = (ref.glu_backward if glu else ref.ep_backward)(dy, h, L, SILU, r)
    ref.close(d, rd, ref.tol_d(rd, dt), "d")
    ref.close(dx, rx, ref.tol_dx(rx, rd, L, dt), "dx")
    ref.close(db, rb, 2.0 ** -20 * (rd.abs().sum(0) + rd.abs().amax()), "dbias")


def large_x(D, M, size):
    """A product of x of the given size and scales near 2^-38 against 64 bits: y, x W
    and what a sum in fp32 is off by."""
    x = ref.normal(M, D.L.K, size, BF16, 1)
    y, _ = run_ep(D, x, NONE)
    yr, _ = ref.ep(x, D.L, NONE)
    terms = (x.double().square() @ D.L.weights().square()).sqrt()
    ref.close(y, yr, ref.ULP[BF16] * 1.01 * yr.abs() + 8 * ref.SUM * terms, f"x of size {size}")


def scaled_layer(K, N, factor, seed=8):
    L = ref.layer(K, N, 128, BF16, True, bias=False, seed=seed)
    L.scale = (L.scale.float() * factor).bfloat16()
    return L


@pytest.mark.parametrize("size", [2.0 ** 117, 2.0 ** 125])
@pytest.mark.parametrize("M", [2, 20])
def test_large_finite_x_on_few_rows(M, size):
    """Finite x up to the type's largest values (normal numbers of size 2^125 reach
    2^127) times small scales, and as small ones times large scales: what the terms
    of the sum allow is finite and keeps its bits."""
    large_x(Dev(scaled_layer(256, 128, 2.0 ** -30)), M, size)
    large_x(Dev(scaled_layer(256, 128, 2.0 ** 30)), M, 2.0 ** -118)


@pytest.mark.parametrize("size", [2.0 ** 117, 2.0 ** 125])
@pytest.mark.parametrize("shape", range(SHAPES))
def test_large_finite_x_in_every_tile_shape(plan, shape, size):
    plan(shape, 1)
    D = Dev(scaled_layer(256, 128, 2.0 ** -30))
    large_x(D, 150, size)
    # a falling scale may not carry the sums past the type's range
    D.L.scale[0] *= 2.0 ** 10
    D.L.scale[1] *= 2.0 ** -40
    large_x(Dev(D.L), 150, 2.0 ** 100)


@pytest.mark.parametrize("shape", [-1, *range(SHAPES)])
def test_scales_far_apart_and_x_zero_between_them(plan, shape):
    """Groups of scales that lie 2^100 and more apart, subnormal ones among them, and
    x zero in the groups of the larger: the rest is the whole result."""
    K, N, M = 512, 128, 20 if shape < 0 else 150
    L = ref.layer(K, N, 128, BF16, True, bias=False, seed=8)
    s = L.scale
    s[0, :32], s[1:3, :32], s[3, :32] = 2.0 ** 10, 2.0 ** -70, 2.0 ** 20
    s[0, 32:64], s[1, 32:64], s[2, 32:64], s[3, 32:64] = 2.0 ** -3, 2.0 ** -66, 2.0 ** -110, 2.0 ** 30
    s[1:3, 64:96] = 3 * 2.0 ** -132
    s[1, 96:112], s[2, 96:112] = 3 * 2.0 ** -131, 0
    plan(shape, int(shape >= 0))
    x = ref.normal(M, K, 2.0 ** 24, BF16, 1)
    x[:, :128], x[:, 384:] = 0, 0
    y, _ = run_ep(Dev(L), x, NONE)
    yr, _ = ref.ep(x, L, NONE)
    terms = (x.double().square() @ L.weights().square()).sqrt()
    ref.close(y, yr, ref.ULP[BF16] * 1.01 * yr.abs() + 8 * ref.SUM * terms, "far apart")


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("M", [3, 300])
def test_gelu_keeps_its_lower_tail(M, dt):
    """GELU and its derivative at pre-activations from -12 to -2 that are exact (x = 0, the
    bias is all there is): relative to the result's own size.  The exponent's
    rounding (v^2 / 2 = 72 at most, a few 2^-24 of it) stays below 2^-14; fp16 has
    its subnormal spacing on top."""
    v = -2 - 10 * torch.arange(256) / 255
    L = ref.layer(128, 512, 128, dt, seed=1)
    L.bias = torch.cat((v, torch.full((256,), 512.0))).to(ref.TD[dt])
    v = L.bias[:256].double()
    cdf, pdf = torch.exp(torch.special.log_ndtr(v)), torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    D, tiny = Dev(L), 2.0 ** -25 * 1.01 if dt == F16 else 0.0

    def near(got, want, what):
        want = want.expand(M, 256)
        ref.close(got, want, (ref.ULP[dt] * 1.01 + 2.0 ** -14) * want.abs() + tiny, what)

    x = torch.zeros((M, 128), dtype=ref.TD[dt])
    near(run_ep(D, x, GELU)[0][:, :256], v * cdf, "gelu")
    near(run_glu(D, x, GELU)[0], v * cdf * 512, "gelu times 512")
    dy = torch.ones((M, 512), dtype=ref.TD[dt])
    h = L.bias.expand(M, 512).contiguous()
    near(run_bwd(D, False, dy, h, GELU)[1][:, :256], cdf + v * pdf, "gelu'")
    near(run_bwd(D, True, dy[:, :256].contiguous(), h, GELU)[1][:, 256:], v * cdf, "gelu, up half")
