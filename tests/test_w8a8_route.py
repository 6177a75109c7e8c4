"""W8A8 products and the MoE router on the host: refusals before any device
call, size queries, and the 64-bit references against other forms."""
import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4

F = 1 << 40          # never dereferenced: validation fails first


def quant(x=F, ldx=0, rc=None, qx=F, sx=F, M=4, K=256, dt=1):
    return w4.lib().w8a8_quantize(x, ldx, rc, qx, sx, M, K, dt, None)


def pre(qx=F, sx=F, wp=F, sw=F, bias=None, y=F, ldy=0, M=4, K=256, N=256, dt=1):
    return w4.lib().w8a8_gemm_prequant(qx, sx, wp, sw, bias, y, ldy, M, K, N, dt, None)


def gemm(x=F, ldx=0, wp=F, sw=F, bias=None, y=F, ldy=0, M=4, K=256, N=256, dt=1, ws=F, nb=1 << 40):
    return w4.lib().w8a8_gemm(x, ldx, wp, sw, bias, y, ldy, M, K, N, dt, ws, nb, None)


def grouped(x=F, srt=None, topk=1, off=F, wp=F, sw=F, y=F, E=4, R=8, K=256, N=256, dt=1, ws=F, nb=1 << 40):
    return w4.lib().w8a8_grouped_gemm(x, srt, topk, off, wp, sw, y, E, R, K, N, dt, ws, nb, None)


@pytest.mark.parametrize("f", [quant, pre, gemm, grouped])
@pytest.mark.parametrize("kw,status", [(dict(dt=2), 3), (dict(dt=-1), 3), (dict(K=0), 2), (dict(K=100), 2),
                                       (dict(K=-128), 2), (dict(K=1 << 17), 2)])
def test_refuses_sizes_and_types(f, kw, status):
    assert f(**kw) == status


@pytest.mark.parametrize("f", [pre, gemm, grouped])
@pytest.mark.parametrize("kw,status", [(dict(N=0), 2), (dict(N=96), 2), (dict(N=(1 << 22) + 64), 2), (dict(wp=None), 1),
                                       (dict(sw=None), 1), (dict(y=None), 1), (dict(wp=F + 8), 4), (dict(sw=F + 2), 4),
                                       (dict(y=F + 8), 4)])
def test_refuses_weights_and_results(f, kw, status):
    assert f(**kw) == status


@pytest.mark.parametrize("f,kw,status", [
    (quant, dict(M=-1), 2), (quant, dict(M=1 << 31), 2), (quant, dict(x=None), 1), (quant, dict(qx=None), 1),
    (quant, dict(sx=None), 1), (quant, dict(x=F + 2), 4), (quant, dict(qx=F + 8), 4), (quant, dict(sx=F + 2), 4),
    (quant, dict(rc=F + 1), 4), (quant, dict(ldx=248), 2), (quant, dict(ldx=257), 4), (quant, dict(ldx=1 << 23), 2),
    (pre, dict(M=-1), 2), (pre, dict(M=1 << 31), 2), (pre, dict(qx=None), 1), (pre, dict(sx=None), 1),
    (pre, dict(qx=F + 8), 4), (pre, dict(sx=F + 2), 4), (pre, dict(bias=F + 1), 4), (pre, dict(ldy=248), 2),
    (pre, dict(ldy=260), 4),
    (gemm, dict(M=-1), 2), (gemm, dict(x=None), 1), (gemm, dict(x=F + 8), 4), (gemm, dict(ldx=8), 2),
    (gemm, dict(ldx=260), 4), (gemm, dict(ldy=8), 2), (gemm, dict(ldy=257), 4), (gemm, dict(ws=None), 5),
    (gemm, dict(nb=1024 + 255 + (32 << 20)), 5), (gemm, dict(ws=F + 8), 4), (gemm, dict(bias=F + 1), 4),
    (grouped, dict(R=-1), 2), (grouped, dict(E=0), 2), (grouped, dict(E=(1 << 20) + 1), 2), (grouped, dict(x=None), 1),
    (grouped, dict(off=None), 1), (grouped, dict(off=F + 2), 4), (grouped, dict(srt=F + 2), 4),
    (grouped, dict(srt=F, topk=0), 2), (grouped, dict(srt=F, topk=3), 2), (grouped, dict(srt=F, topk=1 << 33), 2),
    (grouped, dict(ws=None), 5), (grouped, dict(nb=2048 + 31), 5), (grouped, dict(x=F + 8), 4),
])
def test_refuses(f, kw, status):
    assert f(**kw) == status


def test_workspace_sizes():
    for q in (w4.w8a8_workspace_bytes, w4.w8a8_grouped_workspace_bytes):
        assert q(0, 256) == 0 and q(-1, 256) == 0 and q(4, 100) == 0 and q(4, 1 << 17) == 0
        assert q(1 << 20, 14336) == (1 << 20) * (14336 + 4)
    assert w4.w8a8_grouped_workspace_bytes(4, 256) == 1024 + 16
    assert w4.w8a8_grouped_workspace_bytes(3, 128) == 512 + 12
    # up to 1024 rows: 32 MiB for the sums of K slices, behind the scales
    assert w4.w8a8_workspace_bytes(4, 256) == 1024 + 256 + (32 << 20)
    assert w4.w8a8_workspace_bytes(1024, 256) == 1024 * 256 + 4096 + (32 << 20)
    assert w4.w8a8_workspace_bytes(1025, 256) == 1025 * 256 + 4100


def test_no_rows_is_a_no_op():
    none = dict(x=None, wp=None, sw=None, y=None, ws=None, nb=0)
    assert gemm(M=0, **none) == 0 and grouped(R=0, off=None, **none) == 0
    assert quant(M=0, x=None, qx=None, sx=None) == 0 and pre(M=0, qx=None, sx=None, wp=None, sw=None, y=None) == 0


def route(z=F, ld=0, mask=None, T=8, E=64, topk=4, renorm=1, ids=F, w=F, cnt=F, loss=F, dt=2, ws=F, nb=1 << 40):
    return w4.lib().w4a16_moe_route(z, ld, mask, T, E, topk, renorm, ids, w, cnt, loss, dt, ws, nb, None)


def back(z=F, ld=0, mask=None, ids=F, w=F, cnt=F, dw=F, dloss=F, T=8, E=64, topk=4, renorm=1, dz=F, lddl=0, dt=2):
    return w4.lib().w4a16_moe_route_backward(z, ld, mask, ids, w, cnt, dw, dloss, T, E, topk, renorm, dz, lddl, dt,
                                             None)


@pytest.mark.parametrize("f", [route, back])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), 3), (dict(dt=-1), 3), (dict(E=1025), 3), (dict(E=0), 2), (dict(T=-1), 2), (dict(topk=0), 2),
    (dict(topk=65), 2), (dict(T=1 << 29), 2), (dict(ld=63), 2), (dict(ld=(1 << 22) + 1), 2), (dict(z=None), 1),
    (dict(z=F + 2), 4), (dict(z=F + 1, dt=0), 4), (dict(ids=F + 2), 4), (dict(w=F + 2), 4), (dict(cnt=F + 2), 4),
    (dict(cnt=None), 1),
])
def test_router_refuses(f, kw, status):
    assert f(**kw) == status


def test_router_refuses_the_rest():
    assert route(ids=None) == 1 and route(w=None) == 1 and route(loss=F + 2) == 4
    need = w4.w4a16_moe_route_workspace_bytes(4096, 64)
    assert need > 0 and route(T=4096, nb=need - 1) == 5 and route(T=4096, ws=None) == 5
    assert route(T=4096, ws=F + 8) == 4
    assert back(dz=None) == 1 and back(ids=None) == 1 and back(w=None) == 1
    assert back(dz=F + 2) == 4 and back(dw=F + 2) == 4 and back(dloss=F + 2) == 4 and back(lddl=63) == 2
    for T, E in ((0, 64), (-1, 64), (8, 0), (8, 1025), (1 << 31, 64)):
        assert w4.w4a16_moe_route_workspace_bytes(T, E) == 0


def test_router_without_tokens_is_a_no_op():
    assert route(T=0, z=None, ids=None, w=None, cnt=None, loss=None, ws=None, nb=0) == 0
    assert back(T=0, z=None, ids=None, w=None, cnt=None, dw=None, dloss=None, dz=None) == 0


# ---- the references themselves -------------------------------------------------------

def test_reference_codes_are_the_nearest():
    for td in (torch.float16, torch.bfloat16):
        x = torch.randn((6, 64), generator=torch.Generator().manual_seed(1)).to(td)
        q, s = ref.quantize(x)
        lattice = torch.arange(-127, 128, dtype=torch.float64)
        d = (x.double()[..., None] - lattice * s.double()[:, None, None]).abs()
        assert torch.equal(lattice[d.argmin(-1)], q)


@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(renorm):
    """The gradient's formula against central differences of the forward definitions (the
    choice and the counts held fixed)."""
    T, E, topk = 5, 7, 3
    g = torch.Generator().manual_seed(4)
    z = torch.randn((T, E), generator=g, dtype=torch.float64)
    z[1, 2] = float("-inf")
    mask = torch.tensor([1, 1, 0, 1, 1], dtype=torch.uint8)
    ids, w, cnt, _ = ref.route(z, topk, renorm, mask)
    dw, dloss = torch.randn((T, topk), generator=g, dtype=torch.float64), 0.3
    live = mask.bool()

    def total(v):
        p = ref.softmax_parts(v)
        wk = p.gather(1, ids.long().clamp(min=0))
        wk = wk / wk.sum(1, keepdim=True) if renorm else wk
        c = cnt[:E].double()
        loss = E * (c / c.sum() * p[live].sum(0) / int(cnt[E])).sum()
        return float((wk * dw)[live].sum() + dloss * loss)
    got, _ = ref.route_backward(z, ids, w, cnt, dw, dloss, renorm, mask)
    for t in range(T):
        for e in range(E):
            if z[t, e] == float("-inf"):
                assert got[t, e] == 0
                continue
            a, b = z.clone(), z.clone()
            a[t, e] += 1e-5
            b[t, e] -= 1e-5
            # third derivatives of order 1 times 1e-10, and 64-bit sums' rounding over 2e-5
            assert abs((total(a) - total(b)) / 2e-5 - float(got[t, e])) < 1e-9


def test_packed_layout_reference():
    w = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(128 * 64 // 256).view(1, 128, 64)
    p = ref.pack8(w).reshape(-1)
    for k, n in ((0, 0), (5, 3), (37, 17), (127, 63)):
        at = 2048 * (n // 16) + 32 * (16 * (k // 32) + n % 16) + k % 32
        assert int(p[at]) == int(w[0, k, n]) + 128
