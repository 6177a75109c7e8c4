"""Fused linear operators on the host: refusals before any device call, size
queries, and the 64-bit reference's gradients against differences."""
import ctypes as C

import pytest
import torch

import linear_ref as ref
import weight_only_quantized_amd as w4

F = 1 << 40          # never dereferenced: validation fails first


def lin(**kw):
    a = dict(K=256, N=256, w_packed=F, scale=F, zero=None, bias=None, group_size=128)
    a.update(kw)
    return w4.linear(**a)


def fwd(glu, L, x=F, ldx=0, act=1, res=None, ldr=0, pre=None, y=F, ldy=0, M=4, dt=1, ws=None, nb=0):
    if glu:
        return w4.lib().w4a16_glu_gemm(x, ldx, L, act, pre, y, ldy, M, dt, ws, nb, None)
    return w4.lib().w4a16_gemm_ep(x, ldx, L, act, res, ldr, pre, y, ldy, M, dt, ws, nb, None)


def bwd(glu, L, dy=F, lddy=0, h=F, act=2, add=None, ldadd=0, d=F, db=None, dx=F, lddx=0, M=4, dt=1, ws=F, nb=1 << 40):
    f = w4.lib().w4a16_glu_gemm_backward if glu else w4.lib().w4a16_gemm_ep_backward
    return f(dy, lddy, h, L, act, add, ldadd, d, db, dx, lddx, M, dt, ws, nb, None)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(K=100), 2), (dict(K=0), 2), (dict(N=96), 2), (dict(N=0), 2),
    (dict(group_size=32), 3), (dict(group_size=64), 3), (dict(group_size=192), 3), (dict(group_size=0), 3),
    (dict(group_size=512), 2),
    (dict(w_packed=None), 1), (dict(scale=None), 1),
    (dict(w_packed=F + 8), 4), (dict(scale=F + 1), 4),
])
def test_refuses_bad_weights(glu, kw, status):
    assert fwd(glu, lin(**kw)) == status
    assert bwd(glu, lin(**kw)) == status


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), 3), (dict(act=5), 3), (dict(act=-1), 3), (dict(M=-1), 2), (dict(M=1 << 31), 2),
    (dict(x=None), 1), (dict(y=None), 1), (dict(x=F + 8), 4), (dict(y=F + 8), 4), (dict(pre=F + 2), 4),
    (dict(ldx=248), 2), (dict(ldx=260), 4), (dict(ldy=64), 2), (dict(ldy=260), 4), (dict(ldx=1 << 40), 2),
])
def test_forward_refuses(glu, kw, status):
    assert fwd(glu, lin(), **kw) == status


def test_forward_refuses_misplaced_operands():
    assert fwd(False, lin(bias=F + 2)) == 4
    assert fwd(False, lin(), res=F + 2) == 4
    assert fwd(False, lin(), res=F, ldr=100) == 2
    assert fwd(False, lin(), res=F, ldr=257) == 4
    assert fwd(True, lin(N=192)) == 2               # gate and up halves need a multiple of 64 columns each
    assert w4.lib().w4a16_gemm_ep(F, 0, None, 0, None, 0, None, F, 0, 4, 1, None, 0, None) == 1


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(dt=7), 3), (dict(act=9), 3), (dict(M=-1), 2), (dict(dy=None), 1), (dict(h=None), 1), (dict(d=None), 1),
    (dict(dx=None), 1), (dict(ws=None), 5), (dict(nb=8), 5), (dict(ws=F + 8), 4), (dict(dy=F + 8), 4),
    (dict(h=F + 2), 4), (dict(d=F + 2), 4), (dict(dx=F + 4), 4), (dict(add=F + 8), 4), (dict(db=F + 2), 4),
    (dict(lddy=8), 2), (dict(lddy=261), 4), (dict(lddx=128), 2), (dict(lddx=257), 4), (dict(add=F, ldadd=8), 2),
])
def test_backward_refuses(glu, kw, status):
    assert bwd(glu, lin(), **kw) == status


def test_workspace_queries():
    L = lin(K=14336, N=4096)
    assert w4.w4a16_gemm_ep_workspace_bytes(L, 1) == 0
    need = w4.w4a16_gemm_ep_workspace_bytes(L, 77)
    assert need >= 2 * 77 * 4096 * 4 and need % (77 * 4096 * 4) == 0     # whole fp32 partial results
    assert fwd(False, L, M=77, ws=F, nb=need - 1) == 5
    assert fwd(False, L, M=77) == 5
    for q in (w4.w4a16_gemm_ep_workspace_bytes, w4.w4a16_glu_gemm_workspace_bytes,
              w4.w4a16_gemm_ep_backward_workspace_bytes, w4.w4a16_glu_gemm_backward_workspace_bytes):
        assert q(L, 0) == 0 and q(L, -1) == 0 and q(lin(K=100), 4) == 0 and q(lin(group_size=64), 4) == 0
    assert w4.w4a16_glu_gemm_workspace_bytes(lin(N=192), 77) == 0
    assert bwd(False, L, M=77, nb=w4.w4a16_gemm_ep_backward_workspace_bytes(L, 77) - 1) == 5


def test_no_rows_is_a_no_op():
    L = lin(w_packed=None, scale=None)
    assert fwd(False, L, x=None, y=None, M=0) == 0
    assert fwd(True, L, x=None, y=None, M=0) == 0
    for glu in (False, True):
        assert bwd(glu, L, dy=None, h=None, d=None, dx=None, ws=None, nb=0, M=0) == 0


def test_struct_matches_the_header():
    assert C.sizeof(w4.Linear) == 56
    t = torch.zeros(4)
    assert lin(bias=t).bias == t.data_ptr()         # and the description keeps its tensors
    assert lin(bias=t).tensors[3] is t
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_gemm_ep(F, lin(K=100), F, 4, stream=0)
    assert e.value.status == 2


@pytest.mark.parametrize("a", ref.ACTS)
def test_reference_gradients_match_differences(a):
    """ep_backward and glu_backward of the 64-bit reference against central
    differences of its forward functions: with step e the truncation error is
    O(e^2), the cancellation 2^-53 / e, so e = 2^-14 leaves 1e-7 and less (RELU's
    kink at 0 is not crossed: no pre-activation is that near)."""
    K, N, M, e = 128, 128, 3, 2.0 ** -14
    L = ref.layer(K, N, bias=True, seed=3)
    x = ref.normal(M, K, 1.0, ref.BF16, 4).double()
    v = torch.randn((M, K), dtype=torch.float64, generator=torch.Generator().manual_seed(5))
    for f, back, width in ((ref.ep, ref.ep_backward, N), (ref.glu, ref.glu_backward, N // 2)):
        dy = torch.randn((M, width), dtype=torch.float64, generator=torch.Generator().manual_seed(6))
        p = f(x, L, a)[1]
        dx, d, db = back(dy, p, L, a)
        num = ((f(x + e * v, L, a)[0] - f(x - e * v, L, a)[0]) * dy).sum() / (2 * e)
        assert abs(num - (dx * v).sum()) <= 1e-6 * (dx * v).abs().sum()
        b = L.bias
        L.bias = b.double() + e * torch.ones(N, dtype=torch.float64)
        up = f(x, L, a)[0]
        L.bias = b.double() - e * torch.ones(N, dtype=torch.float64)
        num = ((up - f(x, L, a)[0]) * dy).sum() / (2 * e)
        L.bias = b
        assert abs(num - db.sum()) <= 1e-6 * d.abs().sum()


def test_few_rows_backward_takes_the_faster_kernel():
    """dx of few rows: the decode kernel (no slices here) where it is the faster one, past
    that the tile kernel, whose slices the workspace shows (eight for 32 rows of 4096^2:
    12.5 us against 13.7; one row 11.2 against 8.5, 24 rows of 8192 x 4096 13.9 against 12.6)."""
    for M, K, N, slices in ((32, 4096, 4096, 8), (1, 4096, 4096, 0), (24, 8192, 4096, 0), (32, 4096, 14336, 8)):
        rows = 4 * N * ((M + 3) // 4)                # partial column sums, one row per block of four
        need = w4.w4a16_gemm_ep_backward_workspace_bytes(lin(K=K, N=N), M)
        assert need == rows + slices * M * K * 4, (M, K, N)


@pytest.mark.parametrize("refused,words", [
    (lambda: fwd(False, lin(group_size=64)), ("fused linear operators", "multiple of 128")),
    (lambda: fwd(False, lin(), act=9), ("w4a16_act",)),
    (lambda: fwd(False, lin(), ldx=248), ("row strides", "2^22")),
    (lambda: fwd(True, lin(N=192)), ("gated N%128",)),
    (lambda: fwd(False, lin(K=1 << 23)), ("up to 2^22",)),
    (lambda: fwd(False, lin(group_size=384)), ("group_size dividing K",)),
    (lambda: fwd(False, lin(), ldx=260), ("multiple of 8",)),
    (lambda: fwd(False, lin(), y=F + 2), ("fused linear operators: 16 bytes",)),
    (lambda: bwd(False, lin(), db=F + 2), ("dbias, 4",)),
])
def test_a_refusal_names_its_rule(refused, words):
    text = w4.w4a16_status_str(refused())
    assert all(w in text for w in words), text
