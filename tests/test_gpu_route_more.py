"""MoE router on the GPU: what the sizes, strides and spreads of the other file leave out."""
import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4
from test_gpu_route import check, check_bwd, logits_of, run, run_bwd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = ref.F16, ref.BF16, ref.F32


def spread_logits(T, E, dt, width):
    g = torch.Generator().manual_seed(T + E + width)
    return (torch.rand((T, E), generator=g) * -width + torch.randn((T, 1), generator=g) * 5).to(ref.TORCH[dt])


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,topk", [(300, 8, 8), (200, 16, 16), (300, 64, 8), (100, 40, 12), (100, 256, 8), (50, 1000, 16)])
@pytest.mark.parametrize("width", [3, 80])
def test_weights_of_far_choices(T, E, topk, renorm, dt, width):
    """A chosen weight is as exact far from the row's largest logit as next to it.

    In half steps of fp32: its exponential 3 1/8 (exp2 within a step, 2; one rounding of the corrected
    value, 1; the correction, at most 2^-16 of it, is itself off by some 2^-16 of a step).  Renormalized: the
    same again for the sum's terms, at most 6 + 4 additions (lanes of a token, choices of a lane),
    a reciprocal and a product.  Else: the row's sum, whose terms carry 2.25 d + 2 each for their
    distance d, weighted by their probabilities; 15 + 6 additions, a reciprocal and a product."""
    z = spread_logits(T, E, dt, width)
    _, w, _, _ = run(z.to(DEV), topk, renorm, dt)
    _, want, _, _ = ref.route(z, topk, renorm)
    d = z.double().amax(1, keepdim=True) - z.double()
    assert float(d.max()) < 87                             # nothing below fp32's normal numbers
    if renorm:
        steps = torch.full((T, 1), 2 * 3.125 + 10 + 2, dtype=torch.float64)
    else:
        steps = 3.125 + 2.25 * (ref.softmax_parts(z) * d).sum(1, keepdim=True) + 2 + 21 + 2
    rel = (w.cpu().double() - want).abs() / want
    assert bool((rel <= steps * ref.U32).all()), float((rel / (steps * ref.U32)).max())


def test_choices_whose_distance_leaves_fp32():
    """Differences past fp32's range give the weight 0."""
    z = torch.zeros((2, 8))
    z[0, 3], z[0, 5] = 3e38, -3e38
    z[1, :4] = -3e38
    ids, w, cnt, loss = run(z.to(DEV), 8, True, F32)
    ri, rw, rc, _ = ref.route(z, 8, True)
    assert torch.equal(ids.cpu(), ri) and torch.equal(cnt.cpu(), rc)
    assert bool(((w.cpu().double() - rw).abs() <= 2.0 ** -22 * rw).all())


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("E,pad,lpad", [(16, 8, 16), (64, 8, 16), (120, 40, 8), (256, 8, 24), (512, 16, 8), (1000, 24, 8)])
def test_wide_rows_inside_wider_buffers(E, pad, lpad, dt):
    """Rows of whole 16-byte pieces with gaps between them: the gaps are neither read (NaN) nor written."""
    T, topk = 70, 6
    z = logits_of(T, E, dt, seed=4)
    wide = torch.full((T, E + pad), float("nan"), dtype=z.dtype)
    wide[:, :E] = z
    g = torch.Generator().manual_seed(E)
    dw, dloss = torch.randn((T, topk), generator=g).to(DEV), torch.tensor([0.6], device=DEV)
    for renorm in (False, True):
        ids, w, cnt, loss = run(wide.to(DEV), topk, renorm, dt, ld=E + pad, E=E)
        check(z, (ids, w, cnt, loss), topk, renorm)
        for ld, lddl in ((E + pad, E + lpad), (0, E + lpad), (E + pad, 0)):
            dz = run_bwd((wide if ld else z).to(DEV), ids, w, cnt, dw, dloss, topk, renorm, dt, ld=ld, lddl=lddl, E=E)
            check_bwd(z, dz[:, :E], ids, w, cnt, dw, dloss, renorm)
            assert bool((dz[:, E:] == 9.0).all())


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("T,E,topk", [(3000, 40, 20), (500, 8, 8), (90, 600, 40)])
def test_backward_of_more_choices_than_lanes(T, E, topk, dt):
    """Several tokens per wave and loops over the tokens, some of them padding."""
    z = logits_of(T, E, dt, seed=6)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(E)) > 0.2).to(torch.uint8)
    dw = torch.randn((T, topk), generator=torch.Generator().manual_seed(T)).to(DEV)
    for renorm in (False, True):
        ids, w, cnt, _ = run(z.to(DEV), topk, renorm, dt, mask=mask.to(DEV))
        dz = run_bwd(z.to(DEV), ids, w, cnt, dw, None, topk, renorm, dt, mask=mask.to(DEV))
        # (the other file's bound counts 16 chosen ones: topk - 16 additions more)
        want, size = ref.route_backward(z, ids.cpu(), w.cpu(), cnt.cpu(), dw.cpu(), None, renorm, mask)
        td = z.dtype
        bound = (ref.prob_bound(z) + (48 + topk) * ref.U32) * size * (1 + ref.half_step(td)) + ref.half_step(td) * want.abs()
        bound = bound + torch.finfo(td).smallest_normal * torch.finfo(td).eps
        assert bool(((dz.cpu().double() - want).abs() <= bound).all())
