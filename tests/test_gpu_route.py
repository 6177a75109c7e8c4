"""MoE router on the GPU against 64-bit references."""
import math

import pytest
import torch

import w8a8_ref as ref
import weight_only_quantized_amd as w4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = ref.F16, ref.BF16, ref.F32


def logits_of(T, E, dt, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed * 100 + T + E)
    return (torch.randn((T, E), generator=g) * spread + torch.randn(E, generator=g) * 0.5).to(ref.TORCH[dt])


def run(z, topk, renorm, dt, mask=None, ld=0, want_counts=True, E=None):
    T, E = z.shape[0], E or z.shape[1]
    ids = torch.full((T, topk), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T, topk), 7.0, device=DEV)
    nb = w4.w4a16_moe_route_workspace_bytes(T, E)
    ws = torch.full((max(nb, 4),), 0xA5, dtype=torch.uint8, device=DEV)
    cnt = torch.full((E + 1,), 77, dtype=torch.int32, device=DEV) if want_counts else None
    loss = torch.full((1,), 7.0, device=DEV) if want_counts else None
    w4.w4a16_moe_route(z, T, E, topk, ids, w, counts=cnt, loss=loss, token_mask=mask, renormalize=renorm, dt=dt,
                       ld=ld, workspace=ws if want_counts else None, workspace_bytes=nb if want_counts else 0)
    return ids, w, cnt, loss


def check(z, got, topk, renorm, mask=None):
    ids, w, cnt, loss = got
    ri, rw, rc, rl = ref.route(z, topk, renorm, mask)
    assert torch.equal(ids.cpu(), ri)
    rel = ref.prob_bound(z)
    nan = torch.isnan(rw)
    assert torch.equal(torch.isnan(w.cpu()), nan)
    err = (w.cpu().double() - rw).abs()[~nan]
    assert bool((err <= rel * rw[~nan] + 2.0 ** -126).all()), float(err.max())
    if cnt is None:
        return
    assert torch.equal(cnt.cpu(), rc)
    if math.isnan(rl):
        assert math.isnan(float(loss))
    else:
        # a probability's error, and additions of at most T / 256 + 64 of them in fp32
        assert abs(float(loss) - rl) <= (rel + ref.U32 * (z.shape[0] / 256 + 64)) * rl


SHAPES = [(1, 1, 1), (1, 4, 2), (3, 8, 8), (16, 64, 8), (5, 9, 3), (33, 60, 6), (257, 64, 8), (100, 128, 4),
          (519, 65, 2), (64, 256, 8), (40, 318, 10), (21, 512, 1), (9, 1000, 16), (7, 1024, 70), (4000, 32, 4),
          (2049, 16, 16), (1500, 200, 6)]


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,topk", SHAPES)
def test_route(T, E, topk, renorm, dt):
    z = logits_of(T, E, dt)
    check(z, run(z.to(DEV), topk, renorm, dt), topk, renorm)


@pytest.mark.parametrize("E", [8, 64, 100, 256, 700])
def test_ties_go_to_the_lowest_index(E):
    g = torch.Generator().manual_seed(E)
    z = torch.randint(-2, 3, (300, E), generator=g).float()
    z[0] = 0
    z[1] = -0.0
    z[2, ::2] = -0.0
    z[2, 1::2] = 0.0
    for dt in (F16, BF16, F32):
        zz = z.to(ref.TORCH[dt])
        check(zz, run(zz.to(DEV), min(E, 9), True, dt), min(E, 9), True)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("E", [6, 64, 300])
def test_masks_infinities_and_padding(E, dt):
    T, topk = 120, 5
    z = logits_of(T, E, dt, seed=2)
    low = torch.finfo(z.dtype).min
    z[3] = float("-inf")                                  # no expert
    z[4, 2:] = float("-inf")                              # two experts for five entries
    z[5, 1:] = low                                        # masked with the type's lowest value: still a choice
    z[6] = low
    z[7, 1] = float("-inf")
    z[8] = torch.finfo(z.dtype).max
    mask = (torch.arange(T) % 7 != 1).to(torch.uint8) * 3
    mask[3:9] = 1
    for renorm in (False, True):
        check(z, run(z.to(DEV), topk, renorm, dt, mask=mask.to(DEV)), topk, renorm, mask)
        check(z, run(z.to(DEV), topk, renorm, dt, want_counts=False), topk, renorm)
    z[10, 0] = float("nan")
    z[11, 3] = float("inf")
    z[12, 1] = float("nan")                               # token 12 is kept by the mask below
    z[12, 0] = float("-inf")
    mask[10:13] = 1
    z[15] = float("nan")                                  # padding may hold anything
    mask[15] = 0
    check(z, run(z.to(DEV), topk, True, dt, mask=mask.to(DEV)), topk, True, mask)


def test_no_token_and_only_padding():
    z = logits_of(6, 12, F32)
    mask = torch.zeros(6, dtype=torch.uint8)
    got = run(z.to(DEV), 3, True, F32, mask=mask.to(DEV))
    check(z, got, 3, True, mask)
    assert float(got[3]) == 0.0
    cnt, loss = torch.full((13,), 5, dtype=torch.int32, device=DEV), torch.full((1,), 5.0, device=DEV)
    w4.w4a16_moe_route(None, 0, 12, 3, None, None, counts=cnt, loss=loss)
    assert int(cnt.abs().sum()) == 0 and float(loss) == 0.0


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_row_strides(dt):
    T, E = 50, 30
    z = logits_of(T, E, dt)
    for pad in (1, 2, 34):
        wide = torch.full((T, E + pad), float("nan"), dtype=z.dtype)
        wide[:, :E] = z
        check(z, run(wide.to(DEV), 4, True, dt, ld=E + pad, E=E), 4, True)
    odd = torch.full((T * E + 1,), float("nan"), dtype=z.dtype)      # starts one element into a buffer
    odd[1:] = z.reshape(-1)
    check(z, run(odd.to(DEV)[1:].view(T, E), 4, True, dt), 4, True)


def test_equal_calls_give_equal_bits():
    z = logits_of(3000, 64, BF16).to(DEV)
    a = run(z, 8, True, BF16)
    for _ in range(3):
        for u, v in zip(a, run(z, 8, True, BF16)):
            assert torch.equal(u, v)


# ---- backward ------------------------------------------------------------------------

def run_bwd(z, ids, w, cnt, dw, dloss, topk, renorm, dt, mask=None, ld=0, lddl=0, E=None):
    T, E = z.shape[0], E or z.shape[1]
    dz = torch.full((T, lddl or E), 9.0, dtype=ref.TORCH[dt], device=DEV)
    w4.w4a16_moe_route_backward(z, ids, w, dz, T, E, topk, counts=cnt, dtopk_w=dw, dloss=dloss, token_mask=mask,
                                renormalize=renorm, dt=dt, ld=ld, lddl=lddl)
    return dz


def check_bwd(z, dz, ids, w, cnt, dw, dloss, renorm, mask=None):
    cpu = [None if t is None else t.cpu() for t in (ids, w, cnt, dw)]
    want, size = ref.route_backward(z, *cpu, None if dloss is None else float(dloss), renorm, mask)
    got = dz.cpu().double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    td = dz.dtype
    # probabilities as in the forward pass, the sum over up to 1024 experts, up to 16 chosen
    # ones and a few products; then one rounding to the logits' type
    bound = (ref.prob_bound(z) + 48 * ref.U32) * size * (1 + ref.half_step(td)) + ref.half_step(td) * want.abs()
    bound = bound + torch.finfo(td).smallest_normal * torch.finfo(td).eps
    err = (got - want).abs()
    assert bool((err <= bound)[~nan].all()), float((err / bound)[~nan].max())


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,topk", [s for s in SHAPES if s[2] <= 16])
def test_backward(T, E, topk, renorm, dt):
    z = logits_of(T, E, dt)
    ids, w, cnt, _ = run(z.to(DEV), topk, renorm, dt)
    g = torch.Generator().manual_seed(T)
    dw, dloss = torch.randn((T, topk), generator=g).to(DEV), torch.tensor([0.7], device=DEV)
    for a, b in ((dw, dloss), (dw, None), (None, dloss), (None, None)):
        dz = run_bwd(z.to(DEV), ids if a is not None else None, w if a is not None else None,
                     cnt if b is not None else None, a, b, topk, renorm, dt)
        check_bwd(z, dz, ids, w, cnt, a, b, renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_backward_masks_and_infinities(renorm):
    T, E, topk, dt = 60, 40, 4, F32
    z = logits_of(T, E, dt)
    z[3] = float("-inf")
    z[4, 2:] = float("-inf")
    z[5, 7] = float("-inf")
    z[9] = float("nan")
    z[10, 0] = float("inf")
    mask = (torch.arange(T) % 5 != 2).to(torch.uint8)
    mask[9] = 0
    ids, w, cnt, _ = run(z.to(DEV), topk, renorm, dt, mask=mask.to(DEV))
    dw, dloss = torch.randn((T, topk), generator=torch.Generator().manual_seed(3)).to(DEV), torch.tensor([0.5], device=DEV)
    dw[ids < 0] = float("nan")                            # gradients of entries that went nowhere are not read
    dz = run_bwd(z.to(DEV), ids, w, cnt, dw, dloss, topk, renorm, dt, mask=mask.to(DEV))
    check_bwd(z, dz, ids, w, cnt, torch.nan_to_num(dw), dloss, renorm, mask)


def test_backward_strides_leave_the_gaps():
    T, E, topk = 30, 20, 3
    z = logits_of(T, E, BF16)
    ids, w, cnt, _ = run(z.to(DEV), topk, True, BF16)
    dw, dloss = torch.randn((T, topk), generator=torch.Generator().manual_seed(3)).to(DEV), torch.tensor([0.5], device=DEV)
    wide = torch.full((T, E + 3), float("nan"), dtype=z.dtype)
    wide[:, :E] = z
    dz = run_bwd(wide.to(DEV), ids, w, cnt, dw, dloss, topk, True, BF16, ld=E + 3, lddl=E + 5, E=E)
    check_bwd(z, dz[:, :E], ids, w, cnt, dw, dloss, True)
    assert bool((dz[:, E:] == 9.0).all())


@pytest.mark.parametrize("E", [12, 64, 100, 256])
def test_repeated_ids_add_up(E):
    """Choices made elsewhere may name an expert twice: both entries' gradients arrive."""
    T, topk = 5, 4
    z = logits_of(T, E, F32)
    ids = torch.tensor([[1, 1, 3, -1], [0, 0, 0, 0], [11, 2, 11, 5], [4, 5, 6, 7], [-1, -1, -1, -1]], dtype=torch.int32)
    w = torch.rand((T, topk), generator=torch.Generator().manual_seed(1))
    dw = torch.randn((T, topk), generator=torch.Generator().manual_seed(2))
    for renorm in (False, True):
        dz = run_bwd(z.to(DEV), ids.to(DEV), w.to(DEV), None, dw.to(DEV), None, topk, renorm, F32)
        check_bwd(z, dz, ids, w, None, dw, None, renorm)


def test_graph_of_both_passes():
    """Captured together and replayed with eager work between the replays."""
    T, E, topk, dt = 300, 64, 6, F32
    zs = [logits_of(T, E, dt, seed=s).to(DEV) for s in range(3)]
    dw, dloss = torch.randn((T, topk), generator=torch.Generator().manual_seed(3)).to(DEV), torch.tensor([0.5], device=DEV)

    def eager(z):
        ids, w, cnt, loss = run(z, topk, True, dt)
        return [ids, w, cnt, loss, run_bwd(z, ids, w, cnt, dw, dloss, topk, True, dt)]
    want = [eager(z) for z in zs]
    nb = w4.w4a16_moe_route_workspace_bytes(T, E)
    ws, static = torch.empty(max(nb, 4), dtype=torch.uint8, device=DEV), zs[0].clone()
    out = [torch.zeros_like(t) for t in want[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.w4a16_moe_route(static, T, E, topk, out[0], out[1], counts=out[2], loss=out[3], workspace=ws,
                           workspace_bytes=nb)
        w4.w4a16_moe_route_backward(static, out[0], out[1], out[4], T, E, topk, counts=out[2], dtopk_w=dw, dloss=dloss)
    torch.cuda.synchronize()
    for i in (0, 1, 2, 1, 0):
        static.copy_(zs[i])
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, want[i]):
            assert torch.equal(u, v)
            u.zero_()
        for u, v in zip(eager(zs[2 - i]), want[2 - i]):
            assert torch.equal(u, v)
